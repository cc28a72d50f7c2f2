// Writing the 8-bit paged cache: rows of composed bf16 caches (fill) and new
// tokens rotated on the way (append).
//
// A page holds `page` tokens of one layer; for each kv head its codes are
// e4m3 and share one scale 2^e.  With a = the largest finite magnitude of
// the rows written, e is the smallest integer with a <= 448 * 2^e, so no
// code saturates, and code = e4m3(x * 2^-e), to nearest even.  A power of two
// makes the scaling itself exact.  When later rows need a larger e than the
// page has, its codes c become e4m3(c * 2^(e_old - e)): exact but for codes
// that fall below e4m3's normal range.  A value that is not finite is held as
// NaN and takes no part in a.
//
// A CTA of 8 warps owns 128 consecutive rows of one (sequence, kv head), of K
// or of V: a whole number of pages whatever the page size (16 to 128), so a
// page's largest magnitude never leaves the CTA.  A warp owns 16 rows and
// keeps them in registers between the two steps (largest magnitude, codes),
// so the data are read once.  Bound by the bytes moved.
#include "pages8.h"

namespace c2kv {

namespace {

constexpr int PUT_THREADS = 256;
constexpr int PUT_ROWS = 128;
constexpr int PUT_WARP_ROWS = 16;

// 8 bf16 bit patterns in a uint4 -> fp32, NaN where not finite.
__device__ __forceinline__ void finite_or_nan8(const uint4& u, float (&f)[8]) {
  unpack8(u, f);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if ((__float_as_uint(f[e]) & 0x7F800000u) == 0x7F800000u) f[e] = __uint_as_float(0x7FFFFFFFu);
}

__device__ __forceinline__ uint32_t max_finite8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(f[e]) & 0x7FFFFFFFu;
    if (b < 0x7F800000u) m = max(m, b);
  }
  return m;
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
  return make_uint2(e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16),
                    e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16));
}

__device__ __forceinline__ uint32_t rescale4(uint32_t c, float by) {
  const float2 a = e4m3x2_to_float2(c & 0xFFFFu), b = e4m3x2_to_float2(c >> 16);
  return e4m3x2(a.x * by, a.y * by) | (e4m3x2(b.x * by, b.y * by) << 16);
}

// D: head_dim.  APPEND: rows [n_cached, n_cached + new) from the new tokens,
// K rotated; else rows [0, n_rows) from the bf16 caches.
template <int D, bool APPEND>
__global__ void __launch_bounds__(PUT_THREADS) put_kernel(const __grid_constant__ PutParams p) {
  constexpr int CH = D / 16;              // 8-element chunks of half a row
  constexpr int IT = D / 32;              // items (one chunk of each half) per lane
  __shared__ uint32_t warp_max[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y / p.pool.n_kv, h = blockIdx.y % p.pool.n_kv;
  const int kv = blockIdx.z & 1, layer = blockIdx.z >> 1;
  int first = 0, count;
  if (APPEND) {
    first = p.n_cached[b];
    count = p.n_new ? p.n_new[b] : p.t_len;
    if (first < 0) return;   // an empty place of the batch
    const int rr = p.rope_row[b];
    if (count < 0 || count > p.t_len || (int64_t)first + count > (int64_t)p.max_pages * p.pool.page ||
        (count > 0 && (rr < 0 || (int64_t)rr + count > p.table_rows))) {
      if (threadIdx.x == 0) atomicOr(p.err, kErrLength);
      return;
    }
  } else {
    count = p.n_rows[b];
  }
  const int row0 = (first / PUT_ROWS + (int)blockIdx.x) * PUT_ROWS;   // of this CTA's 128 rows
  const int end = first + count;
  if (row0 >= end || count == 0) return;
  const int page = p.pool.page;
  const int wrow = row0 + warp * PUT_WARP_ROWS;
  const int prow = wrow / page * page;                  // first row of this warp's page
  const bool touched = prow < end && prow + page > first;
  const int pid = touched ? p.page_table[(size_t)b * p.max_pages + wrow / page] : -1;
  const bool ok = touched && pid >= 0 && pid < p.pool.n_pages;
  if (touched && !ok && lane == 0) atomicOr(p.err, kErrLength);
  const size_t block = ok ? (size_t)layer * p.scale_layer + (size_t)pid * p.pool.n_kv + h : 0;
  uint8_t* codes = p.pool.codes[kv] + block * (size_t)page * D;
  float* scale = p.pool.scales[kv] + block;
  const bool has_old = APPEND && ok && prow < first;    // the page holds earlier rows
  const float old = has_old ? *scale : 0.f;

  float lo[IT][8], hi[IT][8];
  uint32_t m = 0;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int item = it * 32 + lane;
    const int r = wrow + item / CH, c = item % CH;
    if (!ok || r < first || r >= end) continue;
    const __nv_bfloat16* src;
    if (APPEND)
      src = p.fresh[kv] + (((size_t)b * p.t_len + (r - first)) * p.pool.n_kv + h) * D;
    else
      src = p.src[kv][b] + (((size_t)layer * p.pool.n_kv + h) * p.cap + r) * D;
    uint4 x = reinterpret_cast<const uint4*>(src)[c], y = reinterpret_cast<const uint4*>(src)[c + CH];
    if (APPEND && kv == 0) {
      float xf[8], yf[8];
      unpack8(x, xf);
      unpack8(y, yf);
      rotate8_df(x, y, p.tab + (size_t)(p.rope_row[b] + (r - first)) * (D / 2) + c * 8);
      finite_or_nan8(x, lo[it]);
      finite_or_nan8(y, hi[it]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(fabsf(xf[e]) < INFINITY && fabsf(yf[e]) < INFINITY)) lo[it][e] = hi[it][e] = __uint_as_float(0x7FFFFFFFu);
    } else {
      finite_or_nan8(x, lo[it]);
      finite_or_nan8(y, hi[it]);
    }
    m = max(m, max(max_finite8(lo[it]), max_finite8(hi[it])));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();
  if (!ok) return;
  const int per = page / PUT_WARP_ROWS;   // warps of a page
  const int w0 = warp / per * per;
  for (int w = 0; w < per; ++w) m = max(m, warp_max[w0 + w]);
  int e = scale_exponent(m);
  int e_old = e;
  if (has_old) {
    e_old = exponent_of_scale(old);
    e = max(e, e_old);
  }
  const float inv = pow2_float(-e);
  const float by = pow2_float(max(e_old - e, -100));
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int item = it * 32 + lane;
    const int r = wrow + item / CH, c = item % CH;
    uint2* dst = reinterpret_cast<uint2*>(codes + (size_t)(r - prow) * D);
    if (r >= first && r < end) {
      dst[c] = codes8(lo[it], inv);
      dst[c + CH] = codes8(hi[it], inv);
    } else if (APPEND && r < first && e > e_old) {
      uint2 u = dst[c], v = dst[c + CH];
      dst[c] = make_uint2(rescale4(u.x, by), rescale4(u.y, by));
      dst[c + CH] = make_uint2(rescale4(v.x, by), rescale4(v.y, by));
    }
  }
  if (warp == w0 && lane == 0) *scale = pow2_float(e);
}

}  // namespace

cudaError_t launch_pages8_fill(const PutParams& p, int head_dim, int max_rows, cudaStream_t st) {
  const dim3 grid((max_rows + PUT_ROWS - 1) / PUT_ROWS, p.batch * p.pool.n_kv, 2 * p.n_layers);
  if (head_dim == 128) put_kernel<128, false><<<grid, PUT_THREADS, 0, st>>>(p);
  else put_kernel<64, false><<<grid, PUT_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages8_append(const PutParams& p, int head_dim, cudaStream_t st) {
  // rows [n, n + t_len) meet at most this many groups of 128 rows
  const dim3 grid((p.t_len + 2 * PUT_ROWS - 2) / PUT_ROWS, p.batch * p.pool.n_kv, 2);
  if (head_dim == 128) put_kernel<128, true><<<grid, PUT_THREADS, 0, st>>>(p);
  else put_kernel<64, true><<<grid, PUT_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace c2kv
