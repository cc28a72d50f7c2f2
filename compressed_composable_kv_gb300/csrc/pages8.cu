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
    const uint4 x = reinterpret_cast<const uint4*>(src)[c], y = reinterpret_cast<const uint4*>(src)[c + CH];
    const CosSin2* t = APPEND && kv == 0 ? p.tab + (size_t)(p.rope_row[b] + (r - first)) * (D / 2) + c * 8 : nullptr;
    new_row8(x, y, t, lo[it], hi[it]);
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
