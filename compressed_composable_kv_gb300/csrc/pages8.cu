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
// A CTA owns 64 consecutive rows of one (sequence, kv head), of K or of V (128
// where a page is that long): a whole number of pages, so a page's largest
// magnitude never leaves the CTA.  A warp owns 16 rows and keeps them, as bf16,
// in registers between the two steps (largest magnitude, codes), so the data
// are read once, with all loads of a warp in flight.
//
// Fill is bound by the bytes moved: 32 layers of 8000 rows, 8 kv heads of 128
// (1.57 GB) 224 us, 7.0 TB/s (a plain copy: 6.8).  Append is bound by the
// rotation and by latency: the two halves of a pair must round as the exact
// values do, which costs a test for each and cos/sin in two parts, 1 KB of table
// for each token of each kv head (from L2).  1 x 4000 tokens 11.5 us (28 MB), 8
// ragged sequences of up to 128 7.5 us, 16 x 1 4.9 us, which is a launch and four
// dependent reads.
//
// In a chunk's call further CTAs of the append's launch rotate the queries (put_queries),
// bound by their bytes: 4000 tokens of 32 heads 65 MB, of 8 kv heads' rows 29 MB more.
#include "pages8.h"

namespace c2kv {

namespace {

constexpr int PUT_MAX_ROWS = 128;
constexpr int PUT_MIN_ROWS = 64;
constexpr int PUT_WARP_ROWS = 16;
constexpr int PUT_SLICES = 4;     // CTAs that share the queries of the same rows

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Bits (as fp32) of the larger half.
__device__ __forceinline__ uint32_t larger_half(uint32_t v) { return max(v & 0xFFFF0000u, v << 16); }

// The pair (x, y) rotated, in fp32; whether rounding these to bf16 gives what
// rounding the exact values does: rot_key_bits' test, with the bound |x| + |y|
// >= |x cos| + |y sin| that serves both, about half its work.
__device__ __forceinline__ bool turn_pair(float x, float y, float c, float s, float& a, float& b) {
  a = fmaf(x, c, -__fmul_rn(y, s));
  b = fmaf(y, c, __fmul_rn(x, s));
  const float m = fabsf(x) + fabsf(y), near = m * 0x1p-21f, small = m * 0x1p-11f;
  const float mid_a = __uint_as_float((__float_as_uint(a) & 0xFFFF0000u) | 0x8000u);
  const float mid_b = __uint_as_float((__float_as_uint(b) & 0xFFFF0000u) | 0x8000u);
  return fabsf(a - mid_a) > near && fabsf(b - mid_b) > near && fabsf(a) > small && fabsf(b) > small;
}

// The codes of the two values of a word.
__device__ __forceinline__ uint32_t codes2(uint32_t w, float inv) {
  return e4m3x2(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xFFFF0000u) * inv);
}

// A word's halves that are not finite become NaN and take no part in m.
__device__ __forceinline__ void tame(uint32_t& w, uint32_t& m) {
  const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  if (lo >= 0x7F80u) w |= 0x7FFFu;
  else m = max(m, lo << 16);
  if (hi >= 0x7F80u) w |= 0x7FFF0000u;
  else m = max(m, hi << 16);
}

// The queries of new tokens at rows wrow + slice, + PUT_SLICES, ... before wrow + 16 and
// `end` (the sequence's first new token is at row `first`), all heads of group h: rotated
// and scaled in fp32, then fp16 over a power of two that brings the largest element of a
// head to (224, 448].  A lane has two neighbouring pairs of a head's halves, a warp
// (at head_dim 64, half a warp) a head: loads and stores are whole lines, and a token's
// RoPE row is read once for the group (16 elements a lane, a head at a time, took 79 us
// for 4000 tokens of 32 heads, most of it for the table's lines in L1).
template <int D>
__device__ __noinline__ void put_queries(const PutParams& p, int b, int h, int slice, int first, int wrow, int end, int rr) {
  constexpr int LPR = D / 4, RPI = 32 / LPR;   // lanes of a row, rows at a time
  const int lane = threadIdx.x & 31, c = lane % LPR;
#pragma unroll 1
  for (int r0 = wrow + slice * RPI; r0 < min(end, wrow + PUT_WARP_ROWS); r0 += PUT_SLICES * RPI) {
    const int r = r0 + lane / LPR, t = r - first;
    const bool on = t >= 0 && r < end;
    const size_t at = (((size_t)b * p.t_len + (on ? t : 0)) * p.n_q + h * p.group) * D;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + at) + c;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.q16 + at) + c;
    float* scale = p.q_scale + ((size_t)b * p.pool.n_kv + h) * p.t_len * p.group + (size_t)(on ? t : 0) * p.group;
    float2 c0 = {}, c1 = {};   // cos, sin
    if (on) {
      const CosSin2* cs = p.tab + (size_t)(rr + t) * (D / 2) + 2 * c;
      c0 = make_float2(cs[0].ch, cs[0].sh);
      c1 = make_float2(cs[1].ch, cs[1].sh);
    }
#pragma unroll 1
    for (int g0 = 0; g0 < p.group; g0 += 4) {
      uint32_t u[4], v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool some = on && g0 + k < p.group;
        u[k] = some ? src[(g0 + k) * (D / 2)] : 0;
        v[k] = some ? src[(g0 + k) * (D / 2) + D / 4] : 0;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (g0 + k >= p.group) break;
        const float x0 = __uint_as_float(u[k] << 16), x1 = __uint_as_float(u[k] & 0xFFFF0000u);
        const float y0 = __uint_as_float(v[k] << 16), y1 = __uint_as_float(v[k] & 0xFFFF0000u);
        const float a0 = (x0 * c0.x - y0 * c0.y) * p.scale_log2, b0 = (y0 * c0.x + x0 * c0.y) * p.scale_log2;
        const float a1 = (x1 * c1.x - y1 * c1.y) * p.scale_log2, b1 = (y1 * c1.x + x1 * c1.y) * p.scale_log2;
        uint32_t top = max(max(__float_as_uint(a0) & 0x7FFFFFFFu, __float_as_uint(b0) & 0x7FFFFFFFu),
                           max(__float_as_uint(a1) & 0x7FFFFFFFu, __float_as_uint(b1) & 0x7FFFFFFFu));
        if (LPR == 32) {
          top = __reduce_max_sync(0xffffffffu, top);
        } else {
#pragma unroll
          for (int off = LPR / 2; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        }
        const int e = top < 0x7F800000u ? scale_exponent(top) : 0;   // a query that is not finite answers NaN
        const float inv = pow2_float(-e);
        if (on) {
          dst[(g0 + k) * (D / 2)] = f16x2(a0 * inv, a1 * inv);
          dst[(g0 + k) * (D / 2) + D / 4] = f16x2(b0 * inv, b1 * inv);
          if (c == 0) scale[g0 + k] = top < 0x7F800000u ? pow2_float(e) : __uint_as_float(0x7FFFFFFFu);
        }
      }
    }
  }
}

// D: head_dim.  APPEND: rows [n_cached, n_cached + new) from the new tokens,
// K rotated; else rows [0, n_rows) from the bf16 caches.
// CTAs per SM: append takes 11.5 us at 2 and 12.4 at 3 for 1 x 4000 tokens
// (registers for the rows in flight); fill is fastest at 3, and so is an append with
// queries (Q), most of whose CTAs have those: a chunk of 1 x 4000 203 us at 2, 195 at 3.
template <int D, bool APPEND, bool Q = false>
__global__ void __launch_bounds__(PUT_MAX_ROWS / PUT_WARP_ROWS * 32, APPEND && !Q ? 2 : 3) put_kernel(const __grid_constant__ PutParams p) {
  constexpr int CH = D / 16;              // items (16 elements) of a row
  constexpr int IT = D / 32;              // items of a lane
  __shared__ uint32_t warp_max[8];
  __shared__ uint64_t rope_bar[8];
  extern __shared__ __align__(128) CosSin2 rope_rows[];   // APPEND: 8 KB for each warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y / p.pool.n_kv, h = blockIdx.y % p.pool.n_kv;
  const int kv = blockIdx.z & 1, layer = blockIdx.z >> 1;   // an append has one layer, and its queries behind V
  const int rows = blockDim.x / 32 * PUT_WARP_ROWS;   // of a CTA
  grid_wait();
  grid_release();
  int first = 0, count, rr = 0;
  if (APPEND) {
    first = p.n_cached[b];
    count = p.n_new ? p.n_new[b] : p.t_len;
    const int64_t row = (int64_t)p.rope_row[b] + (p.row_at_length ? first : 0);
    if (first < 0) return;   // an empty place of the batch
    if (count < 0 || count > p.t_len || (int64_t)first + count > p.max_rows ||
        (count > 0 && (row < 0 || row + count > p.table_rows))) {
      if (threadIdx.x == 0) atomicOr(p.err, kErrLength);
      return;
    }
    rr = (int)row;
  } else {
    count = p.n_rows[b];
  }
  const int row0 = (first / rows + (int)blockIdx.x) * rows;   // of this CTA
  const int end = first + count;
  if (row0 >= end || count == 0) return;
  const int page = p.pool.page;
  const int wrow = row0 + warp * PUT_WARP_ROWS;
  if (Q && (int)blockIdx.z + p.z0 >= 2) {
    put_queries<D>(p, b, h, (int)blockIdx.z + p.z0 - 2, first, wrow, end, rr);
    return;
  }
  const int prow = wrow / page * page;                  // first row of this warp's page
  const bool touched = prow < end && prow + page > first;
  const int pid = touched ? p.page_table[(size_t)b * p.max_pages + wrow / page] : -1;
  bool ok = touched && pid >= 0 && pid < p.pool.n_pages;
  if (touched && !ok && lane == 0) atomicOr(p.err, kErrLength);
  const size_t block = ok ? (size_t)layer * p.scale_layer + (size_t)pid * p.pool.n_kv + h : 0;
  uint8_t* codes = p.pool.codes[kv] + block * (size_t)page * D;
  float* scale = p.pool.scales[kv] + block;
  const bool has_old = APPEND && ok && prow < first;    // the page holds earlier rows
  const float old = has_old ? *scale : 0.f;
  auto source = [&](int r) {
    return APPEND ? p.fresh[kv] + (((size_t)b * p.t_len + (r - first)) * p.pool.n_kv + h) * D
                  : p.src[kv][b] + (((size_t)layer * p.pool.n_kv + h) * p.cap + r) * D;
  };
  auto in = [&](int r) { return r >= first && r < end; };   // read whether or not its page is there yet
  // The values of the 16 rows, as bf16.  Rows to be rotated are held by pairs
  // of a head's halves, two to a lane (w[2i] and w[2i + 1]: of the lane's i-th
  // row), so that a warp reads a row of the RoPE table end to end; other rows
  // by 16 neighbouring elements to a lane (w[8i..]: of its i-th item).
  const bool turn = APPEND && kv == 0;
  constexpr int LPR = D / 4, RPI = 32 / LPR, NI = PUT_WARP_ROWS / RPI;   // lanes of a row, rows at a time, times
  uint32_t w[8 * IT];
  static_assert(8 * IT == 2 * NI, "both forms hold 16 rows");
#pragma unroll
  for (int i = 0; i < 8 * IT; ++i) w[i] = 0;
  if (turn) {
    const int pr = lane % LPR;   // the lane's pairs of the row: 2 pr, 2 pr + 1
    // The RoPE rows come by bulk copies, 8 KB at a time, the first while the
    // keys are read (the rows are most of what this path reads, and registers
    // would hold a few of them at a time, a wait for each few).
    constexpr int CROWS = 8192 / (D / 2 * 16);   // rows of a copy
    CosSin2* tab = rope_rows + warp * 512;
    bool late = false;   // a copy did not come in time
    auto copy = [&](int c0) {   // rows c0 .. c0 + CROWS of the warp's, those of them that are new
      const int lo = max(wrow + c0, first), hi = min(wrow + c0 + CROWS, end);
      if (late) return false;
      if (lane == 0 && lo < hi) {
        const uint32_t bytes = (uint32_t)(hi - lo) * (D / 2) * sizeof(CosSin2);
        mbar_arrive_expect_tx(&rope_bar[warp], bytes);
        bulk_g2s(tab + (lo - wrow - c0) * (D / 2), p.tab + (size_t)(rr + lo - first) * (D / 2), bytes, &rope_bar[warp]);
      }
      return lo < hi;
    };
    if (lane == 0) {
      mbar_init(&rope_bar[warp], 1);
      fence_barrier_init();
    }
    __syncwarp();
    bool coming = copy(0);
    int phase = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = wrow + i * RPI + lane / LPR;
      if (in(r)) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(source(r));
        w[2 * i] = src[pr];
        w[2 * i + 1] = src[D / 4 + pr];
      }
    }
    // Rows whose fp32 evaluation does not decide (a pair in 300 or so) are put
    // off to the end of their copy, where each lane takes its own: the exact
    // evaluation takes as long for one lane as for all.  Values that are not
    // finite never decide, and come out as NaN in both of the pair.
    constexpr int PER = CROWS / RPI;   // times of a copy
    static_assert(NI % PER == 0, "whole copies");
#pragma unroll
    for (int i0 = 0; i0 < NI; i0 += PER) {
      if (i0 > 0) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        coming = copy(i0 * RPI);
      }
      if (coming && !mbar_wait(&rope_bar[warp], phase & 1)) {
        atomicOr(p.err, kErrTimeout);
        ok = false;
        late = true;
        mbar_wait(&rope_bar[warp], phase & 1);   // let it land before the shared memory is released
      }
      if (coming) ++phase;
      late = __any_sync(0xffffffffu, late);
      const CosSin2* t = tab + lane / LPR * (D / 2) + 2 * pr;
      uint32_t open = 0;
#pragma unroll
      for (int i = i0; i < i0 + PER; ++i) {
        if (!in(wrow + i * RPI + lane / LPR)) continue;
        // every other four lanes read their two entries in the other order: eight
        // neighbours then read all banks once
        const bool odd = lane & 4;
        const CosSin2 ta = t[(i - i0) * RPI * (D / 2) + odd], tb = t[(i - i0) * RPI * (D / 2) + !odd];
        const float c0 = odd ? tb.ch : ta.ch, s0 = odd ? tb.sh : ta.sh, c1 = odd ? ta.ch : tb.ch, s1 = odd ? ta.sh : tb.sh;
        const float x0 = __uint_as_float(w[2 * i] << 16), x1 = __uint_as_float(w[2 * i] & 0xFFFF0000u);
        const float y0 = __uint_as_float(w[2 * i + 1] << 16), y1 = __uint_as_float(w[2 * i + 1] & 0xFFFF0000u);
        float a0, b0, a1, b1;
        const bool clear0 = turn_pair(x0, y0, c0, s0, a0, b0), clear1 = turn_pair(x1, y1, c1, s1, a1, b1);
        if (clear0 && clear1) {
          w[2 * i] = pack2(a0, a1);
          w[2 * i + 1] = pack2(b0, b1);
        } else {
          open |= 1u << (i - i0);
        }
      }
      while (__any_sync(0xffffffffu, open != 0)) {
        if (open == 0) continue;
        const int k = __ffs(open) - 1;
        open &= open - 1;
        uint32_t wx = 0, wy = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i == k) wx = w[2 * (i0 + i)], wy = w[2 * (i0 + i) + 1];
        const CosSin2 t0 = t[k * RPI * (D / 2)], t1 = t[k * RPI * (D / 2) + 1];
        const float x0 = __uint_as_float(wx << 16), x1 = __uint_as_float(wx & 0xFFFF0000u);
        const float y0 = __uint_as_float(wy << 16), y1 = __uint_as_float(wy & 0xFFFF0000u);
        wx = rot_key_slow(x0, t0.ch, t0.cl, -y0, t0.sh, t0.sl) | (rot_key_slow(x1, t1.ch, t1.cl, -y1, t1.sh, t1.sl) << 16);
        wy = rot_key_slow(y0, t0.ch, t0.cl, x0, t0.sh, t0.sl) | (rot_key_slow(y1, t1.ch, t1.cl, x1, t1.sh, t1.sl) << 16);
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i == k) w[2 * (i0 + i)] = wx, w[2 * (i0 + i) + 1] = wy;
      }
    }
  } else {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int item = it * 32 + lane;
      const int r = wrow + item / CH;
      if (in(r)) {
        const uint4* src = reinterpret_cast<const uint4*>(source(r)) + 2 * (item % CH);
        const uint4 x = __ldcs(src), y = __ldcs(src + 1);
        w[8 * it + 0] = x.x, w[8 * it + 1] = x.y, w[8 * it + 2] = x.z, w[8 * it + 3] = x.w;
        w[8 * it + 4] = y.x, w[8 * it + 5] = y.y, w[8 * it + 6] = y.z, w[8 * it + 7] = y.w;
      }
    }
  }
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 8 * IT; ++i) m2 = max_nan_bf16x2(m2, w[i] & 0x7FFF7FFFu);
  uint32_t m = larger_half(m2);
  if (__any_sync(0xffffffffu, m >= 0x7F800000u)) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8 * IT; ++i) tame(w[i], m);
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
  if (turn) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = wrow + i * RPI + lane / LPR;
      if (!in(r)) continue;
      uint16_t* dst = reinterpret_cast<uint16_t*>(codes + (size_t)(r - prow) * D) + lane % LPR;
      dst[0] = (uint16_t)codes2(w[2 * i], inv);
      dst[D / 4] = (uint16_t)codes2(w[2 * i + 1], inv);
    }
  } else {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int item = it * 32 + lane;
      const int r = wrow + item / CH;
      if (!in(r)) continue;
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = codes2(w[8 * it + 2 * k], inv) | (codes2(w[8 * it + 2 * k + 1], inv) << 16);
      reinterpret_cast<uint4*>(codes + (size_t)(r - prow) * D)[item % CH] = make_uint4(c[0], c[1], c[2], c[3]);
    }
  }
  if (APPEND && e > e_old) {   // a larger scale: the page's earlier codes follow
    const float by = pow2_float(max(e_old - e, -100));
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int item = it * 32 + lane;
      const int r = wrow + item / CH;
      uint4* dst = reinterpret_cast<uint4*>(codes + (size_t)(r - prow) * D) + item % CH;
      if (r < first) {
        const uint4 u = *dst;
        *dst = make_uint4(rescale4(u.x, by), rescale4(u.y, by), rescale4(u.z, by), rescale4(u.w, by));
      }
    }
  }
  if (warp == w0 && lane == 0) *scale = pow2_float(e);
}

template <int D, bool APPEND, bool Q = false>
cudaError_t launch_put(const PutParams& p, dim3 grid, int threads, cudaStream_t st) {
  static KernelSetup s;
  const int dev = setup_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (APPEND) {
    std::lock_guard<std::mutex> lk(s.mu);
    if (s.state[dev] == 0) {
      const cudaError_t e = cudaFuncSetAttribute(put_kernel<D, APPEND, Q>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 PUT_MAX_ROWS / PUT_WARP_ROWS * 8192);
      if (e != cudaSuccess) cudaGetLastError();
      s.state[dev] = e == cudaSuccess ? 1 : -(int)e;
    }
    if (s.state[dev] != 1) return (cudaError_t)(-s.state[dev]);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = APPEND ? threads / 32 * 8192 : 0;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, put_kernel<D, APPEND, Q>, p);
}

// Rows of a CTA for this page size.
int put_rows(const PutParams& p) { return p.pool.page > PUT_MIN_ROWS ? PUT_MAX_ROWS : PUT_MIN_ROWS; }

}  // namespace

cudaError_t launch_pages8_fill(const PutParams& p, int head_dim, int max_rows, cudaStream_t st) {
  const int rows = put_rows(p), threads = rows / PUT_WARP_ROWS * 32;
  const dim3 grid((max_rows + rows - 1) / rows, p.batch * p.pool.n_kv, 2 * p.n_layers);
  return head_dim == 128 ? launch_put<128, false>(p, grid, threads, st) : launch_put<64, false>(p, grid, threads, st);
}

cudaError_t launch_pages8_append(const PutParams& p, int head_dim, cudaStream_t st) {
  // rows [n, n + t_len) meet at most this many CTAs' rows
  const int rows = put_rows(p), threads = rows / PUT_WARP_ROWS * 32;
  const dim3 grid((p.t_len + 2 * rows - 2) / rows, p.batch * p.pool.n_kv, (p.q ? 2 + PUT_SLICES : 2) - p.z0);
  if (p.q)
    return head_dim == 128 ? launch_put<128, true, true>(p, grid, threads, st) : launch_put<64, true, true>(p, grid, threads, st);
  return head_dim == 128 ? launch_put<128, true>(p, grid, threads, st) : launch_put<64, true>(p, grid, threads, st);
}

}  // namespace c2kv
