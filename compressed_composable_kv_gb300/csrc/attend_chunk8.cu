// Attention of a chunk of new tokens over the 8-bit paged cache:
//   s_j = (R q . K_j) / sqrt(d),  out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// over the rows j up to the token's own; K_j and V_j = code * scale of their page.
//
// A warp takes one token and query head at a time: 32 rows a step, a lane to a
// row for the scores, a lane to head_dim / 32 columns for the sum.
#include <algorithm>

#include "pages8.h"

namespace c2kv {

namespace {

constexpr int CH_THREADS = 256;

template <int D>
__global__ void __launch_bounds__(CH_THREADS) chunk_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int C = D / 32;
  __shared__ float sq[CH_THREADS / 32][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_wait();
  grid_release();
  const int n_kv = p.pool.n_kv, page = p.pool.page, group = p.n_q / n_kv;
  const int64_t items = (int64_t)p.batch * p.t_len * p.n_q;
  for (int64_t it = (int64_t)blockIdx.x * (CH_THREADS / 32) + warp; it < items; it += (int64_t)gridDim.x * (CH_THREADS / 32)) {
    const int hq = (int)(it % p.n_q), t = (int)(it / p.n_q % p.t_len), b = (int)(it / p.n_q / p.t_len);
    const int n = p.n_cached[b], count = p.n_new ? p.n_new[b] : p.t_len;
    if (n < 0 || (count >= 0 && count <= p.t_len && t >= count)) continue;
    const int64_t rr = (int64_t)p.rope_row[b] + (p.row_at_length ? n : 0);
    if (count < 0 || count > p.t_len || (int64_t)n + count > p.max_keys || rr < 0 || rr + count > p.table_rows) {
      if (lane == 0) atomicOr(p.err, kErrLength);
      continue;
    }
    const __nv_bfloat16* q = p.q + it * D;
    const CosSin2* tab = p.tab + (rr + t) * (D / 2);
    __syncwarp();
    for (int c = lane; c < D / 2; c += 32) {
      const float x = __bfloat162float(q[c]), y = __bfloat162float(q[c + D / 2]);
      const CosSin2 cs = tab[c];
      sq[warp][c] = (x * cs.ch - y * cs.sh) * p.scale_log2;
      sq[warp][c + D / 2] = (y * cs.ch + x * cs.sh) * p.scale_log2;
    }
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
    for (int j0 = 0; j0 <= n + t; j0 += 32) {
      const int j = j0 + lane;
      float s = -INFINITY, vs = 0.f;
      size_t row = 0;
      if (j <= n + t) {
        const int id = p.page_table[(size_t)b * p.max_pages + j / page];
        if (id >= 0 && id < p.pool.n_pages) {
          const size_t block = (size_t)id * n_kv + hq / group;
          row = block * page + j % page;
          vs = p.pool.scales[1][block];
          const uint4* k = reinterpret_cast<const uint4*>(p.pool.codes[0] + row * D);
          float dot = 0.f;
#pragma unroll 2
          for (int i = 0; i < D / 16; ++i) {
            const uint4 u = k[i];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 a = e4m3x2_to_float2(w[e] & 0xFFFFu), c = e4m3x2_to_float2(w[e] >> 16);
              const float* f = sq[warp] + 16 * i + 4 * e;
              dot = fmaf(f[0], a.x, fmaf(f[1], a.y, fmaf(f[2], c.x, fmaf(f[3], c.y, dot))));
            }
          }
          s = dot * p.pool.scales[0][block];
        } else if (lane == 0 || j % page == 0) {
          atomicOr(p.err, kErrLength);
        }
      }
      float top = s;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m - base), w = exp2f(s - base);
      m = mn;
      float sum = w;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l = fmaf(l, alpha, sum);
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] *= alpha;
      const bool seen = s != -INFINITY || vs != 0.f;
      for (int i = 0; i < 32; ++i) {
        if (!__shfl_sync(0xffffffffu, (int)seen, i)) continue;
        const float wi = __shfl_sync(0xffffffffu, w, i), si = __shfl_sync(0xffffffffu, vs, i);
        const uint8_t* v = p.pool.codes[1] + __shfl_sync(0xffffffffu, (unsigned long long)row, i) * D + lane * C;
#pragma unroll
        for (int c = 0; c < C; c += 2) {
          const float2 f = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(v + c));
          o[c] = fmaf(wi, f.x * si, o[c]);
          o[c + 1] = fmaf(wi, f.y * si, o[c + 1]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) p.out[it * D + lane * C + c] = __float2bfloat16_rn(l == 0.f ? 0.f : o[c] / l);
  }
}

}  // namespace

cudaError_t launch_attend_chunk8(const ChunkParams& p, int head_dim, int group, int sms, cudaStream_t st) {
  const int64_t items = (int64_t)p.batch * p.t_len * p.n_q;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(8 * sms, (items + CH_THREADS / 32 - 1) / (CH_THREADS / 32)));
  cfg.blockDim = dim3(CH_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return head_dim == 128 ? cudaLaunchKernelEx(&cfg, chunk_kernel<128>, p) : cudaLaunchKernelEx(&cfg, chunk_kernel<64>, p);
}

}  // namespace c2kv
