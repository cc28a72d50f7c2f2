// One decode step over the 8-bit paged cache.
//
// s_j = (R q . K_j) / sqrt(d), out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// over the rows j of a sequence, K_j and V_j = code * scale of their page.
//
// CTA (split, kv head, sequence): its 8 warps take the split's rows in turn,
// one row at a time, the row's codes spread over the lanes, with a running
// maximum and sum per query head.  The splits' partial (m, l, O) meet in the
// last CTA of the (sequence, kv head) to finish.
#include "pages8.h"

namespace c2kv {

namespace {

constexpr int AT_THREADS = 256;
constexpr int AT_WARPS = AT_THREADS / 32;

template <int D, int G>
__global__ void __launch_bounds__(AT_THREADS) attend_pages8_kernel(const __grid_constant__ AttendPages8Params p) {
  constexpr int E = D / 32;   // elements of a row per lane (2 or 4)
  __shared__ float qs[G][D];
  __shared__ float sm[AT_WARPS][G], sl[AT_WARPS][G], so[AT_WARPS][G][D];
  __shared__ int last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int n = p.n_cached[b];
  if (n < 0) return;
  const int keys = n + p.has_new;
  const int rr = p.rope_row[b];
  if (keys > p.max_keys || rr < 0 || rr >= p.table_rows) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrLength);
    return;
  }
  const size_t head0 = (size_t)b * p.n_q + (size_t)h * G;
  for (int i = threadIdx.x; i < G * D / 2; i += AT_THREADS) {
    const int g = i / (D / 2), f = i % (D / 2);
    const CosSin2 t = p.tab[(size_t)rr * (D / 2) + f];
    const __nv_bfloat16* q = p.q + (head0 + g) * D;
    const float x = __bfloat162float(q[f]), y = __bfloat162float(q[f + D / 2]);
    qs[g][f] = (x * t.ch - y * t.sh) * p.scale_log2;
    qs[g][f + D / 2] = (y * t.ch + x * t.sh) * p.scale_log2;
  }
  __syncthreads();
  float m[G], l[G], o[G][E];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[g][e] = 0.f;
  }
  const int lo = split * p.split_keys, hi = min(keys, lo + p.split_keys);
  for (int j = lo + warp; j < hi; j += AT_WARPS) {
    const int pid = p.page_table[(size_t)b * p.max_pages + j / p.pool.page];
    if (pid < 0 || pid >= p.pool.n_pages) {
      if (lane == 0) atomicOr(p.err, kErrLength);
      continue;
    }
    const size_t block = (size_t)pid * p.pool.n_kv + h;
    const size_t at = (block * p.pool.page + j % p.pool.page) * D + lane * E;
    float kf[E], vf[E];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 a = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p.pool.codes[0] + at + e));
      const float2 c = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p.pool.codes[1] + at + e));
      kf[e] = a.x, kf[e + 1] = a.y;
      vf[e] = c.x, vf[e + 1] = c.y;
    }
    const float ks = p.pool.scales[0][block], vs = p.pool.scales[1][block];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(kf[e], qs[g][lane * E + e], s);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= ks;
      const float mn = fmaxf(m[g], s);
      const float a = m[g] == -INFINITY ? 0.f : exp2f(m[g] - mn), pr = exp2f(s - mn);
      m[g] = mn;
      l[g] = l[g] * a + pr;
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = fmaf(o[g][e], a, pr * vs * vf[e]);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (lane == 0) {
      sm[warp][g] = m[g];
      sl[warp][g] = l[g];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][g][lane * E + e] = o[g][e];
  }
  __syncthreads();
  const size_t unit = (size_t)b * p.pool.n_kv + h;
  for (int i = threadIdx.x; i < G * D; i += AT_THREADS) {
    const int g = i / D, d = i % D;
    float mx = -INFINITY, lt = 0.f, ot = 0.f;
    for (int w = 0; w < AT_WARPS; ++w) mx = fmaxf(mx, sm[w][g]);
    for (int w = 0; w < AT_WARPS; ++w) {
      const float a = sm[w][g] == -INFINITY ? 0.f : exp2f(sm[w][g] - mx);
      lt = fmaf(a, sl[w][g], lt);
      ot = fmaf(a, so[w][g][d], ot);
    }
    const size_t at = (unit * p.splits + split) * G + g;
    p.part_o[at * D + d] = ot;
    if (d == 0) {
      p.part_ml[at * 2] = mx;
      p.part_ml[at * 2 + 1] = lt;
    }
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int prev = atomicAdd(p.counters + unit, 1);
    last = prev == p.splits - 1;
    if (last) p.counters[unit] = 0;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  for (int i = threadIdx.x; i < G * D; i += AT_THREADS) {
    const int g = i / D, d = i % D;
    float mx = -INFINITY, lt = 0.f, ot = 0.f;
    const size_t at0 = unit * p.splits * G + g;
    for (int s = 0; s < p.splits; ++s) mx = fmaxf(mx, __ldcg(p.part_ml + (at0 + (size_t)s * G) * 2));
    for (int s = 0; s < p.splits; ++s) {
      const size_t at = at0 + (size_t)s * G;
      const float ms = __ldcg(p.part_ml + at * 2);
      const float a = ms == -INFINITY ? 0.f : exp2f(ms - mx);
      lt = fmaf(a, __ldcg(p.part_ml + at * 2 + 1), lt);
      ot = fmaf(a, __ldcg(p.part_o + at * D + d), ot);
    }
    p.out[(head0 + g) * D + d] = __float2bfloat16_rn(keys == 0 ? 0.f : ot / lt);
  }
}

template <int D>
void launch_g(const AttendPages8Params& p, int group, dim3 grid, cudaStream_t st) {
  switch (group) {
    case 1: attend_pages8_kernel<D, 1><<<grid, AT_THREADS, 0, st>>>(p); break;
    case 2: attend_pages8_kernel<D, 2><<<grid, AT_THREADS, 0, st>>>(p); break;
    case 4: attend_pages8_kernel<D, 4><<<grid, AT_THREADS, 0, st>>>(p); break;
    case 5: attend_pages8_kernel<D, 5><<<grid, AT_THREADS, 0, st>>>(p); break;
    case 8: attend_pages8_kernel<D, 8><<<grid, AT_THREADS, 0, st>>>(p); break;
  }
}

}  // namespace

cudaError_t launch_attend_pages8(const AttendPages8Params& p, int head_dim, int group, cudaStream_t st) {
  const dim3 grid(p.splits, p.pool.n_kv, p.batch);
  if (head_dim == 128) launch_g<128>(p, group, grid, st);
  else launch_g<64>(p, group, grid, st);
  return cudaGetLastError();
}

}  // namespace c2kv
