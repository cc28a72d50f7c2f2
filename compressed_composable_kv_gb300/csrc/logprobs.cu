// Log probabilities of given tokens, entropy and the top alternatives of rows
// of logits x:
//   m = max x, S = sum exp(x - m), lp(t) = x_t - m - log S,
//   H = log S - sum exp(x - m) (x - m) / S.
//
// One pass over the logits, which is what bounds it: a CTA takes 32 KB of a
// row at a time into registers (128 bytes a thread, every load in flight), and
// the CTAs of a row are a thread-block cluster whose partial (m, S, sum) and
// top lists meet in its first CTA through distributed shared memory.  A thread
// sums against its own maximum, so nothing is waited for before the sums;
// partial sums are brought to a common maximum when they meet, in a fixed
// order.
//
// Top alternatives: the CTA's 64 groups of 4 threads have 64 maxima; the k-th
// largest of them is a bound that at least k logits reach, and as a rule few
// more do.  Those go to a list, whose ranks are counted.  Where too many reach
// it (rows of equal logits, or all but a few ruled out) the k largest are found
// one after another instead.  Logits are ordered as whole numbers, (value,
// lower index first), so that equal ones have one order.
#include <cooperative_groups.h>

#include "pages8.h"

namespace cg = cooperative_groups;

namespace c2kv {

namespace {

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_VECS = 8;                            // 16-byte loads of a thread
constexpr int LP_SLICE = LP_VECS * LP_THREADS;        // vectors of a CTA's step
constexpr int LP_GROUPS = 64;
constexpr int LP_CAND = 1024;                         // list of a step; the cluster's lists: 16 * 64
constexpr int LP_MAX_CLUSTER = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFaint = -200.f;                      // exp of it is 0 in fp32

// Larger logit first (NaN above all, -0 and +0 alike).
__device__ __forceinline__ uint32_t order_bits(float x) {
  uint32_t u = __float_as_uint(x);
  if (x != x) return 0xFFFFFFFFu;
  if (u == 0x80000000u) u = 0;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_order(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float exp_faint(float y) {   // e^y for y >= kFaint
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y * kLog2e));
  return r;
}

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Partial result: s = sum e^(x - m), t = sum e^(x - m) (x - m).
struct Part {
  float m, s, t;
};

// p seen from the maximum M >= p.m.
__device__ __forceinline__ Part at_max(Part p, float M) {
  const float d = p.m == M ? 0.f : max_nan(p.m - M, kFaint);
  const float f = exp_faint(d);
  return {M, p.s * f, (p.t + p.s * d) * f};
}

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xFF80FF80u;   // -inf
  static __device__ __forceinline__ float at(const uint4& v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return __uint_as_float((e & 1) ? w & 0xFFFF0000u : w << 16);
  }
  static __device__ __forceinline__ void set(uint4& v, int e, __nv_bfloat16 x) {
    const uint32_t b = __bfloat16_as_ushort(x);
    uint32_t& w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    w = (e & 1) ? (w & 0xFFFFu) | (b << 16) : (w & 0xFFFF0000u) | b;
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  static __device__ __forceinline__ float at(const uint4& v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ void set(uint4& v, int e, float x) {
    (e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w) = __float_as_uint(x);
  }
};

struct LpShared {
  alignas(16) uint64_t cand[LP_CAND];
  uint64_t top[kMaxTopK];     // the CTA's list so far, largest first; 0: none
  uint64_t red[LP_WARPS];
  Part part[LP_WARPS];
  Part all;                   // the CTA's partial result
  uint32_t group[LP_GROUPS];
  uint32_t bound;
  int count;
};

// The k-th list entries of n candidates, by counting how many are larger.
__device__ __forceinline__ void rank_into(LpShared& sh, int n, int k) {
  for (int i = threadIdx.x; i < n; i += LP_THREADS) {
    const uint64_t key = sh.cand[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += sh.cand[j] > key ? 1 : 0;
    if (rank < k) sh.top[rank] = key;
  }
}

__device__ __forceinline__ uint64_t list_key(float x, int i) {
  return ((uint64_t)order_bits(x) << 32) | (uint32_t)~i;
}

// The same from logits [lo, hi) of the row and the list so far (cand[0..k)),
// one after another: the way out where too many logits reach the bound.
template <typename T>
__device__ __noinline__ void one_by_one(LpShared& sh, const T* x, int lo, int hi, int k) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t before = ~0ull;
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0;
    auto see = [&](uint64_t key) {
      if (key < before && key > best) best = key;
    };
    for (int i = lo + threadIdx.x; i < hi; i += LP_THREADS) see(list_key((float)x[i], i));
    if (threadIdx.x < k) see(sh.cand[threadIdx.x]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xffffffffu, best, off);
      best = o > best ? o : best;
    }
    if (lane == 0) sh.red[warp] = best;
    __syncthreads();
    best = 0;
    for (int w = 0; w < LP_WARPS; ++w) best = sh.red[w] > best ? sh.red[w] : best;
    if (threadIdx.x == 0) sh.top[r] = best;
    before = best;
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(LP_THREADS, 3) token_logprobs_kernel(const __grid_constant__ LogprobParams p) {
  using V = Vec<T>;
  __shared__ LpShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = p.cluster, row = blockIdx.x / cs, rank = blockIdx.x % cs, k = p.top_k;
  const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.row_stride;
  // The row as 16-byte vectors: the first and the last may reach beyond it.
  const int mis = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int end = mis + p.vocab, nvec = (end + V::N - 1) / V::N;
  const uint4* base = reinterpret_cast<const uint4*>(x - mis);
  const int share = (nvec + cs - 1) / cs;
  const int v0 = min(nvec, rank * share), v1 = min(nvec, v0 + share);
  Part mine = {-INFINITY, 0.f, 0.f};
  if (tid < k) sh.top[tid] = 0;
  if (tid == 0) sh.count = 0;

  for (int vb = v0; vb < v1; vb += LP_SLICE) {
    uint4 d[LP_VECS];
#pragma unroll
    for (int c = 0; c < LP_VECS; ++c) {
      const int v = vb + c * LP_THREADS + tid;
      if (v < v1 && v * V::N >= mis && v * V::N + V::N <= end) {
        d[c] = __ldcs(base + v);
      } else {
        d[c] = make_uint4(V::kNone, V::kNone, V::kNone, V::kNone);
        if (v < v1)
          for (int e = 0; e < V::N; ++e) {
            const int i = v * V::N + e;
            if (i >= mis && i < end) V::set(d[c], e, x[i - mis]);
          }
      }
    }
    Part q = {-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < LP_VECS; ++c)
#pragma unroll
      for (int e = 0; e < V::N; ++e) q.m = fmaxf(q.m, V::at(d[c], e));
    const float from = q.m == -INFINITY ? 0.f : q.m;
#pragma unroll
    for (int c = 0; c < LP_VECS; ++c)
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        const float y = max_nan(V::at(d[c], e) - from, kFaint);
        const float w = exp_faint(y);
        q.s += w;
        q.t = fmaf(w, y, q.t);
      }
    const float M = fmaxf(mine.m, q.m);
    const Part a = at_max(mine, M), b = at_max(q, M);
    mine = {M, a.s + b.s, a.t + b.t};
    if (k == 0) continue;

    // ---- top alternatives of this step and the list so far
    const uint32_t most = q.s == q.s ? order_bits(q.m) : 0xFFFFFFFFu;   // NaN or +inf: look
    uint32_t g = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    g = max(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if ((lane & 3) == 0) sh.group[tid >> 2] = g;
    __syncthreads();
    if (tid < LP_GROUPS) {
      const uint32_t v = sh.group[tid];
      int r = 0;
      for (int j = 0; j < LP_GROUPS; ++j) {
        const uint32_t o = sh.group[j];
        r += o > v || (o == v && j < tid) ? 1 : 0;
      }
      if (r == k - 1) sh.bound = v;
    }
    if (tid < k) sh.cand[tid] = sh.top[tid];
    __syncthreads();
    const uint32_t bound = sh.bound;
    if (most >= bound) {
#pragma unroll
      for (int c = 0; c < LP_VECS; ++c) {
        const int v = vb + c * LP_THREADS + tid;
#pragma unroll
        for (int e = 0; e < V::N; ++e) {
          const float xe = V::at(d[c], e);
          const int i = v * V::N + e;
          if (order_bits(xe) >= bound && v < v1 && i >= mis && i < end) {
            const int at = k + atomicAdd(&sh.count, 1);
            if (at < LP_CAND) sh.cand[at] = list_key(xe, i - mis);
          }
        }
      }
    }
    __syncthreads();
    const int found = sh.count;
    const int lo = max(vb * V::N, mis) - mis, hi = min(min(v1, vb + LP_SLICE) * V::N, end) - mis;
    __syncthreads();
    if (tid == 0) sh.count = 0;
    if (k + found <= LP_CAND && found >= min(k, hi - lo))
      rank_into(sh, k + found, k);
    else
      one_by_one<T>(sh, x, lo, hi, k);
    __syncthreads();
  }

  // ---- the CTA's partial result: threads, then warps, in order
  {
    float M = mine.m;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    mine = at_max(mine, M);
    mine.s = warp_sum_f32(mine.s);
    mine.t = warp_sum_f32(mine.t);
    if (lane == 0) sh.part[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      float m = -INFINITY;
      for (int w = 0; w < LP_WARPS; ++w) m = fmaxf(m, sh.part[w].m);
      Part all = {m, 0.f, 0.f};
      for (int w = 0; w < LP_WARPS; ++w) {
        const Part q = at_max(sh.part[w], m);
        all.s += q.s;
        all.t += q.t;
      }
      sh.all = all;
    }
    __syncthreads();
  }
  Part all = sh.all;
  if (cs > 1) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    if (rank == 0) {
      float m = -INFINITY;
      Part q[LP_MAX_CLUSTER];
#pragma unroll
      for (int r = 0; r < LP_MAX_CLUSTER; ++r) {
        q[r] = r < cs ? *cl.map_shared_rank(&sh.all, r) : Part{-INFINITY, 0.f, 0.f};
        m = fmaxf(m, q[r].m);
      }
      all = {m, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < LP_MAX_CLUSTER; ++r) {
        const Part o = at_max(q[r], m);
        all.s += o.s;
        all.t += o.t;
      }
      for (int i = tid; i < cs * k; i += LP_THREADS) sh.cand[i] = cl.map_shared_rank(sh.top, i / k)[i % k];
    }
    cl.sync();   // everything of the other CTAs has been read
    if (rank != 0) return;
    rank_into(sh, cs * k, k);
    __syncthreads();
  }
  const float ls = logf(all.s);
  const bool none = all.m == -INFINITY && all.s == 0.f;   // nothing but -inf
  auto lp = [&](float v) { return none ? -INFINITY : (v - all.m) - ls; };
  if (tid == 0) {
    if (p.logprob) {
      const int tok = p.tokens[row];
      if (tok >= p.vocab) atomicOr(p.err, kErrLength);
      p.logprob[row] = tok < 0 ? 0.f : tok >= p.vocab ? NAN : lp((float)x[tok]);
    }
    if (p.entropy) p.entropy[row] = none ? 0.f : ls - all.t / all.s;
  }
  if (tid < k) {
    const uint64_t key = sh.top[tid];
    p.top_ids[(size_t)row * k + tid] = (int)~(uint32_t)key;
    p.top_logprobs[(size_t)row * k + tid] = lp(from_order((uint32_t)(key >> 32)));
  }
}

template <typename T>
cudaError_t launch_lp(LogprobParams p, int sms, cudaStream_t st) {
  static KernelSetup s;
  const int dev = setup_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(s.mu);
    if (s.state[dev] == 0) {
      const cudaError_t e =
          cudaFuncSetAttribute(token_logprobs_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) cudaGetLastError();
      s.state[dev] = e == cudaSuccess ? 1 : -(int)e;
    }
    if (s.state[dev] != 1) return (cudaError_t)(-s.state[dev]);
  }
  // As many CTAs to a row as leave each one step of it, and where the rows are
  // few, up to 16 for the sake of latency, but at least 2 vectors a thread.
  const int64_t nvec = (p.vocab + Vec<T>::N - 1) / Vec<T>::N;
  int cs = 1;
  while (cs < LP_MAX_CLUSTER &&
         (nvec > (int64_t)cs * LP_SLICE || (p.rows * cs * 2 <= sms && nvec >= (int64_t)cs * 4 * LP_THREADS)))
    cs *= 2;
  while (cs > 1 && (int64_t)p.rows * cs > INT32_MAX) cs /= 2;
  p.cluster = cs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * cs));
  cfg.blockDim = dim3(LP_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, p);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams& p, int sms, cudaStream_t st) {
  return p.is_f32 ? launch_lp<float>(p, sms, st) : launch_lp<__nv_bfloat16>(p, sms, st);
}

}  // namespace c2kv
