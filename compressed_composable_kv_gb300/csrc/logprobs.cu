// Log probabilities of given tokens, entropy and the top alternatives of rows
// of logits x:
//   m = max x, S = sum exp(x - m), lp(t) = x_t - m - log S,
//   H = log S - sum exp(x - m) (x - m) / S.
//
// One pass over the logits, which is what bounds it: a thread takes 128 bytes
// at a time, every load in flight, and sums against its own maximum, so nothing
// is waited for on the way; partial sums are brought to a common maximum when
// they meet, in a fixed order.  Few rows are split over thread-block clusters,
// whose CTAs store their partial results and lists into the first one's shared
// memory.
//
// Top alternatives: in the CTA's first 2048 vectors, the k-th largest of the
// maxima of its 64 groups of 4 threads is a bound that at least k logits reach.
// Vectors that reach it (later ones: that exceed it), a few for each 2048, are
// noted on the way; behind the stream their logits are listed and the list's
// ranks counted.  Where very many do (logits that rise along the row, a mask
// that leaves a late part of it) a second pass takes new bounds on its way, and
// where even these leave too many the k largest are found one after another.
// Logits are ordered as whole numbers,
// (value, lower index first), so that equal ones have one order.
//
// Measured (one call among others in a graph; 6.8 TB/s is a plain copy's rate):
// 256 x 50257 fp32 logits with a fifth masked, top 20: 17.6 us (2.9 TB/s), with
// no alternatives 13 us (4.0 TB/s), all but 50 masked 23 us, rising along the row
// 84 us; 256 x 128256 bf16, top 5: 19.7 us (3.3 TB/s); 4 x 128256: 5.3 us.  About
// 5 us of a call are launch, first loads and the join of a row's CTAs, 5 us more
// the bound and the lists: at these sizes every CTA runs at once, so no logits
// stream meanwhile.
#include "pages8.h"

namespace c2kv {

namespace {

// 512 threads took 1.2 us off 256 rows and added 1 us to 4 rows, steps of 4 vectors
// with the next ones loaded ahead added 4 us to 256 rows (on an earlier form).
constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_VECS = 8;                            // 16-byte loads of a thread
constexpr int LP_GROUPS = 64;
constexpr int LP_CAND = 1024;                         // list of a step; the cluster's lists: 16 * 64
constexpr int LP_HITS = 512;                          // vectors noted
constexpr int LP_MAX_CLUSTER = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFaint = -200.f;                      // exp of it is 0 in fp32

// Larger logit first (NaN above all, -0 and +0 alike).
__device__ __forceinline__ uint32_t order_bits(float x) {
  uint32_t u = __float_as_uint(x);
  if (x != x) return 0xFFFFFFFEu;   // a NaN too; with any index below ~0ull
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

__device__ __forceinline__ float ex2_ftz(float z) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(z));
  return r;
}
__device__ __forceinline__ float exp_faint(float y) { return ex2_ftz(y * kLog2e); }   // e^y for y >= kFaint

// Pairs of fp32 numbers in one register pair, as the packed instructions take them.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
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

// n <= 16 partial results as one, in a fixed order, in every lane of a warp.
__device__ __forceinline__ Part join16(const Part* from, int n, int lane) {
  const int i = lane & 15;
  Part q = {-INFINITY, 0.f, 0.f};
  if (i < n) q = from[i];
  float M = q.m;
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  q = at_max(q, M);
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) {
    q.s += __shfl_xor_sync(0xffffffffu, q.s, off);
    q.t += __shfl_xor_sync(0xffffffffu, q.t, off);
  }
  return q;
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
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float largest(const uint4& v) {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  static __device__ __forceinline__ float at(const uint4& v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ float largest(const uint4& v) {
    return max_nan(max_nan(at(v, 0), at(v, 1)), max_nan(at(v, 2), at(v, 3)));
  }
};

struct alignas(16) LpShared {
  uint64_t cand[LP_CAND];                      // a CTA's list
  uint64_t lists[LP_MAX_CLUSTER * kMaxTopK];   // in a row's first CTA: the cluster's top lists, k each
  uint64_t top[kMaxTopK];                      // the largest, in order; 0: none
  uint4 hit[LP_HITS];                          // vectors that reach the bound
  int hit_at[LP_HITS];                         // and where they are
  uint64_t red[LP_WARPS];
  Part part[LP_WARPS];
  Part all[LP_MAX_CLUSTER];                    // in a row's first CTA: the partial results of the cluster
  alignas(16) uint32_t group[LP_GROUPS];
  float bound;
  int count, n_hits;
};

// A CTA's part of a row: vectors [v0, v1) behind its first `head` logits and,
// in the row's first CTA, the `extra` logits before and behind the vectors.
template <typename T>
struct Piece {
  const T* x;
  const uint4* vec;
  int head, v0, v1, extra, vocab;

  __device__ __forceinline__ int extra_at(int i) const { return i < head ? i : vocab - extra + i; }
  __device__ __forceinline__ int index(int v, int e) const { return head + v * Vec<T>::N + e; }
};

// top[0..k) from n candidates (16-byte aligned), by counting how many are
// larger; four threads to a candidate.
__device__ __forceinline__ void rank_into(LpShared& sh, const uint64_t* cand, int n, int k) {
  for (int i0 = 0; i0 < n; i0 += LP_THREADS / 4) {
    const int i = i0 + (threadIdx.x >> 2);
    const uint64_t key = i < n ? cand[i] : ~0ull;
    int rank = 0;
    if (i0 + (int)(threadIdx.x >> 5) * 8 < n) {   // the same for a warp
#pragma unroll 2
      for (int j = 2 * (threadIdx.x & 3); j < n; j += 8) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(cand + j);
        rank += (o.x > key ? 1 : 0) + (j + 1 < n && o.y > key ? 1 : 0);
      }
      rank += __shfl_xor_sync(0xffffffffu, rank, 1);
      rank += __shfl_xor_sync(0xffffffffu, rank, 2);
      if (i < n && (threadIdx.x & 3) == 0 && rank < k) sh.top[rank] = key;
    }
  }
}

__device__ __forceinline__ uint64_t list_key(float x, int i) {
  return ((uint64_t)order_bits(x) << 32) | (uint32_t)~i;
}

// The same from all logits of the piece, one after another: the way out where
// too many reach every bound.
template <typename T>
__device__ __noinline__ void one_by_one(LpShared& sh, const Piece<T>& pc, int k) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t before = ~0ull;
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0;
    auto see = [&](int i) {
      const uint64_t key = list_key((float)pc.x[i], i);
      if (key < before && key > best) best = key;
    };
    for (int i = pc.index(pc.v0, 0) + threadIdx.x; i < pc.index(pc.v1, 0); i += LP_THREADS) see(i);
    if (threadIdx.x < pc.extra) see(pc.extra_at(threadIdx.x));
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

// A thread's LP_VECS vectors v, v + LP_THREADS, ... of the piece; -inf behind its end.
template <typename T>
__device__ __forceinline__ void load_vecs(const Piece<T>& pc, int v, uint4 (&d)[LP_VECS]) {
#pragma unroll
  for (int c = 0; c < LP_VECS; ++c) {
    const uint32_t none = Vec<T>::kNone;
    d[c] = v + c * LP_THREADS < pc.v1 ? __ldg(pc.vec + v + c * LP_THREADS) : make_uint4(none, none, none, none);
  }
}

// A value that at least k logits of the CTA's first vectors reach (all of them,
// if they are fewer): the k-th largest of the maxima of groups of 4 threads.
// vm: the thread's maxima, -inf where it has no vector.
__device__ __forceinline__ float group_bound(LpShared& sh, const float (&vm)[LP_VECS], int tid, int k) {
  float most = vm[0];
#pragma unroll
  for (int c = 1; c < LP_VECS; ++c) most = max_nan(most, vm[c]);
  uint32_t g = order_bits(most);
  g = max(g, __shfl_xor_sync(0xffffffffu, g, 1));
  g = max(g, __shfl_xor_sync(0xffffffffu, g, 2));
  if ((tid & 3) == 0) sh.group[tid >> 2] = g;
  __syncthreads();
  const int i = tid >> 2;   // four threads to a group
  const uint32_t v = sh.group[i];
  int r = 0;
#pragma unroll
  for (int j0 = 0; j0 < LP_GROUPS; j0 += 16) {
    const int j = j0 + (tid & 3) * 4;
    const uint4 o = *reinterpret_cast<const uint4*>(&sh.group[j]);
    r += (o.x > v || (o.x == v && j < i)) + (o.y > v || (o.y == v && j + 1 < i)) +
         (o.z > v || (o.z == v && j + 2 < i)) + (o.w > v || (o.w == v && j + 3 < i));
  }
  r += __shfl_xor_sync(0xffffffffu, r, 1);
  r += __shfl_xor_sync(0xffffffffu, r, 2);
  if ((tid & 3) == 0 && r == k - 1) sh.bound = from_order(v);
  __syncthreads();
  return sh.bound;
}

// A vector that reaches the bound; n_hits says if there was room for all.
__device__ __forceinline__ void note(LpShared& sh, const uint4& d, int v) {
  const int at = atomicAdd(&sh.n_hits, 1);
  if (at < LP_HITS) {
    sh.hit[at] = d;
    sh.hit_at[at] = v;
  }
}

// What the logits x that reach a bound (in the order of order_bits) exceed, as
// !(x <= it): the next value below the bound. A NaN bound (k groups hold one) is
// reached by NaN alone, which exceed +inf so; -inf by all, which exceed NaN so.
__device__ __forceinline__ float below(float bound) {
  if (bound != bound) return INFINITY;
  const uint32_t o = order_bits(bound) - 1;
  return from_order(o == 0x7FFFFFFFu ? o - 1 : o);   // below 0 comes no -0
}

// Notes a step's vectors that reach the step's bound.  Where many equal it (a
// mask's value, say, or NaN) the first k of these in order will do: each holds
// one logit at least that no later one precedes.
template <typename T>
__device__ __forceinline__ void note_step(LpShared& sh, const Piece<T>& pc, const uint4 (&d)[LP_VECS],
                                          const float (&vm)[LP_VECS], int vb, float bound, int k) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float least = below(bound);
  auto reaches = [&](int c) { return vb + c * LP_THREADS + tid < pc.v1 && !(vm[c] <= least); };
  auto above = [&](int c) { return reaches(c) && bound == bound && !(vm[c] <= bound); };
#pragma unroll
  for (int c = 0; c < LP_VECS; ++c)
    if (reaches(c)) note(sh, d[c], vb + c * LP_THREADS + tid);
  __syncthreads();
  const int noted = sh.n_hits;
  __syncthreads();   // every thread has read it before one that goes on notes the next step's
  if (noted <= LP_HITS) return;
#pragma unroll
  for (int c = 0; c < LP_VECS; ++c) {
    const uint32_t eq = __ballot_sync(0xffffffffu, reaches(c) && !above(c));
    if (lane == 0) sh.group[c * LP_WARPS + warp] = __popc(eq);
  }
  __syncthreads();
  if (tid == 0) sh.n_hits = 0;
  __syncthreads();
#pragma unroll
  for (int c = 0; c < LP_VECS; ++c) {
    const bool is = reaches(c) && !above(c);
    int place = __popc(__ballot_sync(0xffffffffu, is) & ((1u << lane) - 1u));
    for (int j = 0; j < c * LP_WARPS + warp; ++j) place += sh.group[j];
    if (above(c) || (is && place < k)) note(sh, d[c], vb + c * LP_THREADS + tid);
  }
}

// top[0..k) in a second pass that takes a bound of its own for every 2048
// vectors: where logits rise along the row, or a mask leaves a later part of
// it.  False where still too many reach it.
template <typename T>
__device__ __noinline__ bool step_by_step(LpShared& sh, const Piece<T>& pc, int k) {
  const int tid = threadIdx.x;
  constexpr int STEP = LP_VECS * LP_THREADS, N = Vec<T>::N;
  int have = 0;
  for (int vb = pc.v0; vb < pc.v1; vb += STEP) {
    const int w = max(pc.v0, min(vb, pc.v1 - STEP));   // a whole step, vectors before vb again
    uint4 d[LP_VECS];
    load_vecs(pc, w + tid, d);
    float vm[LP_VECS];
#pragma unroll
    for (int c = 0; c < LP_VECS; ++c) vm[c] = Vec<T>::largest(d[c]);
    __syncthreads();   // the list of the step before has been ranked
    if (tid == 0) {
      sh.n_hits = 0;
      sh.count = have;
    }
    if (tid < have) sh.cand[tid] = sh.top[tid];
    const float bound = group_bound(sh, vm, tid, k);
    const float least = below(bound);
    note_step(sh, pc, d, vm, w, bound, k);
    __syncthreads();
    if (sh.n_hits > LP_HITS) return false;
    if (tid < k) sh.top[tid] = 0;
    auto list = [&](float v, int i) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < LP_CAND) sh.cand[at] = list_key(v, i);
    };
    for (int i = tid; i < sh.n_hits * N; i += LP_THREADS) {
      const float v = (float)reinterpret_cast<const T*>(sh.hit)[i];
      if (sh.hit_at[i / N] >= vb && !(v <= least)) list(v, pc.index(sh.hit_at[i / N], i % N));
    }
    if (vb == pc.v0 && tid < pc.extra) list((float)pc.x[pc.extra_at(tid)], pc.extra_at(tid));
    __syncthreads();
    const int found = sh.count;
    if (found > LP_CAND) return false;
    rank_into(sh, sh.cand, found, k);
    have = min(k, found);
  }
  return true;
}

// The address of `p` of this CTA's shared memory in the cluster's first CTA.
__device__ __forceinline__ uint32_t in_first_cta(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
  return r;
}

template <typename T>
__global__ void __launch_bounds__(LP_THREADS, 4) token_logprobs_kernel(const __grid_constant__ LogprobParams p) {
  using V = Vec<T>;
  __shared__ LpShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = p.cluster, row = blockIdx.x / cs, rank = blockIdx.x % cs, k = p.top_k;
  // every CTA of a cluster runs before another stores into its shared memory
  if (cs > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  Piece<T> pc;
  pc.x = static_cast<const T*>(p.logits) + (int64_t)row * p.row_stride;
  pc.vocab = p.vocab;
  grid_wait();
  grid_release();
  pc.head = min(p.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(pc.x) & 15)) / sizeof(T)) % V::N);
  pc.vec = reinterpret_cast<const uint4*>(pc.x + pc.head);
  const int nvec = (p.vocab - pc.head) / V::N, share = (nvec + cs - 1) / cs;
  pc.v0 = min(nvec, rank * share);
  pc.v1 = min(nvec, pc.v0 + share);
  pc.extra = rank == 0 ? p.vocab - nvec * V::N : 0;

  if (tid < k) sh.top[tid] = 0;
  if (tid == 0) sh.count = sh.n_hits = 0;
  // the given token is asked for here, its logit behind the stream, both needed at the end
  int tok = -1;
  if (tid == 0 && rank == 0 && p.logprob) tok = p.tokens[row];

  Part mine = {-INFINITY, 0.f, 0.f};
  auto add = [&](Part q) {
    const float M = fmaxf(mine.m, q.m);
    const Part a = at_max(mine, M), b = at_max(q, M);
    mine = {M, a.s + b.s, a.t + b.t};
  };
  float bound = -INFINITY;
  for (int vb = pc.v0; vb < pc.v1; vb += LP_VECS * LP_THREADS) {
    uint4 d[LP_VECS];
    load_vecs(pc, vb + tid, d);
    float vm[LP_VECS];
    Part q = {-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < LP_VECS; ++c) {
      vm[c] = V::largest(d[c]);
      q.m = fmaxf(q.m, vm[c]);
    }
    if (k > 0) {
      if (vb == pc.v0) {
        bound = group_bound(sh, vm, tid, k);
        note_step(sh, pc, d, vm, vb, bound, k);
      } else {   // k logits at or above the bound lie before these: they have to be above it
#pragma unroll
        for (int c = 0; c < LP_VECS; ++c) {
          const int v = vb + c * LP_THREADS + tid;
          if (v < pc.v1 && bound == bound && !(vm[c] <= bound)) note(sh, d[c], v);
        }
      }
    }
    const float from = q.m == -INFINITY ? 0.f : q.m;
    // two logits at a time: the sums of the even and of the odd ones
    const uint64_t minus = pair(-from, -from), scale = pair(kLog2e, kLog2e);
    uint64_t s2 = 0, t2 = 0;
#pragma unroll
    for (int c = 0; c < LP_VECS; ++c) {
      if (vb + c * LP_THREADS >= pc.v1) break;   // the same for the whole CTA
#pragma unroll
      for (int e = 0; e < V::N; e += 2) {
        const float2 y = halves(add2(pair(V::at(d[c], e), V::at(d[c], e + 1)), minus));
        const uint64_t yc = pair(max_nan(y.x, kFaint), max_nan(y.y, kFaint));
        const float2 z = halves(mul2(yc, scale));
        const uint64_t w = pair(ex2_ftz(z.x), ex2_ftz(z.y));
        s2 = add2(s2, w);
        t2 = fma2(w, yc, t2);
      }
    }
    const float2 sh2 = halves(s2), th2 = halves(t2);
    q.s = sh2.x + sh2.y;
    q.t = th2.x + th2.y;
    add(q);
  }
  float xe = -INFINITY;
  if (tid < pc.extra) {
    xe = (float)pc.x[pc.extra_at(tid)];
    add({xe == xe ? xe : -INFINITY, xe == -INFINITY ? 0.f : xe - xe + 1.f, 0.f});   // NaN and +inf sum up to NaN
  }

  float xt = NAN;
  if (tok >= 0 && tok < p.vocab) xt = (float)pc.x[tok];

  // ---- the CTA's partial result: threads, then warps
  {
    float M = mine.m;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    Part w = at_max(mine, M);
    w.s = warp_sum_f32(w.s);
    w.t = warp_sum_f32(w.t);
    if (lane == 0) sh.part[warp] = w;
  }
  __syncthreads();
  if (warp == 0) {
    const Part all = join16(sh.part, LP_WARPS, lane);
    if (lane == 0) sh.all[0] = all;
  }
  if (k > 0) {
    const int n_hits = sh.n_hits;
    const float least = below(bound);
    auto list = [&](float v, int i) {
      if (v <= least) return;
      const int at = atomicAdd(&sh.count, 1);
      if (at < LP_CAND) sh.cand[at] = list_key(v, i);
    };
    if (n_hits <= LP_HITS) {
      for (int i = tid; i < n_hits * V::N; i += LP_THREADS)
        list((float)reinterpret_cast<const T*>(sh.hit)[i], pc.index(sh.hit_at[i / V::N], i % V::N));
      if (tid < pc.extra) list(xe, pc.extra_at(tid));
    }
    __syncthreads();
    const int found = sh.count, there = (pc.v1 - pc.v0) * V::N + pc.extra;
    if (n_hits <= LP_HITS && found <= LP_CAND && found >= min(k, there)) rank_into(sh, sh.cand, found, k);
    else if (!step_by_step(sh, pc, k)) one_by_one(sh, pc, k);
  }
  __syncthreads();

  if (cs > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank > 0) {
      if (tid < k)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_first_cta(&sh.lists[rank * k + tid])), "l"(sh.top[tid])
                     : "memory");
      if (tid == 0) {
        const uint32_t at = in_first_cta(&sh.all[rank]);
        const Part q = sh.all[0];
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(q.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(q.s) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 8), "f"(q.t) : "memory");
      }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
  }
  const Part all = join16(sh.all, cs, lane);   // in every warp
  if (cs > 1) {
    if (k > 0) {
      if (tid < k) sh.lists[tid] = sh.top[tid];
      if (tid == 0) sh.count = 0;
      __syncthreads();
      if (cs * k <= LP_THREADS / 4) {   // one round
        rank_into(sh, sh.lists, cs * k, k);
      } else {
        uint64_t least = 1;   // every list's last entry has k logits at or above it
        for (int r = 0; r < cs; ++r) least = max(least, sh.lists[r * k + k - 1]);
        for (int i = tid; i < cs * k; i += LP_THREADS)
          if (sh.lists[i] >= least) sh.cand[atomicAdd(&sh.count, 1)] = sh.lists[i];
        __syncthreads();
        rank_into(sh, sh.cand, sh.count, k);
      }
      __syncthreads();
    }
  }
  const float ls = logf(all.s);
  const bool none = all.m == -INFINITY && all.s == 0.f;   // nothing but -inf
  auto lp = [&](float v) { return none ? -INFINITY : (v - all.m) - ls; };
  if (tid == 0) {
    if (p.logprob) {
      if (tok >= p.vocab) atomicOr(p.err, kErrLength);
      p.logprob[row] = tok < 0 ? 0.f : tok >= p.vocab ? NAN : lp(xt);
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
  // Two CTAs for each SM where the rows are fewer, but at least two vectors for
  // each thread and at most 16 CTAs to a row (256 x 50257 fp32: 21.2 us with half
  // as many CTAs, 17.6 so, 21.2 with twice as many).
  const int64_t nvec = p.vocab / Vec<T>::N;
  int cs = 1;
  while (cs < LP_MAX_CLUSTER && (int64_t)p.rows * cs < 2 * sms && nvec >= (int64_t)cs * 4 * LP_THREADS) cs *= 2;
  p.cluster = cs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * cs));
  cfg.blockDim = dim3(LP_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, p);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams& p, int sms, cudaStream_t st) {
  return p.is_f32 ? launch_lp<float>(p, sms, st) : launch_lp<__nv_bfloat16>(p, sms, st);
}

}  // namespace c2kv