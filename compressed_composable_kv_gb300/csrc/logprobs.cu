// Log probabilities of given tokens, entropy and the top alternatives of rows
// of logits x:
//   m = max x, S = sum exp(x - m), lp(t) = x_t - m - log S,
//   H = log S - sum exp(x - m) (x - m) / S      (a term with x = -inf is 0).
// One CTA per row; sums in 32 bits.  The top alternatives are found one after
// another: each is the largest (value, then lowest index) behind the last.
#include "pages8.h"

namespace c2kv {

namespace {

constexpr int LP_THREADS = 512;

__device__ __forceinline__ float logit_at(const LogprobParams& p, size_t i) {
  return p.is_f32 ? static_cast<const float*>(p.logits)[i]
                  : __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[i]);
}

// Orders of logits as whole numbers: larger logit first (NaN above all, -0 and
// +0 alike), then the lower index.
__device__ __forceinline__ uint64_t order_key(float x, int i) {
  uint32_t u = __float_as_uint(x);
  if (x != x) u = 0x7FFFFFFFu;
  if (u == 0x80000000u) u = 0;
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((uint64_t)u << 32) | (uint32_t)~i;
}

template <typename T, typename F>
__device__ T block_reduce(T v, T* buf, F f) {
  for (int off = 16; off >= 1; off >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, off));
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = buf[threadIdx.x & (LP_THREADS / 32 - 1)];
  for (int off = 8; off >= 1; off >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, off));
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(LP_THREADS) token_logprobs_kernel(const __grid_constant__ LogprobParams p) {
  __shared__ float fb[16];
  __shared__ uint64_t kb[16];
  const int row = blockIdx.x;
  const size_t base = (size_t)row * p.row_stride;
  float m = -INFINITY;
  bool nan = false;
  for (int i = threadIdx.x; i < p.vocab; i += LP_THREADS) {
    const float x = logit_at(p, base + i);
    nan |= x != x || x == INFINITY;
    m = fmaxf(m, x);
  }
  nan = __syncthreads_or(nan);
  m = block_reduce(m, fb, [](float a, float b) { return fmaxf(a, b); });
  float s = 0.f, t = 0.f;
  if (m != -INFINITY)
    for (int i = threadIdx.x; i < p.vocab; i += LP_THREADS) {
      const float y = logit_at(p, base + i) - m, e = expf(y);
      s += e;
      if (e > 0.f) t = fmaf(e, y, t);
    }
  s = block_reduce(s, fb, [](float a, float b) { return a + b; });
  t = block_reduce(t, fb, [](float a, float b) { return a + b; });
  const float ls = logf(s);
  const bool none = m == -INFINITY;
  auto lp = [&](float x) { return nan ? NAN : none ? -INFINITY : (x - m) - ls; };
  if (threadIdx.x == 0) {
    if (p.logprob) {
      const int tok = p.tokens[row];
      if (tok >= p.vocab) atomicOr(p.err, kErrLength);
      p.logprob[row] = tok < 0 ? 0.f : tok >= p.vocab ? NAN : lp(logit_at(p, base + tok));
    }
    if (p.entropy) p.entropy[row] = nan ? NAN : none ? 0.f : ls - t / s;
  }
  uint64_t before = ~0ull;
  for (int k = 0; k < p.top_k; ++k) {
    uint64_t best = 0;
    for (int i = threadIdx.x; i < p.vocab; i += LP_THREADS) {
      const uint64_t key = order_key(logit_at(p, base + i), i);
      if (key < before && key > best) best = key;
    }
    before = block_reduce(best, kb, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
    if (threadIdx.x == 0) {
      const int i = (int)~(uint32_t)before;
      p.top_ids[(size_t)row * p.top_k + k] = i;
      p.top_logprobs[(size_t)row * p.top_k + k] = lp(logit_at(p, base + i));
    }
  }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams& p, cudaStream_t st) {
  token_logprobs_kernel<<<p.rows, LP_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace c2kv
