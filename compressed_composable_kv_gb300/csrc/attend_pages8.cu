// One decode step (one layer) over the 8-bit paged cache on the 5th-generation
// tensor cores, the append of each sequence's new token included.
//
//   s_j = (R q . K_j) / sqrt(d),  out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// over the rows j of a sequence; K_j and V_j = code * scale of their page.
//
// The step is bound by the bytes of the pages (one byte per key, kv head and
// element of K and of V), so the codes go from HBM to the tensor cores as they
// are: pages by TMA into shared memory, K and V as e4m3 operands of
// tcgen05.mma (kind::f8f6f4), and no thread touches them.  What is not e4m3 is
// split: the query, and the softmax weights, are sums of three e4m3 numbers,
//   x = x1 + 2^-4 x2 + 2^-9 x3,
// each part the rounding of what the parts before it leave (a part leaves at
// most 2^-4 of it), which holds the query to 2^-14.8 of its largest element
// and a weight to 2^-12 of itself and 2^-27 of the largest.  The parts are
// separate columns of the same product, which is nearly free: M = 128 rows of
// K against N = 16 to 48 columns.  The K scale multiplies the score, the V
// scale the weight, per key.
//
// A tile is 128 rows of 128 bytes of K and of V: 128 keys at head_dim 128, 256
// keys at head_dim 64, where a row holds two keys, the query takes one column
// with zeros in the upper half and one with zeros in the lower half, and each
// output lane reads the columns of its own half.  A page of 16 to 128 tokens
// is 1 to 16 KB of a tile and one TMA load.
//
// Work: two CTAs to an SM share the tiles of all (sequence, kv head) units, from
// the device-side lengths.  Where the CTAs suffice every unit is cut into parts
// of about one length, a CTA to a part, so that no CTA works on two units and
// holds up the loads of one while it ends the other; else (more units than
// CTAs, or lengths so mixed that the longest part would be 1.5 times an even
// share) the tiles are laid end to end and cut into one equal range per CTA.
// 8 x 8000 keys of 5 heads to a kv head: 32.2 us by parts, 34.6 us by ranges; 16
// sequences of 1 to 8 thousand keys 33.8 and 34.3; 4 x 32768 49.5 and 51.7; 1 x
// 8000 12.1 and 12.8; but 32 sequences of 200 to 6000 keys 54 and 43 (44 with the
// search that finds parts too long).  (A cluster to a unit, merged in shared
// memory, took 40, 34 and 68 us for the first three on an earlier form: its CTAs
// stream slower.)
// A unit that one CTA holds whole is written at once; else its CTAs write
// partial (m, l, O), and the one whose tiles complete the unit's counter merges
// them, in the order of the keys whoever it is.
//
// Measured (one call among others in a graph; 6.8 TB/s is a plain copy's rate):
//   4 x 32768 keys, 8 kv heads of 4 (269 MB)   50 us   5.4 TB/s
//   8 x 8000 keys, 8 kv heads of 5 (131 MB)    32 us   4.1 TB/s
//   16 ragged, 8 kv heads of 4 (142 MB)        34 us   4.2 TB/s
//   64 of up to 1560 keys, as these (105 MB)   32 us   3.3 TB/s
//   4 x 16384 keys, 8 heads of 64 (67 MB)      20 us   3.4 TB/s
//   1 x 8000 keys, 8 kv heads of 4 (16 MB)     12.1 us
//   16 sequences of up to 300 keys, 2 heads     7.9 us
// While tiles stream they come at 6.9 TB/s.  What is left is the latency of a
// call: 2.5 to 3.5 us for a launch that finds nothing to do, about 2 us to the
// first tile (page ids, the load itself), 1.5 us from the last tile to the
// CTA's partial, 2 us for arrival and merge, and at mixed lengths the wait for
// the longest part.
//
// Roles: warps 0-3 softmax and epilogue (thread t owns row t of a tile, then
// lane t of O^T), warp 4 K's pages and the scales, warp 5 MMA, warp 6 the
// rotated query of each unit, warp 7 V's pages and the last tile of a unit:
// the new token, and zeros in V's places behind it (they may hold any bits,
// NaN among them, and 0 * NaN would reach the sum).
#include <float.h>

#include <algorithm>

#include "pages8.h"
#include "tcgen05.h"

namespace c2kv {

namespace {

constexpr int AP_THREADS = 256;
constexpr int AP_SM_THREADS = 128;
constexpr int AP_PARTS = 3;
constexpr int AP_KV_BYTES = 128 * 128;          // K (or V) of one tile
constexpr int AP_STAGE = 2 * AP_KV_BYTES;
constexpr int AP_MAX_PPT = 16;                  // pages of a tile

// Tiles of a CTA below which fewer CTAs work: more partials cost the merge more
// than they save the stream (at 2, 3, 4: 1 x 8000 keys 12.5, 12.5, 12.1 us; 8000
// keys beside 15 x 100 13.0, 13.0, 13.4).
constexpr int kMinTiles = 4;
// What the end of a unit costs a CTA, in tiles (see PageCut): 64 sequences of up to
// 1560 keys take 42.9, 34.6, 32.2, 31.8, 31.9 us at 0 to 4.
constexpr int kUnitTiles = 3;
constexpr int kMergeRows = 64;   // partials of one round of a merge

// The tiles of a launch, from the device-side lengths (fewer than 2^31, which
// the host checks for max_keys).
struct PageMap {
  int32_t start[kMaxPagedSeqs + 1];   // first tile of each sequence; the last one is the total
  int32_t part[kMaxPagedSeqs + 1];    // split by unit: first CTA of each sequence; evenly: its first place
  int32_t keys[kMaxPagedSeqs];        // rows attended over; -1: left out
  int32_t rope[kMaxPagedSeqs];        // the sequence's row of the RoPE table
  int32_t most;                       // split by unit: tiles of a part at most; 0: split evenly
};

template <int D, int G>
struct ApCfg {
  static constexpr int KPR = 128 / D;                   // keys per row of a tile
  static constexpr int TILE_KEYS = 128 * KPR;
  static constexpr int TILE_LG = KPR == 1 ? 7 : 8;      // its log2
  static constexpr int HCOL = AP_PARTS * G;             // columns of one key of a row
  static constexpr int NCOL = KPR * HCOL;
  static constexpr int NPAD = (NCOL + 15) / 16 * 16;
  // Two CTAs to an SM hide each other's softmax (a tile's chain of steps takes
  // about 0.8 us, an SM's share of HBM brings one in 0.73 us); each has as many
  // stages as half an SM holds.
  static constexpr int STAGES = NPAD == 16 ? 3 : 2;
  // A tile's scales are read until its s_free, a stage of K may be filled again
  // from QK on: twice the slots.
  static constexpr int SCALES = 2 * STAGES;
  static constexpr int OP_BYTES = NPAD * 128;           // query or P^T operand [NPAD][128 bytes]
  static constexpr int RED = 12;                        // per warp: G maxima (or sums), the largest V scale
  static constexpr int OFF_Q = STAGES * AP_STAGE;       // two buffers each
  static constexpr int OFF_P = OFF_Q + 2 * OP_BYTES;
  static constexpr int OFF_MAP = OFF_P + 2 * OP_BYTES;
  static constexpr int OFF_RED = OFF_MAP + (int)((sizeof(PageMap) + 15) / 16 * 16);
  static constexpr int OFF_SC = OFF_RED + 2 * 4 * RED * 4;                  // [SCALES][2][AP_MAX_PPT] scales
  static constexpr int OFF_QS = OFF_SC + SCALES * 2 * AP_MAX_PPT * 4;       // [4][8] the query's scales: read
  // until s_free, two units behind q_free
  static constexpr int OFF_X = OFF_QS + 4 * 8 * 4;                          // KPR == 2: [G][128] output exchange
  static constexpr int OFF_BAR = OFF_X + (KPR == 2 ? G * 128 * 4 : 0);
  static constexpr int N_BAR = 6 * STAGES + 2 * 8 + 2;
  static constexpr int OFF_MISC = OFF_BAR + N_BAR * 8;
  static constexpr int SMEM = OFF_MISC + 64 + 1024;     // + slack for 1024-byte alignment
  static_assert(OP_BYTES % 1024 == 0, "swizzled operands need 1024-byte alignment");
  static_assert(SMEM <= 113 * 1024, "shared memory per CTA");
  static constexpr int TMEM_O = 2 * NPAD;               // two S^T buffers, then two O^T buffers
  static constexpr int TMEM_COLS = 4 * NPAD <= 64 ? 64 : 4 * NPAD <= 128 ? 128 : 256;
  static constexpr int LD = (HCOL + 3) / 4 * 4;         // columns loaded of one key
  static constexpr int MERGE = G > 4 ? 4 : 8;           // partials whose loads are in flight together
  static_assert(kMergeRows * G * 4 <= 2 * OP_BYTES, "the weights of a merge are kept in P^T's buffers");
};

// Instruction descriptor, kind::f8f6f4: e4m3 A and B, fp32 D, M = 128.
__host__ __device__ constexpr uint32_t idesc_e4m3_m128(int n, bool a_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// N consecutive TMEM columns (N a multiple of 4) of the thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, float* r) {
  if constexpr (N >= 16) {
    float t[16];
    tmem_ld_cols<16>(addr, t);
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = t[i];
    tmem_ld_n<N - 16>(addr + 16, r + 16);
  } else if constexpr (N >= 8) {
    float t[8];
    tmem_ld_cols<8>(addr, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = t[i];
    tmem_ld_n<N - 8>(addr + 8, r + 8);
  } else if constexpr (N >= 4) {
    float t[4];
    tmem_ld_cols<4>(addr, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = t[i];
  }
}

// Three e4m3 parts of two values: the codes of part k of a in the low byte of
// out[k], of b in the high byte.
__device__ __forceinline__ void split3(float a, float b, uint32_t (&out)[3]) {
  out[0] = e4m3x2(a, b);
  float2 f = e4m3x2_to_float2(out[0]);
  a = (a - f.x) * 16.f;
  b = (b - f.y) * 16.f;
  out[1] = e4m3x2(a, b);
  f = e4m3x2_to_float2(out[1]);
  out[2] = e4m3x2((a - f.x) * 32.f, (b - f.y) * 32.f);
}

// Bounded wait that gives up once another thread has aborted the CTA.  Waiting
// is kept out of line: the kernel's loops have to stay in the instruction cache.
__device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
  return wait_or_abort(bar, parity, abort_flag, err);
}
__device__ __forceinline__ bool ap_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
  return mbar_try_wait(bar, parity) || slow_wait(bar, parity, abort_flag, err);
}

// Barrier of the softmax warps (all of them reach it on every path, their
// waits being bounded); true if any thread brings `failed`.
__device__ __forceinline__ bool softmax_sync(bool failed) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(failed ? 1u : 0u)
      : "memory");
  return any != 0;
}

// Max over the warp; a NaN is passed over.
__device__ __forceinline__ float warp_max_f32(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

struct PageTile {
  int32_t b, h, t;   // sequence, kv head, tile of the unit
};

// The last sequence b < batch with from[b] <= x.
__device__ __forceinline__ int seq_of(const int32_t* from, int batch, int x) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (from[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ PageTile tile_at(const PageMap& m, int batch, int tile_lg, int x) {
  PageTile d;
  d.b = seq_of(m.start, batch, x);
  const uint32_t r = (uint32_t)(x - m.start[d.b]), tb = (uint32_t)((m.keys[d.b] - 1) >> tile_lg) + 1;
  d.h = (int)(r / tb);
  d.t = (int)(r % tb);
  return d;
}

// The part of one unit that the CTA owns: its tiles [j0, j0 + n), starting at
// tile t0 of unit (b, h).
struct PageSeg {
  int b, h, t0, j0, n;
};

// An even split: a unit's tiles take a place each and its end kUnitTiles more;
// CTA c owns the tiles in places [first(c), first(c + 1)).
struct PageCut {
  int base, rem, ctas;   // the first rem CTAs own base + 1 places, the others base

  __device__ __forceinline__ int first(int c) const { return c * base + min(c, rem); }
  __device__ __forceinline__ int of(int x) const {   // the CTA that owns place x
    const int big = rem * (base + 1);
    return x < big ? (int)((uint32_t)x / (uint32_t)(base + 1)) : rem + (int)((uint32_t)(x - big) / (uint32_t)base);
  }
};

template <int D, int G>
__global__ void __launch_bounds__(AP_THREADS, 2)
    attend_pages8_kernel(const __grid_constant__ AttendPages8Params p) {
  using C = ApCfg<D, G>;
  constexpr int KPR = C::KPR, CH = D / 16;   // CH: 8-element chunks of half a head, 16-byte chunks of a row
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sP = smem + C::OFF_P;
  PageMap& M = *reinterpret_cast<PageMap*>(smem + C::OFF_MAP);
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  float* sc = reinterpret_cast<float*>(smem + C::OFF_SC);
  float* qs = reinterpret_cast<float*>(smem + C::OFF_QS);
  float* xo = reinterpret_cast<float*>(smem + C::OFF_X);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* v_full = k_full + C::STAGES;
  uint64_t* fix_k = v_full + C::STAGES;    // a unit's last tile: the new key is in it
  uint64_t* fix_v = fix_k + C::STAGES;     // and the new value, and V's tail is zero
  uint64_t* k_empty = fix_v + C::STAGES;
  uint64_t* v_empty = k_empty + C::STAGES;
  uint64_t* s_full = v_empty + C::STAGES;
  uint64_t* s_free = s_full + 2;
  uint64_t* p_full = s_free + 2;
  uint64_t* p_free = p_full + 2;
  uint64_t* o_full = p_free + 2;
  uint64_t* o_free = o_full + 2;
  uint64_t* q_full = o_free + 2;
  uint64_t* q_free = q_full + 2;
  uint64_t* mma_done = q_free + 2;    // every MMA of the CTA has completed
  uint64_t* never = mma_done + 1;     // test hook: nothing arrives
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
  volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);
  volatile int* none_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 24);

  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  auto stage_k = [&](int s) { return smem + s * AP_STAGE; };
  auto stage_v = [&](int s) { return smem + s * AP_STAGE + AP_KV_BYTES; };

  if (warp == 0) {
    // The map, 32 sequences at a time.
    if (!p.early) grid_wait();
    int at = 0;
    bool bad = false, none = false;
    auto scan = [&](int v, int& sum) {   // exclusive prefix over the warp on top of sum, which takes the total
      int incl = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      const int before = sum + incl - v;
      sum += __shfl_sync(0xffffffffu, incl, 31);
      return before;
    };
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      int32_t n = -1, keys = -1;
      int64_t rr = 0;
      if (b < p.batch) {
        n = p.n_cached[b];
        rr = (int64_t)p.rope_row[b] + (p.row_at_length ? n : 0);
      }
      if (n >= 0) {
        if (n > p.max_keys - p.has_new || rr < 0 || rr >= p.table_rows) bad = true;
        else keys = n + p.has_new;
      }
      none |= keys == 0;
      M.keys[b] = keys;
      M.rope[b] = (int32_t)rr;   // of an empty or bad place: not used
      M.start[b] = scan((((keys - 1) >> C::TILE_LG) + 1) * p.pool.n_kv, at);
    }
    // Split by unit where there are CTAs enough: every unit in parts of at most
    // `most` tiles, so that no CTA works on two units and waits for the end of
    // one before it goes on.  `most` is the smallest that the CTAs suffice for;
    // where that is over 1.5 times an even share (units of very different
    // lengths), an even split it is.
    int most = 0;
    if (p.batch * p.pool.n_kv <= ctas && at > 0) {
      const int even = (at + ctas - 1) / ctas;
      for (int t = max(even, kMinTiles); most == 0 && t <= even + even / 2 + kMinTiles; t += 1 + t / 16) {
        int parts = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
          const int tb = b0 + lane < p.batch ? ((M.keys[b0 + lane] - 1) >> C::TILE_LG) + 1 : 0;
          parts += __reduce_add_sync(0xffffffffu, (tb + t - 1) / t);
        }
        if (parts * p.pool.n_kv <= ctas) most = t;
      }
      if (most > 0) {
        int sum = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
          const int tb = b0 + lane < p.batch ? ((M.keys[b0 + lane] - 1) >> C::TILE_LG) + 1 : 0;
          const int first = scan((tb + most - 1) / most * p.pool.n_kv, sum);
          M.part[b0 + lane] = first;
        }
        if (lane == 0) M.part[kMaxPagedSeqs] = sum;
      }
    }
    if (most == 0) {
      int sum = 0;
      for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int tb = b0 + lane < p.batch ? ((M.keys[b0 + lane] - 1) >> C::TILE_LG) + 1 : 0;
        const int first = scan(tb > 0 ? (tb + kUnitTiles) * p.pool.n_kv : 0, sum);
        M.part[b0 + lane] = first;
      }
      if (lane == 0) M.part[kMaxPagedSeqs] = sum;
    }
    bad = __any_sync(0xffffffffu, bad);
    none = __any_sync(0xffffffffu, none);
    if (lane == 0) {
      M.start[kMaxPagedSeqs] = at;
      M.most = most;
      *none_flag = none;
      if (bad && cta == 0) atomicOr(p.err, kErrLength);
    }
  } else if (warp == 4) {
    if (lane < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(&p.tm[lane]) : "memory");
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr((const void*)tmem_slot)),
                 "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 5) {
    if (lane == 0) {
      for (int s = 0; s < C::STAGES; ++s) {
        mbar_init(&k_full[s], 1);
        mbar_init(&v_full[s], 1);
        mbar_init(&fix_k[s], 1);
        mbar_init(&fix_v[s], 1);
        mbar_init(&k_empty[s], 1);
        mbar_init(&v_empty[s], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&s_free[i], 4);   // one arrival per softmax warp
        mbar_init(&p_full[i], 4);
        mbar_init(&p_free[i], 1);
        mbar_init(&o_full[i], 1);
        mbar_init(&o_free[i], 4);
        mbar_init(&q_full[i], 1);
        mbar_init(&q_free[i], 1);
      }
      mbar_init(mma_done, 1);
      mbar_init(never, 1);
      *abort_flag = 0;
      fence_barrier_init();
    }
  } else {
    // rows and halves of the operands that nothing writes stay zero
    for (int i = (warp >= 6 ? warp - 3 : warp - 1) * 32 + lane; i < 4 * C::OP_BYTES / 16; i += 160)
      reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto unit_tiles = [&](int b) { return ((M.keys[b] - 1) >> C::TILE_LG) + 1; };   // 0 for -1 and 0 keys
  const int total = M.start[kMaxPagedSeqs], most = M.most;
  PageCut cut;
  auto tile_from = [&](int place) {   // the first tile at this place or behind it
    if (place >= M.part[kMaxPagedSeqs]) return total;
    const int b = seq_of(M.part, p.batch, place), tb = unit_tiles(b);
    const uint32_t r = (uint32_t)(place - M.part[b]), h = r / (uint32_t)(tb + kUnitTiles);
    return M.start[b] + (int)h * tb + min((int)(r - h * (uint32_t)(tb + kUnitTiles)), tb);
  };
  int x0 = 0, x1 = 0;
  if (most > 0) {
    if (cta < M.part[kMaxPagedSeqs]) {
      const int b = seq_of(M.part, p.batch, cta), tb = unit_tiles(b), parts = (tb + most - 1) / most;
      const int r = cta - M.part[b], h = r / parts, i = r - h * parts;
      x0 = M.start[b] + h * tb + (int)((uint32_t)i * (uint32_t)tb / (uint32_t)parts);
      x1 = M.start[b] + h * tb + (int)((uint32_t)(i + 1) * (uint32_t)tb / (uint32_t)parts);
    }
  } else {
    const int places = M.part[kMaxPagedSeqs];
    cut.ctas = min(ctas, max(1, total / kMinTiles));
    cut.base = places / cut.ctas;
    cut.rem = places - cut.base * cut.ctas;
    x0 = tile_from(cut.first(cta));
    x1 = tile_from(cut.first(cta + 1));
  }
  const int ntiles = x1 - x0;
  if (*none_flag) {
    // sequences without a row: their output is zero (out need not be 16-byte aligned)
    grid_wait();
    for (int b = cta; b < p.batch; b += ctas)
      if (M.keys[b] == 0)
        for (int i = tid; i < p.n_q * D; i += AP_THREADS) p.out[(size_t)b * p.n_q * D + i] = __float2bfloat16_rn(0.f);
  }
  if (ntiles == 0) {   // uniform over the CTA
    grid_wait();
    if (warp == 4)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
    return;
  }
  auto seg_at = [&](int j) {
    const PageTile d = tile_at(M, p.batch, C::TILE_LG, x0 + j);
    PageSeg s;
    s.b = d.b;
    s.h = d.h;
    s.t0 = d.t;
    s.j0 = j;
    s.n = min(unit_tiles(d.b) - d.t, ntiles - j);
    return s;
  };
  const int page = p.pool.page;
  const int lg = 31 - __clz(page);            // log2 of the page
  const int prows = page / KPR;               // rows of 128 bytes of a page
  int issued = 0;                             // a loading warp's count of tiles requested

  // ---------------- the loads of K (kv 0, with the scales of both) or V (kv 1)
  // of every tile.  The pages of the CTA's tiles, laid end to end, are taken 32
  // at a time, one to a lane: while a batch is loaded, the scales of the next
  // and the ids of the one after are on their way (two dependent reads, about
  // a microsecond).  K and V have a warp each: a warp issues a TMA load in about
  // 140 cycles whatever its size, so one warp with 16-token pages (16 loads a
  // tile) was what bounded the kernel.  before(j) runs before tile j is asked for.
  auto load_tiles = [&](int kv, auto&& before) -> bool {
    const int lgp = C::TILE_LG - lg;                   // log2 of a tile's pages
    const int ppt = 1 << lgp, per = 32 >> lgp;         // pages of a tile, tiles of a batch
    uint64_t* full = kv == 0 ? k_full : v_full;
    uint64_t* empty = kv == 0 ? k_empty : v_empty;
    struct Ref {
      int32_t id, h;   // id: -1 no page here, -2 outside the pool
      float ks, vs;
    };
    auto ask = [&](int batch0) {
      Ref r;
      r.id = -1;
      r.h = 0;
      r.ks = r.vs = 0.f;
      const int j = batch0 + (lane >> lgp);
      if (j < ntiles) {
        const PageTile d = tile_at(M, p.batch, C::TILE_LG, x0 + j);
        const int pg = (d.t << lgp) + (lane & (ppt - 1));
        r.h = d.h;
        if (pg <= (M.keys[d.b] - 1) >> lg) {
          r.id = p.page_table[(size_t)d.b * p.max_pages + pg];
          if (r.id < 0) r.id = -2;
        }
      }
      return r;
    };
    auto ask_scales = [&](Ref& r) {
      if (r.id >= p.pool.n_pages) r.id = -2;
      if (r.id >= 0 && kv == 0) {
        const size_t block = (size_t)r.id * p.pool.n_kv + r.h;
        r.ks = p.pool.scales[0][block];
        r.vs = p.pool.scales[1][block];
      }
    };
    // The scales' reads go out ahead of the loads: they would wait behind the
    // megabytes that all CTAs ask for at once.
    Ref cur = ask(0), nxt = ask(per);
    ask_scales(cur);
    for (int j0 = 0; j0 < ntiles; j0 += per) {
      ask_scales(nxt);
      const Ref third = ask(j0 + 2 * per);
      if (kv == 0 && cur.id == -2) atomicOr(p.err, kErrLength);
      const int i = lane & (ppt - 1);
      auto request = [&](int j) {
        if ((lane >> lgp) != j - j0) return;
        // no page, or one outside the pool: a load from before the pool, which
        // TMA fills with zeros; its scale 0 masks the keys
        const int s = j % C::STAGES, y = cur.id >= 0 ? (cur.id * p.pool.n_kv + cur.h) * prows : -prows;
        tma_load_2d((kv == 0 ? stage_k(s) : stage_v(s)) + i * prows * 128, &p.tm[kv], 0, y, &full[s]);
      };
      auto settle = [&](int j) {   // its scales, and what its loads will bring
        if (kv == 0 && (lane >> lgp) == j - j0) {
          float* scs = sc + j % C::SCALES * 2 * AP_MAX_PPT;
          scs[i] = cur.ks;
          scs[AP_MAX_PPT + i] = cur.vs;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[j % C::STAGES], AP_KV_BYTES);
        ++issued;
      };
      int j = j0;
      const int end = min(ntiles, j0 + per);
      if (j0 == 0) {
        // the first stages are asked for before the first scales are waited for
        const int n0 = min(end, C::STAGES);
        for (int t = 0; t < n0; ++t) request(t);
        for (; j < n0; ++j) settle(j);
      }
      for (; j < end; ++j) {
        if (!before(j)) return false;
        if (j >= C::STAGES && !__all_sync(0xffffffffu, ap_wait(&empty[j % C::STAGES],
                                                               ((j - C::STAGES) / C::STAGES) & 1, abort_flag, p.err)))
          return false;
        request(j);
        settle(j);
      }
      cur = nxt;
      nxt = third;
    }
    return true;
  };

  if (warp == 4) {
    load_tiles(0, [](int) { return true; });
  } else if (warp == 5) {
    if (lane == 0) {
      // ---------------- MMA issuer
      constexpr uint32_t idesc_qk = idesc_e4m3_m128(C::NPAD, false);   // A = K (K-major), B = query (K-major)
      constexpr uint32_t idesc_pv = idesc_e4m3_m128(C::NPAD, true);    // A = V^T (MN-major), B = P^T (K-major)
      uint32_t fix_par = 0;   // phase of each stage's fix barriers
      auto issue_pv = [&](int i, bool last_tile) -> bool {
        const int pb = i & 1, s = i % C::STAGES;
        if (!ap_wait(&v_full[s], (i / C::STAGES) & 1, abort_flag, p.err)) return false;
        if (last_tile) {
          if (!ap_wait(&fix_v[s], (fix_par >> s) & 1, abort_flag, p.err)) return false;
          fix_par ^= 1u << s;
        }
        if (!ap_wait(&p_full[pb], (i >> 1) & 1, abort_flag, p.err)) return false;
        if (i >= 2 && !ap_wait(&o_free[pb], ((i - 2) >> 1) & 1, abort_flag, p.err)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)   // 32 rows of V at a time
          mma_e4m3(tmem + C::TMEM_O + pb * C::NPAD, sw128_desc(smem_addr(stage_v(s)) + kk * 4096, AP_KV_BYTES, 1024),
                   sw128_desc(smem_addr(sP + pb * C::OP_BYTES) + kk * 32, 16, 1024), idesc_pv, kk > 0 ? 1u : 0u);
        mma_commit(&v_empty[s]);
        mma_commit(&p_free[pb]);
        mma_commit(&o_full[pb]);
        return true;
      };
      bool ok = true, before = false;   // before: tile j - 1 is the last of its unit
      int j = 0;
      for (int seg = 0; ok && j < ntiles; ++seg) {
        const PageSeg sg = seg_at(j);
        const bool ends = sg.t0 + sg.n == unit_tiles(sg.b);
        for (int tt = 0; ok && tt < sg.n; ++tt, ++j) {
          const int s = j % C::STAGES;
          const bool last_tile = ends && tt == sg.n - 1;
          ok = ap_wait(&k_full[s], (j / C::STAGES) & 1, abort_flag, p.err);
          if (ok && tt == 0) ok = ap_wait(&q_full[seg & 1], (seg >> 1) & 1, abort_flag, p.err);
          if (ok && last_tile) ok = ap_wait(&fix_k[s], (fix_par >> s) & 1, abort_flag, p.err);
          if (ok && j >= 2) ok = ap_wait(&s_free[j & 1], ((j - 2) >> 1) & 1, abort_flag, p.err);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)   // 32 bytes of the rows at a time
            mma_e4m3(tmem + (j & 1) * C::NPAD, sw128_desc(smem_addr(stage_k(s)) + kk * 32, 16, 1024),
                     sw128_desc(smem_addr(sQ + (seg & 1) * C::OP_BYTES) + kk * 32, 16, 1024), idesc_qk,
                     kk > 0 ? 1u : 0u);
          mma_commit(&s_full[j & 1]);
          mma_commit(&k_empty[s]);
          if (tt == sg.n - 1) mma_commit(&q_free[seg & 1]);
          if (j >= 1) ok = issue_pv(j - 1, before);
          before = last_tile;
        }
      }
      if (ok) issue_pv(ntiles - 1, before);
      // every MMA issued above must complete before TMEM is released
      mma_commit(mma_done);
      mbar_wait(mma_done, 0);
    }
  } else if (warp == 6) {
    grid_wait();
    grid_release();
    // ---------------- the query of each unit: rotated, times log2(e)/sqrt(d),
    // over a power of two that brings its largest element into (224, 448], in
    // three parts.  Item (g, c): elements 8c.. and D/2 + 8c.. of head g.
    auto prep_q = [&](int i, const PageSeg& sg) -> bool {
      if (i >= 2 && !__all_sync(0xffffffffu, ap_wait(&q_free[i & 1], ((i - 2) >> 1) & 1, abort_flag, p.err)))
        return false;
      const CosSin2* trow = p.tab + (size_t)M.rope[sg.b] * (D / 2);
      uint8_t* qb = sQ + (i & 1) * C::OP_BYTES;
#pragma unroll
      for (int it = 0; it < (G * CH + 31) / 32; ++it) {
        const int item = it * 32 + lane;
        const int g = item / CH, c = item % CH;
        const bool on = g < G;
        float x[8], y[8];
        uint32_t m = 0;
        if (on) {
          const uint4* row = reinterpret_cast<const uint4*>(p.q + ((size_t)sg.b * p.n_q + sg.h * G + g) * D);
          unpack8(row[c], x);
          unpack8(row[c + CH], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const CosSin2 t = trow[c * 8 + e];
            const float a = (x[e] * t.ch - y[e] * t.sh) * p.scale_log2;
            y[e] = (y[e] * t.ch + x[e] * t.sh) * p.scale_log2;
            x[e] = a;
            m = max(m, max(__float_as_uint(x[e]) & 0x7FFFFFFFu, __float_as_uint(y[e]) & 0x7FFFFFFFu));
          }
        }
#pragma unroll
        for (int off = CH / 2; off >= 1; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        const int e = m < 0x7F800000u ? scale_exponent(m) : 0;   // a query that is not finite answers NaN
        const float inv = pow2_float(-e);
        if (on) {
          uint32_t cx[4][3], cy[4][3];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            split3(x[2 * k] * inv, x[2 * k + 1] * inv, cx[k]);
            split3(y[2 * k] * inv, y[2 * k + 1] * inv, cy[k]);
          }
#pragma unroll
          for (int par = 0; par < KPR; ++par)
#pragma unroll
            for (int k = 0; k < AP_PARTS; ++k) {
              const int r = par * C::HCOL + k * G + g;
              const int b0 = par * D + 8 * c, b1 = b0 + D / 2;   // bytes of the row
              *reinterpret_cast<uint2*>(qb + r * 128 + (((b0 >> 4) ^ (r & 7)) << 4) + (b0 & 8)) =
                  make_uint2(cx[0][k] | (cx[1][k] << 16), cx[2][k] | (cx[3][k] << 16));
              *reinterpret_cast<uint2*>(qb + r * 128 + (((b1 >> 4) ^ (r & 7)) << 4) + (b1 & 8)) =
                  make_uint2(cy[0][k] | (cy[1][k] << 16), cy[2][k] | (cy[3][k] << 16));
            }
          if (c == 0) qs[(i & 3) * 8 + g] = m < 0x7F800000u ? pow2_float(e) : __uint_as_float(0x7FFFFFFFu);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[i & 1]);
      return true;
    };
    bool ok = true;
    for (int i = 0, j = 0; ok && j < ntiles; ++i) {
      const PageSeg sg = seg_at(j);
      ok = prep_q(i, sg);
      j += sg.n;
    }
  } else if (warp == 7) {
    // ---------------- V's loads, and the last tile of a unit, tile j of the CTA.
    // A lane holds elements 2 lane, 2 lane + 1 of each half of the new key and of
    // the new value (at head_dim 64 the first 16 lanes do).
    const bool on = lane < D / 4;
    float fresh[2][4];    // [K, V][lower half, upper half] of the unit whose turn is next, as held
    uint32_t m[2];        // bits of their largest magnitudes, over the row
    int id = -1;          // and the row's page
    auto ask_row = [&](const PageSeg& sg) {
      id = p.page_table[(size_t)sg.b * p.max_pages + ((M.keys[sg.b] - 1) >> lg)];
      m[0] = m[1] = 0;
      if (!p.has_new) return;
      if (on) {
        const size_t at = ((size_t)sg.b * p.pool.n_kv + sg.h) * D;
        const uint32_t* ks = reinterpret_cast<const uint32_t*>(p.fresh[0] + at);
        const uint32_t* vs = reinterpret_cast<const uint32_t*>(p.fresh[1] + at);
        const uint32_t kx = ks[lane], ky = ks[D / 4 + lane], vx = vs[lane], vy = vs[D / 4 + lane];
        const CosSin2* t = p.tab + (size_t)M.rope[sg.b] * (D / 2) + 2 * lane;
        const CosSin2 t0 = t[0], t1 = t[1];
        const float x0 = __uint_as_float(kx << 16), x1 = __uint_as_float(kx & 0xFFFF0000u);
        const float y0 = __uint_as_float(ky << 16), y1 = __uint_as_float(ky & 0xFFFF0000u);
        // a pair with a member that is not finite comes out as NaN in both
        const uint32_t bits[2][4] = {{rot_key_bits(x0, t0.ch, t0.cl, -y0, t0.sh, t0.sl) << 16,
                                      rot_key_bits(x1, t1.ch, t1.cl, -y1, t1.sh, t1.sl) << 16,
                                      rot_key_bits(y0, t0.ch, t0.cl, x0, t0.sh, t0.sl) << 16,
                                      rot_key_bits(y1, t1.ch, t1.cl, x1, t1.sh, t1.sl) << 16},
                                     {vx << 16, vx & 0xFFFF0000u, vy << 16, vy & 0xFFFF0000u}};
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a = bits[kv][e] & 0x7FFFFFFFu;
            fresh[kv][e] = __uint_as_float(a < 0x7F800000u ? bits[kv][e] : 0x7FFFFFFFu);
            if (a < 0x7F800000u) m[kv] = max(m[kv], a);
          }
      }
      m[0] = __reduce_max_sync(0xffffffffu, m[0]);
      m[1] = __reduce_max_sync(0xffffffffu, m[1]);
    };
    auto fixup = [&](int j, const PageSeg& sg) -> bool {
      const int s = j % C::STAGES;
      const int n = M.keys[sg.b] - 1;                            // the last row
      const int at = n - (sg.t0 + (j - sg.j0)) * C::TILE_KEYS;   // its key in the tile
      const int pi = at >> lg, pl = n & (page - 1);              // its page of the tile, its place there
      const bool in = id >= 0 && id < p.pool.n_pages;
      // this warp has asked for V's part of the tile, so the stage's phases are
      // this tile's
      if (!__all_sync(0xffffffffu, ap_wait(&k_full[s], (j / C::STAGES) & 1, abort_flag, p.err))) return false;
      if (!__all_sync(0xffffffffu, ap_wait(&v_full[s], (j / C::STAGES) & 1, abort_flag, p.err))) return false;
      // byte `byte` of key `key` of the tile
      auto place = [&](uint8_t* tile, int key, int byte) {
        const int row = key / KPR, b = key % KPR * D + byte;
        return tile + row * 128 + (((b >> 4) ^ (row & 7)) << 4) + (b & 15);
      };
      const size_t block = in ? (size_t)id * p.pool.n_kv + sg.h : 0;
      int grow[2] = {0, 0};
      if (p.has_new && in) {   // uniform over the warp
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          float* scs = sc + (j % C::SCALES * 2 + kv) * AP_MAX_PPT + pi;
          int e = scale_exponent(m[kv]), e_old = e;
          if (pl > 0) {
            e_old = exponent_of_scale(*scs);
            e = max(e, e_old);
          }
          grow[kv] = e_old - e;
          __syncwarp();
          if (on) {
            const float inv = pow2_float(-e);
            const uint16_t a = (uint16_t)e4m3x2(fresh[kv][0] * inv, fresh[kv][1] * inv);
            const uint16_t b = (uint16_t)e4m3x2(fresh[kv][2] * inv, fresh[kv][3] * inv);
            uint8_t* tile = kv == 0 ? stage_k(s) : stage_v(s);
            *reinterpret_cast<uint16_t*>(place(tile, at, 2 * lane)) = a;
            *reinterpret_cast<uint16_t*>(place(tile, at, D / 2 + 2 * lane)) = b;
            uint8_t* dst = p.pool.codes[kv] + (block * page + pl) * D;
            *reinterpret_cast<uint16_t*>(dst + 2 * lane) = a;
            *reinterpret_cast<uint16_t*>(dst + D / 2 + 2 * lane) = b;
            if (lane == 0) {
              *scs = pow2_float(e);
              p.pool.scales[kv][block] = pow2_float(e);
            }
          }
        }
      }
      // a larger scale: the page's earlier codes follow (rare)
      auto rescale = [&](int k) {
        const float by = pow2_float(max(grow[k], -100));
        uint8_t* t = k == 0 ? stage_k(s) : stage_v(s);
#pragma unroll 1
        for (int i = lane; i < pl * CH; i += 32) {
          const int key = i / CH, byte = i % CH * 16;
          uint4* u = reinterpret_cast<uint4*>(place(t, at - pl + key, byte));
          const uint4 r = make_uint4(rescale4(u->x, by), rescale4(u->y, by), rescale4(u->z, by), rescale4(u->w, by));
          *u = r;
          *reinterpret_cast<uint4*>(p.pool.codes[k] + (block * page + key) * D + byte) = r;
        }
      };
      if (grow[0] < 0) rescale(0);
      // the other key of the last row of K would reach this one's score
      if (KPR == 2 && (pl & 1) == 0 && lane < CH)
        *reinterpret_cast<uint4*>(place(stage_k(s), at + 1, lane * 16)) = make_uint4(0, 0, 0, 0);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&fix_k[s]);
      if (grow[1] < 0) rescale(1);
      for (int i = lane; i < (page - 1 - pl) * CH; i += 32)
        *reinterpret_cast<uint4*>(place(stage_v(s), at + 1 + i / CH, i % CH * 16)) = make_uint4(0, 0, 0, 0);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&fix_v[s]);
      return true;
    };
    // Tile t's stage is free for tile t + STAGES once PV(t) has run, so nothing
    // waits for this warp while it completes tile t before it asks for V of tile
    // t + STAGES - 1.
    auto ends = [&](const PageSeg& sg) { return sg.t0 + sg.n == unit_tiles(sg.b); };
    PageSeg next = seg_at(0);
    bool ready = false, done = false;
    auto fix_to = [&](int t) -> bool {   // the units' last tiles up to tile t
      if (t < 0) return true;            // the first stages' loads come first
      if (!ready) {
        grid_wait();
        grid_release();
        if (ends(next)) ask_row(next);
        ready = true;
      }
      while (!done && next.j0 + next.n - 1 <= t) {
        if (ends(next) && !fixup(next.j0 + next.n - 1, next)) return false;
        done = next.j0 + next.n >= ntiles;
        if (!done) {
          next = seg_at(next.j0 + next.n);
          if (ends(next)) ask_row(next);
        }
      }
      return true;
    };
    if (load_tiles(1, [&](int j) { return fix_to(j - C::STAGES + 1); })) fix_to(ntiles - 1);
  } else {
    // ---------------- softmax and epilogue: thread tid owns row tid of each
    // tile (lane tid of S^T) and lane tid of O^T
    grid_wait();
    grid_release();
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t o_col = C::TMEM_O + (tid / D) * C::HCOL;   // the columns of this lane's half
    // A wait that runs out is noted by the thread that waited (`failed`; its
    // neighbours may have been in time), which goes on with what is there. The
    // next softmax_sync tells all four warps (`gave_up`, the same in each thread),
    // and that alone decides who leaves: a barrier or a tensor memory load that
    // some had left before would never end.
    bool failed = false, gave_up = false;
    int k_red = 0;      // uses of red, whose two halves take turns
    int arrived = -1;   // last segment whose tiles were added to its unit's counter
    // out[b][h * G + g] from the lanes' o[g] over l[g]
    auto write_out = [&](int b, int h, const float (&o)[G], const float (&l)[G]) {
      __nv_bfloat16* out = p.out + ((size_t)b * p.n_q + (size_t)h * G) * D;
      if constexpr (KPR == 1) {
#pragma unroll
        for (int g = 0; g < G; ++g) out[g * D + tid] = __float2bfloat16_rn(l[g] == 0.f ? 0.f : o[g] / l[g]);
      } else {
#pragma unroll
        for (int g = 0; g < G; ++g) xo[g * 128 + tid] = l[g] == 0.f ? 0.f : o[g] / l[g];
        gave_up = softmax_sync(failed);
        for (int i = tid; i < G * D; i += AP_SM_THREADS)
          out[i] = __float2bfloat16_rn(xo[i / D * 128 + i % D] + xo[i / D * 128 + D + i % D]);
        gave_up = softmax_sync(failed);
      }
    };
    uint32_t p_at[8];   // this thread's byte of row r of P^T, less 128 r, by r & 7
#pragma unroll
    for (int r = 0; r < 8; ++r) p_at[r] = smem_addr(sP) + (((tid >> 4) ^ r) << 4) + (tid & 15);
    auto put_p = [&](int buf, int r, uint32_t code) {
      asm volatile("st.shared.u8 [%0], %1;" ::"r"(p_at[r & 7] + buf * C::OP_BYTES + r * 128), "r"(code) : "memory");
    };
    int i = 0;
    PageSeg sg = seg_at(0);
    for (;; ++i) {
      const int nkeys = M.keys[sg.b];
      const bool whole = sg.t0 == 0 && sg.n == unit_tiles(sg.b);
      float m_ref[G], l_part[G], o_acc[G], a_prev[G];
      float v_prev = 0.f;   // V factor of the tile before
#pragma unroll
      for (int g = 0; g < G; ++g) {
        m_ref[g] = -INFINITY;
        l_part[g] = 0.f;
        o_acc[g] = 0.f;
        a_prev[g] = 0.f;
      }
      auto consume_o = [&](int jj) {
        failed |= !ap_wait(&o_full[jj & 1], (jj >> 1) & 1, abort_flag, p.err);
        __syncwarp();
        tc_fence_after();
        float ov[C::LD];
        tmem_ld_n<C::LD>(lane_base + o_col + (jj & 1) * C::NPAD, ov);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[jj & 1]);
#pragma unroll
        for (int g = 0; g < G; ++g)
          o_acc[g] = fmaf(o_acc[g], a_prev[g], fmaf(fmaf(ov[2 * G + g], 0x1p-5f, ov[G + g]), 0x1p-4f, ov[g]) * v_prev);
      };
      for (int tt = 0; tt < sg.n; ++tt) {
        const int j = sg.j0 + tt;
        const int sb = j & 1;
        const float* scs = sc + j % C::SCALES * 2 * AP_MAX_PPT;
        const int key0 = (sg.t0 + tt) * C::TILE_KEYS + tid * KPR;
        if (p.inject_timeout && (cta & 1) == 0 && j == 0) {
          failed = !mbar_wait(never, 0, kInjectWaitCycles);
          if (tid == 0) {
            *abort_flag = 1;
            atomicOr(p.err, kErrTimeout);
          }
        }
        failed |= !ap_wait(&s_full[sb], (j >> 1) & 1, abort_flag, p.err);
        __syncwarp();
        tc_fence_after();
        float s[KPR][G], vs[KPR];
        float vmax = 0.f;
#pragma unroll
        for (int par = 0; par < KPR; ++par) {
          float sv[C::LD];
          tmem_ld_n<C::LD>(lane_base + sb * C::NPAD + par * C::HCOL, sv);
          const int pg = (tid * KPR + par) >> lg;
          const float ks = scs[pg];
          vs[par] = scs[AP_MAX_PPT + pg];
          const bool valid = key0 + par < nkeys && ks > 0.f;
          if (!valid) vs[par] = 0.f;
          vmax = fmaxf(vmax, vs[par]);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float f = fmaf(fmaf(sv[2 * G + g], 0x1p-5f, sv[G + g]), 0x1p-4f, sv[g]);
            s[par][g] = valid ? f * (ks * qs[(i & 3) * 8 + g]) : -INFINITY;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[sb]);
        float* rb = red + (k_red++ & 1) * 4 * C::RED;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float t = s[0][g];
          if constexpr (KPR == 2) t = fmaxf(t, s[1][g]);
          t = warp_max_f32(t);
          if (lane == 0) rb[warp * C::RED + g] = t;
        }
        vmax = warp_max_f32(vmax);
        if (lane == 0) rb[warp * C::RED + 8] = vmax;
        if (gave_up = softmax_sync(failed)) break;
        vmax = fmaxf(fmaxf(rb[8], rb[C::RED + 8]), fmaxf(rb[2 * C::RED + 8], rb[3 * C::RED + 8]));
        float alpha[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float tmax =
              fmaxf(fmaxf(rb[g], rb[C::RED + g]), fmaxf(rb[2 * C::RED + g], rb[3 * C::RED + g]));
          const float mn = fmaxf(m_ref[g], tmax);
          // -inf: every key masked so far
          const float base = mn == -INFINITY ? 0.f : mn;
          alpha[g] = ex2_approx(m_ref[g] - base);
          m_ref[g] = mn;
          l_part[g] *= alpha[g];
#pragma unroll
          for (int par = 0; par < KPR; ++par) {
            s[par][g] = ex2_approx(s[par][g] - base);
            l_part[g] += s[par][g];
          }
        }
        // the test hook, in every other CTA: one warp gives up, where no barrier follows before the unit's end
        if (p.inject_timeout && (cta & 1) != 0 && tt == sg.n - 1 && warp == 2) {
          failed = true;
          *abort_flag = 1;
        }
        if (j >= 2) failed |= !ap_wait(&p_free[sb], ((j - 2) >> 1) & 1, abort_flag, p.err);
        // weights are written as 256 p (V scale / the tile's largest): at most 256
        const float v_inv = vmax > 0.f ? 1.f / vmax : 0.f;
#pragma unroll
        for (int par = 0; par < KPR; ++par) {
          const float w = vs[par] * v_inv * 256.f;
#pragma unroll
          for (int g = 0; g < G; g += 2) {
            constexpr int last = G - 1;
            uint32_t part[3];
            split3(s[par][g] * w, g < last ? s[par][g < last ? g + 1 : g] * w : 0.f, part);
#pragma unroll
            for (int k = 0; k < AP_PARTS; ++k) {
              const int r = par * C::HCOL + k * G + g;
              put_p(sb, r, part[k]);
              if (g < last) put_p(sb, r + 1, part[k] >> 8);
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb]);
        if (tt > 0) consume_o(j - 1);
        v_prev = vmax * 0x1p-8f;
#pragma unroll
        for (int g = 0; g < G; ++g) a_prev[g] = alpha[g];
      }
      if (gave_up) break;
      consume_o(sg.j0 + sg.n - 1);

      // ---------------- segment epilogue
      const int u = sg.b * p.pool.n_kv + sg.h;
      float L[G];
      float* rb = red + (k_red++ & 1) * 4 * C::RED;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float ls = warp_sum(l_part[g]);
        if (lane == 0) rb[warp * C::RED + g] = ls;
      }
      if (gave_up = softmax_sync(failed)) break;
#pragma unroll
      for (int g = 0; g < G; ++g) L[g] = (rb[g] + rb[C::RED + g]) + (rb[2 * C::RED + g] + rb[3 * C::RED + g]);
      if (whole) {
        write_out(sg.b, sg.h, o_acc, L);
      } else {
        const int slot = 2 * cta + (i == 0 ? 0 : 1);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          p.part_o[((size_t)slot * G + g) * 128 + tid] = o_acc[g];
          if (tid == g) {
            p.part_ml[((size_t)slot * G + g) * 2 + 0] = m_ref[g];
            p.part_ml[((size_t)slot * G + g) * 2 + 1] = L[g];
          }
        }
        // every partial store of the CTA is ordered before tid 0's arrival
        // (a release at GPU scope, cumulative over the barrier)
        if (gave_up = softmax_sync(failed)) break;
        if (tid == 0) {
          int prev;
          asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;"
                       : "=r"(prev)
                       : "l"(p.counters + u), "r"(sg.n)
                       : "memory");
          const bool last = prev + sg.n == unit_tiles(sg.b);
          if (last) p.counters[u] = 0;   // every CTA of the unit has arrived
          *last_flag = last ? 1 : 0;
        }
        arrived = i;
        if (gave_up = softmax_sync(failed)) break;
        if (*last_flag) {
          // ---- merge: the CTAs from the one with the unit's first tile to the
          // one with its last, in that order whoever merges; a CTA's slot is
          // 2c, or 2c + 1 if the unit is not where its range starts.  A round
          // takes kMergeRows of them: warp w turns the (m, l) of heads w, w + 4
          // into weights, then thread tid adds up its lane of O, with the
          // loads of C::MERGE partials in flight (the first of them since
          // before the weights).
          const int tb = unit_tiles(sg.b), uf = M.start[sg.b] + sg.h * tb;
          int cf, nctr, slot0;
          if (most > 0) {
            nctr = (tb + most - 1) / most;
            cf = M.part[sg.b] + sg.h * nctr;
            slot0 = 2 * cf;
          } else {
            const int place = M.part[sg.b] + sg.h * (tb + kUnitTiles);
            cf = cut.of(place);
            nctr = cut.of(place + tb - 1) - cf + 1;
            slot0 = 2 * cf + (tile_from(cut.first(cf)) < uf ? 1 : 0);
          }
          auto slot = [&](int k) { return k == 0 ? slot0 : 2 * (cf + k); };
          float* wts = reinterpret_cast<float*>(sP);   // [kMergeRows][G]; every PV that read P has completed
          float* tot = red;                            // [G] (scale of what is summed so far, sum of weights)
          float mx[(G + 3) / 4];                       // of heads warp, warp + 4
          float lt[G], ot[G];
#pragma unroll
          for (int g = 0; g < G; ++g) lt[g] = ot[g] = 0.f;
#pragma unroll
          for (int q = 0; q < (G + 3) / 4; ++q) mx[q] = -INFINITY;
          for (int k0 = 0; k0 < nctr; k0 += kMergeRows) {
            const int nk = min(kMergeRows, nctr - k0);
            float ov[C::MERGE][G];
            auto fetch = [&](int k) {
#pragma unroll
              for (int r = 0; r < C::MERGE; ++r)
#pragma unroll
                for (int g = 0; g < G; ++g)
                  ov[r][g] = k + r < nk ? __ldcg(&p.part_o[((size_t)slot(k0 + k + r) * G + g) * 128 + tid]) : 0.f;
            };
            fetch(0);
#pragma unroll
            for (int q = 0; q < (G + 3) / 4; ++q) {
              const int g = warp + 4 * q;
              if (g >= G) break;
              float2 a = make_float2(-INFINITY, 0.f), b = a;
              if (lane < nk) a = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (size_t)slot(k0 + lane) * G + g);
              if (lane + 32 < nk)
                b = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (size_t)slot(k0 + lane + 32) * G + g);
              const float cm = fmaxf(mx[q], warp_max_f32(fmaxf(a.x, b.x)));
              const float base = cm == -INFINITY ? 0.f : cm;
              const float wa = ex2_approx(a.x - base), wb = ex2_approx(b.x - base);
              const float sum = warp_sum(wa * a.y + wb * b.y);
              wts[lane * G + g] = wa;
              wts[(lane + 32) * G + g] = wb;
              if (lane == 0) {
                tot[2 * g] = ex2_approx(mx[q] - base);
                tot[2 * g + 1] = sum;
              }
              mx[q] = cm;
            }
            softmax_sync(false);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              lt[g] = fmaf(lt[g], tot[2 * g], tot[2 * g + 1]);
              ot[g] *= tot[2 * g];
            }
            for (int k = 0; k < nk; k += C::MERGE) {
              if (k > 0) fetch(k);
#pragma unroll
              for (int r = 0; r < C::MERGE; ++r)
#pragma unroll
                for (int g = 0; g < G; ++g) ot[g] = fmaf(wts[(k + r) * G + g], ov[r][g], ot[g]);
            }
            softmax_sync(false);   // wts and tot are free again
          }
          write_out(sg.b, sg.h, ot, lt);
        }
      }
      if (gave_up) break;
      if (sg.j0 + sg.n >= ntiles) break;
      sg = seg_at(sg.j0 + sg.n);
    }
    if (gave_up && tid == 0) {
      // The CTA gave up: still add the tiles of its remaining shared units to
      // their counters (their outputs are undefined), so that every counter is
      // back at zero when the launch ends.
      PageSeg q = seg_at(0);
      for (int k = 0;; ++k) {
        if (k > arrived && !(q.t0 == 0 && q.n == unit_tiles(q.b))) {
          const int prev = atomicAdd(p.counters + q.b * p.pool.n_kv + q.h, q.n);
          if (prev + q.n == unit_tiles(q.b)) p.counters[q.b * p.pool.n_kv + q.h] = 0;
        }
        if (q.j0 + q.n >= ntiles) break;
        q = seg_at(q.j0 + q.n);
      }
    }
  }

  // ---------------- teardown
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && (warp == 4 || warp == 7) && lane == 0) {
    // let the copies in flight land before the shared memory is released
    uint64_t* full = warp == 4 ? k_full : v_full;
    for (int j = max(0, issued - C::STAGES); j < issued; ++j) mbar_wait(&full[j % C::STAGES], (j / C::STAGES) & 1);
  }
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
  }
}

template <int D, int G>
cudaError_t launch_ap(const AttendPages8Params& p, int sms, cudaStream_t st) {
  using C = ApCfg<D, G>;
  static KernelSetup s;
  const int dev = setup_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(s.mu);
    if (s.state[dev] == 0) {
      const cudaError_t e =
          cudaFuncSetAttribute(attend_pages8_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
      if (e != cudaSuccess) cudaGetLastError();
      s.state[dev] = e == cudaSuccess ? 1 : -(int)e;
    }
    if (s.state[dev] != 1) return (cudaError_t)(-s.state[dev]);
  }
  // Two CTAs to an SM, but no more than the longest sequences could use (1 x 8000
  // keys: 12.1 us with 128 CTAs, 12.5 with 304; 16 of up to 300: 7.9 and 8.5).
  const int64_t parts = ((p.max_keys - 1) / C::TILE_KEYS + kMinTiles) / kMinTiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(2 * sms, parts * p.batch * p.pool.n_kv));
  cfg.blockDim = dim3(AP_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_pages8_kernel<D, G>, p);
}

template <int D>
cudaError_t launch_group(const AttendPages8Params& p, int group, int sms, cudaStream_t st) {
  switch (group) {
    case 1: return launch_ap<D, 1>(p, sms, st);
    case 2: return launch_ap<D, 2>(p, sms, st);
    case 4: return launch_ap<D, 4>(p, sms, st);
    case 5: return launch_ap<D, 5>(p, sms, st);
    case 8: return launch_ap<D, 8>(p, sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_attend_pages8(const AttendPages8Params& p, int head_dim, int group, int sms, cudaStream_t st) {
  return head_dim == 128 ? launch_group<128>(p, group, sms, st) : launch_group<64>(p, group, sms, st);
}

}  // namespace c2kv
