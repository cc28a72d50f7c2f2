// Attention of a chunk of new tokens over the 8-bit paged cache (one layer) on
// the 5th-generation tensor cores:
//   s_j = (R q . K_j) / sqrt(d),  out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// over the rows j up to the token's own; K_j and V_j = code * scale of their page.
//
// A unit is 256 (token, query head) rows of one (sequence, kv head), token-major,
// against the key tiles (128 rows) that they see.  Every e4m3 code is an fp16
// number, so a tile's codes are brought to fp16 once for all 256 rows, and both
// products run as kind::f16 (fp32 accumulators): the keys and values lose
// nothing; a query row is held in fp16 times a power of two of its own, 2^-11 of
// each element, and so is a weight (2^7 exp(s - m), so that weights down to 2^-21
// of the largest keep their 11 bits), which is well below what the bf16 output
// itself rounds away.  Pages of one tile with different scales meet at the largest
// of them by an exact multiplication in fp16; the tile's K scale multiplies the
// scores, its V scale, over the largest so far, the weights.
//
// The places of all units (their tiles, and kUnitTiles for the end of each) are
// laid end to end, from the device-side lengths, and cut into one even range per
// CTA (one to an SM).  A unit that one CTA holds whole is written at once; else its
// CTAs write partial (m, l, O) and merge_kernel joins them in the order of the keys.
//
// Roles: warps 0-3 and 4-7 softmax and epilogue of the unit's two 128-row tiles
// (a thread to a row), warps 8-11 codes to fp16, warp 12 page ids and scales ahead
// of them, warp 13 the MMAs, warp 14 tensor memory.
#include <float.h>

#include <algorithm>

#include "pages8.h"
#include "tcgen05.h"

namespace c2kv {

namespace {

constexpr int CK_THREADS = 512;
constexpr int CK_ROWS = 256;       // rows of a unit
constexpr int CK_KEYS = 128;       // keys of a tile
constexpr int kSlots = 8;          // tiles whose pages are known ahead
constexpr int kChunkMinTiles = 2;  // tiles of a CTA below which fewer CTAs work
constexpr int kChunkUnitTiles = 2; // what a unit's begin and end cost, in tiles
constexpr int kNoScale = -1000;    // exponent of a tile without a page
constexpr float kRescaleLog2 = 8.f;   // a row's maximum may lag behind by this (weights up to 2^15, sums exact)
constexpr float kWeightLog2 = 7.f;

// What warp 12 finds out about a tile.
struct TileSlot {
  int32_t grp[8];      // 16 rows each: index of the first of them in the layer, in 16s; -1: no page
  uint32_t kf[8];      // half2: the page's scale over the tile's, of K and of V
  uint32_t vf[8];
  float k_scale;       // the tile's
  int32_t v_exp;
  uint32_t bad;        // bit g: the rows of grp[g] take no part
  int32_t rows;        // keys of the tile that any row of the unit sees
  int32_t diag;        // keys below this are seen by every row
  int32_t seg;
  uint32_t flags;      // 1: kf are not all 1, 2: vf, 4: the CTA's last tile
  int32_t pad;
};

struct ChunkMap {
  int32_t start[kMaxPagedSeqs + 1];   // first place of each sequence; the last one is the total
  int32_t per[kMaxPagedSeqs];         // places of one kv head of it
  int32_t n[kMaxPagedSeqs];           // rows held before the chunk
  int32_t count[kMaxPagedSeqs];       // new tokens
  int32_t rope[kMaxPagedSeqs];
  int32_t tiles;                      // of the launch
};

template <int D>
struct CkCfg {
  static constexpr int TILE = 128 * D * 2;             // a query, K or V tile in fp16
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = 4 * TILE;
  static constexpr int OFF_SLOT = 6 * TILE;
  static constexpr int OFF_MAP = OFF_SLOT + kSlots * (int)sizeof(TileSlot);
  static constexpr int OFF_BAR = OFF_MAP + (int)((sizeof(ChunkMap) + 15) / 16 * 16);
  static constexpr int N_BAR = 2 * 8 + 2 * kSlots + 2;
  static constexpr int OFF_MISC = OFF_BAR + N_BAR * 8;
  static constexpr int SMEM = OFF_MISC + 64 + 1024;    // + slack for 1024-byte alignment
  static_assert(SMEM <= 232448, "shared memory per CTA");
  static constexpr int TMEM_O = 256;                   // two S tiles of 128 columns, then two O tiles
};

__host__ __device__ constexpr uint32_t idesc_f16_m128(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __noinline__ bool ck_slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
  return wait_or_abort(bar, parity, abort_flag, err);
}
__device__ __forceinline__ bool ck_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
  return mbar_try_wait(bar, parity) || ck_slow_wait(bar, parity, abort_flag, err);
}

// Two fp32 values to fp16, `a` in the low half.
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Two e4m3 codes to fp16 (exact).
__device__ __forceinline__ uint32_t f16x2_of_codes(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

__device__ __forceinline__ void tmem_st_cols16(uint32_t taddr, const float (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(__float_as_uint(r[0])), "r"(__float_as_uint(r[1])), "r"(__float_as_uint(r[2])), "r"(__float_as_uint(r[3])),
      "r"(__float_as_uint(r[4])), "r"(__float_as_uint(r[5])), "r"(__float_as_uint(r[6])), "r"(__float_as_uint(r[7])),
      "r"(__float_as_uint(r[8])), "r"(__float_as_uint(r[9])), "r"(__float_as_uint(r[10])), "r"(__float_as_uint(r[11])),
      "r"(__float_as_uint(r[12])), "r"(__float_as_uint(r[13])), "r"(__float_as_uint(r[14])), "r"(__float_as_uint(r[15]))
      : "memory");
}

// ---------------------------------------------------------------- work
// Unit i of a sequence (n rows held, `count` new tokens, G heads of a group)
// sees n + e(i) keys, e(i) = floor((256 i + 255) / G) + 1 tokens having rows up to
// its end, `count` for the last: ceil((n + e(i)) / 128) = floor((2 i + c) / G)
// tiles with c = floor((255 + G (n + 128)) / 128).
struct UnitMath {
  int c, q, r, G, units, last;   // c = G q + r; last: tiles of the last unit

  __device__ __forceinline__ UnitMath(int n, int count, int g) : G(g) {
    c = (int)((255 + (int64_t)g * (n + 128)) >> 7);
    q = c / g;
    r = c - q * g;
    units = (int)(((int64_t)count * g + CK_ROWS - 1) / CK_ROWS);
    last = (n + count + CK_KEYS - 1) / CK_KEYS;
  }
  __device__ __forceinline__ int tiles(int i) const { return i == units - 1 ? last : (2 * i + c) / G; }
  // sum of floor((2 k + r) / G) over k < v <= G: the terms are 0, 1 or 2
  __device__ __forceinline__ int part(int v) const { return max(0, v - (G - r + 1) / 2) + max(0, v - (2 * G - r + 1) / 2); }
  // places before unit i, with i = G u + v
  __device__ __forceinline__ int before(int i) const {
    const int m = min(i, units - 1), u = m / G, v = m - u * G;
    return m * q + G * u * (u - 1) + 2 * u * v + u * part(G) + part(v) + (i == units ? last : 0) + i * kChunkUnitTiles;
  }
};

struct CkCut {   // CTA c owns places [first(c), first(c + 1))
  int base, rem, ctas;
  __device__ __forceinline__ int first(int c) const { return c * base + min(c, rem); }
  __device__ __forceinline__ int of(int x) const {
    const int big = rem * (base + 1);
    return x < big ? (int)((uint32_t)x / (uint32_t)(base + 1)) : rem + (int)((uint32_t)(x - big) / (uint32_t)base);
  }
};

__device__ __forceinline__ int ck_seq_of(const int32_t* from, int batch, int x) {   // the last b with from[b] <= x
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (from[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Tiles [t0, t0 + n) of unit i of (b, h); the unit has `tiles`, its first place is `place`.
struct CkSeg {
  int b, h, i, t0, n, tiles, place;
  __device__ __forceinline__ bool whole() const { return n == tiles; }
};

// The CTA's next segment at place x or behind it; false: none before x1.
__device__ __noinline__ bool ck_seg_at(const ChunkMap& m, int batch, int G, int x, int x1, CkSeg& s) {
  for (;;) {
    if (x >= x1) return false;
    s.b = ck_seq_of(m.start, batch, x);
    const UnitMath um(m.n[s.b], m.count[s.b], G);
    const int per = m.per[s.b], r = x - m.start[s.b];
    s.h = (int)((uint32_t)r / (uint32_t)per);
    const int at = r - s.h * per;
    int lo = 0, hi = um.units;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (um.before(mid) <= at) lo = mid;
      else hi = mid;
    }
    s.i = lo;
    s.tiles = um.tiles(lo);
    s.t0 = at - um.before(lo);
    s.place = x - s.t0;
    if (s.t0 < s.tiles) {
      s.n = min(s.tiles - s.t0, x1 - x);
      return true;
    }
    x = s.place + s.tiles + kChunkUnitTiles;
  }
}
__device__ __forceinline__ bool ck_next(const ChunkMap& m, int batch, int G, int x1, CkSeg& s) {
  const int x = s.place + s.t0 + s.n;
  return ck_seg_at(m, batch, G, s.t0 + s.n == s.tiles ? x + kChunkUnitTiles : x, x1, s);
}

template <int D>
__global__ void __launch_bounds__(CK_THREADS, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
  using C = CkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TileSlot* slots = reinterpret_cast<TileSlot*>(smem + C::OFF_SLOT);
  ChunkMap& M = *reinterpret_cast<ChunkMap*>(smem + C::OFF_MAP);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);   // two each: of a row tile, or of a stage
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* k_full = o_done + 2;
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* slot_full = v_empty + 2;
  uint64_t* slot_empty = slot_full + kSlots;
  uint64_t* mma_done = slot_empty + kSlots;
  uint64_t* never = mma_done + 1;   // test hook: nothing arrives
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
  volatile int* nan_seg = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);   // [4]: segment + 1 with NaN values some rows do not see

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, G = p.group;

  if (warp == 14) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr((const void*)tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 13 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);   // one arrival per warp
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&slot_full[i], 1);
      mbar_init(&slot_empty[i], 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(never, 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) nan_seg[i] = 0;
    fence_barrier_init();
  }
  grid_wait();
  grid_release();
  if (warp == 0) {
    // the map, 32 sequences at a time
    int at = 0, tiles = 0;
    bool bad = false;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      int32_t n = -1, count = 0;
      int64_t rr = 0;
      if (b < p.batch) {
        n = p.n_cached[b];
        count = p.n_new ? p.n_new[b] : p.t_len;
        rr = (int64_t)p.rope_row[b] + (p.row_at_length ? n : 0);
        if (n >= 0 && (count < 0 || count > p.t_len || (int64_t)n + count > p.max_keys ||
                       (count > 0 && (rr < 0 || rr + count > p.table_rows)))) {
          bad = true;
          count = 0;
        }
        if (n < 0) count = 0;
      }
      int per = 0, all = 0;
      if (count > 0) {
        const UnitMath um(n, count, G);
        per = um.before(um.units);
        all = (per - um.units * kChunkUnitTiles) * p.pool.n_kv;
      }
      const int v = per * p.pool.n_kv;
      int incl = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      M.start[b] = at + incl - v;
      M.per[b] = per;
      M.n[b] = n;
      M.count[b] = count;
      M.rope[b] = (int32_t)rr;   // of an empty or bad place: not used
      at += __shfl_sync(0xffffffffu, incl, 31);
      tiles += __reduce_add_sync(0xffffffffu, all);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      M.start[kMaxPagedSeqs] = at;
      M.tiles = tiles;
      if (bad && cta == 0) atomicOr(p.err, kErrLength);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  CkCut cut;
  const int places = M.start[kMaxPagedSeqs];
  cut.ctas = min((int)gridDim.x, max(1, M.tiles / kChunkMinTiles));
  cut.base = places / cut.ctas;
  cut.rem = places - cut.base * cut.ctas;
  const int x0 = cta < cut.ctas ? cut.first(cta) : places, x1 = cta < cut.ctas ? cut.first(cta + 1) : places;
  if (tid == 0) p.desc[cta * 8] = 0;   // no unit to merge, so far

  if (warp >= 12) {
    if (warp == 12) {
      // ---------------- page ids and scales: lane 8 k + g has group g of the k-th
      // tile of four; the ids of the next four are on their way meanwhile
      const int g = lane & 7;
      CkSeg sg;
      int seg = 0, at = lane >> 3, j = lane >> 3;   // tile `at` of segment `seg`, the CTA's j-th
      bool more = ck_seg_at(M, p.batch, G, x0, x1, sg);
      struct Ref {
        int32_t id, key0, rows, diag, h, seg;   // id: -1 no page here, -2 outside the pool
        bool on, last;
      };
      auto ask = [&]() {
        Ref r;
        r.id = -1;
        while (more && at >= sg.n) {
          at -= sg.n;
          ++seg;
          more = ck_next(M, p.batch, G, x1, sg);
        }
        r.on = more;
        r.last = false;
        if (more) {
          const int n = M.n[sg.b], tok0 = sg.i * CK_ROWS / G;
          const int end = n + min((sg.i * CK_ROWS + CK_ROWS - 1) / G + 1, M.count[sg.b]);
          r.key0 = (sg.t0 + at) * CK_KEYS;
          r.rows = min(end - r.key0, CK_KEYS);
          r.diag = n + tok0 + 1 - r.key0;
          r.h = sg.h;
          r.seg = seg;
          if (16 * g < r.rows) {
            r.id = p.page_table[(size_t)sg.b * p.max_pages + (r.key0 + 16 * g) / p.pool.page];
            if (r.id < 0) r.id = -2;
          }
          if (at == sg.n - 1) {
            CkSeg t = sg;
            r.last = !ck_next(M, p.batch, G, x1, t);
          }
        }
        at += 4;
        return r;
      };
      Ref cur = ask();
      bool ok = true;
      while (__any_sync(0xffffffffu, cur.on)) {
        const Ref nxt = ask();
        if (cur.id >= p.pool.n_pages) cur.id = -2;
        float ks = 0.f, vs = 0.f;
        const size_t block = cur.id >= 0 ? (size_t)cur.id * p.pool.n_kv + cur.h : 0;
        if (cur.id >= 0) {
          ks = p.pool.scales[0][block];
          vs = p.pool.scales[1][block];
        }
        if (cur.id == -2) atomicOr(p.err, kErrLength);
        const int ke = cur.id >= 0 ? exponent_of_scale(ks) : kNoScale, ve = cur.id >= 0 ? exponent_of_scale(vs) : kNoScale;
        int km = ke, vm = ve;
        uint32_t bad = cur.id == -2 ? 1u << g : 0;
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) {
          km = max(km, __shfl_xor_sync(0xffffffffu, km, off));
          vm = max(vm, __shfl_xor_sync(0xffffffffu, vm, off));
          bad |= __shfl_xor_sync(0xffffffffu, bad, off);
        }
        const bool mixed_k = cur.id >= 0 && ke != km, mixed_v = cur.id >= 0 && ve != vm;
        const uint32_t mk = __ballot_sync(0xffffffffu, mixed_k) >> (lane & 24), mv = __ballot_sync(0xffffffffu, mixed_v) >> (lane & 24);
        TileSlot& s = slots[j % kSlots];
        ok = !cur.on || j < kSlots || ck_wait(&slot_empty[j % kSlots], ((j / kSlots) - 1) & 1, abort_flag, p.err);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (cur.on) {
          s.grp[g] = cur.id >= 0 ? (int32_t)((block * p.pool.page + (cur.key0 + 16 * g) % p.pool.page) >> 4) : -1;
          const float kf = pow2_float(max(ke - km, -126)), vf = pow2_float(max(ve - vm, -126));
          s.kf[g] = f16x2(kf, kf);
          s.vf[g] = f16x2(vf, vf);
          if (g == 0) {
            s.k_scale = km == kNoScale ? 1.f : pow2_float(km);
            s.v_exp = vm;
            s.bad = bad;
            s.rows = cur.rows;
            s.diag = cur.diag;
            s.seg = cur.seg;
            s.flags = ((mk & 0xFF) ? 1u : 0u) | ((mv & 0xFF) ? 2u : 0u) | (cur.last ? 4u : 0u);
          }
        }
        __syncwarp();
        if (cur.on && g == 0) mbar_arrive(&slot_full[j % kSlots]);
        cur = nxt;
        j += 4;
      }
    } else if (warp == 13 && lane == 0) {
      // ---------------- MMA issuer.  The two row tiles take turns: while the
      // softmax of one works, the products of the other run.
      constexpr uint32_t idesc_qk = idesc_f16_m128(CK_KEYS, false);   // B = K (K-major)
      constexpr uint32_t idesc_pv = idesc_f16_m128(D, true);          // B = V (MN-major)
      auto qk = [&](int m, int j) {
        tc_fence_after();
        const uint32_t q = smem_addr(smem + C::OFF_Q + m * C::TILE), k = smem_addr(smem + C::OFF_K + (j & 1) * C::TILE);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * 16384 + (kk % 4) * 32;
          mma_bf16(tmem + m * 128, sw128_desc(q + off, 16, 1024), sw128_desc(k + off, 16, 1024), idesc_qk, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[m]);
      };
      auto pv = [&](int m, int j, bool first) {
        tc_fence_after();
        const uint32_t v = smem_addr(smem + C::OFF_V + (j & 1) * C::TILE);
#pragma unroll
        for (int kk = 0; kk < CK_KEYS / 16; ++kk)
          mma_bf16_tmem_a(tmem + C::TMEM_O + m * 128, tmem + m * 128 + kk * 8, sw128_desc(v + kk * 2048, 16384, 1024),
                          idesc_pv, !first || kk > 0 ? 1u : 0u);
        mma_commit(&o_done[m]);
      };
      int j = 0, n0 = 0, n1 = 0, seg0 = 0, seg1 = 0;   // tiles and segments of each row tile
      CkSeg sg;
      bool ok = true;
      for (bool more = ck_seg_at(M, p.batch, G, x0, x1, sg); ok && more; more = ck_next(M, p.batch, G, x1, sg)) {
        const bool two = M.count[sg.b] * G - sg.i * CK_ROWS > 128;
        ok = ck_wait(&k_full[j & 1], (j >> 1) & 1, abort_flag, p.err) && ck_wait(&q_full[0], seg0++ & 1, abort_flag, p.err);
        if (!ok) break;
        qk(0, j);
        if (two) {
          ok = ck_wait(&q_full[1], seg1++ & 1, abort_flag, p.err);
          if (!ok) break;
          qk(1, j);
        }
        mma_commit(&k_empty[j & 1]);
        for (int t = 0; t < sg.n; ++t, ++j) {
          const bool next = t + 1 < sg.n;
          ok = ck_wait(&v_full[j & 1], (j >> 1) & 1, abort_flag, p.err) && ck_wait(&p_full[0], n0++ & 1, abort_flag, p.err);
          if (!ok) break;
          pv(0, j, t == 0);
          if (next) {
            ok = ck_wait(&k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, abort_flag, p.err);
            if (!ok) break;
            qk(0, j + 1);
          }
          if (two) {
            ok = ck_wait(&p_full[1], n1++ & 1, abort_flag, p.err);
            if (!ok) break;
            pv(1, j, t == 0);
          }
          mma_commit(&v_empty[j & 1]);
          mbar_arrive(&slot_empty[j % kSlots]);   // the softmax has its part of it, the codes are in fp16
          if (next) {
            if (two) qk(1, j + 1);
            mma_commit(&k_empty[(j + 1) & 1]);
          }
        }
      }
      // every MMA issued above must complete before TMEM is released
      mma_commit(mma_done);
      mbar_wait(mma_done, 0);
    }
  } else if (warp >= 8) {
    // ---------------- codes to fp16: a thread has 16 codes of a row, 8 (at
    // head_dim 64, 4) times a tile of K and as often of V; the codes of the next
    // tile are asked for as soon as this one's registers are free
    constexpr int LPR = D / 16, RPP = 128 / LPR, NP = 128 / RPP;   // lanes of a row, rows at a time, times
    const int ct = tid - 256, c = ct % LPR, r0 = ct / LPR;
    // the 16-byte units of the row in fp16 that the codes go to; at head_dim 128 the
    // upper half of a row writes its second unit first, so that the eight lanes of a
    // row meet different banks
    const bool swap = c >= 4;
    const uint32_t sub = (uint32_t)(c / 4) * 16384;
    const int u0 = 2 * (c % 4);
    uint4 kc[NP], vc[NP];
    auto ask = [&](int j, int kv, uint4 (&u)[NP]) {
      const TileSlot& s = slots[j % kSlots];
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int row = k * RPP + r0, grp = s.grp[row >> 4];
        u[k] = make_uint4(0, 0, 0, 0);
        if (grp >= 0 && row < s.rows) u[k] = load_codes(p.pool.codes[kv] + (size_t)grp * (16 * D) + (row & 15) * D + c * 16);
      }
    };
    auto put = [&](int j, uint4 (&u)[NP], uint8_t* tile, const uint32_t* factors, bool mixed, int diag) {
      bool nan = false;
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int row = k * RPP + r0;
        uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
        if (row >= diag) {   // a NaN that some rows do not see must not reach them: see the epilogue
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t is = __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            nan |= is != 0;
            w[i] &= ~is;
          }
        }
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[2 * i] = f16x2_of_codes(w[i]);
          h[2 * i + 1] = f16x2_of_codes(w[i] >> 16);
        }
        if (mixed) {
          const uint32_t f = factors[row >> 4];
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = mul_f16x2(h[i], f);
        }
        const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
        uint8_t* at = tile + sub + row * 128;
        *reinterpret_cast<uint4*>(at + (((u0 + swap) ^ (row & 7)) << 4)) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(at + (((u0 + !swap) ^ (row & 7)) << 4)) = swap ? lo : hi;
      }
      return nan;
    };
    bool ok = x0 < x1;
    if (ok) {
      CkSeg sg;
      ok = ck_seg_at(M, p.batch, G, x0, x1, sg);   // a tile at all
    }
    if (ok) {
      ok = ck_wait(&slot_full[0], 0, abort_flag, p.err);
      if (__all_sync(0xffffffffu, ok)) {
        ask(0, 0, kc);
        ask(0, 1, vc);
      } else {
        ok = false;
      }
    }
    for (int j = 0; ok; ++j) {
      const TileSlot& s = slots[j % kSlots];
      const uint32_t flags = s.flags;
      const int diag = s.diag, seg = s.seg;
      if (j >= 2) ok = ck_wait(&k_empty[j & 1], ((j >> 1) - 1) & 1, abort_flag, p.err);
      put(j, kc, smem + C::OFF_K + (j & 1) * C::TILE, s.kf, flags & 1, CK_KEYS);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[j & 1]);
      if (!(flags & 4)) {
        ok = ck_wait(&slot_full[(j + 1) % kSlots], ((j + 1) / kSlots) & 1, abort_flag, p.err) && ok;
        if (!__all_sync(0xffffffffu, ok)) break;
        ask(j + 1, 0, kc);
      }
      if (j >= 2) ok = ck_wait(&v_empty[j & 1], ((j >> 1) - 1) & 1, abort_flag, p.err);
      if (put(j, vc, smem + C::OFF_V + (j & 1) * C::TILE, s.vf, flags & 2, diag)) nan_seg[seg & 3] = seg + 1;
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[j & 1]);
      if (flags & 4) break;
      ok = __all_sync(0xffffffffu, ok);
      if (ok) ask(j + 1, 1, vc);
    }
  } else {
    // ---------------- softmax and epilogue: row `row` of the unit
    const int m = warp >> 2;                      // row tile
    const int row = tid;                          // 0 .. 255
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_base + m * 128, o_at = lane_base + C::TMEM_O + m * 128;
    int j = 0, nt = 0, seg = 0;                   // the CTA's tiles, this row tile's, segments
    bool ok = true;
    CkSeg sg;
    for (bool more = ck_seg_at(M, p.batch, G, x0, x1, sg); ok && more; ++seg, more = ck_next(M, p.batch, G, x1, sg)) {
      const int n = M.n[sg.b], count = M.count[sg.b];
      const int first = sg.i * CK_ROWS, rows = min(count * G - first, CK_ROWS);   // of the unit
      if (sg.t0 == 0 && !sg.whole() && tid == 0) {
        // this CTA has the unit's first tile: it says who has the others
        int32_t* d = p.desc + cta * 8;
        d[1] = sg.b;
        d[2] = sg.h;
        d[3] = first;
        d[4] = cut.of(sg.place + sg.tiles - 1) - cta + 1;   // CTAs
        d[0] = rows;
      }
      if (m == 1 && rows <= 128) {   // nothing in this row tile
        j += sg.n;
        continue;
      }
      const int tok = (first + row) / G, head = sg.h * G + (first + row) % G;
      const bool live = row < rows;
      const bool warp_live = (row & ~31) < rows;
      // ---- the queries: rotated, times log2(e)/sqrt(d), over a power of two of
      // the row, in fp16.  8 (4) lanes to a row.
      float qs = 0.f;
      {
        constexpr int CH = D / 16, RPW = 32 / CH;   // lanes of a row, rows at a time
        const int c = lane % CH;
        uint8_t* qt = smem + C::OFF_Q + m * C::TILE;
#pragma unroll 2
        for (int k = 0; k < CH; ++k) {
          const int r = (row & ~31) + k * RPW + lane / CH;   // of the unit
          float x[8], y[8];
          uint32_t top = 0;
          if (r < rows) {
            const int rq = first + r, tk = rq / G;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (((size_t)sg.b * p.t_len + tk) * p.n_q + sg.h * G + rq % G) * D);
            unpack8(src[c], x);
            unpack8(src[c + CH], y);
            const CosSin2* t = p.tab + ((size_t)M.rope[sg.b] + tk) * (D / 2) + c * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 co = *reinterpret_cast<const float2*>(t + e), si = *reinterpret_cast<const float2*>(&t[e].sh);
              const float a = (x[e] * co.x - y[e] * si.x) * p.scale_log2;
              y[e] = (y[e] * co.x + x[e] * si.x) * p.scale_log2;
              x[e] = a;
              top = max(top, max(__float_as_uint(x[e]) & 0x7FFFFFFFu, __float_as_uint(y[e]) & 0x7FFFFFFFu));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
          }
#pragma unroll
          for (int off = CH / 2; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
          const int e = top < 0x7F800000u ? scale_exponent(top) : 0;   // a query that is not finite answers NaN
          const float inv = pow2_float(-e);
          uint32_t hx[4], hy[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hx[i] = f16x2(x[2 * i] * inv, x[2 * i + 1] * inv);
            hy[i] = f16x2(y[2 * i] * inv, y[2 * i + 1] * inv);
          }
          const int rt = r & 127, ux = c, uy = D == 128 ? c : c + 4;
          *reinterpret_cast<uint4*>(qt + rt * 128 + ((ux ^ (rt & 7)) << 4)) = make_uint4(hx[0], hx[1], hx[2], hx[3]);
          *reinterpret_cast<uint4*>(qt + (D == 128 ? 16384 : 0) + rt * 128 + ((uy ^ (rt & 7)) << 4)) =
              make_uint4(hy[0], hy[1], hy[2], hy[3]);
          const float scale = top < 0x7F800000u ? pow2_float(e) : __uint_as_float(0x7FFFFFFFu);
          const float mine = __shfl_sync(0xffffffffu, scale, lane % RPW * CH);
          if (lane / RPW == k) qs = mine;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[m]);
      }
      float m_run = -INFINITY, l_run = 0.f;
      int v_ref = kNoScale;
      const int lim = n + tok + 1;   // keys that the row sees
      if (p.inject_timeout && (cta & 1) == 0 && seg == 0) {
        ok = mbar_wait(never, 0, kInjectWaitCycles);
        *abort_flag = 1;
        if (tid == 0) atomicOr(p.err, kErrTimeout);
        break;
      }
      for (int t = 0; t < sg.n; ++t, ++j, ++nt) {
        ok = __all_sync(0xffffffffu, ck_wait(&s_full[m], nt & 1, abort_flag, p.err));
        if (!ok) break;
        if (warp_live) {
          tc_fence_after();
          const TileSlot& ts = slots[j % kSlots];
          const int nvis = live ? lim - (sg.t0 + t) * CK_KEYS : 0;
          float sc = qs * ts.k_scale;   // in range, so that a masked score stays -inf; NaN stays
          sc = sc < FLT_MIN ? FLT_MIN : sc > FLT_MAX ? FLT_MAX : sc;
          const uint32_t bad = ts.bad;
          const int v_exp = ts.v_exp;
          // the scores are read twice, 32 at a time: once for the maximum, once for
          // the weights, which take the place of the scores read before them
          const bool partial = nvis < CK_KEYS || bad;
          auto mask = [&](int i0, float (&x)[32]) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i0 + i >= nvis || (bad >> ((i0 + i) >> 4) & 1)) x[i] = -INFINITY;
          };
          float top = -INFINITY;
#pragma unroll
          for (int i0 = 0; i0 < CK_KEYS; i0 += 64) {
            float x[32], y[32];
            tmem_ld32(s_at + i0, x);
            tmem_ld32(s_at + i0 + 32, y);
            tmem_wait_ld();
            if (partial) {
              mask(i0, x);
              mask(i0 + 32, y);
            }
            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              t0 = fmaxf(t0, x[i]);
              t1 = fmaxf(t1, y[i]);
            }
            top = fmaxf(top, fmaxf(t0, t1));
          }
          top = top == -INFINITY ? top : top * sc;
          float alpha = 1.f;
          bool rescale = false;
          if (top > m_run) {
            if (m_run == -INFINITY) {
              m_run = top;   // nothing accumulated yet: O holds zeros
            } else if (top - m_run > kRescaleLog2) {
              alpha = ex2_approx(m_run - top);
              m_run = top;
              rescale = true;
            }
          }
          l_run *= alpha;
          if (v_exp > v_ref) {   // the same in every row
            if (v_ref != kNoScale) {
              alpha *= pow2_float(max(v_ref - v_exp, -126));
              rescale = true;
            }
            v_ref = v_exp;
          }
          const float v_mul = v_exp == kNoScale || v_exp < v_ref - 126 ? 0.f : pow2_float(v_exp - v_ref);
          const float mu = (m_run == -INFINITY ? 0.f : m_run) - kWeightLog2;
          if (__any_sync(0xffffffffu, rescale) && t > 0) {
            ok = __all_sync(0xffffffffu, ck_wait(&o_done[m], (nt - 1) & 1, abort_flag, p.err));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
              float o[32];
              tmem_ld32(o_at + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= alpha;
              tmem_st32(o_at + c0, o);
            }
          }
          float l0 = 0.f, l1 = 0.f;
          float x[2][32];
          tmem_ld32(s_at, x[0]);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            tmem_wait_ld();
            if (q4 < 3) tmem_ld32(s_at + (q4 + 1) * 32, x[(q4 + 1) & 1]);
            float (&y)[32] = x[q4 & 1];
            if (partial) mask(q4 * 32, y);
            float w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float a = ex2_approx(fmaf(y[i], sc, -mu)), b = ex2_approx(fmaf(y[i + 1], sc, -mu));
              l0 += a;
              l1 += b;
              w[i / 2] = __uint_as_float(f16x2(a * v_mul, b * v_mul));
            }
            tmem_st_cols16(s_at + q4 * 16, w);
          }
          l_run += l0 + l1;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[m]);
      }
      if (!ok) break;
      // ---- epilogue
      ok = __all_sync(0xffffffffu, ck_wait(&o_done[m], (nt - 1) & 1, abort_flag, p.err));
      if (!ok) break;
      if (!warp_live) continue;
      tc_fence_after();
      const bool nan = nan_seg[seg & 3] == seg + 1;
      const bool whole = sg.whole();
      const float scale = v_ref == kNoScale ? 0.f : pow2_float(v_ref);
      const float f = whole ? (l_run == 0.f ? 0.f : scale / l_run) : scale;
      const int slot = 2 * cta + (sg.t0 == 0 ? 1 : 0);   // of a unit's first part: see the merge
      if (!whole && live) p.part_ml[(size_t)slot * p.part_rows + row] = make_float2(m_run, l_run);
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        tmem_ld32(o_at + c0, o);
        tmem_wait_ld();
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= f;
        if (nan) {   // values that are not numbers, for the rows that see them
          const int end = min(lim, (sg.t0 + sg.n) * CK_KEYS);
          for (int key = max(n + first / G + 1, sg.t0 * CK_KEYS); key < end; ++key) {
            const int id = p.page_table[(size_t)sg.b * p.max_pages + key / p.pool.page];
            if (id < 0 || id >= p.pool.n_pages) continue;
            const uint8_t* v = p.pool.codes[1] + (((size_t)id * p.pool.n_kv + sg.h) * p.pool.page + key % p.pool.page) * D + c0;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((v[i] & 0x7F) == 0x7F) o[i] = __uint_as_float(0x7FFFFFFFu);
          }
        }
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + (((size_t)sg.b * p.t_len + tok) * p.n_q + head) * D + c0);
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            const float e[8] = {o[i], o[i + 1], o[i + 2], o[i + 3], o[i + 4], o[i + 5], o[i + 6], o[i + 7]};
            dst[i / 8] = pack8(e);
          }
        } else {
          float4* dst = p.part_o + ((size_t)slot * (D / 4) + c0 / 4) * p.part_rows + row;
#pragma unroll
          for (int i = 0; i < 32; i += 4) dst[(size_t)(i / 4) * p.part_rows] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 14) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the parts of the units that several CTAs hold.  blockIdx.x: the CTA with
// the unit's first tile (its part is slot 2 c + 1, those of the CTAs behind it slot
// 2 c'); blockIdx.y: 32 rows; a lane to a row, a warp to D / 8 columns.
constexpr int MG_THREADS = 256;
template <int D>
__global__ void __launch_bounds__(MG_THREADS) merge_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int C4 = D / 4 / 8;
  __shared__ float wts[kMaxChunkCtas][32];
  __shared__ float red[8][32];
  grid_wait();
  grid_release();
  const int32_t* d = p.desc + blockIdx.x * 8;
  const int rows = d[0], row = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)blockIdx.y * 32 >= rows) return;
  const int b = d[1], h = d[2], rq = d[3] + row, parts = d[4], G = p.group;
  auto slot = [&](int k) { return (size_t)(2 * ((int)blockIdx.x + k) + (k == 0 ? 1 : 0)); };
  const bool live = row < rows;
  float mx = -INFINITY;
  for (int k = warp; k < parts; k += 8) {
    const float m = live ? p.part_ml[slot(k) * p.part_rows + row].x : -INFINITY;
    wts[k][lane] = m;
    mx = fmaxf(mx, m);
  }
  red[warp][lane] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = fmaxf(mx, red[i][lane]);
  __syncthreads();
  const float base = mx == -INFINITY ? 0.f : mx;
  float l = 0.f;
  for (int k = warp; k < parts; k += 8) {
    const float w = ex2_approx(wts[k][lane] - base);
    wts[k][lane] = w;
    l = fmaf(w, live ? p.part_ml[slot(k) * p.part_rows + row].y : 0.f, l);
  }
  red[warp][lane] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) l += red[i][lane];
  if (!live) return;
  float4 acc[C4];
#pragma unroll
  for (int i = 0; i < C4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const float w = wts[k][lane];
    const float4* o = p.part_o + (slot(k) * (D / 4) + warp * C4) * p.part_rows + row;
#pragma unroll
    for (int i = 0; i < C4; ++i) {
      const float4 v = o[(size_t)i * p.part_rows];
      acc[i].x = fmaf(w, v.x, acc[i].x);
      acc[i].y = fmaf(w, v.y, acc[i].y);
      acc[i].z = fmaf(w, v.z, acc[i].z);
      acc[i].w = fmaf(w, v.w, acc[i].w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2* dst = reinterpret_cast<uint2*>(p.out + (((size_t)b * p.t_len + rq / G) * p.n_q + h * G + rq % G) * D) + warp * C4;
#pragma unroll
  for (int i = 0; i < C4; ++i) dst[i] = make_uint2(pack2(acc[i].x * inv, acc[i].y * inv), pack2(acc[i].z * inv, acc[i].w * inv));
}

template <int D>
cudaError_t launch_chunk(const ChunkParams& p, int sms, cudaStream_t st) {
  using C = CkCfg<D>;
  static KernelSetup s;
  const int dev = setup_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(s.mu);
    if (s.state[dev] == 0) {
      const cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
      if (e != cudaSuccess) cudaGetLastError();
      s.state[dev] = e == cudaSuccess ? 1 : -(int)e;
    }
    if (s.state[dev] != 1) return (cudaError_t)(-s.state[dev]);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(CK_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_kernel<D>, p);
}

template <int D>
cudaError_t launch_merge(const ChunkParams& p, int sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms, p.part_rows / 32);
  cfg.blockDim = dim3(MG_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel<D>, p);
}

}  // namespace

int chunk_part_rows(int t_len, int group) {
  return (int)std::min<int64_t>(CK_ROWS, ((int64_t)t_len * group + 31) / 32 * 32);
}

int64_t chunk_places(int batch, int n_kv, int t_len, int group, int max_keys) {
  const int64_t units = ((int64_t)t_len * group + CK_ROWS - 1) / CK_ROWS;
  return batch * (int64_t)n_kv * units * ((max_keys + CK_KEYS - 1) / CK_KEYS + kChunkUnitTiles);
}

cudaError_t launch_attend_chunk8(const ChunkParams& p, int head_dim, int sms, cudaStream_t st) {
  return head_dim == 128 ? launch_chunk<128>(p, sms, st) : launch_chunk<64>(p, sms, st);
}

cudaError_t launch_attend_chunk8_merge(const ChunkParams& p, int head_dim, int sms, cudaStream_t st) {
  return head_dim == 128 ? launch_merge<128>(p, sms, st) : launch_merge<64>(p, sms, st);
}

}  // namespace c2kv
