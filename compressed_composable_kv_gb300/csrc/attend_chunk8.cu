// Attention of a chunk of new tokens over the 8-bit paged cache (one layer) on
// the 5th-generation tensor cores:
//   s_j = (R q . K_j) / sqrt(d),  out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// over the rows j up to the token's own; K_j and V_j = code * scale of their page.
//
// A unit is 256 or 128 (token, query head) rows of one (sequence, kv head), token-major,
// against the key tiles (128 rows) that they see.  Every e4m3 code is an fp16
// number, so a tile's codes are brought to fp16 once for all rows of the unit, and both
// products run as kind::f16 (fp32 accumulators): the keys and values lose
// nothing; a query row is held in fp16 times a power of two of its own, 2^-11 of
// each element, and so is a weight (2^7 exp(s - m), so that weights down to 2^-15
// of the largest keep their 11 bits).  The bf16 output itself rounds away 2^-8: answers are
// 0.00161 to 0.00172 off the exact ones in the mean square, most where logits are large (a query
// moves one by up to 2^-11 sum |q_i K_i| / sqrt(d)), sums of bf16 queries in fp32 0.00159 to 0.00166.
// Twice the query's bits would be twice the scores' products, and their tiles do not fit beside
// those of K and V with 256 rows.  Pages
// of one tile with different scales meet at the largest of them by an exact multiplication
// in fp16 (apart_tile has what is too far apart for that); the tile's K scale multiplies the
// scores, its V scale the weights, over a unit that each row of O has for itself.
//
// The places of all units (their tiles, and some for the end of each) are laid end to
// end, from the device-side lengths, and cut into one even range per CTA (one to an SM).
// A unit that one CTA holds whole is written at once; else its CTAs write partial
// (m, l, O / l) and merge_kernel joins them in the order of the keys.
//
// A call is two launches, or three: the append, whose further CTAs rotate the queries
// into the output buffer (fp16, pages8.cu), this kernel, and the join where units are
// cut.  Each is set up, and reads what the one before does not write, while that one runs.
//
// Roles: warps 0-3 and 4-7 softmax and epilogue, a thread to a row (of a unit of 256 rows
// each four have 128; of a smaller one each four have every other key tile), warps 8-11
// and 12-15 the codes of K and V to fp16, warp 16 page ids and scales ahead of them and
// their codes to L2, warps 17 and 18 the MMAs of a half each, warp 19 tensor memory.
//
// What bounds it.  256 rows: scores, weights and products of 64 keys go round in two parts
// of a tile for each half, and the two halves fill each other's waits.  A tile takes
// 2.3 to 2.4 us of an SM, against 1.3 at the bf16 rate that a library product reaches: left out,
// the conversion is worth 4 %, three quarters of the scores' products 5 %, the exponentials
// 5 %, all of the softmax 15 %, so no part alone is the limit; N = 64 costs the scores'
// products half again as much (Q's rows come from shared memory, 128 bytes a cycle), but
// N = 128 leaves a half nothing to do while its scores are made (4 x 512 tokens over 32768
// 974-1040 us against 990, 8 x 128 137 against 132, 16 x 5 75 against 73).  128 rows: a
// tile takes 1.5 us, the halves' chains of scores, weights, products and the next stage's
// codes, of which none can be left out for more than 7 %.  Few rows over short caches: the
// launches, 3 to 4 us each, and the way through the first tile, 4 us.
//
// 32 query heads of 128 over 8 kv heads: 4 x 512 tokens over 32768 1008 us (1.10 PFLOP/s),
// 1 x 4000 over nothing 202 us, 16 x 5 over 1000 to 8000 74 us (1.9 TB/s), 1 x 64 over 8000
// 35 us; 40 heads over 8, 8 x 128 over 7000 to 8000 119 us (0.53 PFLOP/s).
// Figures beside a choice, here and below, are of both sides at the time it was made.
#include <float.h>

#include <algorithm>

#include "pages8.h"
#include "tcgen05.h"

namespace c2kv {

namespace {

constexpr int CK_THREADS = 640;
constexpr int CK_KEYS = 128;       // keys of a tile
constexpr int kSlots = 8;          // tiles whose pages are known ahead
// Tiles of a CTA below which fewer CTAs work, where units are cut: a part costs its sums
// and their joining (7 x 7 tokens over 58 to 847 rows 23.4 us at 1, 21.0 at 2, 24.8 at 3).
constexpr int kChunkMinTiles = 2;
// What a unit's begin and end cost, in tiles (16 x 5 over 1000 to 8000 72 us at 1, 67 at 2;
// 1 x 4000 222 and 203 us).
constexpr int kChunkUnitTiles = 2;
// What a tile of a 256-row unit counts, and one of up to 128 rows among them (8 x 128 of
// group 5, whose units have 256, 256 and 128 rows: 124 us where both count the same, 115 at
// 8 to 5, 114 at 3 to 2).
constexpr int kChunkWidePlaces = 3, kChunkNarrowPlaces = 2;
constexpr int kChunkFewTiles = 16; // see chunk_wide
constexpr int kChunkWholeKeys = 512, kChunkMergeTiles = 4;  // see chunk_whole
constexpr int kNoScale = -1000;    // exponent of a tile without a page
// A code times 2^-15 is an fp16 number, times less it may not be (codes are multiples of
// 2^-9, fp16 numbers of 2^-24).
constexpr int kMostBelow = 15;
constexpr float kRescaleLog2 = 8.f;   // a row's maximum may lag behind by this (weights up to 2^15, sums exact)
constexpr float kWeightLog2 = 7.f;
// How far a tile's V scale may be below the unit of a row's O before the unit is brought
// down to it: weights below 2^-21 of the row's largest lose bits, with this 2^-15.
constexpr int kUnitAbove = 6;
// ... or above it before its products are made in fp32 (see apart_tile): to raise the unit by
// more costs columns that only other pages have values in their place in fp32's range.
constexpr int kUnitBelow = 60;
constexpr int kMostLog2 = 120;        // O's largest element stays below 2^this when its unit is brought down,
constexpr int kLeastLog2 = 100;       // its least above 2^-this when the unit is raised for a tile's scale
constexpr int kSumLog2 = 80;          // weights in fp32 are up to 2^(kWeightLog2 + this)

// What warp 16 finds out about a tile, and the segment that it belongs to.
enum : uint32_t { kWhole = 2, kEnd = 4, kWide = 8, kNone = 16, kFresh = 32 };
struct TileSlot {
  int32_t grp[8];      // 16 rows each: index of the first of them in the layer, in 16s; -1: no page
  uint32_t kf[8];      // half2: the page's scale over the tile's, of K and of V
  uint32_t vf[8];
  float k_scale;       // the tile's
  int32_t v_exp;
  uint32_t bad;        // bit g: the rows of grp[g] take no part, bit 8 + g: their keys' codes
                       // are held as they are, their scores times k_by[g], bit 16 + g: their V
                       // scale is further below v_exp than fp16 has room for (see apart_tile)
  float k_by[8];
  int32_t v_of[8];     // exponents of the V scales
  int32_t rows;        // keys of the tile that any row of the unit sees
  int32_t diag;        // keys below this are seen by every row
  // from here on known (seg_full) before the rest (slot_full)
  uint32_t flags;      // kWhole: the segment is a whole unit, kEnd: it is
                       // the CTA's last, kWide: a unit of more than 128 rows, kNone: the CTA has no
                       // tile, kFresh: the tile has rows that the append writes
  int32_t seg;         // segments of the CTA before this one
  int32_t b, h, first; // sequence, kv head, the unit's first row
  int32_t tile, n;     // of the unit, and how many of the segment are left
  int32_t ctas;        // CTAs that hold the unit, if this is the first
  int32_t pad[3];
};

struct ChunkMap {
  int32_t start[kMaxPagedSeqs + 1];   // first place of each sequence; the last one is the total
  int32_t per[kMaxPagedSeqs];         // places of one kv head of it
  int32_t n[kMaxPagedSeqs];           // rows held before the chunk
  int32_t count[kMaxPagedSeqs];       // new tokens
  int32_t tiles;                      // of the launch
};

template <int D, int W>
struct CkCfg {
  static constexpr int TILE = 128 * D * 2;             // a query, K or V tile in fp16
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = W * TILE;
  static constexpr int OFF_V = OFF_K + 2 * TILE;
  // what the second softmax half hands to the first (W == 1): O of 64 rows, column
  // by column of four; then (m, l, scale) of 128
  static constexpr int OFF_HO = OFF_V + 2 * TILE;
  static constexpr int OFF_X = OFF_HO + (W == 1 ? 64 * D * 4 : 0);
  static constexpr int OFF_SLOT = OFF_X + 128 * 16;
  static constexpr int OFF_MAP = OFF_SLOT + kSlots * (int)sizeof(TileSlot);
  static constexpr int OFF_BARS = OFF_MAP + (int)((sizeof(ChunkMap) + 15) / 16 * 16);
  static constexpr int N_BAR = 2 * 9 + 3 * kSlots + 5;
  static constexpr int OFF_MISC = OFF_BARS + N_BAR * 8;
  static constexpr int SMEM = OFF_MISC + 64 + 1024;    // + slack for 1024-byte alignment
  static_assert(SMEM <= 232448, "shared memory per CTA");
  static constexpr int TMEM_O = 256;                   // two S tiles of 128 columns, then two O tiles
};

__host__ __device__ constexpr uint32_t idesc_f16_m128(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// A bounded wait that gives up once another thread has aborted the CTA.  The thread
// sleeps some microseconds at a time: warps that poll take issue slots from the rest.
__device__ __forceinline__ bool ck_slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
  const long long t0 = clock64();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (done) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort_flag = 1;
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool ck_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
  return mbar_try_wait(bar, parity) || ck_slow_wait(bar, parity, abort_flag, err);
}

// Two e4m3 codes to fp16 (exact).
__device__ __forceinline__ uint32_t f16x2_of_codes(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ uint64_t pack_f32x2(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack_f32x2(a)), "l"(pack_f32x2(b)), "l"(pack_f32x2(c)));
  return unpack_f32x2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack_f32x2(a)), "l"(pack_f32x2(b)));
  return unpack_f32x2(r);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// 16 codes, or zeros.  One instruction sequence: where the compiler joins the two
// cases it waits for the load there and then.
__device__ __forceinline__ uint4 load_codes(const uint8_t* p, bool on) {
  uint4 u;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(u.x), "=&r"(u.y), "=&r"(u.z), "=&r"(u.w)
      : "l"(p), "r"((uint32_t)on));
  return u;
}

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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
// Unit i of a sequence (n rows held, `count` new tokens, G heads of a group) has
// 128 w rows, w = 1 or 2, and sees n + e(i) keys, e(i) = floor((128 w (i + 1) - 1) / G)
// + 1 tokens having rows up to its end, `count` for the last: ceil((n + e(i)) / 128) =
// floor((w i + c) / G) tiles with c = floor((128 w - 1 + G (n + 128)) / 128).
// A tile of a unit is `full` places of the work, one of the last unit `cost` (in a batch
// of 256-row units a unit of up to 128 rows takes two thirds of the time), and the end
// of a unit `end`.
struct UnitMath {
  int c, q, r, G, w, units, last;   // c = G q + r; last: tiles of the last unit
  int full, cost, end;

  __device__ __forceinline__ UnitMath(int n, int count, int g, int wide) : G(g), w(wide) {
    c = (int)((128 * w - 1 + (int64_t)g * (n + 128)) >> 7);
    q = c / g;
    r = c - q * g;
    units = (int)(((int64_t)count * g + 128 * w - 1) / (128 * w));
    last = (n + count + CK_KEYS - 1) / CK_KEYS;
    full = w == 1 ? 1 : kChunkWidePlaces;
    cost = w == 2 && (int64_t)count * g - 256 * (int64_t)(units - 1) <= 128 ? kChunkNarrowPlaces : full;
    end = full * kChunkUnitTiles;
  }
  __device__ __forceinline__ int tiles(int i) const { return i == units - 1 ? last : (w * i + c) / G; }
  // sum of floor((w k + r) / G) over k < v <= G: the terms are 0 to w
  __device__ __forceinline__ int part(int v) const {
    return w == 1 ? max(0, v - (G - r)) : max(0, v - (G - r + 1) / 2) + max(0, v - (2 * G - r + 1) / 2);
  }
  // tiles of units before unit i < units, with i = G u + v
  __device__ __forceinline__ int tiles_before(int i) const {
    const int u = i / G, v = i - u * G;
    return i * q + w * (G * (u * (u - 1) / 2) + u * v) + u * part(G) + part(v);
  }
  __device__ __forceinline__ int all_tiles() const { return tiles_before(units - 1) + last; }
  __device__ __forceinline__ int cost_of(int i) const { return i == units - 1 ? cost : full; }
  // places before unit i
  __device__ __forceinline__ int before(int i) const {
    return full * tiles_before(min(i, units - 1)) + (i == units ? last * cost : 0) + i * end;
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
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (from[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Tiles [t0, t0 + n) of unit i of (b, h); the unit has `tiles` of `cost` places each,
// its first place is `place`, the next unit's `next`.  A tile is the CTA's that has its
// first place.  Where units are left whole, each is one place.
struct CkSeg {
  int b, h, i, t0, n, tiles, place, cost, next;
  __device__ __forceinline__ bool whole() const { return n == tiles; }
};

// The unit at place x, and its first tile at x or behind it (t0 >= tiles: none is).
template <int W>
__device__ __forceinline__ void ck_locate(const ChunkMap& m, int batch, int G, bool whole, int x, CkSeg& s) {
  s.b = ck_seq_of(m.start, batch, x);
  const UnitMath um(m.n[s.b], m.count[s.b], G, W);
  const int per = m.per[s.b], r = x - m.start[s.b];
  s.h = (int)((uint32_t)r / (uint32_t)per);
  const int at = r - s.h * per;
  if (whole) {
    s.i = at;
    s.tiles = um.tiles(at);
    s.t0 = 0;
    s.cost = 1;
    s.place = x;
    s.next = x + 1;
    return;
  }
  int lo = 0, hi = um.units;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (um.before(mid) <= at) lo = mid;
    else hi = mid;
  }
  s.i = lo;
  s.tiles = um.tiles(lo);
  s.cost = um.cost_of(lo);
  const int off = at - um.before(lo);
  s.t0 = (int)((uint32_t)(off + s.cost - 1) / (uint32_t)s.cost);
  s.place = x - off;
  s.next = s.place + s.tiles * s.cost + um.end;
}

// The CTA's next segment at place x or behind it; false: none before x1.
template <int W>
__device__ __forceinline__ bool ck_seg_at(const ChunkMap& m, int batch, int G, bool whole, int x, int x1, CkSeg& s) {
#pragma unroll 1
  for (;;) {
    if (x >= x1) return false;
    ck_locate<W>(m, batch, G, whole, x, s);
    if (s.t0 < s.tiles) {
      s.n = whole ? s.tiles : min(s.tiles, (int)((uint32_t)(x1 - s.place + s.cost - 1) / (uint32_t)s.cost)) - s.t0;
      return s.n > 0;
    }
    x = s.next;
  }
}
template <int W>
__device__ __forceinline__ bool ck_next(const ChunkMap& m, int batch, int G, bool whole, int x1, CkSeg& s) {
  return s.t0 + s.n == s.tiles && ck_seg_at<W>(m, batch, G, whole, s.next, x1, s);
}

// Rows begin, begin + 2 (at head_dim 64: 4) - 1 by a warp, and so on before `end`, of the
// unit that begins at row `first` of (b, h): its queries, as the launch before left
// them, to row rt0 + r mod 128 of their tile.
template <int D>
__device__ __forceinline__ void ck_copy_queries(const ChunkParams& p, uint32_t q_smem, int b, int h, int first, int begin, int end, int rt0) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;   // lanes of a row, rows at a time
  const int lane = threadIdx.x & 31, c = lane % LPR, G = p.group;
  int r = begin + lane / LPR, t = (first + r) / G, g = first + r - t * G;
  const __nv_bfloat16* src = p.out + ((size_t)b * p.t_len * p.n_q + h * G) * D + c * 8;
#pragma unroll 4
  for (; r < end; r += RPI) {
    const int rt = rt0 + (r & 127);
    const uint32_t dst = q_smem + (r >> 7) * (128 * D * 2) + (c >> 3) * 16384 + rt * 128 + (((c & 7) ^ (rt & 7)) << 4);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + ((size_t)t * p.n_q + g) * D) : "memory");
    for (g += RPI; g >= G; g -= G) ++t;
  }
}

// Lane l of each four has row l's four pieces: afterwards piece l of the four rows.
__device__ __forceinline__ void transpose4(uint4 (&a)[4]) {
  const bool b0 = threadIdx.x & 1, b1 = threadIdx.x & 2;
  auto swap = [](uint4& keep0, uint4& keep1, bool hi, int by) {
    const uint4 give = hi ? keep0 : keep1;
    uint4 got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, by);
    got.y = __shfl_xor_sync(0xffffffffu, give.y, by);
    got.z = __shfl_xor_sync(0xffffffffu, give.z, by);
    got.w = __shfl_xor_sync(0xffffffffu, give.w, by);
    if (hi) keep0 = got;
    else keep1 = got;
  };
  swap(a[0], a[1], b0, 1);
  swap(a[2], a[3], b0, 1);
  swap(a[0], a[2], b1, 2);
  swap(a[1], a[3], b1, 2);
}

// O (D columns of a row in each lane of the warp, all of it there) to a unit 2^-down of its
// present one, `down` of either sign, or as far in that direction as keeps it in fp32's
// range.  Returns how far.
template <int D>
__device__ __forceinline__ int move_unit(uint32_t o_at, int down) {
  float most = 0.f, least = INFINITY;   // of what is not 0
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 16) {
    float o[16];
    tmem_ld_cols<16>(o_at + c0, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      most = fmaxf(most, fabsf(o[i]));
      if (o[i] != 0.f) least = fminf(least, fabsf(o[i]));
    }
  }
  if (most > 0.f) {
    down = min(down, max(kMostLog2 - exponent_of_scale(most), 0));
    down = max(down, min(-kLeastLog2 - exponent_of_scale(least), 0));
  }
  const int half = min(max(down, -120), 120);
  const float by = pow2_float(half), more = pow2_float(down - half);
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 16) {
    float o[16];
    tmem_ld_cols<16>(o_at + c0, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = o[i] * by * more;
    tmem_st_cols16(o_at + c0, o);
  }
  tmem_wait_st();
  return down;
}

// Rows 16 g, 16 g + 1, ... of the tile that any row of the unit sees, and where their values are.
template <int D>
__device__ __forceinline__ const uint4* values_of(const ChunkParams& p, const TileSlot& s, int g, int& rows) {
  rows = s.grp[g] < 0 || (s.bad >> g & 1) ? 0 : min(max(s.rows - 16 * g, 0), 16);
  return reinterpret_cast<const uint4*>(p.pool.codes[1] + (int64_t)s.grp[g] * (16 * D));
}

// Whether any value of these groups of 16 rows is not 0 (the same in every lane).
template <int D>
__device__ __forceinline__ bool any_value(const ChunkParams& p, const TileSlot& s, uint32_t groups) {
  uint32_t some = 0;
#pragma unroll 1
  for (; groups; groups &= groups - 1) {
    int rows;
    const uint4* v = values_of<D>(p, s, __ffs(groups) - 1, rows);
    for (int i = threadIdx.x & 31; i < rows * (D / 16); i += 32) {
      const uint4 u = v[i];
      some |= (u.x | u.y | u.z | u.w) & 0x7F7F7F7Fu;
    }
  }
  return __any_sync(0xffffffffu, some != 0);
}

// Adds rows 16 g, ... of the tile to O in fp32, each lane for its own row of the unit.
// The unit of O moves as before a tile's products.  s_at: the group's scores.
template <int D>
__device__ __forceinline__ void add_values(const ChunkParams& p, const TileSlot& s, int g, uint32_t s_at, uint32_t o_at,
                                           int nvis, float sc, float m_run, int& v_ref) {
  int rows;
  const uint4* v = values_of<D>(p, s, g, rows);
  if (rows == 0 || !any_value<D>(p, s, 1u << g)) return;
  if (v_ref == kNoScale) v_ref = s.v_of[g];
  int v_by = s.v_of[g] - v_ref;
  sc *= s.bad >> (8 + g) & 1 ? s.k_by[g] : 1.f;
  if (__any_sync(0xffffffffu, v_by < -60)) {
    const int down = move_unit<D>(o_at, v_by < -60 ? -v_by : 0);
    v_ref -= down;
    v_by += down;
  }
  float x[16], top = -INFINITY;
  tmem_ld_cols<16>(s_at, x);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, 16 * g + i < nvis ? x[i] : -INFINITY);
  const int room = (int)fmaxf(floorf(m_run - top * sc), 0.f), up = top != -INFINITY ? max(v_by - room - kSumLog2, 0) : 0;
  float by = up > 126 ? 0.f : pow2_float(-up);   // what O is multiplied by, once
  v_ref += up;
  v_by -= up;
#pragma unroll 1
  for (int i = 0; i < rows; i += 2) {
    float e[2];
    tmem_ld_cols<2>(s_at + i, e);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 2; ++k)
      e[k] = i + k < rows && 16 * g + i + k < nvis ? ex2_approx(fmaf(e[k], sc, kWeightLog2 + (float)v_by - m_run)) : 0.f;
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
      float o[16];
      tmem_ld_cols<16>(o_at + 16 * c, o);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 u = i + k < rows ? v[(i + k) * (D / 16) + c] : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          // NaN that some rows of the unit do not see: see the epilogue
          const uint32_t codes = w[n] & ~(16 * g + i + k < s.diag ? 0u : __vcmpeq4(w[n] & 0x7F7F7F7Fu, 0x7F7F7F7Fu));
          const float2 a = e4m3x2_to_float2(codes & 0xFFFFu), b = e4m3x2_to_float2(codes >> 16);
          float* to = o + 4 * n;
          if (k == 0) to[0] *= by, to[1] *= by, to[2] *= by, to[3] *= by;
          to[0] = fmaf(e[k], a.x, to[0]);
          to[1] = fmaf(e[k], a.y, to[1]);
          to[2] = fmaf(e[k], b.x, to[2]);
          to[3] = fmaf(e[k], b.y, to[3]);
        }
      }
      tmem_st_cols16(o_at + 16 * c, o);
      tmem_wait_st();
    }
    by = 1.f;
  }
}

// A tile some of whose pages have V scales more than 2^15 apart, which share no fp16 scale
// that all fit, or one whose scale is too far from O's unit for that to be moved: its values are added in fp32, page by page, and its weights are 0 for the
// products that the issuer makes of them all the same (60 to 80 us a tile: right, not fast).
// From the scores of its first part, which are there, to the end of its second.
struct RowSums {
  float m, l;
  int v_ref;
};
template <int D, int W>
__device__ __forceinline__ bool apart_tile(const ChunkParams& p, const TileSlot& s, uint64_t* s_full, uint64_t* p_full, uint64_t* k_empty,
                                        uint64_t* v_empty, int step, bool has_o, volatile uint32_t* o_set, uint32_t s_at,
                                        uint32_t o_at, int nvis, float sc, int ns, volatile int* abort_flag, RowSums& r) {
  const int lane = threadIdx.x & 31;
  auto wait = [&](uint64_t* bar, int phase) {
    return __all_sync(0xffffffffu, ck_wait(bar, (uint32_t)phase & 1, abort_flag, p.err)) != 0;
  };
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    if (part == 1) {
      if (!wait(s_full + 1, ns)) return false;
      if (W == 2 && lane == 0) {
        mbar_arrive_n(k_empty, step);
        if (has_o) mbar_arrive_n(v_empty, step);
      }
    }
    tc_fence_after();
    float x[16] = {}, top = -INFINITY, l = 0.f;
    auto score = [&](int g, int i) {   // of the row's key 16 g + i
      return 16 * g + i < nvis && !(s.bad >> g & 1) ? x[i] * (s.bad >> (8 + g) & 1 ? s.k_by[g] : 1.f) * sc : -INFINITY;
    };
#pragma unroll 1
    for (int g = 4 * part; g < 4 * part + 4; ++g) {
      tmem_ld_cols<16>(s_at + 16 * g, x);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, score(g, i));
    }
    const float m = fmaxf(r.m, top), by = m == -INFINITY ? 1.f : ex2_approx(r.m - m), base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
    for (int g = 4 * part; g < 4 * part + 4; ++g) {
      tmem_ld_cols<16>(s_at + 16 * g, x);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) l += ex2_approx(score(g, i) + (kWeightLog2 - base));
    }
    r.m = m;
    r.l = fmaf(r.l, by, l);
    // O is there once the other part's next scores are
    const bool begins = part == 0 && !has_o;
    if (!begins) {
      if (!wait(s_full + 1 - part, ns + part)) return false;
      tc_fence_after();
    } else if (lane == 0) {
      *o_set = 1;
    }
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 16) {
      tmem_ld_cols<16>(o_at + c0, x);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = begins ? 0.f : x[i] * by;
      tmem_st_cols16(o_at + c0, x);
    }
    tmem_wait_st();
#pragma unroll 1
    for (int g = 4 * part; g < 4 * part + 4; ++g) add_values<D>(p, s, g, s_at + 16 * g, o_at, nvis, sc, base, r.v_ref);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    tmem_st_cols16(s_at + part * 64, x);
    tmem_st_cols16(s_at + part * 64 + 16, x);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(p_full + part);
  }
  return true;
}

// The same by calls, for 256-row units: what is in line there slows the tiles that do not need it
// (4 x 512 over 32768 1030 us, not 1010; with 128-row units a call does, 16 x 5 75 us, not 72).
template <int D>
__device__ __noinline__ int move_unit_call(uint32_t o_at, int down) {
  return move_unit<D>(o_at, down);
}
template <int D>
__device__ __noinline__ bool any_value_call(const ChunkParams& p, const TileSlot& s, uint32_t groups) {
  return any_value<D>(p, s, groups);
}
template <int D>
__device__ __noinline__ bool apart_tile_call(const ChunkParams& p, const TileSlot& s, uint64_t* s_full, uint64_t* p_full, uint64_t* k_empty,
                                             uint64_t* v_empty, int step, bool has_o, volatile uint32_t* o_set, uint32_t s_at,
                                             uint32_t o_at, int nvis, float sc, int ns, volatile int* abort_flag, RowSums& r) {
  return apart_tile<D, 2>(p, s, s_full, p_full, k_empty, v_empty, step, has_o, o_set, s_at, o_at, nvis, sc, ns, abort_flag, r);
}

// W: units of 128 W rows.
template <int D, int W>
__global__ void __launch_bounds__(CK_THREADS, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
  using C = CkCfg<D, W>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TileSlot* slots = reinterpret_cast<TileSlot*>(smem + C::OFF_SLOT);
  ChunkMap& M = *reinterpret_cast<ChunkMap*>(smem + C::OFF_MAP);
  float4* hand = reinterpret_cast<float4*>(smem + C::OFF_X);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);   // two each: of a row tile, or of a stage
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 4;
  uint64_t* k_full = p_full + 4;
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* slot_full = v_empty + 2;
  uint64_t* slot_empty = slot_full + kSlots;
  uint64_t* seg_full = slot_empty + kSlots;
  uint64_t* handed = seg_full + kSlots;
  uint64_t* q_free = handed + 1;
  uint64_t* mma_done = q_free + 1;
  uint64_t* never = mma_done + 2;   // test hook: nothing arrives
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
  volatile int* nan_seg = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);   // [4]: segment + 1 with NaN values some rows do not see
  // [2]: flags and tiles of a segment, for the MMA issuers: with q_full, and there until
  // both have arrived at q_free (a tile's slot may be filled anew before an issuer that
  // has none of its scores to make comes to it)
  volatile uint2* seg_word = reinterpret_cast<volatile uint2*>(smem + C::OFF_MISC + 32);
  volatile uint32_t* o_set = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 48);   // [2]: O has sums before a half's first products

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int cta = blockIdx.x, G = p.group;

  if (warp == 19) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr((const void*)tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 17 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);   // one arrival per warp
      for (int k = 0; k < 2; ++k) {
        mbar_init(&s_full[2 * i + k], 1);
        mbar_init(&p_full[2 * i + k], 4);
      }
      mbar_init(&k_full[i], 4);
      // an MMA issuer's commit; with 256-row units the softmax warps, of a smaller one four,
      // twice (there the commits cost more than the wait: 4 x 512 over 32768 1112 us, not
      // 1013; here 16 x 5 70 us, not 73)
      mbar_init(&k_empty[i], W == 1 ? 1 : 8);
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], W == 1 ? 1 : 8);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&slot_full[i], 1);
      mbar_init(&slot_empty[i], 12);   // 8 softmax warps, 4 of V's
      mbar_init(&seg_full[i], 1);
    }
    mbar_init(handed, 4);
    mbar_init(q_free, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&mma_done[i], 1);
    }
    mbar_init(never, 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) nan_seg[i] = 0;
    o_set[0] = o_set[1] = 0;
    fence_barrier_init();
  }
  // The launch before is the call's own, of the append and the queries, and itself
  // began behind what came before it: what it does not write is read without a wait,
  // everything but the queries and the pages from the one that the length ends in on.
  // What comes behind is let go where the append is known to be done, so that a launch
  // that reads some of its data early finds that, too.
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
        const UnitMath um(n, count, G, W);
        per = p.whole ? um.units : um.before(um.units);
        all = um.all_tiles() * p.pool.n_kv;
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  CkCut cut;
  const int places = M.start[kMaxPagedSeqs];
  // (where units are cut, a CTA's range holds a tile's first place, so that none between
  // a unit's first and last CTA is left out)
  cut.ctas = min((int)gridDim.x,
                 max(1, p.whole ? places : min(M.tiles / kChunkMinTiles, places / (W == 1 ? 1 : kChunkWidePlaces))));
  cut.base = places / cut.ctas;
  cut.rem = places - cut.base * cut.ctas;
  if (tid == 0) p.desc[cta * 8] = 0;   // no unit to merge, so far

  if (warp >= 16) {
    regs_down<64>();
    if (warp == 16) {
      // ---------------- page ids and scales: lane 8 k + g has group g of the k-th
      // tile of four; the ids of the next four are on their way meanwhile
      const int g = lane & 7;
      CkSeg sg;
      const int x0 = cta < cut.ctas ? cut.first(cta) : places, x1 = cta < cut.ctas ? cut.first(cta + 1) : places;
      int seg = 0, at = lane >> 3, j = lane >> 3;   // tile `at` of segment `seg`, the CTA's j-th
      bool more = ck_seg_at<W>(M, p.batch, G, p.whole, x0, x1, sg);
      int done = 0;   // tiles of the segments before
      struct Ref {
        int32_t id, key0, rows, diag, ctas;   // id: -1 no page here, -2 outside the pool
        int32_t b, h, first, tile, n, seg;
        uint32_t flags;
        bool on;
      };
      auto ask = [&]() {
        Ref r;
        r.id = -1;
        while (more && at - done >= sg.n) {
          done += sg.n;
          ++seg;
          more = ck_next<W>(M, p.batch, G, p.whole, x1, sg);
        }
        r.on = more;
        if (more) {
          const int n = M.n[sg.b], unit = 128 * W, first = sg.i * unit, t = at - done, all = M.count[sg.b] * G;
          const int end = n + min((first + unit - 1) / G + 1, M.count[sg.b]);
          r.b = sg.b;
          r.h = sg.h;
          r.first = first;
          r.tile = sg.t0 + t;
          r.n = sg.n - t;
          r.seg = seg;
          r.key0 = r.tile * CK_KEYS;
          r.rows = min(end - r.key0, CK_KEYS);
          r.diag = n + first / G + 1 - r.key0;
          r.ctas = sg.t0 == 0 && !sg.whole() ? cut.of(sg.place + (sg.tiles - 1) * sg.cost) - cta + 1 : 0;
          const bool ends = sg.t0 + sg.n < sg.tiles || sg.next >= x1;
          r.flags = (r.key0 + r.rows > n / p.pool.page * p.pool.page ? kFresh : 0u) | (sg.whole() ? kWhole : 0u) | (ends ? kEnd : 0u) | (min(all - first, unit) > 128 ? kWide : 0u);
          if (16 * g < r.rows) {
            r.id = p.page_table[(size_t)sg.b * p.max_pages + (r.key0 + 16 * g) / p.pool.page];
            if (r.id < 0) r.id = -2;
          }
        }
        at += 4;
        return r;
      };
      Ref cur = ask();
      if (!__any_sync(0xffffffffu, cur.on)) {
        if (lane == 0) {
          slots[0].flags = kNone;
          mbar_arrive(&seg_full[0]);
          mbar_arrive(&slot_full[0]);
        }
      }
      while (__any_sync(0xffffffffu, cur.on)) {
        const Ref nxt = ask();
        if (cur.id >= p.pool.n_pages) cur.id = -2;
        float ks = 0.f, vs = 0.f;
        const size_t block = cur.id >= 0 ? (size_t)cur.id * p.pool.n_kv + cur.h : 0;
        const size_t row = block * p.pool.page + (cur.key0 + 16 * g) % p.pool.page;
        if (__any_sync(0xffffffffu, cur.on && (cur.flags & kFresh))) grid_wait();
        if (cur.id >= 0) {
          ks = p.pool.scales[0][block];
          vs = p.pool.scales[1][block];
          // the codes to L2, some tiles before the warps that read them
          prefetch_l2(p.pool.codes[0] + row * D, 16 * D);
          prefetch_l2(p.pool.codes[1] + row * D, 16 * D);
        }
        if (cur.id == -2) atomicOr(p.err, kErrLength);
        TileSlot& s = slots[j % kSlots];
        const bool ok = !cur.on || j < kSlots || ck_wait(&slot_empty[j % kSlots], ((j / kSlots) - 1) & 1, abort_flag, p.err);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (cur.on && g == 0) {
          s.rows = cur.rows;
          s.diag = cur.diag;
          s.flags = cur.flags;
          s.seg = cur.seg;
          s.b = cur.b;
          s.h = cur.h;
          s.first = cur.first;
          s.tile = cur.tile;
          s.n = cur.n;
          s.ctas = cur.ctas;
          mbar_arrive(&seg_full[j % kSlots]);
        }
        const int ke = cur.id >= 0 ? exponent_of_scale(ks) : kNoScale, ve = cur.id >= 0 ? exponent_of_scale(vs) : kNoScale;
        int km = ke, vm = ve;
        uint32_t bad = cur.id == -2 ? 1u << g : 0;
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) {
          km = max(km, __shfl_xor_sync(0xffffffffu, km, off));
          vm = max(vm, __shfl_xor_sync(0xffffffffu, vm, off));
          bad |= __shfl_xor_sync(0xffffffffu, bad, off);
        }
        const bool k_far = cur.id >= 0 && ke - km < -kMostBelow;
        const bool v_far = cur.id >= 0 && ve - vm < -kMostBelow;
        bad |= (__ballot_sync(0xffffffffu, k_far) >> (lane & 24) & 0xFFu) << 8;
        bad |= (__ballot_sync(0xffffffffu, v_far) >> (lane & 24) & 0xFFu) << 16;
        if (cur.on) {
          s.grp[g] = cur.id >= 0 ? (int32_t)(row >> 4) : -1;
          const float kf = k_far ? 1.f : pow2_float(max(ke - km, -126)), vf = pow2_float(max(ve - vm, -126));
          s.kf[g] = f16x2(kf, kf);
          s.vf[g] = f16x2(vf, vf);
          s.v_of[g] = ve;
          s.k_by[g] = k_far ? pow2_float(max(ke - km, -126)) : 1.f;
          if (g == 0) {
            s.k_scale = km == kNoScale ? 1.f : pow2_float(km);
            s.v_exp = vm;
            s.bad = bad;
          }
        }
        __syncwarp();
        if (cur.on && g == 0) mbar_arrive(&slot_full[j % kSlots]);
        cur = nxt;
        j += 4;
      }
    } else if (warp < 19 && lane == 0) {
      // ---------------- MMA issuers, one to each half of the softmax: a few MMAs fill
      // the tensor core's queue, so that a single issuer's waits were time that it stood
      // still.  A wide unit has two row tiles, one to an issuer.  A narrow one has a
      // single row tile: one issuer has its even key tiles, the other the odd ones, each
      // with sums of its own.  Scores are made 64 keys at a time, the two parts of a tile
      // by turns, so that a part's scores are there while the softmax works on the other
      // (tensor memory holds no second set of 128; N = 64 costs the scores half again as
      // much: at 128 bytes of shared memory a cycle Q's operand is what bounds them).
      constexpr uint32_t idesc_qk = idesc_f16_m128(64, false);   // B = K (K-major)
      constexpr uint32_t idesc_pv = idesc_f16_m128(D, true);          // B = V (MN-major)
      const int m = warp - 17;
      const uint32_t base = smem_addr(smem), o_col = tmem + C::TMEM_O + m * 128;
      const uint64_t q_desc = sw128_desc(base + C::OFF_Q, 16, 1024), k_desc = sw128_desc(base + C::OFF_K, 16, 1024),
                     v_desc = sw128_desc(base + C::OFF_V, 16384, 1024);
      auto wait = [&](uint64_t* bar, uint32_t parity) { return ck_wait(bar, parity, abort_flag, p.err); };
      bool ok = true;
      int np = 0;   // tiles whose weights were seen
      for (int j = 0, seg = 0; ok; ++seg) {
        ok = wait(&q_full[0], seg & 1) && wait(&q_full[1], seg & 1);
        if (!ok) break;
        const uint32_t flags = seg_word[seg & 1].x;
        if (flags & kNone) break;
        const int n = (int)seg_word[seg & 1].y, wide = W == 2 && (flags & kWide) ? 1 : 0, step = 2 - wide, t0 = wide ? 0 : m;
        const uint64_t q = q_desc + (uint32_t)(wide ? m : 0) * (C::TILE >> 4);
        if (t0 >= n) mbar_arrive(q_free);
        // P V of a part of tile t, then the same part's scores of the next, which take
        // the weights' place
#pragma unroll 1
        for (int t = t0 - step; ok && t < n; t += step) {
          const int jt = j + t, tn = t + step, jn = j + tn;
          const uint64_t v = v_desc + (uint32_t)(jt & 1) * (C::TILE >> 4), k = k_desc + (uint32_t)(jn & 1) * (C::TILE >> 4);
          if (t >= t0) ok = wait(&v_full[jt & 1], (jt >> 1) & 1);
#pragma unroll 1
          for (int part = 0; ok && part < 2; ++part) {
            const uint32_t s_col = tmem + m * 128 + part * 64;
            if (t >= t0) {
              ok = wait(&p_full[2 * m + part], np & 1);
              if (!ok) break;
              tc_fence_after();
              uint32_t onto = t > t0 || part > 0 ? 1 : 0;
              if (!onto) {
                onto = o_set[m];
                o_set[m] = 0;
              }
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16_tmem_a(o_col, s_col + kk * 8, v + (uint32_t)(4 * part + kk) * (2048 >> 4), idesc_pv, kk > 0 ? 1u : onto);
              // the next tile of this half takes the same stage
              if (W == 1 && part == 1) mma_commit(&v_empty[jt & 1]);
            }
            // (the products above do not wait for the next keys)
            if (tn < n && part == 0) ok = wait(&k_full[jn & 1], (jn >> 1) & 1);
            if (!ok) break;
            if (tn < n) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk / 4) * (16384 >> 4) + (kk % 4) * 2;
                mma_bf16(s_col, q + off, k + off + (uint32_t)part * (8192 >> 4), idesc_qk, kk > 0 ? 1u : 0u);
              }
            }
            if (tn < n || t >= t0) mma_commit(&s_full[2 * m + part]);
            if (W == 1 && tn < n && part == 1) mma_commit(&k_empty[jn & 1]);
          }
          if (t >= t0) ++np;
          if (tn < n && tn + step >= n) mma_commit(q_free);
        }
        j += n;
        if (flags & kEnd) break;
      }
      // every MMA issued above must complete before TMEM is released
      mma_commit(&mma_done[m]);
      mbar_wait(&mma_done[m], 0);
    }
  } else if (warp >= 8) {
    regs_down<64>();
    // ---------------- codes to fp16, warps 8-11 of K, 12-15 of V: a thread has 16
    // codes of a row, 8 (at head_dim 64, 4) times a tile; the next tile's are asked
    // for as soon as the registers are free.  Eight neighbouring lanes have two rows'
    // neighbouring chunks: their stores meet all banks.
    const int kv = (warp - 8) >> 2;
    constexpr int LPR = D / 16, RPP = 128 / LPR, NP = 128 / RPP;   // lanes of a row, rows at a time, times
    const int c = D == 128 ? (lane & 3) + (lane >> 1 & 4) : lane & 3;
    const int r0 = D == 128 ? (lane >> 2 & 1) + (lane >> 3 & 2) + (warp & 3) * 4 : (lane >> 2) + (warp & 3) * 8;
    // a chunk's two 16-byte units of the row in fp16; rows of a thread are a multiple of 8 apart
    const int u0 = 2 * (c & 3);
    const uint32_t at0 = (uint32_t)(c >> 2) * 16384 + r0 * 128 + ((u0 ^ (r0 & 7)) << 4);
    const uint32_t at1 = (uint32_t)(c >> 2) * 16384 + r0 * 128 + (((u0 + 1) ^ (r0 & 7)) << 4);
    const uint8_t* codes = p.pool.codes[kv] + (r0 & 15) * D + c * 16;
    uint64_t* full = kv == 0 ? k_full : v_full;
    uint64_t* empty = kv == 0 ? k_empty : v_empty;
    uint8_t* ring = smem + (kv == 0 ? C::OFF_K : C::OFF_V);
    uint4 u[NP];
    bool ok = true;
    auto ask = [&](int j) {
      ok = ck_wait(&slot_full[j % kSlots], (j / kSlots) & 1, abort_flag, p.err);
      if (!__all_sync(0xffffffffu, ok)) return false;
      const TileSlot& s = slots[j % kSlots];
      const int rows = (s.flags & kNone) ? 0 : s.rows;
      if (s.flags & kFresh) grid_wait();
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int row = k * RPP + r0, grp = s.grp[row >> 4];
        u[k] = load_codes(codes + (int64_t)grp * (16 * D), grp >= 0 && row < rows);
      }
      return true;
    };
    if (ask(0)) {
      for (int j = 0;; ++j) {
        const TileSlot& s = slots[j % kSlots];
        const bool last = (s.flags & kEnd) && s.n == 1;
        if (s.flags & kNone) break;
        if (kv == 1 && s.diag < CK_KEYS) {
          // a NaN that some rows of the unit do not see must not reach them: see the epilogue
          bool nan = false;
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t is = k * RPP + r0 < s.diag ? 0 : __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              nan |= is != 0;
              w[i] &= ~is;
            }
            u[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (nan) nan_seg[s.seg & 3] = s.seg + 1;
        }
        if (j >= 2) ok = ck_wait(&empty[j & 1], ((j >> 1) - 1) & 1, abort_flag, p.err);
        if (!__all_sync(0xffffffffu, ok)) break;
        uint8_t* tile = ring + (j & 1) * C::TILE;
        const uint32_t* factors = kv == 0 ? s.kf : s.vf;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w}, f = factors[(k * RPP + r0) >> 4];
          uint32_t h[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[2 * i] = mul_f16x2(f16x2_of_codes(w[i]), f);
            h[2 * i + 1] = mul_f16x2(f16x2_of_codes(w[i] >> 16), f);
          }
          *reinterpret_cast<uint4*>(tile + at0 + k * RPP * 128) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(tile + at1 + k * RPP * 128) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[j & 1]);
          if (kv == 1) mbar_arrive(&slot_empty[j % kSlots]);
        }
        if (last || !ask(j + 1)) break;
      }
    }
  } else {
    regs_up<144>();
    // ---------------- softmax and epilogue: row `row` of the unit
    const int m = warp >> 2;                      // row tile, or parity of the key tiles
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_base + m * 128, o_at = lane_base + C::TMEM_O + m * 128;
    int ns = 0;                                   // phases of s_full so far: a tile each, and one for a segment's end
    int hands = 0;                                // narrow segments that both halves had tiles of
    bool ok = true;
    struct Seg {
      uint32_t flags;
      int b, h, first, t0, tiles, rows;
    } sg;
    float qs = 0.f, qs_next = 0.f;   // the row's power of two
    // The thread's row of the unit.  Up to 64 rows stand twice in a tile, the second
    // half works on the second 64 lanes: on other parts of the SM than the first (16 x 5
    // 67 us, not 70).
    auto row_of = [&](bool wide, bool twice) { return wide ? tid : twice ? (tid & 127) - 64 * m : tid & 127; };
    int j = 0, seg = 0;
    // The segment that begins with tile j, and its queries, as the launch before left them.
    auto take = [&]() -> bool {
      if (!__all_sync(0xffffffffu, ck_wait(&seg_full[j % kSlots], (j / kSlots) & 1, abort_flag, p.err))) return false;
      const TileSlot& s = slots[j % kSlots];
      sg.flags = s.flags;
      if (sg.flags & kNone) return true;
      sg.b = s.b;
      sg.h = s.h;
      sg.first = s.first;
      sg.t0 = s.tile;
      sg.tiles = s.n;
      sg.rows = min(M.count[sg.b] * G - sg.first, 128 * W);   // of the unit
      if (tid == 0 && s.ctas > 0) {
        // this CTA has the unit's first tile: it says who has the others
        int32_t* d = p.desc + cta * 8;
        d[1] = sg.b;
        d[2] = sg.h;
        d[3] = sg.first;
        d[4] = s.ctas;
        d[0] = sg.rows;
      }
      return true;
    };
    // The segment's queries are asked for ...
    auto ask_queries = [&](int before) -> bool {   // `before`: segments whose queries these take the place of
      if (before > 0 && !__all_sync(0xffffffffu, ck_wait(q_free, (before - 1) & 1, abort_flag, p.err))) return false;
      const bool wide = W == 2 && (sg.flags & kWide), twice = W == 1 && sg.rows <= 64;
      // rows behind the last one are left as they are: what comes of them is not used
      const int begin = (wide ? m * 128 : twice ? 0 : m * 64) + (warp & 3) * (wide ? 32 : 16), row = row_of(wide, twice);
      grid_wait();
      ck_copy_queries<D>(p, smem_addr(smem + C::OFF_Q), sg.b, sg.h, sg.first, begin, min(sg.rows, begin + (wide ? 32 : 16)),
                         twice ? m * 64 : 0);
      qs_next = (uint32_t)row < (uint32_t)sg.rows ? p.q_scale[((size_t)sg.b * p.pool.n_kv + sg.h) * p.t_len * G + sg.first + row] : 0.f;
      return true;
    };
    // ... and are there.
    auto queries_here = [&](int of) {   // `of`: the segment
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async();
      __syncwarp();
      if (tid == 0) {
        seg_word[of & 1].x = sg.flags;
        seg_word[of & 1].y = (uint32_t)sg.tiles;
      }
      if (lane == 0) mbar_arrive(&q_full[m]);
    };
    sg.flags = 0;
    sg.tiles = 0;
    ok = take();
    if (ok && !(sg.flags & kNone)) ok = ask_queries(0);
    if (ok) queries_here(0);
    if (sg.flags & kNone) ok = false;
    if (ok && p.inject_timeout && (cta & 1) == 0) {
      ok = mbar_wait(never, 0, kInjectWaitCycles);
      *abort_flag = 1;
      if (tid == 0) atomicOr(p.err, kErrTimeout);
    }
    for (; ok; ++seg) {
      const bool wide = W == 2 && (sg.flags & kWide), twice = W == 1 && sg.rows <= 64;
      const int t0 = sg.t0, tiles = sg.tiles;
      const int row = row_of(wide, twice);
      const bool live = (uint32_t)row < (uint32_t)sg.rows;
      const bool warp_live = (uint32_t)(row & ~31) < (uint32_t)sg.rows;
      const int lim = M.n[sg.b] + (sg.first + row) / G + 1;   // keys that the row sees
      qs = qs_next;
      float m_run = -INFINITY, l_run = 0.f;
      int v_ref = kNoScale;
      const int step = wide ? 1 : 2;
      for (int t = 0; t < tiles; ++t, ++j) {
        if (!wide && (t & 1) != m) {   // the other half's: only let it go
          ok = __all_sync(0xffffffffu, ck_wait(&seg_full[j % kSlots], (j / kSlots) & 1, abort_flag, p.err));
          if (!ok) break;
          if (lane == 0) mbar_arrive(&slot_empty[j % kSlots]);
          continue;
        }
        float sc = 0.f;
        uint32_t bad = 0;
        int nvis = 0, v_by = 0;   // 2^v_by: the tile's V scale over the unit of the row's O
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          ok = __all_sync(0xffffffffu, ck_wait(&s_full[2 * m + part], ns & 1, abort_flag, p.err));
          if (!ok) break;
          // The products behind these scores have read K, those before them V.  (Before
          // the wait below: the other part's next scores may need these stages.)
          if (W == 2 && lane == 0 && part == 1) {
            mbar_arrive_n(&k_empty[j & 1], step);
            if (t >= step) mbar_arrive_n(&v_empty[(j - step) & 1], step);
          }
          if (warp_live) {
            tc_fence_after();
            // The row's maximum may lag behind by kRescaleLog2; where it is further
            // behind (seldom), the sum and O are brought down.  The weights take the
            // place of the scores.  (The loop is rolled: unrolled code did not stay in
            // the instruction cache.)
            if (part == 0) {
              const TileSlot& ts = slots[j % kSlots];
              nvis = live ? lim - (t0 + t) * CK_KEYS : 0;
              sc = qs * ts.k_scale;   // in range, so that a masked score stays -inf; NaN stays
              sc = sc < FLT_MIN ? FLT_MIN : sc > FLT_MAX ? FLT_MAX : sc;
              bad = ts.bad;
              // The weights hold the tile's V scale over 2^v_ref, the unit of the row's O.  Where
              // the scale is far below it, O is brought to a smaller unit first (as far as
              // its largest element stays in range), so that these weights keep their bits; where it
              // is above, the unit is raised below, by as much as the row's weights need, or far above, here,
              // by as much as leaves all of O in range.  So a large scale costs a row nothing that gives
              // its page no weight.
              const int v_exp = ts.v_exp;
              bool apart = bad >> 16 && (W == 1 ? any_value<D>(p, ts, bad >> 16) : any_value_call<D>(p, ts, bad >> 16));   // (seldom)
              if (!apart) {
                if (v_ref == kNoScale) v_ref = v_exp;
                v_by = v_exp == kNoScale ? 0 : v_exp - v_ref;
                if (__any_sync(0xffffffffu, (uint32_t)(v_by + kUnitAbove) > (uint32_t)(kUnitAbove + kUnitBelow))) {
                  ok = __all_sync(0xffffffffu, ck_wait(&s_full[2 * m + 1], ns & 1, abort_flag, p.err));   // O is there
                  if (!ok) break;
                  tc_fence_after();
                  const int by = v_by < -kUnitAbove || v_by > kUnitBelow ? -v_by : 0;
                  const int down = W == 1 ? move_unit<D>(o_at, by) : move_unit_call<D>(o_at, by);
                  v_ref -= down;
                  v_by += down;
                  // (O has no room to be moved so far)
                  apart = __any_sync(0xffffffffu, (uint32_t)(v_by + kUnitAbove) > (uint32_t)(kUnitAbove + kUnitBelow));
                }
              }
              if (apart) {
                RowSums sums = {m_run, l_run, v_ref};
                auto* tile = W == 1 ? apart_tile<D, 1> : apart_tile_call<D>;
                ok = tile(p, ts, s_full + 2 * m, p_full + 2 * m, &k_empty[j & 1], &v_empty[(j - step) & 1], step, t >= step, o_set + m, s_at, o_at,
                          nvis, sc, ns, abort_flag, sums);
                m_run = sums.m;
                l_run = sums.l;
                v_ref = sums.v_ref;
                break;
              }
            }
            float x[2][32];
            tmem_ld32(s_at + part * 64, x[0]);
            tmem_ld32(s_at + part * 64 + 32, x[1]);
            float alpha = 1.f;   // what O is multiplied by
            tmem_wait_ld();
            if (nvis < CK_KEYS || bad) {
              if (bad >> 8 & 0xFFu) {   // pages whose K scales are far below the tile's (seldom)
#pragma unroll
                for (int i = 0; i < 64; ++i) x[i / 32][i % 32] *= slots[j % kSlots].k_by[4 * part + i / 16];
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int i1 = 64 * part + 32 * k, left = nvis - i1;
                uint32_t vis = left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1;
                if (bad >> (i1 >> 4) & 1) vis &= 0xFFFF0000u;
                if (bad >> (i1 >> 4) & 2) vis &= 0x0000FFFFu;
#pragma unroll
                for (int i = 0; i < 32; ++i) x[k][i] = (vis >> i & 1) ? x[k][i] : -INFINITY;
              }
            }
            // The weights are computed from the maximum so far while these scores' is
            // found, and once more where it is too far above.
            float w[32];
            float2 l4[4];
            const float2 sc2 = make_float2(sc, sc);
#pragma unroll 1
            for (;;) {
              const float mu = kWeightLog2 + (float)max(v_by, -60) - (m_run == -INFINITY ? 0.f : m_run);
              const float2 mu2 = make_float2(mu, mu);
              float tops[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                l4[i] = make_float2(0.f, 0.f);
                tops[i] = -INFINITY;
              }
#pragma unroll
              for (int i = 0; i < 64; i += 2) {
                const float a = x[i / 32][i % 32], b = x[i / 32][i % 32 + 1];
                tops[i / 2 % 4] = fmaxf(tops[i / 2 % 4], fmaxf(a, b));
                float2 e = fma2(make_float2(a, b), sc2, mu2);
                e.x = ex2_approx(e.x);
                e.y = ex2_approx(e.y);
                l4[i / 2 % 4] = add2(l4[i / 2 % 4], e);
                w[i / 2] = __uint_as_float(f16x2(e.x, e.y));
              }
              const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
              // (a weight is at most 2^(kWeightLog2 + kRescaleLog2), with the V scale in it, too)
              const bool up = top != -INFINITY && top * sc > m_run + (kRescaleLog2 - (float)max(v_by, 0));
              if (!__any_sync(0xffffffffu, up)) break;
              if (up) {
                if (top * sc > m_run + kRescaleLog2) {
                  const float by = ex2_approx(m_run - top * sc);   // 0 for the first scores of a row
                  m_run = top * sc;
                  alpha *= by;
                  l_run *= by;
                }
                const int room = (int)fmaxf(floorf(m_run - top * sc), 0.f);   // NaN: 0
                if (v_by > room) {
                  v_ref += v_by - room;
                  alpha *= v_by - room > 126 ? 0.f : pow2_float(room - v_by);
                  v_by = room;
                }
              }
            }
            if ((t >= step || part == 1) && __any_sync(0xffffffffu, alpha != 1.f)) {
              // what was added to O is there once the other part's next scores are
              ok = __all_sync(0xffffffffu, ck_wait(&s_full[2 * m + 1 - part], (ns + part) & 1, abort_flag, p.err));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 16) {
                float o[16];
                tmem_ld_cols<16>(o_at + c0, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= alpha;
                tmem_st_cols16(o_at + c0, o);
              }
            }
            tmem_st32(s_at + part * 64, w);
            const float2 l2 = add2(add2(l4[0], l4[1]), add2(l4[2], l4[3]));
            l_run = fmaf(l2.x + l2.y, pow2_float(min(max(-v_by, -126), 60)), l_run);
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * m + part]);
        }
        if (!ok) break;
        ++ns;
        if (lane == 0) mbar_arrive(&slot_empty[j % kSlots]);
      }
      if (!ok) break;
      // ---- epilogue
      // The next segment's queries are copied while the last products are made.
      const Seg was = sg;
      const bool ends = was.flags & kEnd;
      if (!ends) {
        ok = take() && ask_queries(seg + 1);
        if (!ok) break;
      }
      const bool mine = wide || m == 0 || tiles > 1;   // this half had a tile
      if (mine) {
        ok = __all_sync(0xffffffffu, ck_wait(&s_full[2 * m + 1], ns & 1, abort_flag, p.err));
        if (!ok) break;
        ++ns;
        // this half's last tile: j - 1, or the one before it
        if (W == 2 && lane == 0) mbar_arrive_n(&v_empty[(j - 1 - (wide || ((tiles - 1) & 1) == m ? 0 : 1)) & 1], step);
      }
      const bool two = !wide && tiles > 1;   // a narrow unit's halves are added up by the first
      float4 other = make_float4(-INFINITY, 0.f, (float)kNoScale, 0.f);   // m, l, v_ref of the second half
      float4* hand_o = reinterpret_cast<float4*>(smem + C::OFF_HO);
      if (two && m == 1) {
        // its sums are complete; the first half cannot read tensor memory of other lanes
        if (twice && warp_live) {
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            float o[16];
            tmem_ld_cols<16>(o_at + c0, o);
            tmem_wait_ld();
            if (live) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) hand_o[(c0 + i) / 4 * 64 + row] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
        }
        tc_fence_before();
        if (live) hand[row] = make_float4(m_run, l_run, (float)v_ref, 0.f);
        __syncwarp();
        if (lane == 0) mbar_arrive(handed);
      }
      if (two && m == 0) {
        ok = __all_sync(0xffffffffu, ck_wait(handed, hands++ & 1, abort_flag, p.err));
        if (!ok) break;
        if (live) other = hand[row];
      }
      // The next scores are made meanwhile; but not while the first half still reads the
      // second half's sums.
      if (!ends && !two) queries_here(seg + 1);
      if (warp_live && (wide || m == 0)) {
        tc_fence_after();
        const bool whole = was.flags & kWhole;
        const int n = M.n[was.b];
        const bool nan = nan_seg[seg & 3] == seg + 1;
        // A part's O is divided by its own sum, too: what is stored is a mean of values, and
        // in range as they are.  Its unit 2^v_ref is multiplied in where that stays in range.
        float f = 1.f, f1 = 0.f, g = 1.f, g1 = 1.f;
        int unit = v_ref;
        if (two) {   // O's common unit: the larger of the halves', with the weight that each has
          const float top = fmaxf(m_run, other.x), base = top == -INFINITY ? 0.f : top;
          const float a = m_run - base, a1 = other.x - base;
          const float top_unit = ceilf(fmaxf((float)v_ref + a, other.z + a1));
          unit = (int)fminf(fmaxf(top_unit, -120.f), 120.f);
          const float d = (float)(v_ref - unit) + a, d1 = other.z - (float)unit + a1;
          f = ex2_approx(fmaxf(d, -100.f));
          g = ex2_approx(fminf(d + 100.f, 0.f));   // (far below the other, and still all that some columns have)
          f1 = ex2_approx(fmaxf(d1, -100.f));
          g1 = ex2_approx(fminf(d1 + 100.f, 0.f));
          l_run = l_run * ex2_approx(a) + other.y * ex2_approx(a1);
          m_run = top;
        }
        if (unit == kNoScale) unit = 0;
        const int near = min(max(unit, -64), 64);
        const float inv = l_run == 0.f ? 0.f : pow2_float(near) / l_run, rest = pow2_float(unit - near);
        const bool far = __any_sync(0xffffffffu, unit != near || g * g1 != 1.f);
        f *= inv;
        f1 *= inv;
        const int t_of = (was.first + row) / G;
        const uint32_t to = live ? (uint32_t)((was.b * p.t_len + t_of) * p.n_q + was.h * G + was.first + row - t_of * G) : ~0u;   // row of out
        const int slot = 2 * cta + (t0 == 0 ? 1 : 0);   // of a unit's first part: see the merge
        if (!whole && live) p.part_ml[(size_t)slot * p.part_rows + row] = make_float2(m_run, l_run);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
          tmem_ld32(o_at + c0, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= f;
          if (far) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= g;
          }
          if (two && !twice) {
            float y[32];
            tmem_ld32(o_at + 128 + c0, y);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(y[i] * g1, f1, o[i]);
          }
          if (live && two && twice) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float4 y = hand_o[(c0 + i) / 4 * 64 + row];
              if (far) y.x *= g1, y.y *= g1, y.z *= g1, y.w *= g1;
              o[i] = fmaf(y.x, f1, o[i]);
              o[i + 1] = fmaf(y.y, f1, o[i + 1]);
              o[i + 2] = fmaf(y.z, f1, o[i + 2]);
              o[i + 3] = fmaf(y.w, f1, o[i + 3]);
            }
          }
          if (far) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= rest;
          }
          if (live && nan) {   // values that are not numbers, for the rows that see them
            const int end = min(lim, (t0 + tiles) * CK_KEYS);
            for (int key = max(n + was.first / G + 1, t0 * CK_KEYS); key < end; ++key) {
              const int id = p.page_table[(size_t)was.b * p.max_pages + key / p.pool.page];
              if (id < 0 || id >= p.pool.n_pages) continue;
              const uint8_t* v =
                  p.pool.codes[1] + (((size_t)id * p.pool.n_kv + was.h) * p.pool.page + key % p.pool.page) * D + c0;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((v[i] & 0x7F) == 0x7F) o[i] = __uint_as_float(0x7FFFFFFFu);
            }
          }
          if (whole) {
            uint4 out[4];
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              const float e[8] = {o[i], o[i + 1], o[i + 2], o[i + 3], o[i + 4], o[i + 5], o[i + 6], o[i + 7]};
              out[i / 8] = pack8(e);
            }
            // four lanes have a row's 64 bytes, and so whole sectors: a lane's own row is
            // 16 bytes of 32 lines a store (a unit of 256 rows then took 2 us longer)
            transpose4(out);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t at = __shfl_sync(0xffffffffu, to, (lane & ~3) + k);
              if (at != ~0u) reinterpret_cast<uint4*>(p.out)[(size_t)at * (D / 8) + c0 / 8 + (lane & 3)] = out[k];
            }
          } else if (live) {
            float4* dst = p.part_o + ((size_t)slot * (D / 4) + c0 / 4) * p.part_rows + row;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              dst[(size_t)(i / 4) * p.part_rows] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        tc_fence_before();
      }
      if (ends) break;
      if (two) queries_here(seg + 1);
    }
  }
  grid_wait();   // the launch completes only behind the append
  grid_release();
  tc_fence_before();
  __syncthreads();
  if (warp == 19) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the parts of the units that several CTAs hold.  blockIdx.x: the CTA with
// the unit's first tile (its part is slot 2 c + 1, those of the CTAs behind it slot
// 2 c'); blockIdx.y: 32 rows, blockIdx.z: 32 columns; a lane to a row, a warp to four
// columns.
// Bound by the parts' bytes (1 x 4000 tokens 34 MB: 22 us from memory, less where they
// are in L2) and, where they are few, by its launch and two dependent reads (5 us).
constexpr int MG_THREADS = 256;
template <int D>
__global__ void __launch_bounds__(MG_THREADS) merge_kernel(const __grid_constant__ ChunkParams p) {
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
  const int c4 = blockIdx.z * 8 + warp;
  auto part = [&](int k) { return live ? p.part_o[(slot(k) * (D / 4) + c4) * p.part_rows + row] : make_float4(0.f, 0.f, 0.f, 0.f); };
  constexpr int AHEAD = 8;   // parts whose loads are in flight, the first since before the weights
  float4 v[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (i < parts) v[i] = part(i);
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
    const float w = ex2_approx(wts[k][lane] - base) * (live ? p.part_ml[slot(k) * p.part_rows + row].y : 0.f);
    wts[k][lane] = w;
    l += w;
  }
  red[warp][lane] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) l += red[i][lane];
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k0 = 0; k0 < parts; k0 += AHEAD) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (k0 + i >= parts) break;
      const float w = wts[k0 + i][lane] * inv;
      acc.x = fmaf(w, v[i].x, acc.x);
      acc.y = fmaf(w, v[i].y, acc.y);
      acc.z = fmaf(w, v[i].z, acc.z);
      acc.w = fmaf(w, v[i].w, acc.w);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (k0 + AHEAD + i < parts) v[i] = part(k0 + AHEAD + i);
  }
  if (!live) return;
  uint2* dst = reinterpret_cast<uint2*>(p.out + (((size_t)b * p.t_len + rq / G) * p.n_q + h * G + rq % G) * D) + c4;
  *dst = make_uint2(pack2(acc.x, acc.y), pack2(acc.z, acc.w));
}

template <int D, int W>
cudaError_t launch_chunk(const ChunkParams& p, int sms, cudaStream_t st) {
  using C = CkCfg<D, W>;
  static KernelSetup s;
  const int dev = setup_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(s.mu);
    if (s.state[dev] == 0) {
      const cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
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
  return cudaLaunchKernelEx(&cfg, chunk_kernel<D, W>, p);
}

template <int D>
cudaError_t launch_merge(const ChunkParams& p, int sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms, p.part_rows / 32, D / 32);
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

// 128-row tiles of a unit: one where that leaves each CTA few tiles (a part's sums are
// half as much to store and to join, which then is much of the time), else two, whose
// rows share the work of bringing the codes to fp16.  3 x 333 tokens over 100 to 4999 rows,
// 10 tiles of 256 rows to a CTA: 29 us by 128 rows, 32 by 256; 16 x 64 over 4000, 27 tiles:
// 122 and 113 us.
int chunk_wide(int batch, int n_kv, int t_len, int group, int max_keys, int ctas) {
  const int64_t rows = (int64_t)t_len * group;
  if (rows <= 128) return 1;
  const int64_t tiles = batch * (int64_t)n_kv * ((rows + 255) / 256) * ((max_keys + CK_KEYS - 1) / CK_KEYS);
  return tiles < (int64_t)kChunkFewTiles * ctas ? 1 : 2;
}

// Whether units are left whole: the call then has no third launch, and no CTA a second
// end.  In tiles, of the longest CTA: its units one after another, against an even
// share, another end and what the third launch takes (kChunkMergeTiles).  Whole and cut,
// in us, 32 query heads over 8: 8 x 128 tokens over 4000 rows 90 and 108, 4 x 200 over 4000
// 88 and 95, 16 x 30 over 1000 31 and 42, 4 x 33 over 1800 41 and 35, 2 x 100 over 900 31
// and 30.  (All units count as long as max_keys allows, so lengths that differ mislead it: 32 x 5
// over 100 to 2000 70 and 62; 152 units, 19 x 5, are whole at any max_keys, and with one sequence of
// 32768 rows and the others of 500 that is 359 us, where 16 x 5 of such lengths, cut, are 56.)
// Units of few tiles are whole in any case: 8 x 4 over 300 rows, head_dim 64, 15.2 and 19.4, 3 x 100
// over 400 17.7 and 19.4, 2 x 30 over 480 of llama8b's heads 22.3 and 23.5, 16 x 8 over 400 23.1
// and 23.2, but 4 x 4 over 500 22.7 and 21.7, 1 x 5 over 500 of qwen14b's 22.2 and 20.9.
bool chunk_whole(int batch, int n_kv, int t_len, int group, int max_keys, int wide, int ctas) {
  if (max_keys <= kChunkWholeKeys) return true;
  const int64_t units = batch * (int64_t)n_kv * (((int64_t)t_len * group + 128 * wide - 1) / (128 * wide));
  const int64_t tiles = (max_keys + CK_KEYS - 1) / CK_KEYS + kChunkUnitTiles;
  const int64_t each = (units + ctas - 1) / ctas;
  return each * tiles * ctas <= units * tiles + std::min<int64_t>(units, ctas) * kChunkUnitTiles + ctas * (int64_t)kChunkMergeTiles;
}

int chunk_part_rows(int t_len, int group, int wide) {
  return (int)std::min<int64_t>(128 * wide, ((int64_t)t_len * group + 31) / 32 * 32);
}

int64_t chunk_places(int batch, int n_kv, int t_len, int group, int max_keys, int wide) {
  const int64_t units = ((int64_t)t_len * group + 128 * wide - 1) / (128 * wide);
  return batch * (int64_t)n_kv * units * ((max_keys + CK_KEYS - 1) / CK_KEYS + kChunkUnitTiles) * (wide == 1 ? 1 : kChunkWidePlaces);
}

cudaError_t launch_attend_chunk8(const ChunkParams& p, int head_dim, int sms, cudaStream_t st) {
  if (p.wide == 2) return head_dim == 128 ? launch_chunk<128, 2>(p, sms, st) : launch_chunk<64, 2>(p, sms, st);
  return head_dim == 128 ? launch_chunk<128, 1>(p, sms, st) : launch_chunk<64, 1>(p, sms, st);
}

cudaError_t launch_attend_chunk8_merge(const ChunkParams& p, int head_dim, int sms, cudaStream_t st) {
  return head_dim == 128 ? launch_merge<128>(p, sms, st) : launch_merge<64>(p, sms, st);
}

}  // namespace c2kv
