// The 8-bit paged cache: device layout, parameters and launchers shared by
// its kernels (pages8.cu, attend_pages8.cu) and entry points (api_pages8.cu).
#pragma once

#include "c2kv_internal.h"

namespace c2kv {

constexpr int kMaxPagedSeqs = 256;      // sequences in one append or attention call over pages
constexpr int kMinScaleExponent = -120;

// Largest magnitude of e4m3 and the smallest exponent e with a <= 448 * 2^e
// (448 = 1.75 * 2^8), for finite a >= 0 given by its fp32 bits.  The clamp
// keeps both 2^e and 2^-e normal fp32 numbers (the largest e is 120).
__device__ __forceinline__ int scale_exponent(uint32_t abs_bits) {
  const int e = (int)(abs_bits >> 23) - 127 - 8 + ((abs_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, kMinScaleExponent);
}

__device__ __forceinline__ float pow2_float(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Exponent of a scale that the library wrote (a power of two).
__device__ __forceinline__ int exponent_of_scale(float s) { return (int)((__float_as_uint(s) >> 23) & 0xFFu) - 127; }

// Two fp32 values -> two e4m3 codes (nearest even), `a` in the low byte; NaN
// becomes the NaN code.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Two e4m3 codes -> fp32 (every e4m3 value is an fp16 value).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// a (bh + bl) + c (dh + dl), one element of a rotated key, rounded to fp32 and
// from there to bf16 (the two roundings of a conversion that goes by way of
// fp32; they differ from a single one in about 2^-17 of elements).  Where the
// fp32 evaluation decides, it is rot_bf16_bits' fast path; the bounds are its.
static __device__ __noinline__ uint32_t rot_key_slow(float a, float bh, float bl, float c, float dh, float dl) {
  float hi, lo;
  dot2_df(a, bh, bl, c, dh, dl, hi, lo);
  return fabsf(hi) < INFINITY ? bf16_bits_rn(hi) : 0x7FFFu;   // beyond fp32's range: NaN
}

__device__ __forceinline__ uint32_t rot_key_bits(float a, float bh, float bl, float c, float dh, float dl) {
  const float p = __fmul_rn(c, dh);
  const float r = fmaf(a, bh, p);
  const float m = __fadd_rn(fabsf(__fmul_rn(a, bh)), fabsf(p));   // 2^21 times the error bound
  const uint32_t bits = __float_as_uint(r);
  const float mid = __uint_as_float((bits & 0xFFFF0000u) | 0x8000u);
  if (__fmul_rn(fabsf(__fsub_rn(r, mid)), 0x1p21f) > m && __fmul_rn(fabsf(r), 0x1p11f) > m) return bf16_bits_rn(r);
  return rot_key_slow(a, bh, bl, c, dh, dl);
}

// Four codes times a power of two, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float by) {
  const float2 a = e4m3x2_to_float2(c & 0xFFFFu), b = e4m3x2_to_float2(c >> 16);
  return e4m3x2(a.x * by, a.y * by) | (e4m3x2(b.x * by, b.y * by) << 16);
}

// One layer's range of a page pool: codes [n_pages][n_kv][page][d] per layer,
// scales [n_pages][n_kv] per layer; index 0 is K, 1 is V.
struct PagePool {
  uint8_t* codes[2];
  float* scales[2];
  int32_t n_pages, page, n_kv;
};

// Writes rows of sequences into their pages (pages8.cu): bf16 cache rows
// (fill) or new tokens (append).
struct PutParams {
  PagePool pool;                 // of the first layer written
  int64_t scale_layer;           // scales from one layer to the next (fill)
  const int32_t* page_table;     // [batch][max_pages]
  int32_t max_pages, batch, n_layers;
  unsigned* err;
  // fill: rows [0, n_rows[b]) of caches [n_layers][n_kv][cap][d]
  const __nv_bfloat16* src[2][kMaxBatch];
  int32_t n_rows[kMaxBatch];
  int32_t cap;
  // append: [batch][t_len][n_kv][d]; token i of sequence b goes to row
  // n_cached[b] + i and is rotated by row rope_row[b] + i of the table
  const __nv_bfloat16* fresh[2];
  const int32_t* n_cached;
  const int32_t* n_new;          // null: t_len each
  const CosSin2* tab;
  const int32_t* rope_row;
  int32_t t_len, table_rows;
};

// One decode step over the pages of `batch` sequences (attend_pages8.cu).
// tm: the layer's K and V codes as rows of 128 bytes (2-D map {128, rows}, one
// page and kv head per box, 128-byte swizzle).
struct AttendPages8Params {
  CUtensorMap tm[2];
  PagePool pool;
  const int32_t* page_table;
  const int32_t* n_cached;
  const __nv_bfloat16* q;        // [batch][n_q][d]
  const __nv_bfloat16* fresh[2]; // [batch][n_kv][d] new k (before RoPE) and v
  const CosSin2* tab;
  const int32_t* rope_row;
  __nv_bfloat16* out;            // [batch][n_q][d]
  float* part_o;                 // [2 * CTAs][G][128] partial O of shared units
  float* part_ml;                // [2 * CTAs][G][2] their (m, l)
  int32_t* counters;             // [batch * n_kv] tiles merged so far per unit
  unsigned* err;
  int32_t batch, n_q, max_pages, max_keys, table_rows, has_new, inject_timeout;
  int32_t row_at_length;         // a sequence's table row is rope_row + its length
  int32_t early;                 // lengths, page table, RoPE rows and held rows may be read before the wait
  float scale_log2;
};
constexpr int kMaxPageCtas = 512;   // CTAs of one launch (at most two per SM)

struct LogprobParams {
  const void* logits;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  unsigned* err;
  int64_t row_stride;
  int32_t rows, vocab, top_k, is_f32;
  int32_t cluster;               // CTAs of a row (set by the launcher)
};

constexpr int kMaxTopK = 64;

// The launches below may be set up while the kernel before them on the stream
// finishes (programmatic dependent launch), which takes about 2 us off a call
// among others.  Each waits for that kernel before it touches global memory,
// unless its caller says what may be read earlier, and lets the next launch be
// set up from then on.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

cudaError_t launch_pages8_fill(const PutParams& p, int head_dim, int max_rows, cudaStream_t st);
cudaError_t launch_pages8_append(const PutParams& p, int head_dim, cudaStream_t st);
cudaError_t launch_attend_pages8(const AttendPages8Params& p, int head_dim, int group, int sms, cudaStream_t st);
cudaError_t launch_token_logprobs(const LogprobParams& p, int sms, cudaStream_t st);

// What the entry points of another translation unit share with api.cu.
c2kv_status api_fail(c2kv_status st, const char* msg);
c2kv_status api_cuda(cudaError_t e, const char* what);
c2kv_status api_launched(cudaError_t e, const char* what);   // counts the launch if it succeeded
c2kv_status api_check_geom(const c2kv_geometry* g);
c2kv_status api_device_state(unsigned** err, int* num_sms);
int api_sm_count_for_sizing();
int api_take_injected_timeout();
// uint8 tensor map {128, rows} of 128-byte rows, box {128, box_rows}, 128-byte swizzle
c2kv_status api_encode_rows128(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows);

}  // namespace c2kv
