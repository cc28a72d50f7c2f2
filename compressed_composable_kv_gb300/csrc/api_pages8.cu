// C ABI of the 8-bit paged cache and of the token log probabilities: argument
// checks on the host, then one launch.  See include/c2kv.h for each call.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "pages8.h"

using namespace c2kv;

namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The pool of one layer, and the checks every call over pages makes.
c2kv_status check_pages(const c2kv_geometry* g, const c2kv_pages8* pages, int32_t layer, const int32_t* page_table,
                        int32_t max_pages, PagePool* out) {
  const c2kv_status s = api_check_geom(g);
  if (s != C2KV_OK) return s;
  if (pages == nullptr) return api_fail(C2KV_EINVAL, "pages is null");
  if (pages->page != 16 && pages->page != 32 && pages->page != 64 && pages->page != 128)
    return api_fail(C2KV_EINVAL, "page must be 16, 32, 64 or 128 tokens");
  // a layer's rows of 128 bytes are counted in 32 bits
  if (pages->n_pages < 1 ||
      (int64_t)pages->n_pages * g->n_kv_heads * pages->page * g->head_dim / 128 > INT32_MAX)
    return api_fail(C2KV_EINVAL, "n_pages must be >= 1 and one layer's codes below 2^38 bytes");
  if (layer < 0 || layer >= g->n_layers) return api_fail(C2KV_EINVAL, "layer out of range");
  if (!pages->k || !pages->v || !pages->k_scale || !pages->v_scale || !page_table)
    return api_fail(C2KV_EINVAL, "a pages pointer or the page table is null");
  if (!aligned(pages->k, 16) || !aligned(pages->v, 16)) return api_fail(C2KV_EINVAL, "pages must be 16-byte aligned");
  if (max_pages < 1 || (int64_t)max_pages * pages->page > INT32_MAX / 2)
    return api_fail(C2KV_EINVAL, "max_pages must be >= 1 and max_pages * page below 2^30");
  const size_t scales = (size_t)pages->n_pages * g->n_kv_heads;
  const size_t codes = scales * pages->page * g->head_dim;
  out->codes[0] = static_cast<uint8_t*>(pages->k) + layer * codes;
  out->codes[1] = static_cast<uint8_t*>(pages->v) + layer * codes;
  out->scales[0] = pages->k_scale + layer * scales;
  out->scales[1] = pages->v_scale + layer * scales;
  out->n_pages = pages->n_pages;
  out->page = pages->page;
  out->n_kv = g->n_kv_heads;
  return C2KV_OK;
}

c2kv_status check_new_tokens(int32_t batch, const int32_t* n_cached_dev, const void* k_new, const void* v_new,
                             const void* rope_table, int32_t table_rows, const int32_t* rope_row_dev) {
  if (batch < 1 || batch > kMaxPagedSeqs) return api_fail(C2KV_EINVAL, "batch must be in [1, 256]");
  if (!n_cached_dev || !rope_table || !rope_row_dev) return api_fail(C2KV_EINVAL, "null pointer");
  if (table_rows < 1) return api_fail(C2KV_EINVAL, "table_rows must be >= 1");
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(rope_table, 16))
    return api_fail(C2KV_EINVAL, "k_new, v_new and rope_table must be 16-byte aligned");
  return C2KV_OK;
}

// Scratch of the attention: arrival counters at offset 0 (sized for the
// largest batch, so that no call's partials overlap counters another call
// relies on being zero), then two partial results per CTA.
struct AttendWs {
  size_t ml_off, o_off, total;
};

AttendWs attend_workspace(const c2kv_geometry* g, int sms) {
  const size_t rows = (size_t)2 * std::min(2 * sms, kMaxPageCtas) * (g->n_q_heads / g->n_kv_heads);
  AttendWs w;
  w.ml_off = up256((size_t)kMaxPagedSeqs * g->n_kv_heads * sizeof(int32_t));
  w.o_off = w.ml_off + up256(rows * 2 * sizeof(float));
  w.total = w.o_off + up256(rows * 128 * sizeof(float));
  return w;
}

}  // namespace

extern "C" {

c2kv_status c2kv_pages8_fill(const c2kv_geometry* geom, const c2kv_pages8* pages, int32_t layer_begin,
                             int32_t layer_end, int32_t batch, void* const* k_caches, void* const* v_caches,
                             int32_t cap, const int32_t* n_rows, const int32_t* page_table, int32_t max_pages,
                             void* stream) {
  PutParams p;
  std::memset(&p, 0, sizeof(p));
  c2kv_status s = check_pages(geom, pages, layer_begin, page_table, max_pages, &p.pool);
  if (s != C2KV_OK) return s;
  if (layer_end <= layer_begin || layer_end > geom->n_layers || layer_end - layer_begin > 32767)
    return api_fail(C2KV_EINVAL, "need 0 <= layer_begin < layer_end <= n_layers");
  if (batch < 1 || batch > kMaxBatch) return api_fail(C2KV_EINVAL, "batch must be in [1, 16]");
  if (!k_caches || !v_caches || !n_rows) return api_fail(C2KV_EINVAL, "null pointer");
  if (cap < 1) return api_fail(C2KV_EINVAL, "cap must be >= 1");
  int most = 0;
  for (int b = 0; b < batch; ++b) {
    if (!k_caches[b] || !v_caches[b]) return api_fail(C2KV_EINVAL, "null cache pointer");
    if (!aligned(k_caches[b], 16) || !aligned(v_caches[b], 16))
      return api_fail(C2KV_EINVAL, "caches must be 16-byte aligned");
    if (n_rows[b] < 0) return api_fail(C2KV_EINVAL, "n_rows must be >= 0");
    if (n_rows[b] > cap) return api_fail(C2KV_ECAPACITY, "n_rows exceeds cap");
    if (n_rows[b] > max_pages * pages->page) return api_fail(C2KV_ECAPACITY, "n_rows exceeds max_pages * page");
    const size_t at = (size_t)layer_begin * geom->n_kv_heads * cap * geom->head_dim;
    p.src[0][b] = static_cast<const __nv_bfloat16*>(k_caches[b]) + at;
    p.src[1][b] = static_cast<const __nv_bfloat16*>(v_caches[b]) + at;
    p.n_rows[b] = n_rows[b];
    most = std::max(most, n_rows[b]);
  }
  if (most == 0) return C2KV_OK;
  s = api_device_state(&p.err, nullptr);
  if (s != C2KV_OK) return s;
  p.scale_layer = (int64_t)pages->n_pages * geom->n_kv_heads;
  p.page_table = page_table;
  p.max_pages = max_pages;
  p.batch = batch;
  p.n_layers = layer_end - layer_begin;
  p.cap = cap;
  return api_launched(launch_pages8_fill(p, geom->head_dim, most, static_cast<cudaStream_t>(stream)),
                      "c2kv_pages8_fill");
}

c2kv_status c2kv_pages8_append(const c2kv_geometry* geom, const c2kv_pages8* pages, int32_t layer, int32_t batch,
                               int32_t t_len, const int32_t* page_table, int32_t max_pages,
                               const int32_t* n_cached_dev, const int32_t* n_new_dev, const void* k_new,
                               const void* v_new, const void* rope_table, int32_t table_rows,
                               const int32_t* rope_row_dev, void* stream) {
  PutParams p;
  std::memset(&p, 0, sizeof(p));
  c2kv_status s = check_pages(geom, pages, layer, page_table, max_pages, &p.pool);
  if (s != C2KV_OK) return s;
  s = check_new_tokens(batch, n_cached_dev, k_new, v_new, rope_table, table_rows, rope_row_dev);
  if (s != C2KV_OK) return s;
  if (!k_new || !v_new) return api_fail(C2KV_EINVAL, "null pointer");
  if ((int64_t)batch * geom->n_kv_heads > 65535) return api_fail(C2KV_EINVAL, "batch * n_kv_heads must be below 65536");
  if (t_len < 1 || t_len > INT32_MAX / 2) return api_fail(C2KV_EINVAL, "t_len must be >= 1");
  if (t_len > max_pages * pages->page) return api_fail(C2KV_ECAPACITY, "t_len exceeds max_pages * page");
  s = api_device_state(&p.err, nullptr);
  if (s != C2KV_OK) return s;
  p.page_table = page_table;
  p.max_pages = max_pages;
  p.batch = batch;
  p.n_layers = 1;
  p.fresh[0] = static_cast<const __nv_bfloat16*>(k_new);
  p.fresh[1] = static_cast<const __nv_bfloat16*>(v_new);
  p.n_cached = n_cached_dev;
  p.n_new = n_new_dev;
  p.tab = static_cast<const CosSin2*>(rope_table);
  p.rope_row = rope_row_dev;
  p.t_len = t_len;
  p.table_rows = table_rows;
  return api_launched(launch_pages8_append(p, geom->head_dim, static_cast<cudaStream_t>(stream)),
                      "c2kv_pages8_append");
}

size_t c2kv_attend_pages8_workspace_size(const c2kv_geometry* geom, int32_t batch, int32_t max_keys) {
  if (api_check_geom(geom) != C2KV_OK || batch < 1 || batch > kMaxPagedSeqs || max_keys < 1) return 0;
  return attend_workspace(geom, api_sm_count_for_sizing()).total;
}

c2kv_status c2kv_attend_pages8(const c2kv_geometry* geom, const c2kv_pages8* pages, int32_t layer, int32_t batch,
                               const int32_t* page_table, int32_t max_pages, const int32_t* n_cached_dev,
                               int32_t max_keys, const void* q, const void* k_new, const void* v_new,
                               const void* rope_table, int32_t table_rows, const int32_t* rope_row_dev, void* out,
                               void* workspace, size_t workspace_bytes, uint32_t flags, void* stream) {
  AttendPages8Params p;
  std::memset(&p, 0, sizeof(p));
  if (flags & ~uint32_t(C2KV_DECODE_OVERLAP_PREVIOUS | C2KV_DECODE_ROW_AT_LENGTH)) return api_fail(C2KV_EINVAL, "unknown decode flags");
  c2kv_status s = check_pages(geom, pages, layer, page_table, max_pages, &p.pool);
  if (s != C2KV_OK) return s;
  s = check_new_tokens(batch, n_cached_dev, k_new, v_new, rope_table, table_rows, rope_row_dev);
  if (s != C2KV_OK) return s;
  if (!q || !out || !workspace) return api_fail(C2KV_EINVAL, "null pointer");
  if ((k_new == nullptr) != (v_new == nullptr)) return api_fail(C2KV_EINVAL, "k_new and v_new go together");
  if (!aligned(q, 16)) return api_fail(C2KV_EINVAL, "q must be 16-byte aligned");
  if (max_keys < 1 || max_keys > max_pages * pages->page)
    return api_fail(C2KV_EINVAL, "max_keys must be in [1, max_pages * page]");
  // a tile for every 128 rows of 128 bytes, and a few for the end of each head's
  if ((int64_t)batch * geom->n_kv_heads * ((max_keys - 1) / (128 * 128 / geom->head_dim) + 8) > INT32_MAX)
    return api_fail(C2KV_EINVAL, "batch * n_kv_heads * max_keys is above 2^31 tiles of 128 rows of 128 bytes");
  const int sms = std::min(api_sm_count_for_sizing(), kMaxPageCtas / 2);
  const AttendWs w = attend_workspace(geom, sms);
  if (workspace_bytes < w.total || !aligned(workspace, 16))
    return api_fail(C2KV_EINVAL, "workspace too small or not 16-byte aligned");
  s = api_device_state(&p.err, nullptr);
  if (s != C2KV_OK) return s;
  for (int kv = 0; kv < 2; ++kv) {
    s = api_encode_rows128(&p.tm[kv], p.pool.codes[kv],
                           (uint64_t)p.pool.n_pages * p.pool.n_kv * p.pool.page * geom->head_dim / 128,
                           (uint32_t)(p.pool.page * geom->head_dim / 128));
    if (s != C2KV_OK) return s;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.counters = reinterpret_cast<int32_t*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + w.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + w.o_off);
  p.page_table = page_table;
  p.n_cached = n_cached_dev;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.fresh[0] = static_cast<const __nv_bfloat16*>(k_new);
  p.fresh[1] = static_cast<const __nv_bfloat16*>(v_new);
  p.tab = static_cast<const CosSin2*>(rope_table);
  p.rope_row = rope_row_dev;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.batch = batch;
  p.n_q = geom->n_q_heads;
  p.max_pages = max_pages;
  p.max_keys = max_keys;
  p.table_rows = table_rows;
  p.has_new = k_new != nullptr ? 1 : 0;
  p.row_at_length = (flags & C2KV_DECODE_ROW_AT_LENGTH) != 0 ? 1 : 0;
  p.early = (flags & C2KV_DECODE_OVERLAP_PREVIOUS) != 0 ? 1 : 0;
  p.inject_timeout = api_take_injected_timeout();
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)geom->head_dim));
  return api_launched(launch_attend_pages8(p, geom->head_dim, geom->n_q_heads / geom->n_kv_heads, sms,
                                           static_cast<cudaStream_t>(stream)),
                      "c2kv_attend_pages8");
}

c2kv_status c2kv_token_logprobs(const void* logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                                const int32_t* tokens, int32_t top_k, float* logprob, float* entropy,
                                int32_t* top_ids, float* top_logprobs, void* stream) {
  LogprobParams p;
  std::memset(&p, 0, sizeof(p));
  if (dtype != C2KV_BF16 && dtype != C2KV_F32) return api_fail(C2KV_EINVAL, "logits must be C2KV_BF16 or C2KV_F32");
  if (rows < 0 || vocab < 1 || vocab > (1 << 30)) return api_fail(C2KV_EINVAL, "need rows >= 0 and 1 <= vocab <= 2^30");
  if (row_stride < vocab) return api_fail(C2KV_EINVAL, "row_stride must be >= vocab");
  if (top_k < 0 || top_k > kMaxTopK || top_k > vocab) return api_fail(C2KV_EINVAL, "top_k must be in [0, min(64, vocab)]");
  if (rows == 0) return C2KV_OK;
  if (!logits) return api_fail(C2KV_EINVAL, "logits is null");
  if ((logprob == nullptr) != (tokens == nullptr)) return api_fail(C2KV_EINVAL, "tokens and logprob go together");
  if (top_k > 0 && (!top_ids || !top_logprobs)) return api_fail(C2KV_EINVAL, "top_ids / top_logprobs is null");
  if (!aligned(logits, dtype == C2KV_BF16 ? 2 : 4)) return api_fail(C2KV_EINVAL, "logits must be aligned to their type");
  int sms = 0;
  const c2kv_status s = api_device_state(&p.err, &sms);
  if (s != C2KV_OK) return s;
  p.logits = logits;
  p.tokens = tokens;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  p.row_stride = row_stride;
  p.rows = rows;
  p.vocab = vocab;
  p.top_k = top_k;
  p.is_f32 = dtype == C2KV_F32;
  return api_launched(launch_token_logprobs(p, sms, static_cast<cudaStream_t>(stream)), "c2kv_token_logprobs");
}

}  // extern "C"
