/*
 * c2kv.h -- C ABI of the GB300 (sm_103a) C2KV composed-cache hot path.
 *
 * C2KV (compressed, composable, non-prefix KV-cache reuse) stores one
 * compressed, pre-RoPE K/V slot per k document tokens, keeps the stores in
 * host memory, and at request time streams the selected documents to the
 * GPU, re-applies RoPE at their new positions, concatenates them into one
 * cache and then prefills the question and decodes the answer over it.
 *
 * Sources (cited by page title and section):
 *   [EXPL]  "C 2 KV: Compressed and Composable KV Cache Reuse for Efficient
 *           LLM Inference", paper-daily.com explainer.  Sections used:
 *           "the problem" (它到底在解决什么问题？), "pipeline: extract, store,
 *           concatenate" (整体流程：抽取、存储、拼接), "C2 tokens"
 *           (C2 token：用额外的“记忆槽”承载压缩信息), "structured information flow"
 *           (为什么需要“结构化信息流”？), "positions at concatenation"
 *           (拼接时位置怎么处理？), "results" (实验结果：真的又快又准吗？).
 *   [ABS]   arXiv 2607.17715 listing (arxivdaily.com), English abstract.
 *
 * Conventions for every entry point:
 *   - No exception crosses the ABI; each call returns a c2kv_status and, on
 *     failure, c2kv_last_error() (thread-local) describes it.  All argument
 *     checks run on the host before anything is enqueued: a call that fails
 *     validation enqueues nothing.
 *   - All K/V/q tensors are bf16 (raw 16-bit patterns).  Device buffers are
 *     owned by the caller; the library never frees them.  Host inputs are
 *     read during the call only (copied where they must outlive it).
 *   - Device work is enqueued on the caller's `stream` (a cudaStream_t passed
 *     as void*; NULL is the legacy default stream) and is ordered after the
 *     work already on it; calls return after enqueueing.
 *   - Cache layout per sequence: k_cache and v_cache are each
 *     [n_layers][n_kv_heads][cap][head_dim] bf16 (one contiguous key run per
 *     layer and kv head).  q head h reads kv head h / (n_q_heads/n_kv_heads).
 *   - RoPE is the rotate-half form with inv_freq_i = rope_theta^(-2i/d);
 *     angles are formed and reduced in fp64 (once per cache row, into a RoPE
 *     table); stored keys are rotated in double-float arithmetic on the fp32
 *     pipe and rounded once to bf16 (nearest even).
 *   - A kernel that finds a device-side problem (a bounded wait that expired,
 *     a device length beyond the cache capacity) records it in a device error
 *     word and skips the affected output; c2kv_device_error() reads it.
 */
#ifndef C2KV_H_
#define C2KV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct c2kv_store_s* c2kv_store;

typedef struct {
  int32_t n_layers;
  int32_t n_q_heads;
  int32_t n_kv_heads;   /* must divide n_q_heads; group = n_q/n_kv in {1,2,4,5,8} */
  int32_t head_dim;     /* 64 or 128 */
  double rope_theta;
} c2kv_geometry;

typedef enum {
  C2KV_OK = 0,
  C2KV_EINVAL = 1,     /* bad argument (null pointer, bad size, k mismatch, bad order) */
  C2KV_ENOMEM = 2,     /* pinned pool exhausted or host allocation failed */
  C2KV_ENOTFOUND = 3,  /* unknown document id */
  C2KV_ECAPACITY = 4,  /* composed or appended rows exceed the cache capacity */
  C2KV_ECUDA = 5,      /* a CUDA runtime call failed (message in c2kv_last_error) */
  C2KV_ETIMEOUT = 6,   /* a kernel's bounded wait expired (from c2kv_device_error) */
  C2KV_EDEVICE = 7,    /* a kernel rejected a device-side value (from c2kv_device_error) */
  C2KV_EIO = 8         /* a store file could not be opened, read or written */
} c2kv_status;

typedef enum {
  C2KV_MASK_CAUSAL = 0,      /* plain causal mask over the whole sequence */
  C2KV_MASK_STRUCTURED = 1,  /* [EXPL] "structured information flow" rules */
  C2KV_MASK_ANCHOR = 2       /* [EXPL] "results": the anchor-token ablation */
} c2kv_mask;

/* Thread-local description of the last failure on this thread ("" if none). */
const char* c2kv_last_error(void);

/* Library version string. */
const char* c2kv_version(void);

/*
 * Segment store: pinned host memory holding compressed pre-RoPE segments.
 * [EXPL] "the problem": the caches live in host memory and are moved to the
 * GPU when used; [EXPL] "positions at concatenation": they are kept before
 * RoPE so they can be re-rotated wherever they are composed.
 *
 * Creates a store on the current CUDA device with a pinned pool of
 * pinned_bytes (cudaHostAlloc), a non-blocking copy stream and events.
 * Returns C2KV_EINVAL for a bad geometry, C2KV_ENOMEM if the pool cannot be
 * pinned.  *out receives the handle (owned by the caller; free with
 * c2kv_store_destroy).
 */
c2kv_status c2kv_store_create(const c2kv_geometry* geom, size_t pinned_bytes,
                              c2kv_store* out);

/* Waits for the store's copies in flight, then frees the pool and handles. */
void c2kv_store_destroy(c2kv_store store);

/*
 * Copies n_docs compressed segments into the pinned pool.
 * [EXPL] "C2 tokens": one slot per k document tokens, only the slots' K/V
 * are kept.  For document i: doc_ids[i] (unique, not yet stored),
 * n_tokens[i] >= 1 original tokens, 1 <= n_slots[i] <= n_tokens[i] slots
 * stored at compression ratio k >= 1, and host pointers k_pre[i], v[i] to
 * bf16 arrays [n_layers][n_kv_heads][n_slots[i]][head_dim] (K before RoPE).
 * The inputs are copied; the caller keeps ownership.
 * Errors: C2KV_EINVAL (bad sizes, null pointer, duplicate id),
 * C2KV_ENOMEM (pool full; nothing of this call is stored).
 */
c2kv_status c2kv_store_segments(c2kv_store store, int32_t n_docs,
                                const int32_t* doc_ids, const int32_t* n_tokens,
                                const int32_t* n_slots, int32_t k,
                                const void* const* k_pre, const void* const* v);

/*
 * Persists the store.  [EXPL] "pipeline: extract, store, concatenate": each
 * document's compressed cache is extracted once, stored, and reused by any
 * later request; these two calls keep the stored caches across processes.
 *
 * c2kv_store_save writes every stored document (ascending ids: id, original
 * length, slots, k, then its K and V rows [n_layers][n_kv_heads][slot][d]
 * bf16) after a header holding the geometry, in host byte order, to `path`
 * (created or truncated).  Errors: C2KV_EINVAL (null argument), C2KV_EIO.
 *
 * c2kv_store_load adds the documents of such a file to `store`, which must
 * have the geometry the file was saved with.  Documents read before an error
 * stay in the store.  Errors: C2KV_EIO (cannot open, truncated), C2KV_EINVAL
 * (not a store file, another geometry, a bad record, an id already stored),
 * C2KV_ENOMEM (pool full).
 */
c2kv_status c2kv_store_save(c2kv_store store, const char* path);
c2kv_status c2kv_store_load(c2kv_store store, const char* path);

/* Looks up one stored document: its original length, slot count and k. */
c2kv_status c2kv_store_lookup(c2kv_store store, int32_t doc_id,
                              int32_t* n_tokens, int32_t* n_slots, int32_t* k);

/*
 * Host-only composition planner (no device work; usable without a GPU).
 * [EXPL] "positions at concatenation": documents are taken in composed
 * order, composed doc c = input doc order[c] (order NULL = identity; order
 * must be a permutation of 0..n_docs-1).  Each document occupies its
 * original length of positions, so composed doc c starts at position
 * pos_offset[c] = sum of n_tokens of the composed docs before it, and its
 * slots start at row slot_start[c] = sum of their n_slots.  Outputs (host,
 * n_docs entries each, may be NULL): slot_start, pos_offset; totals
 * *total_slots = sum n_slots and *total_tokens = sum n_tokens (the position
 * of the first appended question token).  Slot j of composed doc c sits at
 * pos_offset[c] + min((j+1)k, n_tokens) - 1.
 * Errors: C2KV_EINVAL (bad order, sizes, int32 overflow).
 */
c2kv_status c2kv_plan(int32_t n_docs, const int32_t* n_tokens,
                      const int32_t* n_slots, const int32_t* order,
                      int32_t* slot_start, int32_t* pos_offset,
                      int32_t* total_slots, int32_t* total_tokens);

/*
 * Composes one request's cache.  [EXPL] "pipeline": fetch the documents'
 * compressed caches, re-apply position encoding at their new positions and
 * concatenate them, with no repair step; [EXPL] "positions at
 * concatenation": slot j of composed doc c is rotated at
 * pos_offset[c] + min((j+1)k, n_tokens_c) - 1.
 *
 * doc_ids[n_docs] (repeats allowed), order as in c2kv_plan, k must equal the
 * k every document was stored with.  k_cache/v_cache: caller-owned device
 * buffers [n_layers][n_kv_heads][cap][head_dim] bf16; rows [0, N) of every
 * layer and kv head are written (N = total slots), rows >= N are untouched.
 * rope_table_out (required): caller-owned device buffer of
 * c2kv_rope_table_bytes(geom, cap) bytes receiving, for every cache row r,
 * the cos/sin of its position for the head_dim/2 RoPE frequencies as fp32
 * (hi, lo) pairs, layout [cap][head_dim/2][cos_hi, cos_lo, sin_hi, sin_lo].
 * Row r < N holds slot r's position; row r >= N holds L_tot + (r - N), the
 * position of the (r-N)-th token appended after the documents (reading: the
 * question starts right after the documents' original length L_tot).
 * Prefill and decode rotate with this table.
 * pos_dev_out: optional device int32 [cap] receiving the position of every row.
 * Host outputs (optional): *n_slots_out = N, *next_pos_out = L_tot.
 * The segments are copied host->device on the store's copy stream in layer
 * groups; the table and the re-rotation of each group run on `stream` (the
 * latter once its copy has landed), and all of it is ordered before later
 * work on `stream`.  The store must not be destroyed before that work
 * completes.
 * Errors: C2KV_EINVAL, C2KV_ENOTFOUND, C2KV_ECAPACITY (N > cap), C2KV_ECUDA.
 */
c2kv_status c2kv_compose(c2kv_store store, int32_t n_docs, const int32_t* doc_ids,
                         const int32_t* order, int32_t k, void* k_cache,
                         void* v_cache, int32_t cap, void* rope_table_out,
                         int32_t* pos_dev_out, int32_t* n_slots_out,
                         int32_t* next_pos_out, void* stream);

/*
 * c2kv_compose over the layers [layer_begin, layer_end) only, with flags:
 *
 * C2KV_COMPOSE_NO_REALIGN — the ablation of [EXPL] "results" that drops the
 *   position re-alignment: every document keeps the positions it was
 *   extracted at (slot j at min((j+1)k, n_c) - 1, no offset off_c), so all
 *   documents start at position 0.  Appended tokens still start at L_tot,
 *   the summed original length (reading: the ablation changes the
 *   documents' positions only).  c2kv_plan's pos_offset does not apply.
 *
 * C2KV_COMPOSE_CONTINUE — continue the composition started by the last
 *   c2kv_compose / c2kv_compose_layers call on this store into the same
 *   RoPE table (same doc_ids, order, k, flags other than this one, caches
 *   and cap): the table and pos_dev_out are not rebuilt, and the
 *   copies of these layers are queued behind that call's copies on the
 *   store's copy stream instead of waiting for the caller's stream.  So a
 *   caller can compose layer group 0, enqueue work on those layers (the
 *   question prefill), then compose group 1, and the prefill overlaps the
 *   later groups' host->device copies ([EXPL] "the problem": loading the
 *   cache is the dominant TTFT cost).  The caller guarantees that nothing
 *   issued on `stream` since the first call reads or writes rows [0, N) of
 *   the continued layers.  The re-rotation of the layers is ordered on
 *   `stream` after their copies.
 *
 * 0 <= layer_begin < layer_end <= n_layers.  Other arguments, outputs and
 * errors as c2kv_compose; C2KV_EINVAL also for a CONTINUE that does not
 * follow a composition of the same request (documents, k, flags, caches,
 * cap, table) on this store.  The store remembers the compositions into the
 * 1024 tables most recently composed into; a CONTINUE into an older one is
 * refused the same way.
 */
#define C2KV_COMPOSE_NO_REALIGN 1u
#define C2KV_COMPOSE_CONTINUE 2u
c2kv_status c2kv_compose_layers(c2kv_store store, int32_t n_docs, const int32_t* doc_ids,
                                const int32_t* order, int32_t k, uint32_t flags,
                                int32_t layer_begin, int32_t layer_end, void* k_cache,
                                void* v_cache, int32_t cap, void* rope_table_out,
                                int32_t* pos_dev_out, int32_t* n_slots_out,
                                int32_t* next_pos_out, void* stream);

/* Bytes of a RoPE table of `rows` rows: rows * (head_dim/2) * 16. */
size_t c2kv_rope_table_bytes(const c2kv_geometry* geom, int32_t rows);

/*
 * Builds a RoPE table (layout as in c2kv_compose) for arbitrary positions:
 * row r gets the cos/sin of position pos_dev[r] (device int32 [rows]), for
 * caches filled by other means than c2kv_compose.  Angles pos * inv_freq are
 * formed in fp64 and reduced mod 2*pi before the fp64 sincos.
 */
c2kv_status c2kv_rope_table(const c2kv_geometry* geom, const int32_t* pos_dev,
                            int32_t rows, void* table_out, void* stream);

/*
 * Device scratch (bytes) that c2kv_attend_prefill / c2kv_attend_decode /
 * c2kv_attend_masked need for `batch` sequences of `t_len` new tokens each,
 * with at most `max_keys` keys per sequence (cached + new).  The scratch
 * holds split-K partial results and per-(sequence, head) arrival counters;
 * it must be zeroed once before first use (c2kv_workspace_init) and may then
 * be reused by calls that do not overlap on the GPU.  Returns 0 on bad input.
 */
size_t c2kv_attend_workspace_size(const c2kv_geometry* geom, int32_t batch,
                                  int32_t t_len, int32_t max_keys);

/* Zeroes a workspace on `stream` (cudaMemsetAsync). */
c2kv_status c2kv_workspace_init(void* workspace, size_t bytes, void* stream);

/*
 * Question prefill for one layer of `batch` requests.
 * [EXPL] "pipeline": after composition the question is appended and
 * generation starts.
 *
 * k_caches[b], v_caches[b]: host array of device pointers to request b's
 * cache base (layer 0, layout as above); `layer` selects the layer.
 * rope_tables[b]: host array of device pointers to request b's RoPE table
 * (from c2kv_compose).  n_cached[b] (host): rows already in the cache.
 * q: device [batch][q_len][n_q_heads][head_dim] (before RoPE);
 * k_new, v_new: device [batch][q_len][n_kv_heads][head_dim] (k before RoPE).
 * Question token i lands at row n_cached[b] + i and is rotated with that
 * row of the table (q and k alike); then out[b][i] = softmax(q_i K^T /
 * sqrt(d)) V over the n_cached[b] + i + 1 visible keys (all cached rows plus
 * question tokens 0..i), written to device out [batch][q_len][n_q_heads]
 * [head_dim] bf16.  q_len > 1 runs QK^T and PV on the tcgen05 tensor cores.
 * workspace: device scratch of c2kv_attend_workspace_size(geom, batch,
 * q_len, max_b(n_cached[b] + q_len)) bytes, zeroed once.
 * Errors: C2KV_EINVAL, C2KV_ECAPACITY (n_cached[b] + q_len > cap), C2KV_ECUDA.
 */
c2kv_status c2kv_attend_prefill(const c2kv_geometry* geom, int32_t layer,
                                int32_t batch, void* const* k_caches,
                                void* const* v_caches, const void* const* rope_tables,
                                int32_t cap, const int32_t* n_cached, int32_t q_len,
                                const void* q, const void* k_new, const void* v_new,
                                void* out, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * One decode step for one layer of `batch` sequences.  [EXPL] "results":
 * each generated token reads the whole composed cache, which C2KV shrinks.
 *
 * As prefill with one new token per sequence, except that the lengths live
 * on the device so a captured sequence of calls can be replayed:
 * n_cached_dev[b] (device int32) rows are cached; the new token's key is
 * rotated with table row n_cached_dev[b], stored with its value at that row,
 * and the token attends over n_cached_dev[b] + 1 keys -- all in one kernel
 * launch.  max_keys (host) bounds n_cached_dev[b] + 1 for every b and sizes
 * the grid; a device length over max_keys or cap is recorded in the device
 * error word and that sequence's output is skipped.
 * q: [batch][n_q_heads][head_dim]; k_new, v_new: [batch][n_kv_heads]
 * [head_dim]; out: [batch][n_q_heads][head_dim].  The lengths are not
 * advanced (see c2kv_seq_advance).
 * workspace: c2kv_attend_workspace_size(geom, batch, 1, max_keys) bytes.
 */
c2kv_status c2kv_attend_decode(const c2kv_geometry* geom, int32_t layer,
                               int32_t batch, void* const* k_caches,
                               void* const* v_caches, const void* const* rope_tables,
                               int32_t cap, const int32_t* n_cached_dev, int32_t max_keys,
                               const void* q, const void* k_new, const void* v_new,
                               void* out, void* workspace, size_t workspace_bytes,
                               uint32_t flags, void* stream);

/*
 * Decode flag: the launch may begin while the kernel enqueued just before it
 * on `stream` is still finishing (programmatic dependent launch).  Before it
 * waits for that kernel it reads only n_cached_dev, the RoPE table and the
 * cache rows below n_cached_dev[b] of this layer, so the caller promises that
 * the previous kernel writes none of these (e.g. it is the decode of another
 * layer, or the projection producing q/k_new/v_new -- but not
 * c2kv_seq_advance).  q, k_new, v_new, out and the workspace are touched only
 * after the previous kernel has completed.
 */
#define C2KV_DECODE_OVERLAP_PREVIOUS 1u

/*
 * c2kv_attend_decode without a workspace argument: the paper has no
 * counterpart; this is a convenience of the library.
 *
 * For callers that cannot allocate device memory where they decode -- a
 * plugin whose host framework hands it only a stream and tensors and forbids
 * allocation while enqueueing, or a serving loop that freezes all device
 * allocations at start-up.  The split-K scratch lives instead in one
 * fixed-size array (4 MiB) in the library's device memory; every GPU that
 * loads the library holds that array until the process exits.  This call
 * allocates nothing (no cudaMalloc/cudaFree, no allocating library routine).
 *
 * Arguments and results are those of c2kv_attend_decode (with flags 0).  The first call on
 * a device looks up the array's device address (cudaGetSymbolAddress) with
 * that device current; make that first call before any stream capture.  The
 * array is shared by every call and keeps the previous call's contents: each
 * call clears its arrival counters on `stream` first, so two calls whose GPU
 * work can overlap (for example calls on different streams) race on the
 * array; issue such calls one after the other.  A decode whose scratch would
 * exceed the array is rejected with C2KV_EINVAL before anything is enqueued.
 */
c2kv_status c2kv_attend_decode_noalloc(const c2kv_geometry* geom, int32_t layer,
                                       int32_t batch, void* const* k_caches,
                                       void* const* v_caches, const void* const* rope_tables,
                                       int32_t cap, const int32_t* n_cached_dev,
                                       int32_t max_keys, const void* q, const void* k_new,
                                       const void* v_new, void* out, void* stream);

/* Adds `delta` to n_cached_dev[b] for b < batch <= 1024 (device kernel). */
c2kv_status c2kv_seq_advance(int32_t batch, int32_t* n_cached_dev, int32_t delta,
                             void* stream);

/*
 * Attention over one extraction sequence under a mask (the "mask mode").
 * [EXPL] "structured information flow": n_doc document tokens followed by
 * n_slot slot tokens.  C2KV_MASK_STRUCTURED: document tokens keep the
 * causal mask and see no slot; slot i sees the sink block B(0) (document
 * tokens [0, k)), its own block [i*k, min((i+1)k, n_doc)) and slots 0..i.
 * [EXPL] "positions at concatenation": documents sit at 0..n_doc-1 and slot
 * i at min((i+1)k, n_doc) - 1.  C2KV_MASK_ANCHOR: the anchor-token
 * ablation of [EXPL] "results", read as a change of mask only: the n_slot
 * extra tokens take the slots' positions; document token r sees document
 * tokens 0..r and every extra token; extra token i sees every document
 * token and extra tokens 0..i.  C2KV_MASK_CAUSAL: plain causal attention,
 * token t at position t (n_slot must be 0).
 * q: device [N][n_q_heads][head_dim], kk, v: device [N][n_kv_heads][head_dim]
 * with N = n_doc + n_slot, all before RoPE; out: device [N][n_q_heads][d].
 * workspace: c2kv_attend_workspace_size(geom, 1, N, N) + c2kv_masked_extra_bytes
 * (geom, N) bytes (the sequence's RoPE table and its rotated keys and values
 * are staged there), zeroed once.
 */
c2kv_status c2kv_attend_masked(const c2kv_geometry* geom, int32_t mask,
                               int32_t n_doc, int32_t n_slot, int32_t k,
                               const void* q, const void* kk, const void* v,
                               void* out, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Extra scratch bytes c2kv_attend_masked needs beyond the attention scratch. */
size_t c2kv_masked_extra_bytes(const c2kv_geometry* geom, int32_t n_tokens);

/*
 * The synthetic-weight decoder step around the attention calls: its linear
 * layers and RMSNorm.  [EXPL] "the problem" (Fig. 1): the time to first token
 * and the decode rate of the whole model are what the cache reuse buys, and
 * a decoder layer runs these projections and its MLP around the attention
 * over the composed cache.
 *
 * c2kv_linear: y[t][n] = sum_k x[t][k] * w[n][k] on the tensor cores (fp32
 * accumulation, bf16 result) for t < tokens, then an epilogue:
 *   C2KV_LINEAR_STORE   y [tokens][n_out] = the product;
 *   C2KV_LINEAR_ADD     y [tokens][n_out] = product + residual [tokens][n_out]
 *                       (residual may be y: an in-place residual update);
 *   C2KV_LINEAR_SPLIT3  output columns [0, split1) to y [tokens][split1],
 *                       [split1, split2) to y2, [split2, n_out) to y3 (the
 *                       q, k and v of a fused QKV projection);
 *   C2KV_LINEAR_SWIGLU  rows 128i .. 128i+63 of w are the gate rows of
 *                       features 64i .. 64i+63 and rows 128i+64 .. 128i+127
 *                       their up rows; y [tokens][n_out / 2] =
 *                       silu(gate) * up, silu(g) = g / (1 + e^-g).
 * x: device bf16 [tokens][k_in], w: device bf16 [n_out][k_in] (row-major,
 * as a linear layer's weight), both 16-byte aligned.  1 <= tokens <= 256,
 * k_in a positive multiple of 64, n_out a positive multiple of 128 up to
 * 1048576.  workspace: c2kv_linear_workspace_size(tokens, n_out) bytes of
 * device memory, zeroed once (c2kv_workspace_init); calls of any shapes that
 * fit it may share it as long as their GPU work does not overlap (a launch
 * with C2KV_LINEAR_OVERLAP_PREVIOUS touches it only after the kernel before
 * it has completed).  flags: C2KV_LINEAR_OVERLAP_PREVIOUS lets the launch
 * begin, and request its first weight tiles, while the kernel before it on
 * `stream` finishes (the caller promises that kernel does not write w); x,
 * the residual and the outputs are touched only after it completes.
 * Errors: C2KV_EINVAL, C2KV_ECUDA.
 *
 * c2kv_rmsnorm: y[t] = x[t] / sqrt(mean_i x[t][i]^2 + eps) * w for t < tokens,
 * x and y device bf16 [tokens][dim], w bf16 [dim] (dim a multiple of 8,
 * 16-byte aligned pointers), sums in fp32.  flags as c2kv_linear.
 */
#define C2KV_LINEAR_STORE 0
#define C2KV_LINEAR_ADD 1
#define C2KV_LINEAR_SPLIT3 2
#define C2KV_LINEAR_SWIGLU 3
#define C2KV_LINEAR_OVERLAP_PREVIOUS 1u
size_t c2kv_linear_workspace_size(int32_t tokens, int32_t n_out);
c2kv_status c2kv_linear(const void* x, int32_t tokens, int32_t k_in, const void* w, int32_t n_out,
                        int32_t epilogue, const void* residual, void* y, void* y2, void* y3,
                        int32_t split1, int32_t split2, void* workspace, size_t workspace_bytes,
                        uint32_t flags, void* stream);
c2kv_status c2kv_rmsnorm(const void* x, int32_t tokens, int32_t dim, const void* w, float eps, void* y,
                         uint32_t flags, void* stream);

/*
 * The 8-bit paged cache: half the bytes of the composed bf16 cache, which is
 * what bounds a decode step ([EXPL] "results": every generated token reads the
 * whole composed cache).
 *
 * A pool of n_pages pages; a page holds `page` tokens of one layer: for each
 * kv head, page rows of head_dim e4m3 codes of K (after RoPE) and of V, and
 * one scale each.  A held value is code * scale.  A sequence's rows are in
 * the pages its row of the page table names: row j in entry j / page, place
 * j % page.  page_table: device int32 [batch][max_pages]; entries behind a
 * sequence's last row are never read.  Sequences may share pages that no call
 * writes; a page that a call writes must belong to one sequence of it.
 *
 * Scales: a scale is 2^e.  For the rows first written to a page, e is the
 * smallest integer with a <= 448 * 2^e, a being their largest finite
 * magnitude of that kv head (e >= -120).  Rows added later raise e to what
 * they need, never lower it; when it rises from e to e', the page's earlier
 * codes c become e4m3(c * 2^(e - e')).  Codes are rounded to nearest even; a
 * value that is not finite is held as NaN.  The scales of K and V pages must
 * be ones that these calls wrote.
 *
 * Device-side values (lengths, page ids, table rows) are checked on the
 * device: a bad one is recorded in the device error word (C2KV_EDEVICE) and
 * what it would reach is left out.  A length n_cached_dev[b] < 0 marks an
 * empty place of the batch: nothing of it is read or written, which is no
 * error (c2kv_seq_advance adds to every length: a place that is to stay empty
 * takes one far below 0).
 */
typedef struct {
  void* k;          /* device e4m3 [n_layers][n_pages][n_kv_heads][page][head_dim] */
  void* v;          /* same layout; both 16-byte aligned */
  float* k_scale;   /* device fp32 [n_layers][n_pages][n_kv_heads] */
  float* v_scale;
  int32_t n_pages;
  int32_t page;     /* tokens of a page: 16, 32, 64 or 128 */
} c2kv_pages8;

/*
 * Fills pages from composed bf16 caches, layers [layer_begin, layer_end):
 * rows [0, n_rows[b]) (host array) of sequence b's caches (as for
 * c2kv_attend_prefill, batch <= 16) go to its pages; the places behind them
 * in the last page are left as they were.  One pass over the rows, one
 * launch.  Errors: C2KV_EINVAL, C2KV_ECAPACITY (n_rows above cap or above
 * max_pages * page), C2KV_ECUDA.
 */
c2kv_status c2kv_pages8_fill(const c2kv_geometry* geom, const c2kv_pages8* pages, int32_t layer_begin,
                             int32_t layer_end, int32_t batch, void* const* k_caches, void* const* v_caches,
                             int32_t cap, const int32_t* n_rows, const int32_t* page_table, int32_t max_pages,
                             void* stream);

/*
 * Appends new tokens of one layer: token i of sequence b, i < n_new_dev[b]
 * (device int32 [batch], 0 <= n_new_dev[b] <= t_len; NULL: t_len each), goes
 * to row n_cached_dev[b] + i.  k_new, v_new: device bf16 [batch][t_len]
 * [n_kv_heads][head_dim], k before RoPE.  rope_table: device table of
 * table_rows rows (layout of c2kv_rope_table); token i's key is rotated by its
 * row rope_row_dev[b] + i, rounded to fp32 and from there to bf16, about as a
 * bf16 cache would hold it, before it is rounded to its code.  The lengths are not advanced
 * (c2kv_seq_advance).  batch <= 256, batch * n_kv_heads < 65536.  A sequence whose tokens would not fit
 * max_pages pages, or whose table rows are out of range, is left out whole.
 */
c2kv_status c2kv_pages8_append(const c2kv_geometry* geom, const c2kv_pages8* pages, int32_t layer, int32_t batch,
                               int32_t t_len, const int32_t* page_table, int32_t max_pages,
                               const int32_t* n_cached_dev, const int32_t* n_new_dev, const void* k_new,
                               const void* v_new, const void* rope_table, int32_t table_rows,
                               const int32_t* rope_row_dev, void* stream);

/*
 * One decode step of one layer over the pages, the append of its own token
 * included: as c2kv_pages8_append with t_len 1, then out[b] = softmax(q_b K^T
 * / sqrt(d)) V over the n_cached_dev[b] + 1 held rows, q_b rotated by table
 * row rope_row_dev[b].  k_new and v_new NULL: nothing is appended and the
 * n_cached_dev[b] held rows are attended over; with none, out[b] is 0.
 * q, out: device bf16 [batch][n_q_heads][head_dim].  max_keys bounds the rows
 * attended over by every sequence and sizes the launch; a sequence with more
 * is left out.  workspace: c2kv_attend_pages8_workspace_size bytes, 16-byte
 * aligned, zeroed once (c2kv_workspace_init), then reused by c2kv_attend_pages8
 * calls of the same geometry that do not overlap on the GPU (other calls'
 * scratch would overwrite its counters).  flags: C2KV_DECODE_OVERLAP_PREVIOUS, as in
 * c2kv_attend_decode: the kernel before on `stream` must not write the
 * lengths, the page table, the RoPE table and rope_row_dev, or this layer's
 * held rows and their scales.  C2KV_DECODE_ROW_AT_LENGTH: the table row of
 * sequence b is rope_row_dev[b] + n_cached_dev[b], so that rope_row_dev says
 * where a sequence's rows begin in the table and the lengths are all that
 * advances from step to step.
 */
#define C2KV_DECODE_ROW_AT_LENGTH 4u
size_t c2kv_attend_pages8_workspace_size(const c2kv_geometry* geom, int32_t batch, int32_t max_keys);
c2kv_status c2kv_attend_pages8(const c2kv_geometry* geom, const c2kv_pages8* pages, int32_t layer, int32_t batch,
                               const int32_t* page_table, int32_t max_pages, const int32_t* n_cached_dev,
                               int32_t max_keys, const void* q, const void* k_new, const void* v_new,
                               const void* rope_table, int32_t table_rows, const int32_t* rope_row_dev, void* out,
                               void* workspace, size_t workspace_bytes, uint32_t flags, void* stream);

/*
 * Attention of a chunk of new tokens of one layer over the pages, their append
 * included: a further question on a composed cache, drafted tokens checked at
 * once, a document taken in piece by piece ([EXPL] "pipeline": what is asked
 * goes behind the composed cache).  As c2kv_pages8_append, then for token i of
 * sequence b, i < n_new_dev[b], with q_bi rotated by the token's table row,
 * out[b][i] = softmax(q_bi K^T / sqrt(d)) V over rows [0, n_cached_dev[b] + i].
 * k_new and v_new NULL: nothing is appended, the tokens' rows are held already.
 * q, out: device bf16 [batch][t_len][n_q_heads][head_dim], 16-byte aligned (out
 * holds the rotated queries until their answers take their place; it may be q);
 * out behind a sequence's last new token is left as it was.  max_keys bounds
 * n_cached_dev[b] + n_new_dev[b]; a sequence with more, or one that the append
 * leaves out, is left out whole.  Rows on pages outside the pool are not
 * attended over, and a token that sees no other row gets 0.  workspace:
 * c2kv_attend_pages8_chunk_workspace_size bytes, 16-byte aligned, of any
 * contents; calls that do not overlap on the GPU may share it, whatever their
 * shapes.  flags: C2KV_DECODE_ROW_AT_LENGTH, for the append as well.  The
 * queries are held to 11 bits, in fp16 times a power of two for each head, and
 * so are the softmax weights, down to 2^-15 of a row's largest; sums are in fp32.
 * The scales of a sequence's pages may be as far apart as they get; where V
 * scales among 128 neighbouring rows are more than 2^15 apart, those rows take
 * some 30 times as long.  A query that is not finite gives NaN, a held NaN gives
 * NaN to the tokens that see it.
 */
size_t c2kv_attend_pages8_chunk_workspace_size(const c2kv_geometry* geom, int32_t batch, int32_t t_len,
                                               int32_t max_keys);
c2kv_status c2kv_attend_pages8_chunk(const c2kv_geometry* geom, const c2kv_pages8* pages, int32_t layer, int32_t batch,
                                     int32_t t_len, const int32_t* page_table, int32_t max_pages,
                                     const int32_t* n_cached_dev, const int32_t* n_new_dev, int32_t max_keys,
                                     const void* q, const void* k_new, const void* v_new, const void* rope_table,
                                     int32_t table_rows, const int32_t* rope_row_dev, void* out, void* workspace,
                                     size_t workspace_bytes, uint32_t flags, void* stream);

/*
 * The pages of a pool among its sequences.  refs: device int32 [n_pages], how
 * many sequences hold a page, 0 where it is free.  For these two calls a row of
 * page_table names all the pages that its sequence holds: its entries up to the
 * first negative one.  All layers have one table; all layers are copied.
 *
 * c2kv_pages8_fork makes a new batch of batch_out sequences out of the old one
 * of `batch`: place i goes on with sequence parent_dev[i] (negative, or a
 * sequence with a length below 0: an empty place).  So it forks answers, moves
 * and drops beams, ends sequences and takes pages for new tokens:
 *   - A parent's full pages are shared by its children.  The first of them, by
 *     place, keeps the others as well; the rest get a copy of the page that the
 *     length ends in (its held rows), so that every page that will be written
 *     to belongs to one sequence.  (In the old batch, too, a page that a length
 *     ends in, and those behind it, are their sequence's alone; a length is not
 *     taken back below what a fork has shared.)
 *   - Pages of sequences that no place goes on with are given back.
 *   - Each sequence gets pages until it has room for its length and `room` more
 *     tokens.  Pages are taken in the order of places and entries, the free page
 *     of the lowest index first; what the call itself gives back is free.
 * Written are refs_out, page_table_out [batch_out][max_pages] (entries behind
 * the held pages -1) and n_cached_out [batch_out] (-1: empty); each may be the
 * call's own input, else they must not overlap it.  A parent >= batch, an entry
 * that names no page in use, a length beyond the pages held, more pages than
 * max_pages for a sequence or than are free: C2KV_EDEVICE in the device error
 * word, and nothing is written.
 *
 * c2kv_pages8_compact moves the U pages in use to indices [0, U): the i-th
 * page in use of index >= U goes to the i-th free index, so a pool can be cut
 * off there or a large run of pages be had.  Written are refs_out,
 * page_table_out [batch][max_pages] (entries behind the held pages -1) and, if
 * not NULL, moved_out [n_pages]: the new index of each page, -1 for free ones.
 * Outputs may be inputs, and bad values end the call, as for the fork.
 *
 * batch, batch_out <= 256; batch_out * max_pages < 2^31.  workspace: c2kv_pages8_plan_workspace_size bytes
 * for the larger batch, 16-byte aligned, of any contents, shared by calls that
 * do not overlap on the GPU.  Errors: C2KV_EINVAL, C2KV_ECUDA.
 */
size_t c2kv_pages8_plan_workspace_size(int32_t n_pages, int32_t batch, int32_t max_pages);
c2kv_status c2kv_pages8_fork(const c2kv_geometry* geom, const c2kv_pages8* pages, int32_t batch,
                             const int32_t* page_table, int32_t max_pages, const int32_t* n_cached_dev,
                             int32_t batch_out, const int32_t* parent_dev, int32_t room, const int32_t* refs,
                             int32_t* refs_out, int32_t* page_table_out, int32_t* n_cached_out, void* workspace,
                             size_t workspace_bytes, void* stream);
c2kv_status c2kv_pages8_compact(const c2kv_geometry* geom, const c2kv_pages8* pages, int32_t batch,
                                const int32_t* page_table, int32_t max_pages, const int32_t* refs, int32_t* refs_out,
                                int32_t* page_table_out, int32_t* moved_out, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * Log probabilities from logits x [rows][vocab] (device, C2KV_BF16 or
 * C2KV_F32, row_stride elements from one row to the next): for each row, with
 * m = max x and S = sum exp(x - m),
 *   logprob  = x[tokens[row]] - m - log S   (a negative token: none is given, 0),
 *   entropy  = log S - sum exp(x - m) (x - m) / S,
 *   top_ids, top_logprobs [rows][top_k]: the top_k largest logits, largest
 *              first, equal ones by the lower index (NaN counts as largest).
 * Sums are in fp32; outputs are fp32 and int32.  tokens (device int32) and
 * logprob go together and may both be NULL, entropy may be NULL, top_k is at
 * most 64 and may be 0.  Logits of -inf are tokens ruled out: probability 0,
 * log probability -inf.  A row of nothing else has no distribution: its log
 * probabilities are -inf and its entropy 0.  A row with NaN or +inf gives NaN.
 * A token >= vocab gives NaN and is recorded in the device error word.
 */
#define C2KV_BF16 0
#define C2KV_F32 1
c2kv_status c2kv_token_logprobs(const void* logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                                const int32_t* tokens, int32_t top_k, float* logprob, float* entropy,
                                int32_t* top_ids, float* top_logprobs, void* stream);

/*
 * Reads and clears the device error word of the current device (waits for
 * the device).  *code receives C2KV_OK, C2KV_ETIMEOUT or C2KV_EDEVICE; the
 * return value is C2KV_ECUDA only if the read itself failed.
 */
c2kv_status c2kv_device_error(int32_t* code);

/*
 * Kernel launches this library has enqueued in the process so far, counted
 * once each when the launch call succeeds (a launch enqueued while a stream
 * is being captured into a CUDA graph counts once, at capture, and not at
 * each replay).  Host-only; never fails except for a null count (C2KV_EINVAL).
 */
c2kv_status c2kv_kernel_launches(uint64_t* count);

/*
 * Test hook for the failure path (the pages have no counterpart): the next
 * n_launches decode launches (c2kv_attend_decode, c2kv_attend_decode_noalloc,
 * c2kv_attend_prefill with q_len 1) each wait, at their first key tile, on a
 * barrier nothing arrives on, for ~0.5 ms of GPU clock.  The wait expires and
 * the kernel takes its timeout path: it records C2KV_ETIMEOUT in the device
 * error word, lets its copies in flight land and returns; that launch's
 * outputs are undefined, the cache rows it appends are written, and the
 * context stays usable.  c2kv_attend_pages8_chunk counts among them, and
 * c2kv_attend_pages8: the rows that it appends may then be missing, and in
 * every other of its CTAs one warp alone gives up, at the last tile of a
 * sequence's head.  0 disarms it.  Process-wide; C2KV_EINVAL for n < 0.
 */
c2kv_status c2kv_test_expire_next_waits(int32_t n_launches);

#ifdef __cplusplus
}
#endif

#endif /* C2KV_H_ */
