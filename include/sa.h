/*
 * sa.h -- C ABI of the GB300 KV-cache attention library (libsa.so).
 *
 * Sixteen operations, all computed on the GPU on the caller's stream:
 *
 *   validate_indices     index-row validation with a device error word
 *   build_present_kv     present K/V = past ++ current (concat or in-place append)
 *   sparse_attn_decode   selected-token attention (dense or FP8 hybrid cache)
 *   attn_prefill         dense (causal) prefill with softcap, present K/V out
 *   paged_attn_decode    causal decode over a page table (element or FP8 pages)
 *   rotary_embed         rotary positions of queries and keys
 *   paged_kv_write       new tokens' K/V, rotated and quantised, into their pages
 *   paged_kv_read        a context read back from its pages into packed rows
 *   attn_prefill_packed  causal prefill of packed sequences of different lengths
 *   attn_weights_packed  the attention weight that each key receives from packed queries
 *   paged_attn_decode_weights  the paged decode, its attention weights accumulated
 *   paged_kv_select      the tokens that each head keeps of a context over its budget
 *   paged_kv_compact     the kept rows moved to the front of their pages, in place
 *   sparse_index_select  ratio-4 index scoring + top-k (produces selected indices)
 *   csa_ratio4_attention compressed sparse attention: window store + records + sink
 *   csa_*_compress       the compression stages that produce the CSA records
 *                        (ratio 128, ratio-4 attention records, ratio-4 index keys)
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every tensor pointer is a DEVICE pointer owned by the caller.  The
 *    library never allocates, frees or synchronises; scratch comes from a
 *    caller-provided workspace whose size is given by the matching
 *    *_workspace() query.  Tensors are dense and row-major in the stated
 *    shape (no strides other than the stated capacity strides).
 *  - `stream` is a cudaStream_t passed as void*; NULL means the legacy default
 *    stream.  All work is enqueued on it; the calls return before it runs.
 *  - Host-side argument errors return a negative status before anything is
 *    enqueued.  Data-dependent problems (malformed index rows, out-of-range
 *    page table entries or write positions) never fail the call: they OR bits
 *    into a caller-zeroed device word `err_word` (read it after your own
 *    synchronisation), and the kernels keep every load in bounds.
 *  - The calls are stateless and thread-safe.  No kernel spins or traps.
 *
 * Sources of the semantics (page title, section):
 *  [IS]  onnx-runtime-ep-cuda src/kernels/index_share.rs (IndexShare):
 *        module docs, validate_indices, build_present, index_share_row.
 *  [SA]  onnx-runtime-ep-cuda src/kernels/standard_attention.rs (ONNX
 *        Attention): module docs "Semantics", build_kv, attention_row,
 *        attention_split / attention_combine (FlashDecoding split-KV).
 *  [CSA] onnx-runtime-ep-cpu src/kernels/compressed_sparse_attention.rs:
 *        CacheFormat (hybrid FP8 record), dequantize_cache; onnx-runtime-ep-cuda
 *        compressed_sparse_attention.rs, csa_ratio128_sink_attention.
 *  [PG]  ferrum-kernels vnext_ops/transformer/causal_attention.rs: paged KV
 *        blocks of 16 tokens addressed through a table.
 *  [CSA-CPU] onnx-runtime-ep-cpu compressed_sparse_attention.rs: the ratio-4
 *        index stream (finalize_index_query, select_ratio4_topk) and the
 *        compression stream (compress_ratio4_stream, pool_ratio4_record,
 *        pool_ratio128_record, finalize_attention_record,
 *        finalize_index_record, apply_compressed_rope).
 */
#ifndef SA_H
#define SA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes (return values) ------------------------------------ */
#define SA_OK 0
#define SA_ERR_NULL (-1)        /* a required pointer is NULL                 */
#define SA_ERR_SHAPE (-2)       /* a size is non-positive or inconsistent     */
#define SA_ERR_DTYPE (-3)       /* unsupported dtype or dtype combination     */
#define SA_ERR_ALIGN (-4)       /* a pointer is not 16-byte aligned           */
#define SA_ERR_WORKSPACE (-5)   /* workspace missing or too small             */
#define SA_ERR_OVERLAP (-6)     /* an output overlaps an input illegally      */
#define SA_ERR_UNSUPPORTED (-7) /* valid request this build does not serve    */
#define SA_ERR_LAUNCH (-8)      /* the CUDA runtime refused a launch          */
#define SA_ERR_SCRATCH_LIMIT (-9) /* sparse_attn_decode_noalloc: scratch needed
                                     exceeds SA_NOALLOC_SCRATCH_BYTES          */

/* ---- storage dtypes --------------------------------------------------- */
#define SA_F32 0
#define SA_F16 1
#define SA_BF16 2
#define SA_FP8_E4M3_B64 3 /* hybrid record: blocks of [E8M0, 64 x E4M3FN] + bf16 tail */
/* page format of a quantised pool (pool_format; 0 = pages of plain elements).
 * A pool is uint8 [num_pages, Hkv, page_tokens * (D + 1)]: per page and KV head
 * first page_tokens rows of D E4M3FN codes, then one E8M0 byte per row; an
 * element is code * 2^(byte - 127), and every element of a row whose byte is
 * 255 is NaN.  D is 64, 128 or 256 and page_tokens a multiple of 16, so that
 * a page of one head is one contiguous, 16-byte aligned piece. */
#define SA_FP8_E4M3_PAGE 4
#define SA_MAX_FORMAT 255 /* formats yet to come lie below this */

/* ---- index-row status codes (row_status bytes; OR-ed into err_word) --- */
#define SA_IDX_BELOW_SENTINEL 1  /* a value below -1                          */
#define SA_IDX_AFTER_PADDING 2   /* a non -1 value after a -1                 */
#define SA_IDX_OUT_OF_RANGE 4    /* a value >= the row's bound                */
#define SA_IDX_NOT_INCREASING 8  /* a value smaller than its predecessor      */
#define SA_IDX_DUPLICATE 16      /* a value equal to its predecessor          */
#define SA_IDX_ALL_PADDING 32    /* the row holds only -1                     */
/* other err_word bits */
#define SA_ERRBIT_WRITE_POS 64   /* build_present_kv: write_pos[b] out of range */
#define SA_ERRBIT_PAGE 128       /* paged: ctx_len or block-table entry invalid */
#define SA_ERRBIT_TIMEOUT 256    /* a kernel's bounded wait for a copy ran out  */
#define SA_ERRBIT_RECORD 2048    /* csa_ratio4_attention: a selected record at or
                                    past the valid records (skipped)             */
#define SA_ERRBIT_COMPRESS 4096  /* csa_*_compress: a record met a non-finite
                                    value and was stored as zeros                */
#define SA_ERRBIT_SEQ 8192       /* packed sequences: the starts decrease or leave
                                    the tensor                                   */
#define SA_ERRBIT_NONFINITE 16384 /* paged_kv_write: a row to quantise held a NaN
                                    or an infinity and is stored as NaN          */

/* ---- sa_sparse_params.options bits ------------------------------------- */
#define SA_OPT_ROW_COPIES 1u     /* dense f16/bf16 caches: fetch each K/V row with
                                    its own bulk copy instead of TMA tensor maps */
#define SA_OPT_FP8_WARP_MMA 2u   /* FP8 records: the warp-level MMA kernel (32-head
                                    blocks) for every head count */

/* Human-readable name of a status code (static string). */
const char* sa_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int sa_version(void);

/*
 * sa_set_kernel_events -- measurement hook (no counterpart on the pages).
 *
 * before, after: cudaEvent_t handles (created by the caller, with timing
 * enabled), or both NULL to turn the hook off.  While set, every call made
 * from this host thread records `before` on its stream immediately before it
 * launches its dominant kernel (the gather kernel of a decode, the tensor-core
 * attention kernel of an FP8 decode, the prefill kernel) and `after`
 * immediately after it, so that the events bracket that one kernel.  The
 * handles are not owned; the caller keeps them alive while the hook is set.
 * Recording between two kernels removes their launch overlap, so timings of
 * whole calls are taken with the hook off.  Under stream capture the records
 * become event-record nodes of the graph (cudaEventRecordExternal), so a
 * replayed graph brackets the kernel the same way.
 * Returns SA_OK, or SA_ERR_NULL if exactly one of the two is NULL.
 */
int sa_set_kernel_events(void* before, void* after);

/*
 * sa_graph_kernel_count -- measurement hook (no counterpart on the pages): the
 * number of kernel nodes in a CUDA graph (a cudaGraph_t, not owned), e.g. one
 * library call captured from a stream, so that a benchmark can state how many
 * of the library's kernels one call launches.  Returns the count, or a
 * negative status (SA_ERR_NULL for a NULL graph, SA_ERR_LAUNCH if the graph
 * cannot be read).
 */
int sa_graph_kernel_count(void* graph);

/*
 * sa_check_wait_timeout -- diagnostic (no counterpart on the pages): runs the
 * library's bounded-wait timeout path on purpose, without a fault.
 *
 * Every pipelined kernel waits on its shared-memory barriers for at most about
 * 2e9 SM cycles (about one second), then ORs SA_ERRBIT_TIMEOUT into the
 * caller's error word, sets its CTA's abort flag and returns, leaving the
 * context usable.  A correct call never takes that path; this call makes one
 * warp wait on a barrier that nothing arrives on (no copy or MMA in flight),
 * then wait once more on the abort flag the first wait set.
 *
 * err_word: device pointer to one uint32 (zeroed by the caller), receives
 *           SA_ERRBIT_TIMEOUT.
 * out:      device pointer to four uint32: [0] 1 if the first wait gave up,
 *           [1] 1 if the second returned at once, [2], [3] the first wait's
 *           SM cycles (low, high word).
 * stream:   cudaStream_t or NULL.  Asynchronous; about one second of device
 *           time on one SM.
 * Returns SA_OK, SA_ERR_NULL, SA_ERR_ALIGN (a pointer not 4-byte aligned) or
 * SA_ERR_LAUNCH.
 */
int sa_check_wait_timeout(uint32_t* err_word, uint32_t* out, void* stream);

/*
 * validate_indices -- [IS] validate_indices / validate_index_rows.
 *
 * idx: [B, I, Sq, K] int32 (idx_is_i64 = 0) or int64 (idx_is_i64 = 1).
 * Each row is scanned left to right: -1 marks padding; any other value is
 * checked, in this order, for being below -1, following padding, being
 * >= bound, equal to its predecessor, smaller than it.  The first failing
 * column decides the row's code; a row of only -1 is SA_IDX_ALL_PADDING.
 * bound_per_batch: nullable device int64 [B]; when NULL every row is bounded
 * by `bound`.
 * row_status: nullable device uint8 [B*I*Sq], written with each row's code
 * (0 = valid).  err_word: device uint32, OR-ed with every row's code (the
 * caller zeroes it).  Bit-exact with the definition.
 */
int validate_indices(const void* idx, int idx_is_i64, int64_t B, int64_t I, int64_t Sq,
                     int64_t K, const int64_t* bound_per_batch, int64_t bound,
                     uint8_t* row_status, uint32_t* err_word, void* stream);

/*
 * build_present_kv -- [IS] build_present, [SA] build_kv.  A pure copy
 * (bit-exact), for K and (optionally) V in one launch.
 *
 * Concat mode (write_pos == NULL):
 *   present[b,h,t,:] = past[b,h,t,:]      for t <  P   (past is [B,H,P,D])
 *                    = cur[b,h,t-P,:]     for P <= t < P+C (cur is [B,H,C,D])
 *   present is [B, H, present_stride, D] with present_stride >= P + C;
 *   positions >= P + C are not written.  past may be NULL only when P == 0.
 *   present must not overlap past or cur (SA_ERR_OVERLAP).
 * Append mode (write_pos != NULL, device int64 [B]):
 *   present is a capacity cache [B, H, present_stride, D]; cur[b,h,c,:] is
 *   written at position write_pos[b] + c.  past must be NULL or equal to
 *   present (in place: nothing else moves); another past [B,H,present_stride,D]
 *   is first copied whole.  A write_pos outside [0, present_stride - C] skips
 *   that batch and sets SA_ERRBIT_WRITE_POS in err_word (nullable).
 * past_v/cur_v/present_v: the same for V; present_v NULL means K only.
 * dtype: SA_F32, SA_F16 or SA_BF16 (any 2/4-byte element copies exactly).
 */
int build_present_kv(const void* past_k, const void* cur_k, void* present_k,
                     const void* past_v, const void* cur_v, void* present_v, int dtype,
                     int64_t B, int64_t H, int64_t P, int64_t C, int64_t D,
                     int64_t present_stride, const int64_t* write_pos, uint32_t* err_word,
                     void* stream);

/*
 * Selected-token attention -- [IS] index_share_row (semantics), [SA]
 * Semantics + attention_split/attention_combine (split-KV, fixed-order
 * combine), [CSA] dense window + FP8 records + sink.
 *
 * For every output row (b, h, i) with kvh = h / (Hq/Hkv) and index head
 * ih = 0 (I == 1), kvh (I == Hkv) or h (I == Hq):
 *   C = valid prefix of idx[b, ih, i, :] (entries before the first -1);
 *   with window W > 0: C = [len_b - W, len_b) united with {j in C : j < len_b - W};
 *   s_j = scale * q . k_j;  s_j = softcap * tanh(s_j / softcap) if softcap != 0;
 *   s_j += bias(b, h, i, j) when bias != NULL ([IS] index_share_row / bias_at:
 *         keyed by the cache position j);
 *   s_j = -inf when j >= len_b (len_b = kv_len[b], or T), or causal and
 *         j > past_len + i;
 *   y = sum_j softmax(s)_j v_j, with exp(sink[h] - max) added to the
 *   denominator when sink != NULL; a row whose scores are all -inf gives 0.
 * Layouts:
 *   q  [B, Hq, Sq, D] in q_dtype (F32, F16, BF16);  y [B, Hq, Sq, Dv] same dtype.
 *   dense cache (kv_dtype == q_dtype): k_cache [B, Hkv, T, D], v_cache [B, Hkv, T, Dv].
 *   FP8 cache (kv_dtype SA_FP8_E4M3_B64, q_dtype BF16): k_cache is
 *     [B, Hkv, T, record_stride] bytes, each record (D - n_rope)/64 blocks of
 *     [E8M0 scale, 64 E4M3FN codes] then n_rope little-endian bf16 values;
 *     V is the same decoded record (its first Dv dims); v_cache is ignored.
 *   idx [B, I, Sq, K] int32 or int64.  kv_len: nullable device int64 [B].
 *   sink: nullable device float [Hq] (natural-log logits).
 *   bias: nullable device float32, dense row-major of shape
 *     bias_dims[0 .. bias_rank-1] with 0 <= bias_rank <= 4, broadcast against
 *     [B, Hq, Sq, T] from the right ([IS] validate_bias_shape: every axis is 1
 *     or the extent it lines up with; otherwise SA_ERR_SHAPE).  Entries are
 *     finite or -inf (a -inf masks its key); the bias counts only for the
 *     candidate keys, each read at its cache position.
 * options: 0, or SA_OPT_* bits choosing a kernel variant (the result is the
 * same operation; tests use them to cover every path).
 * scale: 0 means 1/sqrt(D).  Index rows are validated on the device against
 * len_b when err_word != NULL (row_status nullable, as in validate_indices);
 * malformed rows never fault: negative entries are skipped, entries >= len_b
 * are masked, and the other entries of such a row (after padding, repeated or
 * out of order) are attended as they stand.  A malformed row's output is
 * finite; only a well-formed row's output is the definition above.
 * Fused append (dense cache only): when k_cur != NULL, the current token(s)
 * k_cur / v_cur [B, Hkv, cur_len, D] are first written into the cache at
 * positions write_pos[b] .. write_pos[b] + cur_len - 1 (write_pos: nullable
 * device int64 [B], NULL meaning T - cur_len) -- build_present_kv's append
 * mode -- and attention sees them there.  A write position outside
 * [0, T - cur_len] sets SA_ERRBIT_WRITE_POS and skips that batch's write.
 * Workspace: sparse_attn_decode_workspace(p) bytes, 256-byte aligned; its
 * contents on entry do not matter (every word is written before it is read).
 * It holds the planned candidate positions and the key splits' partial
 * results; for the FP8 cache with Hq a multiple of 128 also the decoded
 * candidates (B * Sq * ceil((window + K) / 128) * 128 rows of D bf16 values,
 * e.g. 40 MB for B 16, 2176 candidates, D 576).  Calls that share a workspace
 * must not overlap on the GPU.
 */
typedef struct {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const void* idx;
  const float* sink;
  void* y;
  int32_t q_dtype;
  int32_t kv_dtype;
  int32_t idx_is_i64;
  int32_t causal;
  int64_t B, Hq, Hkv, Sq, D, Dv, T, I, K;
  const int64_t* kv_len;
  int64_t past_len;
  float scale;
  float softcap;
  int64_t window;
  int64_t record_stride;
  int64_t n_rope;
  uint32_t* err_word;
  uint8_t* row_status;
  const void* k_cur;
  const void* v_cur;
  const int64_t* write_pos;
  int64_t cur_len;
  void* workspace;
  size_t workspace_bytes;
  const float* bias;
  int64_t bias_rank;
  int64_t bias_dims[4];
  uint32_t options;
  uint32_t reserved_;   /* must be 0 */
} sa_sparse_params;

size_t sparse_attn_decode_workspace(const sa_sparse_params* p);
int sparse_attn_decode(const sa_sparse_params* p, void* stream);

/*
 * sparse_attn_decode_noalloc -- the same operation as sparse_attn_decode for
 * callers that cannot allocate device memory themselves: runtimes that own a
 * fixed device-memory budget and account for every byte, plugins whose host
 * framework passes them inputs and outputs but no scratch, or code that must
 * not set off cudaMalloc's implicit device synchronisation (or be refused it
 * during a global-mode stream capture).  The pages have no counterpart: it is
 * a deployment variant of this library's own entry point.
 *
 * p->workspace / p->workspace_bytes are ignored.  Scratch comes from one
 * built-in device buffer of SA_NOALLOC_SCRATCH_BYTES, which every GPU that
 * loads the library holds until the process exits; a request needing more
 * (sparse_attn_decode_workspace(p) > SA_NOALLOC_SCRATCH_BYTES) returns
 * SA_ERR_SCRATCH_LIMIT before anything is enqueued.  Nothing is allocated or
 * freed.  The first call on each device looks up that buffer's device
 * address (once, with that device current); make that first call before any
 * stream capture.  The address is kept for the life of the process: a device
 * reset (cudaDeviceReset) while the library is loaded is not supported by this
 * entry point, since the kept address would then be stale.  Every call
 * shares the buffer and it keeps the last call's contents (the call needs
 * none of it cleared: all scratch is written before it is read), so calls
 * that overlap on the GPU -- on different streams, or from different
 * threads, of the same device -- race and must be serialised by the caller.
 */
#define SA_NOALLOC_SCRATCH_BYTES (16u << 20)
int sparse_attn_decode_noalloc(const sa_sparse_params* p, void* stream);

/*
 * sparse_index_select -- ratio-4 index scoring and top-k selection, the step
 * that produces the selected indices: [CSA-CPU] finalize_index_query,
 * hadamard_bf16, fp4_roundtrip, select_ratio4_topk; [CSA]
 * csa_ratio4_index_select, csa_ratio4_index_replicate.
 *
 * For each row (b, s), at position p = query_start (or query_start_b[b]) + s:
 *   q_h = fp4_roundtrip(hadamard_bf16(bf16(query[b, s, h, :])))   per head h,
 *     the Walsh-Hadamard transform with a 1/sqrt(ID) scale rounded to bf16,
 *     then every block of 32 rounded to FP4 E2M1 with an E8M0 scale by the
 *     OCP MX rule (scale 2^(floor(log2 amax) - 2), nearest value, ties to
 *     even, saturating);
 *   score_r = sum_h relu(q_h . k_r) * weight[b, s, h] * c,  c = (1/sqrt(ID))/sqrt(IH),
 *     for the causal records r < min(R, (p + 1) / 4), in binary32: each dot
 *     product summed in ascending dimension order, the heads in ascending
 *     order, every multiply and add rounded on its own (the pages' order; the
 *     result is that definition bit for bit);
 *   the records ranked by score (Rust f32::total_cmp, higher first) and then
 *   by record index; the first topk written, -1 after them.
 * The compressed RoPE of the query's last components is the caller's: the
 * query enters after it.
 *
 * query: float32 [B, S, IH, ID], ID in {32, 64, 128, 256}; weight: float32
 * [B, S, IH]; keys: [B, R, key_stride] bytes, each record ID/32 blocks of
 * [E8M0 scale byte, 16 bytes of E2M1 codes, element 2j in the low nibble of
 * byte j] (68 bytes for ID 128), key_stride a multiple of 4, keys 4-byte
 * aligned.  selected: int32 [B, out_heads, S, topk], the same row for every
 * output head ([CSA] replicate); ascending = 1 writes the selected records
 * in ascending record order instead of score order (the form
 * sparse_attn_decode validates).  1 <= topk <= 4096, 1 <= IH <= 256.
 * row_status (nullable uint8 [B*S]) and err_word (nullable): SA_SEL_TIE when
 * two scores of the row are equal (the pages refuse such input; the ranking
 * still orders them by record), SA_SEL_NONFINITE when a score is NaN or
 * infinite; err_word receives them shifted into SA_ERRBIT_SEL_*.
 * Workspace: sparse_index_select_workspace(p) bytes, 256-byte aligned,
 * contents on entry irrelevant.  Deterministic.
 */
#define SA_SEL_TIE 1
#define SA_SEL_NONFINITE 2
#define SA_ERRBIT_SEL_TIE 512
#define SA_ERRBIT_SEL_NONFINITE 1024
typedef struct {
  const float* query;
  const float* weight;
  const uint8_t* keys;
  int32_t* selected;
  uint8_t* row_status;
  uint32_t* err_word;
  int64_t B, S, IH, ID, R, topk, key_stride, out_heads;
  int64_t query_start;
  const int64_t* query_start_b;
  int32_t ascending;
  int32_t reserved_;    /* must be 0 */
  void* workspace;
  size_t workspace_bytes;
} sa_index_select_params;

size_t sparse_index_select_workspace(const sa_index_select_params* p);
int sparse_index_select(const sa_index_select_params* p, void* stream);

/*
 * csa_ratio4_attention -- compressed sparse attention, ratio 4, in the pages'
 * own form: [CSA-CPU] ratio4_attention (with its call in execute_ratio4),
 * [CSA] csa_ratio4_sink_attention.
 *
 * For query s of batch b at position p = total - S + s, with base = total - L
 * (the position of current_kv row 0):
 *   dense slots c < dense (dense = 128, or min(L, 128) when total == S): the
 *     current_kv row at position max(base, p + 1 - 128) + c when that is <= p
 *     and stored (row < L), else no candidate;
 *   slot dense + k: selected record selected[b, s, k] when it lies in
 *     [0, min(R, total / 4)); a negative entry is no candidate, one at or past
 *     that bound is skipped and sets SA_ERRBIT_RECORD (err_word nullable);
 *   score = scale * q . row + bias(b, h, s, slot) (bias nullable, float32,
 *     rank <= 4, broadcast right-aligned against [B, H, S, dense + topk]);
 *   y = sum softmax(score) row, with exp(sink[h] - max) added to the
 *     denominator (sink nullable); a query with no candidate gives 0.
 * K = V = the row: current_kv is one latent head; a record decodes as
 * (D - n_rope) / 64 blocks of [E8M0 scale, 64 E4M3FN] then n_rope LE bf16
 * (583 bytes at D 512, n_rope 64; any byte alignment).
 * Layouts: query / y [B, S, H, D] (q_dtype SA_F32 or SA_BF16, y the same);
 * current_kv [B, L, D] (kv_dtype SA_F32 or SA_BF16); records [B, R,
 * record_stride] bytes; selected int32 [B, S, topk].  D 128 or 512, H a
 * multiple of 32, n_rope even with D - n_rope a positive multiple of 64.
 * Arithmetic: rows and queries as bf16 (float inputs rounded; FP8 records
 * exact) on the tensor cores with fp32 accumulation and softmax.
 * Workspace: csa_ratio4_attention_workspace(p) bytes, 256-byte aligned,
 * contents on entry irrelevant (the candidate rows, B * S * (dense + topk)
 * rows of D bf16, and split partials).
 */
typedef struct {
  const void* query;
  const void* current_kv;
  const uint8_t* records;
  const int32_t* selected;
  const float* sink;
  const float* bias;
  int64_t bias_rank;
  int64_t bias_dims[4];
  void* y;
  int32_t q_dtype;
  int32_t kv_dtype;
  int64_t B, S, H, D, n_rope, L, R, topk, record_stride, total;
  float scale;          /* 0: 1/sqrt(D) */
  int32_t reserved_;    /* must be 0 */
  uint32_t* err_word;
  void* workspace;
  size_t workspace_bytes;
} sa_csa_params;

size_t csa_ratio4_attention_workspace(const sa_csa_params* p);
int csa_ratio4_attention(const sa_csa_params* p, void* stream);

/*
 * csa_ratio128_compress / csa_ratio4_main_compress / csa_ratio4_index_compress
 * -- the compression stages that produce the CSA records: [CSA-CPU]
 * compress_ratio4_stream, pool_ratio4_record, pool_ratio128_record,
 * finalize_attention_record, finalize_index_record, apply_compressed_rope;
 * [CSA] csa_ratio128_compress, csa_ratio4_main_compress,
 * csa_ratio4_index_compress.
 *
 * One call appends S tokens per sequence at positions start = total - S ..
 * total - 1.  Token p's score row is gate + ape[p % ratio].  Every block of
 * `ratio` tokens that closes in [start, total) emits record k = p / ratio
 * (p its last token), computed at block_start = k * ratio:
 *   pool: per dimension d, over the candidates in order -- ratio 128: the
 *     block's 128 tokens; ratio 4: the previous block's 4 tokens on source
 *     dim d, then the block's 4 tokens on source dim D + d (a token before
 *     position 0 is no candidate) -- the weighted mean sum(w v) / sum(w)
 *     with w = e^(score - max score) (the binary32 rounding of the exact
 *     value), candidates of score -inf left out; then bf16;
 *   RMSNorm: binary32 square sum in dimension order, times
 *     1 / sqrt(sum / D + 1e-6), times norm[d], bf16;
 *   compressed RoPE of the last n_rope dims, pair i = dims (D - n_rope + 2i,
 *     +1): frequency f = b (1 - r) + (b / 16) r with b = 160000^(-2i/n_rope)
 *     and r = clamp((i - 15) / 10, 0, 1), angle = block_start * f (binary32),
 *     cos and sin rounded from their exact values; each component bf16;
 *   attention records (main, ratio 128): (D - n_rope) / 64 blocks of
 *     [E8M0 byte, 64 E4M3FN codes] -- the block exponent is the smallest e
 *     with amax / 2^e <= 448 (0 for a zero block), codes the nearest-even
 *     E4M3FN of x / 2^e -- then the n_rope dims as little-endian bf16:
 *     (D - n_rope) / 64 * 65 + 2 n_rope bytes (583 at D 512, n_rope 64);
 *   index keys: the Walsh-Hadamard transform (butterflies of span 1, 2, 4,
 *     ..., then times 1 / sqrt(D), bf16), then D / 32 blocks of [E8M0 byte,
 *     16 bytes of FP4 E2M1 codes, even element in the low nibble] with the
 *     OCP MX scale 2^(floor(log2 amax) - 2) (byte 0 for a zero block):
 *     D / 32 * 17 bytes (68 at D 128).
 * Every step is one binary32 operation rounded to nearest, in this order.
 * A record that meets a non-finite value (no finite score in a dimension,
 * an unusable sum, a non-finite square sum or result) is stored as zeros and
 * sets SA_ERRBIT_COMPRESS in err_word (nullable).
 *
 * Layouts (float32 unless stated): kv, gate [B, S, W] with W = D (ratio
 * 128) or 2 D (ratio 4); ape [ratio, W]; norm [D]; carry [B, slots, 2, W]
 * with slots 128 (ratio 128) or 8 (ratio 4), channel 0 the value and 1 the
 * score, read and rewritten in place: it holds the open block's tokens (slot
 * p % 128, or 4 + p % 4) and, at ratio 4, the last closed block's (slots
 * 0..3); empty slots hold (0, -inf).  A call with start == 0 ignores the
 * carry's contents.  records [B, rows, record_stride] bytes and logical
 * [B, rows, D] (the record's dequantized values), each nullable but not
 * both: row k is written, the others untouched.  rows >= total / ratio.
 * Shapes: attention records need D % 4 == 0, D <= 1024, (D - n_rope) % 64
 * == 0; index keys D in {32, 64, 128, 256}; n_rope even, <= min(D, 128).
 * kv, gate, ape and carry 16-byte aligned.  No workspace.
 */
typedef struct {
  const float* kv;
  const float* gate;
  const float* ape;
  const float* norm;
  float* carry;
  uint8_t* records;
  float* logical;
  uint32_t* err_word;
  int64_t B, S, D, n_rope, rows, record_stride, total;
  int64_t reserved_;  /* must be 0 */
} sa_compress_params;

int csa_ratio128_compress(const sa_compress_params* p, void* stream);
int csa_ratio4_main_compress(const sa_compress_params* p, void* stream);
int csa_ratio4_index_compress(const sa_compress_params* p, void* stream);

/*
 * csa_pool_weight -- w[i] = e^t[i] rounded to binary32 (nearest even), the
 * pool weight of the compression stages, for checking that rounding on its
 * own: t, w device float32 [n] (t <= 0 is the compression's domain; any
 * value is accepted).  Returns SA_OK or an argument error.
 */
int csa_pool_weight(const float* t, float* w, int64_t n, void* stream);

/* attention-mask element types of sa_prefill_params.mask_kind */
#define SA_MASK_NONE 0
#define SA_MASK_F32 1
#define SA_MASK_F16 2
#define SA_MASK_BF16 3
#define SA_MASK_BOOL 4  /* one byte per element: nonzero keeps the key */

/*
 * attn_prefill -- [SA] Semantics with no past: q [B, Hq, S, D],
 * k/v [B, Hkv, S, D] (GQA, Hq % Hkv == 0), y [B, Hq, S, D]; query i sees
 * keys 0..i when causal; softcap as above, applied before the mask; fp32
 * softmax.  present_k / present_v (nullable, [B, Hkv, S, D]) receive exact
 * copies of k / v (past ++ current with an empty past).  dtype: SA_BF16 or
 * SA_F16, or SA_F32.  Workspace rules as for sparse_attn_decode.
 * bf16 / f16 with D in {64, 128}, a positive scale and 16-byte aligned
 * q / k / v / y run on the tcgen05 tensor-core kernel and need no workspace
 * (a misaligned y there is SA_ERR_ALIGN); other shapes take the general
 * kernel.  err_word (nullable) receives SA_ERRBIT_TIMEOUT if the tensor-core
 * pipeline stalled, in which case y is unspecified.
 * nonpad_kv_seqlen (nullable device int64 [B]; [SA] attention_row's padding
 * frontier): keys j >= nonpad[b] are masked (a negative entry disables that),
 * and a causal query i then sees keys j <= i + nonpad[b] - S; a row left with
 * no key gives 0.  Served by the tcgen05 kernel.
 * attn_mask (nullable device, [SA] mask_bias): mask_kind elements in a dense
 * row-major tensor of shape mask_dims[0 .. mask_rank-1], rank <= 4, broadcast
 * right-aligned against [B, Hq, S, S] (every axis but the last 1 or its
 * target; the last is the key axis: keys at or past its extent take -inf);
 * float masks add their value after the softcap, bool masks keep a key where
 * nonzero.  A request with a mask runs on the per-row kernels (correct, not
 * tuned) and writes present K/V by a separate copy.
 */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  void* y;
  void* present_k;
  void* present_v;
  int32_t dtype;
  int32_t causal;
  int64_t B, Hq, Hkv, S, D;
  float scale;
  float softcap;
  void* workspace;
  size_t workspace_bytes;
  uint32_t* err_word;   /* nullable: SA_ERRBIT_TIMEOUT if a tensor-core pipeline stalled */
  const void* attn_mask;
  int32_t mask_kind;    /* SA_MASK_NONE / _F32 / _F16 / _BF16 / _BOOL */
  int32_t reserved_;    /* must be 0 */
  int64_t mask_rank;
  int64_t mask_dims[4];
  const int64_t* nonpad_kv_seqlen;
} sa_prefill_params;

size_t attn_prefill_workspace(const sa_prefill_params* p);
int attn_prefill(const sa_prefill_params* p, void* stream);

/*
 * paged_attn_decode -- [PG] paged causal decode.  One new query per
 * sequence: q [B, Hq, D], y [B, Hq, D].  Pools k_pool / v_pool are
 * [num_pages, Hkv, page_tokens, D]; token t of sequence b lives at page
 * block_table[b * max_pages + t / page_tokens], slot t % page_tokens.
 * ctx_len[b] (device int32) counts the new token, which attends to all
 * ctx_len[b] tokens.  If k_new / v_new ([B, Hkv, D]) are given they are first
 * written into the pool at token ctx_len[b] - 1.  A ctx_len outside
 * [1, max_pages*page_tokens] or a table entry outside [0, num_pages) sets
 * SA_ERRBIT_PAGE (err_word nullable) and is never dereferenced.
 * dtype SA_F16 / SA_BF16 / SA_F32; scale 0 means 1/sqrt(D).  Workspace rules
 * as for sparse_attn_decode.
 * pool_format SA_FP8_E4M3_PAGE: quantised pages (q and y SA_F16 or SA_BF16, D
 * 64 / 128 / 256, page_tokens a multiple of 16, B <= 4096, q, y and pools 16-byte
 * aligned, options 0); k_new / v_new are quantised as paged_kv_write does.  The codes'
 * values enter the products exactly and the K scales in fp32; a row's weight, its
 * probability times its V scale, is held to 2^-22 of itself or 2^-31 of the largest
 * weight of a row that is not zero, whichever is more (V beyond 2^118 in magnitude
 * may overflow the fp32 sums).  B * Hkv (times the parts that a
 * group of more than 16 heads, 8 for D 256, is cut into) * (max_pages * page_tokens /
 * 16 + 2) has to stay below 2^31 - 2^20.
 */
typedef struct {
  const void* q;
  void* k_pool;
  void* v_pool;
  const void* k_new;
  const void* v_new;
  const int32_t* block_table;
  const int32_t* ctx_len;
  void* y;
  int32_t dtype;
  uint32_t options;     /* 0, or SA_OPT_ROW_COPIES (pages fetched row by row) */
  int64_t B, Hq, Hkv, D, page_tokens, max_pages, num_pages;
  float scale;
  int32_t pool_format;  /* 0: elements of dtype, or SA_FP8_E4M3_PAGE.  Padding before
                           version 0.2: what is no format, 1 .. SA_MAX_FORMAT,
                           counts as 0 */
  uint32_t* err_word;
  void* workspace;
  size_t workspace_bytes;
} sa_paged_params;

size_t paged_attn_decode_workspace(const sa_paged_params* p);
int paged_attn_decode(const sa_paged_params* p, void* stream);

/*
 * Rotary positions -- sa_rope_table fills a table of angles from a
 * configuration (host only, nothing is launched), which rotary_embed and
 * paged_kv_write take.  Pair i (of rotary_dim / 2) turns by the angle
 * position * f_i, with f_i, in 64 bits,
 *   SA_ROPE_NONE    base^(-2i / rotary_dim)
 *   SA_ROPE_LINEAR  that / factor
 *   SA_ROPE_NTK     the same with base * factor^(rotary_dim / (rotary_dim - 2))
 *   SA_ROPE_RAMP    f (g + (1 - g) / factor), f the plain frequency and
 *                   g = clamp((r - ramp_low) / (ramp_high - ramp_low), 0, 1) of the
 *                   pair's turns r = original_len f / (2 pi) over the original
 *                   context: fast pairs keep their frequency, slow ones take the
 *                   linear scaling
 *   SA_ROPE_FREQS   inv_freq[i], given by the caller
 * and (u, v) becomes mscale * (u cos - v sin, u sin + v cos).  The pair is
 * dims (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved; dims from
 * rotary_dim on pass unchanged.  The table keeps f_i as a 64-bit fraction of a
 * turn, so position times that fraction modulo one turn is exact integer arithmetic
 * (int32 or int64 positions, negative ones too); the fraction is f_i rounded to a
 * double, about 2^-53 of itself, an error that grows with the position.
 * rotary_dim: even, 2 .. 256.  mscale 0 means 1.  Returns SA_OK, SA_ERR_NULL,
 * SA_ERR_SHAPE (a size or a parameter out of its range: base <= 0, factor <= 0,
 * ramp_high <= ramp_low, original_len <= 0 where it is used, a frequency that
 * is not finite) or SA_ERR_UNSUPPORTED (an unknown scaling).
 */
#define SA_ROPE_NONE 0
#define SA_ROPE_LINEAR 1
#define SA_ROPE_NTK 2
#define SA_ROPE_RAMP 3
#define SA_ROPE_FREQS 4
#define SA_ROPE_MAX_PAIRS 128
typedef struct {
  int32_t rotary_dim, interleaved, scaling;
  float mscale;
  double base, factor, original_len, ramp_low, ramp_high;
  const double* inv_freq; /* SA_ROPE_FREQS: host [rotary_dim / 2] */
} sa_rope_config;
typedef struct {
  int32_t rotary_dim, interleaved;
  float mscale;
  int32_t reserved_; /* 0 */
  uint64_t turns[SA_ROPE_MAX_PAIRS]; /* f_i / (2 pi) * 2^64 modulo 2^64 */
} sa_rope;
int sa_rope_table(const sa_rope_config* c, sa_rope* out);

/*
 * rotary_embed -- rotary positions of q [B, S, Hq, D] and, when k != NULL,
 * k [B, S, Hk, D], in one launch.  Tensors are given by their batch, token and
 * head strides in elements (the D elements of a head are contiguous), so
 * packed [T, H, D] tensors (B = 1), head-major [B, H, S, D] tensors and views
 * into a fused projection all serve.  positions: device int32 or int64, token
 * s of batch b at positions[b * pos_stride + s] (pos_stride 0: one row of S
 * positions for every batch).  q_out / k_out may be the input itself (same
 * pointer and strides); any other overlap is SA_ERR_OVERLAP.  dtype SA_F32,
 * SA_F16 or SA_BF16; the reduced angle is rounded to fp32 (2^-25 of a half turn),
 * cos and sin and the rotation are fp32, rounded once.  S 0 is a call that does nothing; B * S of 2^31 - 256 and
 * more is SA_ERR_UNSUPPORTED.
 */
typedef struct {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const void* positions;
  const sa_rope* rope; /* host */
  int32_t dtype;
  int32_t pos_is_i64;
  int64_t B, S, Hq, Hk, D;
  int64_t pos_stride;
  int64_t q_strides[3], k_strides[3], q_out_strides[3], k_out_strides[3];
} sa_rotary_params;
int rotary_embed(const sa_rotary_params* p, void* stream);

/*
 * paged_kv_write / paged_kv_read -- packed rows of K and V to and from pages.
 *
 * k / v [T, Hkv, D] in dtype (SA_F32, SA_F16, SA_BF16), given by their token
 * and head strides in elements.  Sequence b owns rows seq_start[b] ..
 * seq_start[b + 1] - 1 (device int32 [B + 1], non-decreasing; rows behind the
 * last sequence belong to nobody).  Pages as for paged_attn_decode.
 *
 * paged_kv_write: the n_b rows of sequence b are the last n_b tokens of its
 * ctx_len[b]: row seq_start[b] + i is written at token ctx_len[b] - n_b + i.
 * seq_start NULL means one row per sequence (T == B).  With rope != NULL, K is
 * rotated at that token's position first, in fp32.  Pages of plain elements
 * take dtype's own elements (an exact copy, or the rotated row rounded once);
 * SA_FP8_E4M3_PAGE rows are quantised from the fp32 row: the exponent is the
 * smallest e with max|row| / 2^e <= 448 (0 for a row of zeros, at least -127),
 * the codes the nearest-even E4M3FN of x / 2^e.  A row that holds a NaN or an
 * infinity is stored with scale byte 255 (reads as NaN) and sets
 * SA_ERRBIT_NONFINITE.  Nothing else in the pools is touched.
 *
 * paged_kv_read: rows seq_start[b] + i receive token i of sequence b (its first
 * n_b tokens); rope must be NULL.  The values are exact products rounded once
 * to dtype.  Rows behind the last sequence stay as they are.
 *
 * A table entry outside [0, num_pages), a token outside [0, ctx_len[b]) or a
 * ctx_len outside [0, max_pages * page_tokens] sets SA_ERRBIT_PAGE, starts that
 * decrease or leave [0, T] set SA_ERRBIT_SEQ (err_word nullable); such rows are
 * skipped, and no access leaves the tensors.  Two rows written to one slot (a
 * page shared by two sequences) leave bytes of both there, in no order.
 * pool_format 0 (pages [num_pages, Hkv, page_tokens, D] of dtype) serves any D
 * up to 1024; the rope then needs rotary_dim <= D.  T below 2^31 - 256.  No
 * workspace.
 */
typedef struct {
  void* k;
  void* v;
  void* k_pool;
  void* v_pool;
  const int32_t* block_table; /* [B, max_pages] */
  const int32_t* ctx_len;     /* [B] */
  const int32_t* seq_start;   /* [B + 1] */
  const sa_rope* rope;        /* host, nullable */
  uint32_t* err_word;
  int32_t dtype;
  int32_t pool_format;
  int64_t T, B, Hkv, D, page_tokens, max_pages, num_pages;
  int64_t k_strides[2], v_strides[2]; /* token, head */
} sa_kv_pages_params;
int paged_kv_write(const sa_kv_pages_params* p, void* stream);
int paged_kv_read(const sa_kv_pages_params* p, void* stream);

/*
 * attn_prefill_packed -- attn_prefill's attention over packed sequences of
 * different lengths: q / y [Tq, Hq, D], k / v [Tk, Hkv, D] (GQA), given by
 * their token and head strides in elements.  Sequence b has the query rows
 * q_start[b] .. q_start[b + 1] - 1 and the key rows k_start[b] .. (device int32
 * [B + 1], non-decreasing; k_start NULL: q_start).  With nq queries and nk
 * keys, query i sees keys j <= i + nk - nq when causal (the ends are aligned:
 * a chunk of a prompt sees the context before it), every key otherwise; a
 * query that sees no key gives 0.  softcap as in attn_prefill, scale 0 means
 * 1/sqrt(D).  Rows of y behind the last sequence stay as they are; rows of q,
 * k and v outside the sequences may hold anything.  Scores, row sums and outputs are
 * summed in fp32; SA_F16 and SA_BF16 on the tensor cores round each probability to
 * that type before its product with v.
 * dtype SA_F16 / SA_BF16 with D 64 or 128, a positive scale, Hq / Hkv <= 128
 * and 16-byte aligned pointers and strides run on the tcgen05 tensor cores;
 * other shapes (SA_F32, D a multiple of 4 up to 256) take a kernel on the fp32
 * pipes.  Malformed starts set SA_ERRBIT_SEQ (err_word nullable), leave y
 * unspecified and read or write nothing outside the tensors.  No workspace.
 */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  void* y;
  const int32_t* q_start;
  const int32_t* k_start;
  uint32_t* err_word;
  int32_t dtype;
  int32_t causal;
  int64_t B, Tq, Tk, Hq, Hkv, D;
  int64_t q_strides[2], k_strides[2], v_strides[2], y_strides[2]; /* token, head */
  float scale;
  float softcap;
} sa_packed_params;
int attn_prefill_packed(const sa_packed_params* p, void* stream);

/*
 * Cache eviction -- the operators that keep a paged cache within a budget of tokens
 * by the attention that its tokens receive.
 *
 * A weights pool is float32 [num_pages, Hkv, page_tokens], addressed like the pages of
 * K and V: the accumulated weight of token t of sequence b and KV head h lies at page
 * block_table[b * max_pages + t / page_tokens], head h, slot t % page_tokens.  A token's
 * weight is the sum of the softmax probabilities that the queries of the KV head's
 * group give it.  Two calls accumulate it.  Both SET the weights of the tokens that
 * are new with them (so that a page that changes hands needs no clearing) and ADD to
 * the others'.  Of a page that two sequences of one call share, a token to which both
 * add receives the weights of both, in no order; one that either sets holds the weights
 * of either, added to or not (let one sequence alone set such tokens).
 * Sums and softmax statistics are fp32.
 *
 * After a compaction a token's place in its pages is no longer its position: rotate
 * with rotary_embed and the true positions, and write with paged_kv_write without a rope.
 */

/*
 * attn_weights_packed -- the weights that packed queries give the keys of their
 * sequences: q [Tq, Hq, D], k [Tk, Hkv, D] (GQA), starts and strides as for
 * attn_prefill_packed, causal: with nq queries and nk keys, query i sees the keys
 * j <= i + nk - nq.  For sequence b and KV head h
 *   w_j = sum over the queries i and the heads of h's group of
 *         softmax_j(scale q_i . k_j)        (a query that sees no key gives nothing)
 * and the weight of token j is set to w_j where j >= nk - nq (the queries' own tokens) or
 * accumulate is 0, else w_j is added to it.  All queries of a prompt, a chunk's, or
 * the last few of a context may be given.  Sequences without queries or keys, and
 * slots that hold no token, are left as they are.  The scores have no softcap: the weights
 * are not those that attn_prefill_packed gives with one.
 * scale 0 means 1/sqrt(D).  dtype SA_F16 / SA_BF16 with D 64 or 128, a positive scale,
 * Hq / Hkv <= 128 and 16-byte aligned pointers and strides run on the tcgen05 tensor
 * cores; other shapes (SA_F32, D a multiple of 4 up to 256) take a kernel on the fp32
 * pipes.  Malformed starts set SA_ERRBIT_SEQ (err_word nullable) and nothing is
 * written; a table entry outside [0, num_pages), or a token past max_pages *
 * page_tokens, sets SA_ERRBIT_PAGE and that token is skipped.  Workspace:
 * attn_weights_packed_workspace(p) bytes, 256-byte aligned, contents on entry
 * irrelevant (the rows' statistics and the partial sums of tiles cut between CTAs).
 * Deterministic, but for shared pages.
 */
typedef struct {
  const void* q;
  const void* k;
  float* weights;
  const int32_t* block_table; /* [B, max_pages] */
  const int32_t* q_start;     /* [B + 1] */
  const int32_t* k_start;     /* [B + 1]; NULL: q_start */
  uint32_t* err_word;
  int32_t dtype;
  int32_t accumulate;
  int64_t B, Tq, Tk, Hq, Hkv, D, page_tokens, max_pages, num_pages;
  int64_t q_strides[2], k_strides[2]; /* token, head */
  float scale;
  int32_t reserved_;          /* must be 0 */
  void* workspace;
  size_t workspace_bytes;
} sa_weights_params;

size_t attn_weights_packed_workspace(const sa_weights_params* p);
int attn_weights_packed(const sa_weights_params* p, void* stream);

/*
 * paged_attn_decode_weights -- paged_attn_decode (the same y) that also accumulates
 * the weights of its queries: of token t < ctx_len[b] - 1 added, of the new token,
 * ctx_len[b] - 1, set.  weights: the pool, with p's num_pages, Hkv and page_tokens; it
 * must overlap nothing else of the call.  options must be 0.  Workspace:
 * paged_attn_decode_weights_workspace(p) bytes: paged_attn_decode's, and the scores,
 * B * Hq * max_pages * page_tokens floats (at most 2^40).
 */
size_t paged_attn_decode_weights_workspace(const sa_paged_params* p);
int paged_attn_decode_weights(const sa_paged_params* p, float* weights, void* stream);

/*
 * paged_kv_select -- the tokens that each KV head keeps.  For sequence b with
 * n = ctx_len[b] tokens and KV head h: all of them when n <= budget, else exactly
 * `budget`: the first `sink`, the last `recent`, and of those between them the
 * budget - sink - recent with the largest weights (ties: the lower token; NaN counts
 * as -inf).  keep: int32 [B, Hkv, budget], ascending, -1 behind the last: an index row as
 * sparse_attn_decode and paged_kv_compact take it.  new_len (nullable int32 [B], not
 * ctx_len itself): min(n, budget).  A ctx_len outside [0, max_pages * page_tokens] sets
 * SA_ERRBIT_PAGE (err_word nullable) and counts as 0; the weight behind a table entry
 * outside [0, num_pages) counts as -inf and sets it too.  sink + recent <= budget;
 * max_pages * page_tokens up to 2^22.  Exact; no workspace.
 */
typedef struct {
  const float* weights;
  const int32_t* block_table;
  const int32_t* ctx_len;
  int32_t* keep;
  int32_t* new_len;
  uint32_t* err_word;
  int64_t B, Hkv, page_tokens, max_pages, num_pages;
  int64_t budget, sink, recent;
} sa_select_params;
int paged_kv_select(const sa_select_params* p, void* stream);

/*
 * paged_kv_compact -- moves the kept rows to the front of their sequence's pages, in
 * place: for every sequence b, KV head h and i < m, with m the entries of keep[b, h, :]
 * before its first -1, token i's row of K, row of V and weight (weights nullable)
 * become those of token keep[b, h, i].  Bit for bit; FP8 rows move with their scale
 * bytes.  Tokens from m on keep what they held.  keep: int32 [B, Hkv, width], each row
 * strictly increasing from 0 on, below ctx_len[b] (the length before), -1 behind;
 * a row that is not stays as it is and ORs its SA_IDX_* codes into err_word (nullable).
 * A ctx_len outside [0, max_pages * page_tokens], or a table entry outside
 * [0, num_pages) that a moved row names, sets SA_ERRBIT_PAGE; such rows stay.  The pages of
 * a sequence must be its own: a page shared with another sequence of the call, or
 * named twice, ends up with rows of either.  pool_format and D as for
 * paged_kv_write.  No workspace.
 */
typedef struct {
  void* k_pool;
  void* v_pool;
  float* weights;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* keep;
  uint32_t* err_word;
  int32_t dtype;              /* of pages of plain elements */
  int32_t pool_format;
  int64_t B, Hkv, D, page_tokens, max_pages, num_pages, width;
} sa_compact_params;
int paged_kv_compact(const sa_compact_params* p, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SA_H */
