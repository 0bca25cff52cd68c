// sa_api_weights.cu -- C ABI of the operators that keep a paged cache within a budget:
// the weights of packed queries, the selection of the tokens to keep and the
// compaction.  Host-side argument checks and launches; nothing here allocates, frees
// or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/sa.h"
#include "strided.h"
#include "weights.h"

namespace {

// Sizes of a paged pool: positive, and small enough for the kernels' 32-bit tokens.
int pages_status(int64_t B, int64_t Hkv, int64_t page_tokens, int64_t max_pages, int64_t num_pages) {
  if (B <= 0 || Hkv <= 0 || page_tokens <= 0 || max_pages <= 0 || num_pages <= 0) return SA_ERR_SHAPE;
  if (B >= kMaxInt || Hkv >= (int64_t(1) << 20) || B * Hkv >= kMaxInt / 64 || page_tokens >= kMaxInt ||
      max_pages >= kMaxInt || num_pages >= kMaxInt || max_pages * page_tokens >= kMaxInt - (int64_t(1) << 17))
    return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

// Bytes of a pool with `row` bytes per token and head; 0 when they leave 62 bits.
size_t pool_bytes(int64_t Hkv, int64_t page_tokens, int64_t num_pages, int64_t row) {
  const int64_t head = page_tokens * row;  // (below 2^31 * 2^13)
  if (num_pages * Hkv > (int64_t(1) << 62) / head) return 0;
  return static_cast<size_t>(num_pages * Hkv * head);
}

// log2(n), or -1 where n is no power of two.
int log2_of(int64_t n) {
  for (int s = 0; s < 31; ++s)
    if (n == int64_t(1) << s) return s;
  return -1;
}

// Checks; fills the kernel's arguments, whether it runs on the tensor cores and its workspace.
int weights_args(const sa_weights_params* p, bool query, sa::WeightsArgs& a, bool& tc, size_t& need) {
  if (!p || !p->q || !p->k || !p->block_table || !p->q_start || (!query && !p->weights)) return SA_ERR_NULL;
  if (p->reserved_ != 0) return SA_ERR_UNSUPPORTED;
  const size_t es = dtype_bytes(p->dtype);
  if (es == 0) return SA_ERR_DTYPE;
  if (p->Tq < 0 || p->Tk < 0 || p->Hq <= 0 || p->D <= 0) return SA_ERR_SHAPE;
  const int rc = pages_status(p->B, p->Hkv, p->page_tokens, p->max_pages, p->num_pages);
  if (rc != SA_OK) return rc;
  if (p->Hq % p->Hkv != 0 || (!p->k_start && p->Tq != p->Tk)) return SA_ERR_SHAPE;
  if (!std::isfinite(p->scale)) return SA_ERR_SHAPE;
  if (p->D > 256 || p->D % 4 != 0 || p->Tq >= (int64_t(1) << 30) || p->Tk >= (int64_t(1) << 30) ||
      p->B >= (int64_t(1) << 24) || p->Hq > 65535)
    return SA_ERR_UNSUPPORTED;
  const size_t pool = pool_bytes(p->Hkv, p->page_tokens, p->num_pages, 4);
  if (pool == 0) return SA_ERR_UNSUPPORTED;
  const Strided q{p->q, es, 2, {p->Tq, p->Hq, 1}, {p->q_strides[0], p->q_strides[1], 0}, p->D};
  const Strided k{p->k, es, 2, {p->Tk, p->Hkv, 1}, {p->k_strides[0], p->k_strides[1], 0}, p->D};
  for (const Strided* t : {&q, &k}) {
    if (!t->strides_ok()) return SA_ERR_SHAPE;
    if (!aligned(t->p, es)) return SA_ERR_ALIGN;
  }
  for (const void* x : {static_cast<const void*>(p->weights), static_cast<const void*>(p->block_table),
                        static_cast<const void*>(p->q_start), static_cast<const void*>(p->k_start),
                        static_cast<const void*>(p->err_word)})
    if (!aligned(x, 4)) return SA_ERR_ALIGN;
  const size_t starts = static_cast<size_t>(p->B + 1) * 4, table = static_cast<size_t>(p->B * p->max_pages) * 4;
  if (p->weights &&
      ((!q.empty() && ranges_meet(p->weights, pool, q.p, q.extent())) ||
       (!k.empty() && ranges_meet(p->weights, pool, k.p, k.extent())) ||
       ranges_meet(p->weights, pool, p->block_table, table) || ranges_meet(p->weights, pool, p->q_start, starts) ||
       (p->k_start && ranges_meet(p->weights, pool, p->k_start, starts)) ||
       (!query && ranges_meet(p->weights, pool, p->workspace, p->workspace ? p->workspace_bytes : 0))))
    return SA_ERR_OVERLAP;
  memset(&a, 0, sizeof(a));
  a.q = p->q;
  a.k = p->k;
  a.weights = p->weights;
  a.block_table = p->block_table;
  a.q_start = p->q_start;
  a.k_start = p->k_start ? p->k_start : p->q_start;
  a.err_word = p->err_word;
  a.workspace = p->workspace;
  a.dtype = p->dtype;
  a.accumulate = p->accumulate ? 1 : 0;
  a.B = p->B;
  a.Tq = p->Tq;
  a.Tk = p->Tk;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.D = p->D;
  for (int i = 0; i < 2; ++i) {
    a.qs[i] = q.st[i];
    a.ks[i] = k.st[i];
  }
  a.page_tokens = p->page_tokens;
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.scale = p->scale != 0.f ? p->scale : 1.0f / sqrtf(static_cast<float>(p->D));
  tc = true;  // 16-byte rows whose strides a tensor map can hold
  for (const Strided* t : {&q, &k}) {
    tc = tc && t->vec16();
    for (int i = 0; i < 2; ++i) tc = tc && (t->n[i] <= 1 || t->st[i] > 0);
  }
  tc = tc && sa::weights_tc_supported(a);
  need = tc ? sa::weights_tc_workspace(a) : sa::weights_simt_workspace(a);
  return SA_OK;
}

}  // namespace

extern "C" {

size_t attn_weights_packed_workspace(const sa_weights_params* p) {
  sa::WeightsArgs a;
  bool tc;
  size_t need;
  return weights_args(p, true, a, tc, need) == SA_OK ? need : 0;
}

int attn_weights_packed(const sa_weights_params* p, void* stream) {
  sa::WeightsArgs a;
  bool tc;
  size_t need;
  const int rc = weights_args(p, false, a, tc, need);
  if (rc != SA_OK) return rc;
  if (p->Tq == 0 || p->Tk == 0) return SA_OK;
  if (!p->workspace || p->workspace_bytes < need) return SA_ERR_WORKSPACE;
  if (!aligned(p->workspace, 256)) return SA_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  sa::mark_event(sa::kernel_event_before(), st);
  const int lrc = tc ? sa::launch_weights_tc(a, st) : sa::launch_weights_simt(a, st);
  sa::mark_event(sa::kernel_event_after(), st);
  return lrc == 0 ? SA_OK : SA_ERR_LAUNCH;
}

int paged_kv_select(const sa_select_params* p, void* stream) {
  if (!p || !p->weights || !p->block_table || !p->ctx_len || !p->keep) return SA_ERR_NULL;
  const int rc = pages_status(p->B, p->Hkv, p->page_tokens, p->max_pages, p->num_pages);
  if (rc != SA_OK) return rc;
  if (p->budget <= 0 || p->sink < 0 || p->recent < 0) return SA_ERR_SHAPE;
  if (p->budget >= kMaxInt - (int64_t(1) << 17) || p->max_pages * p->page_tokens > sa::kSelectMost)
    return SA_ERR_UNSUPPORTED;
  if (p->sink > p->budget || p->recent > p->budget || p->sink + p->recent > p->budget) return SA_ERR_SHAPE;
  const size_t pool = pool_bytes(p->Hkv, p->page_tokens, p->num_pages, 4);
  if (pool == 0) return SA_ERR_UNSUPPORTED;
  for (const void* x : {static_cast<const void*>(p->weights), static_cast<const void*>(p->block_table),
                        static_cast<const void*>(p->ctx_len), static_cast<const void*>(p->keep),
                        static_cast<const void*>(p->new_len), static_cast<const void*>(p->err_word)})
    if (!aligned(x, 4)) return SA_ERR_ALIGN;
  const size_t keep = static_cast<size_t>(p->B * p->Hkv) * static_cast<size_t>(p->budget) * 4;  // (below 2^58)
  const size_t len = static_cast<size_t>(p->B) * 4, table = len * static_cast<size_t>(p->max_pages);
  if (ranges_meet(p->keep, keep, p->weights, pool) || ranges_meet(p->keep, keep, p->block_table, table) ||
      ranges_meet(p->keep, keep, p->ctx_len, len))
    return SA_ERR_OVERLAP;
  if (p->new_len &&
      (ranges_meet(p->new_len, len, p->weights, pool) || ranges_meet(p->new_len, len, p->block_table, table) ||
       ranges_meet(p->new_len, len, p->ctx_len, len) || ranges_meet(p->new_len, len, p->keep, keep)))
    return SA_ERR_OVERLAP;
  sa::SelectArgs a;
  memset(&a, 0, sizeof(a));
  a.weights = p->weights;
  a.block_table = p->block_table;
  a.ctx_len = p->ctx_len;
  a.keep = p->keep;
  a.new_len = p->new_len;
  a.err_word = p->err_word;
  a.B = static_cast<int>(p->B);
  a.Hkv = static_cast<int>(p->Hkv);
  a.budget = static_cast<int>(p->budget);
  a.sink = static_cast<int>(p->sink);
  a.recent = static_cast<int>(p->recent);
  a.page_tokens = static_cast<int>(p->page_tokens);
  a.shift = log2_of(p->page_tokens);
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.vec = p->page_tokens % 4 == 0 && aligned(p->weights, 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  sa::mark_event(sa::kernel_event_before(), st);
  const int lrc = sa::launch_kv_select(a, st);
  sa::mark_event(sa::kernel_event_after(), st);
  return lrc == 0 ? SA_OK : SA_ERR_LAUNCH;
}

int paged_kv_compact(const sa_compact_params* p, void* stream) {
  if (!p || !p->k_pool || !p->v_pool || !p->block_table || !p->ctx_len || !p->keep) return SA_ERR_NULL;
  const bool fp8 = p->pool_format == SA_FP8_E4M3_PAGE;
  const size_t es = fp8 ? 1 : dtype_bytes(p->dtype);
  if (es == 0 || (p->pool_format != 0 && !fp8)) return SA_ERR_DTYPE;
  const int rc = pages_status(p->B, p->Hkv, p->page_tokens, p->max_pages, p->num_pages);
  if (rc != SA_OK) return rc;
  if (p->D <= 0 || p->width <= 0) return SA_ERR_SHAPE;
  if (p->D > 1024 || p->width >= kMaxInt - (int64_t(1) << 17) || p->num_pages * p->Hkv >= kMaxInt) return SA_ERR_UNSUPPORTED;
  if (fp8 && (!(p->D == 64 || p->D == 128 || p->D == 256) || p->page_tokens % 16 != 0)) return SA_ERR_UNSUPPORTED;
  const int64_t row = p->D * static_cast<int64_t>(es);
  const size_t pool = pool_bytes(p->Hkv, p->page_tokens, p->num_pages, row + (fp8 ? 1 : 0));
  const size_t sums = p->weights ? pool_bytes(p->Hkv, p->page_tokens, p->num_pages, 4) : 0;
  if (pool == 0 || (p->weights && sums == 0)) return SA_ERR_UNSUPPORTED;
  if (!aligned(p->k_pool, fp8 ? 16 : es) || !aligned(p->v_pool, fp8 ? 16 : es)) return SA_ERR_ALIGN;
  for (const void* x : {static_cast<const void*>(p->weights), static_cast<const void*>(p->block_table),
                        static_cast<const void*>(p->ctx_len), static_cast<const void*>(p->keep),
                        static_cast<const void*>(p->err_word)})
    if (!aligned(x, 4)) return SA_ERR_ALIGN;
  const size_t keep = static_cast<size_t>(p->B * p->Hkv) * static_cast<size_t>(p->width) * 4;  // (below 2^58)
  const size_t len = static_cast<size_t>(p->B) * 4, table = len * static_cast<size_t>(p->max_pages);
  const void* out[3] = {p->k_pool, p->v_pool, p->weights};
  const size_t bytes[3] = {pool, pool, sums};
  for (int i = 0; i < 3; ++i) {
    if (!out[i]) continue;
    for (int j = 0; j < i; ++j)
      if (ranges_meet(out[i], bytes[i], out[j], bytes[j])) return SA_ERR_OVERLAP;
    if (ranges_meet(out[i], bytes[i], p->keep, keep) || ranges_meet(out[i], bytes[i], p->block_table, table) ||
        ranges_meet(out[i], bytes[i], p->ctx_len, len))
      return SA_ERR_OVERLAP;
  }
  sa::CompactArgs a;
  memset(&a, 0, sizeof(a));
  a.pool[0] = p->k_pool;
  a.pool[1] = p->v_pool;
  a.weights = p->weights;
  a.block_table = p->block_table;
  a.ctx_len = p->ctx_len;
  a.keep = p->keep;
  a.err_word = p->err_word;
  a.fp8 = fp8;
  a.B = static_cast<int>(p->B);
  a.Hkv = static_cast<int>(p->Hkv);
  a.width = static_cast<int>(p->width);
  a.row_bytes = static_cast<int>(row);
  a.align = 2;
  for (int n : {4, 16})
    if (row % n == 0 && aligned(p->k_pool, n) && aligned(p->v_pool, n)) a.align = n;
  a.page_tokens = static_cast<int>(p->page_tokens);
  a.shift = log2_of(p->page_tokens);
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  sa::mark_event(sa::kernel_event_before(), st);
  const int lrc = sa::launch_kv_compact(a, st);
  sa::mark_event(sa::kernel_event_after(), st);
  return lrc == 0 ? SA_OK : SA_ERR_LAUNCH;
}

}  // extern "C"
