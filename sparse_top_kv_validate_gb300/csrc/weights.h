// weights.h -- argument blocks and launchers of the operators that keep a paged
// cache within a budget: attention weights of packed queries, the weights of a
// decode step, the selection of the tokens to keep, and the compaction.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "serving.h"

namespace sa {

// ---- attention weights of packed queries -------------------------------------------------
struct WeightsArgs {
  const void* q;
  const void* k;
  float* weights;             // [num_pages, Hkv, page_tokens]
  const int32_t* block_table;
  const int32_t* q_start;
  const int32_t* k_start;
  uint32_t* err_word;
  void* workspace;
  int dtype, accumulate;
  int64_t B, Tq, Tk, Hq, Hkv, D;
  int64_t qs[2], ks[2];       // element strides: token, head
  int64_t page_tokens, max_pages, num_pages;
  float scale;
};
bool weights_tc_supported(const WeightsArgs& a);
size_t weights_tc_workspace(const WeightsArgs& a);
int launch_weights_tc(const WeightsArgs& a, cudaStream_t st);
size_t weights_simt_workspace(const WeightsArgs& a);
int launch_weights_simt(const WeightsArgs& a, cudaStream_t st);

// ---- weights of a paged decode step --------------------------------------------------------
// a: the decode's arguments, its kernels launched.  launch_row_stats: stats and pref_out
// from the scores, after a decode that has left neither.
int launch_row_stats(const GatherArgs& a, cudaStream_t st);
int launch_decode_weights(const GatherArgs& a, float* weights, int64_t pool_heads, cudaStream_t st);

// ---- selection of the tokens to keep ---------------------------------------------------
struct SelectArgs {
  const float* weights;       // [num_pages, Hkv, page_tokens]
  const int32_t* block_table;
  const int32_t* ctx_len;
  int32_t* keep;              // [B, Hkv, budget]
  int32_t* new_len;           // nullable [B]
  uint32_t* err_word;
  int B, Hkv, budget, sink, recent;
  int page_tokens, shift;     // shift: log2(page_tokens), or -1
  int64_t max_pages, num_pages;
  int vec;                    // four tokens at a time: 16-byte loads stay inside a page
};
constexpr int64_t kSelectTokens = int64_t(1) << 19;  // tokens that a CTA can mark
constexpr int64_t kSelectMost = 8 * kSelectTokens;   // of a context: what a cluster can mark
int launch_kv_select(const SelectArgs& a, cudaStream_t st);

// ---- compaction ------------------------------------------------------------------------
struct CompactArgs {
  void* pool[2];              // K, V
  float* weights;             // nullable
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* keep;        // [B, Hkv, width]
  uint32_t* err_word;
  int fp8;                    // SA_FP8_E4M3_PAGE pages
  int B, Hkv, width;
  int row_bytes;              // of a row of K or V (codes only, for FP8 pages)
  int align;                  // bytes that every row of K and V is aligned to: 16, 4, 2
  int page_tokens, shift;     // shift: log2(page_tokens), or -1
  int64_t max_pages, num_pages;
};
int launch_kv_compact(const CompactArgs& a, cudaStream_t st);

}  // namespace sa
