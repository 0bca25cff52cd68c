// serving.h -- argument blocks and launchers of the serving-step operators:
// rotary positions, the page write and read-back, decode over FP8 pages and
// the packed prefill.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sa.h"
#include "kernels.h"

namespace sa {

// The measurement hook's events of this host thread (sa_set_kernel_events).
void* kernel_event_before();
void* kernel_event_after();

// Let a kernel use up to `bytes` of dynamic shared memory (the same for every call):
// asked once per kernel and device, as the call costs about a microsecond.
constexpr int kAllSmem = 227 * 1024;
bool allow_smem(const void* kernel, int bytes = kAllSmem);

// Multiprocessors of the current device, asked once per device.
int sm_count();

// ---- rotary positions ------------------------------------------------------------
struct RotaryArgs {
  const void* x[2];           // queries, keys (H[1] == 0: queries only)
  void* y[2];
  const void* positions;      // [B or 1, S]
  int pos_is_i64;
  int vec;                    // 16-element chunks and 16-byte accesses everywhere
  int S, T;                   // tokens per batch, B * S
  int D;
  int H[2];
  int in_place[2];            // y is x: the dims past rotary_dim are already there
  int64_t pos_stride;
  int64_t xs[2][3], ys[2][3]; // element strides: batch, token, head
  sa_rope rope;
};
int launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t st);

// ---- packed rows <-> pages ---------------------------------------------------------
struct KvPagesArgs {
  void* x[2];                 // K and V rows
  int64_t xs[2][2];           // element strides: token, head
  void* pool[2];
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* seq_start;   // nullable: one row per sequence
  uint32_t* err_word;
  int fp8;                    // SA_FP8_E4M3_PAGE pages
  int aligned;                // 16-byte accesses to the rows are legal
  int has_rope;
  int T, B, Hkv, D;
  int64_t page_tokens, max_pages, num_pages;
  sa_rope rope;
};
int launch_kv_write(const KvPagesArgs& a, int dtype, cudaStream_t st);
int launch_kv_read(const KvPagesArgs& a, int dtype, cudaStream_t st);

// ---- decode over FP8 pages ------------------------------------------------------------
// GatherArgs of the paged source with Hkv the number of query-head groups
// (KV heads times sub-groups) and g = hpu heads per group.  Launches the attention
// kernel (one CTA per SM) and the merge of the units split across its CTAs.
constexpr int kFp8UnitCost = 2;               // tiles that a change of unit costs a warp
int64_t fp8_pages_max_heads(int D);           // query heads one group can hold
int launch_fp8_pages(const GatherArgs& a, int64_t pool_heads, int dtype, int sms,
                     cudaStream_t st);

// ---- packed prefill --------------------------------------------------------------------
struct PackedArgs {
  const void* q;
  const void* k;
  const void* v;
  void* y;
  const int32_t* q_start;
  const int32_t* k_start;
  uint32_t* err_word;
  int dtype, causal;
  int64_t B, Tq, Tk, Hq, Hkv, D;
  int64_t qs[2], ks[2], vs[2], ys[2];  // element strides: token, head
  float scale, softcap;
};
bool packed_tc_supported(const PackedArgs& a);
int launch_packed_tc(const PackedArgs& a, cudaStream_t st);
int launch_packed_simt(const PackedArgs& a, cudaStream_t st);

}  // namespace sa
