// k_decode_weights.cu -- the attention weights of a paged decode step: after the
// decode's kernels have kept each row's scores (log2 units), maximum m and inverse sum,
// w_t = sum over the group's heads of 2^(s_t - m) / l, added to the pool (set for the new
// token).
//
// The scores are 4 bytes per query head and token against 2 (D + 1) per KV head of the
// FP8 pages, written once and read once here: with groups of 4 and heads of 128, 12% of
// the decode's traffic where a second pass over K would be 50%.  Bound by that
// traffic (64 contexts, 1.08 M tokens, 32 / 8 heads of 128: 460 us for the decode with
// weights, 372 without; 262,144 tokens: this kernel 14.5 us): every warp takes a contiguous range of 16-token tiles of all (sequence, KV
// head)s laid end to end, 128 tokens at a time, four to a lane.
#include "gather_common.cuh"
#include "pool_add.cuh"
#include "weights.h"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kStep = 8;  // tiles of 16 tokens that a warp takes at a time

__device__ __forceinline__ float weight_of(float s, float2 st) {
  return st.x == SA_NEG_INF ? st.y : ex2(s - st.x) * st.y;
}

__global__ void __launch_bounds__(kThreads)
    decode_weights_kernel(const __grid_constant__ GatherArgs a, float* weights, int heads, int vec) {
  pdl_wait();  // the scores, the statistics and the tile space
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int B = static_cast<int>(a.B), g = static_cast<int>(a.Hq / heads);
  const uint32_t pt = static_cast<uint32_t>(a.page_tokens);
  const int64_t total = static_cast<int64_t>(heads) * a.pref_out[B];
  const int64_t R = ((total + warps - 1) / warps + kStep - 1) / kStep * kStep;
  int64_t t = warp * R;
  const int64_t t_end = min(t + R, total);
  if (t >= t_end) return;
  int b;
  {
    int lo = 0, hi = B;  // the last sequence that begins at or before t
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const int k = __popc(__ballot_sync(0xffffffffu, at < hi && static_cast<int64_t>(heads) * a.pref_out[at] <= t));
      lo += (k - 1) * step;
      hi = min(lo + step, hi);
    }
    b = lo;
  }
  bool bad = false;
  while (t < t_end) {
    while (static_cast<int64_t>(heads) * a.pref_out[b + 1] <= t) ++b;
    const int64_t base = static_cast<int64_t>(heads) * a.pref_out[b];
    const int tb = a.pref_out[b + 1] - a.pref_out[b];
    const int h = static_cast<int>((t - base) / tb);
    const int64_t off = base + static_cast<int64_t>(h) * tb, stop = min(t_end, off + tb);
    const int ctx = __ldg(a.ctx_len + b);
    const int64_t row = b * a.Hq + static_cast<int64_t>(h) * g;
    const float* sp = a.scores + row * a.score_stride;
    const float2* st = a.stats + row;
    for (; t < stop; t += kStep) {
      const int tok = static_cast<int>((t - off) * 16) + lane * 4;
      if (t + (lane >> 2) >= stop || tok >= ctx) continue;
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int hh = 0; hh < g; ++hh) {
        const float4 s = *reinterpret_cast<const float4*>(sp + hh * a.score_stride + tok);
        const float2 e = st[hh];
        w.x += weight_of(s.x, e);
        w.y += weight_of(s.y, e);
        w.z += weight_of(s.z, e);
        w.w += weight_of(s.w, e);
      }
      const float ws[4] = {w.x, w.y, w.z, w.w};
      auto place = [&](int x) -> float* {
        const uint32_t pi = static_cast<uint32_t>(x) / pt;
        const int32_t page = __ldg(a.block_table + b * a.max_pages + pi);
        if (page < 0 || page >= a.num_pages) {
          bad = true;
          return nullptr;
        }
        return weights + (page * static_cast<int64_t>(heads) + h) * pt + (static_cast<uint32_t>(x) - pi * pt);
      };
      if (vec) {  // the four tokens lie in one page
        float* at = place(tok);
        if (!at) continue;
        if (tok + 4 < ctx) {
          pool_add4(at, w);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (tok + e < ctx) pool_put(at + e, ws[e], tok + e < ctx - 1);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (tok + e >= ctx) continue;
          float* at = place(tok + e);
          if (at) pool_put(at, ws[e], tok + e < ctx - 1);
        }
      }
    }
    t = stop;
  }
  if (bad && a.err_word) atomicOr(a.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
}

// After the decode on the fp32 pipes, which leaves neither: the tile space and each
// row's maximum and inverse sum, from its scores.  A block per row.
__global__ void __launch_bounds__(kThreads) row_stats_kernel(const __grid_constant__ GatherArgs a) {
  __shared__ float sm_m[kThreads / 32], sm_l[kThreads / 32];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x, cap = a.max_pages * a.page_tokens;
  if (row == 0 && warp == 0) {
    int32_t carry = 0;
    if (lane == 0) a.pref_out[0] = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += 32) {
      int32_t v = 0;
      if (b0 + lane < a.B) {
        const int64_t n = __ldg(a.ctx_len + b0 + lane);
        v = n >= 1 && n <= cap ? static_cast<int32_t>((n + 15) / 16) : 0;
      }
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, v, sh);
        if (lane >= sh) v += x;
      }
      if (b0 + lane < a.B) a.pref_out[b0 + lane + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  int64_t n = __ldg(a.ctx_len + row / a.Hq);
  if (n < 1 || n > cap) n = 0;
  const float* s = a.scores + row * a.score_stride;
  float m = SA_NEG_INF;
  for (int64_t i = tid; i < n; i += kThreads) m = fmaxf(m, s[i]);
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, sh));
  if (lane == 0) sm_m[warp] = m;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, sm_m[w]);
  const float mu = m == SA_NEG_INF ? 0.f : m;
  float l = 0.f;
  for (int64_t i = tid; i < n; i += kThreads) l += ex2(s[i] - mu);
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
  if (lane == 0) sm_l[warp] = l;
  __syncthreads();
  if (tid == 0) {
    l = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) l += sm_l[w];
    a.stats[row] = row_stat(m, l);
  }
}

}  // namespace

int launch_row_stats(const GatherArgs& a, cudaStream_t st) {
  row_stats_kernel<<<static_cast<unsigned>(a.B * a.Hq), kThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_decode_weights(const GatherArgs& a, float* weights, int64_t pool_heads, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sm_count() * 4));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int vec = a.page_tokens % 4 == 0 && reinterpret_cast<uintptr_t>(weights) % 16 == 0;
  return cudaLaunchKernelEx(&cfg, decode_weights_kernel, a, weights, static_cast<int>(pool_heads), vec) == cudaSuccess ? 0 : -1;
}

}  // namespace sa
