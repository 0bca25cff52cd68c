// k_kv_select.cu -- the tokens that a head keeps of a context that has outgrown its
// budget: the first `sink`, the last `recent`, and of those between them the ones
// whose accumulated attention weight is largest (ties: the lower token).
//
// A row is a (sequence, KV head) with n tokens.  The weights are compared as unsigned
// keys (sign and exponent turned so that a larger weight is a larger key; NaN like
// -inf, -0 like 0; the first and the latest tokens above every weight).  The key T of the
// last token kept is found digit by digit, from a histogram of the upper 11 bits on.  A
// second pass over the weights, from L2, marks the tokens above the digit found, four
// to a byte in shared memory, and lists the few that share it; the list's histograms of
// the 11 bits below and of the last 10 give T and their marks.  (A digit with more
// tokens than the list holds, as in a fresh pool of zeros, takes two more passes over
// all.)  Token t is kept when key > T, or key == T and fewer than `ties` equal keys lie
// before it: the number kept before a token is G + min(E, ties), with G the greater and
// E the equal keys before it, so one scan over the marks places every token in
// ascending order.
//
// Bound by issue slots: some 30 instructions a token, and what a warp does once per
// row.  So a row has one CTA where there are enough rows (keys kept in registers by
// clusters of four CTAs a row, 64 warps instead of 16: 178 us for 2.16 M tokens in 8
// heads), and a cluster of up to 8, which share their histograms, lists and counts
// through distributed shared memory, where there are few.
#include "cluster.cuh"
#include "weights.h"

namespace sa {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kQuads = 4;                          // of four tokens, that a thread has in flight
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;                        // of the first two digits (the third: 1,024)
constexpr int kList = 2048;                        // tokens that share the first digit found
constexpr uint32_t kLowest = 0x007fffffu;          // the key of -inf
constexpr uint32_t kNone = 0u, kAlways = 0xffffffffu;  // no token; one kept whatever its weight

__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 becomes 0
  if (w != w) return kLowest;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct Shared {
  uint32_t hist[3][kBins];
  uint32_t list[kList], token[kList];
  uint32_t listed;                  // tokens in the list
  uint32_t sum[kWarps];             // of a block-wide scan
  uint32_t bin, above, inside;      // the digit found, the keys above it, its own
  uint2 total;                      // greater and equal keys of the CTA
};

// Dynamic shared memory: Shared, then a byte per four tokens of the CTA: greater in the
// low half, equal in the high one.
template <bool kCluster>
__global__ void __launch_bounds__(kThreads, 3)
    kv_select_kernel(const __grid_constant__ SelectArgs a, int ctas) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw);
  uint8_t* map = smem_raw + sizeof(Shared);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int row = static_cast<int>(blockIdx.x / static_cast<uint32_t>(ctas));
  const int rank = kCluster ? static_cast<int>(cluster_rank()) : 0;
  const int b = row / a.Hkv, h = row - b * a.Hkv;
  const int64_t n64 = __ldg(a.ctx_len + b);
  const bool ok = n64 >= 0 && n64 <= a.max_pages * a.page_tokens;
  const int n = ok ? static_cast<int>(n64) : 0;
  if (tid == 0 && rank == 0) {
    if (!ok && a.err_word) atomicOr(a.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
    if (h == 0 && a.new_len) a.new_len[b] = min(n, a.budget);
  }
  int32_t* keep = a.keep + static_cast<int64_t>(row) * a.budget;
  if (n <= a.budget) {  // everything
    for (int64_t i = rank * kThreads + tid; i < a.budget; i += ctas * kThreads)
      keep[i] = i < n ? static_cast<int32_t>(i) : -1;
    return;
  }

  uint32_t need = static_cast<uint32_t>(a.budget - a.sink - a.recent);  // of the middle
  const int seg = ((n + ctas - 1) / ctas + 15) & ~15;
  const int begin = min(rank * seg, n), end = min(begin + seg, n), end16 = begin + ((end - begin + 15) & ~15);
  bool bad = false;
  const int32_t* table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  const uint32_t pt = static_cast<uint32_t>(a.page_tokens);
  auto weight_at = [&](uint32_t t) -> const float* {
    const uint32_t pi = a.shift >= 0 ? t >> a.shift : t / pt;
    const int32_t p = __ldg(table + pi);
    if (p < 0 || p >= a.num_pages) {
      bad = true;
      return nullptr;
    }
    return a.weights + (p * static_cast<int64_t>(a.Hkv) + h) * pt + (t - pi * pt);
  };
  // f(t, keys of t .. t + 3) for all quads of this CTA, those of a thread 4 * kThreads apart.
  auto quads = [&](auto&& f) {
#pragma unroll 1
    for (int t0 = begin + 4 * tid; t0 < end16; t0 += 4 * kThreads * kQuads) {
      float w[kQuads][4];
#pragma unroll
      for (int r = 0; r < kQuads; ++r) {
        const int t = t0 + 4 * kThreads * r;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[r][e] = SA_NEG_INF;
        if (a.vec) {
          const float* x = t < end ? weight_at(static_cast<uint32_t>(t)) : nullptr;
          if (x) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(x));
            w[r][0] = v.x;
            w[r][1] = v.y;
            w[r][2] = v.z;
            w[r][3] = v.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* x = t + e < end ? weight_at(static_cast<uint32_t>(t + e)) : nullptr;
            if (x) w[r][e] = __ldg(x);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kQuads; ++r) {
        const int t = t0 + 4 * kThreads * r;
        if (t >= end16) break;
        uint32_t key[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) key[e] = key_of(w[r][e]);
        if (t < a.sink || t + 3 >= n - a.recent || t + 3 >= end) {  // (few: the row's ends)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (t + e < a.sink || t + e >= n - a.recent) key[e] = kAlways;
            if (t + e >= end) key[e] = kNone;
          }
        }
        f(t, key);
      }
    }
  };
  auto middle = [](uint32_t k) { return k - 1u < kAlways - 1u; };

  for (int i = tid; i < 3 * kBins; i += kThreads) (&sm.hist[0][0])[i] = 0;
  if (tid == 0) {
    sm.listed = 0;
    sm.total = make_uint2(0u, 0u);
  }
  __syncthreads();

  // The digit whose keys hold the last one kept: `c` the counts of the bins at .. at + 3, all
  // threads' together (the largest bins with the first threads).
  const int at = kBins - 4 - 4 * tid;
  auto find_digit = [&](uint4 c) {
    const uint32_t sum = c.x + c.y + c.z + c.w;
    uint32_t before = sum;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, before, sh);
      if (lane >= sh) before += x;
    }
    if (lane == 31) sm.sum[warp] = before;
    __syncthreads();
    before -= sum;
    for (int w = 0; w < warp; ++w) before += sm.sum[w];
    if (before < need && need <= before + sum) {  // one thread
      uint32_t up = before;
      int i = 3;
      uint32_t v = c.w;
      if (up + v < need) up += v, v = c.z, i = 2;
      if (i == 2 && up + v < need) up += v, v = c.y, i = 1;
      if (i == 1 && up + v < need) up += v, v = c.x, i = 0;
      sm.bin = static_cast<uint32_t>(at + i);
      sm.above = up;
      sm.inside = v;
    }
    __syncthreads();
    need -= sm.above;
  };
  auto counts = [&](int p) {  // over the cluster
    uint32_t* h4 = sm.hist[p] + at;
    if (!kCluster) {
      __syncthreads();
      return *reinterpret_cast<const uint4*>(h4);
    }
    cluster_sync();
    uint4 c = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t addr = smem_u32(h4);
    for (int q = 0; q < ctas; ++q) {
      const uint4 v = ld_cluster4(cluster_addr(addr, static_cast<uint32_t>(q)));
      c.x += v.x;
      c.y += v.y;
      c.z += v.z;
      c.w += v.w;
    }
    return c;
  };
  auto sync = [&]() {
    if (kCluster) cluster_sync();
    else __syncthreads();
  };

  // ---- the key of the last one kept, and the marks -------------------------------------------
  uint32_t ties = 0;
  // tokens of at least `from` are greater; those of `to` .. from - 1 go to the list
  auto mark = [&](uint32_t from, uint32_t to) {
    quads([&](int t, const uint32_t(&key)[4]) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (key[e] >= from) m |= 1u << e;
        else if (key[e] >= to) {
          const uint32_t i = atomicAdd(&sm.listed, 1u);
          sm.list[i] = key[e];
          sm.token[i] = static_cast<uint32_t>(t + e - begin);
        }
      }
      map[(t - begin) >> 2] = static_cast<uint8_t>(m);
    });
  };
  if (need == 0) {
    mark(kAlways, kAlways);
  } else {
    quads([&](int, const uint32_t(&key)[4]) {
      const uint32_t d = key[0] >> 21;
      if ((key[1] >> 21) == d && (key[2] >> 21) == d && (key[3] >> 21) == d && middle(key[0]) && d != kBins - 1) {
        atomicAdd(sm.hist[0] + d, 4u);  // (a pool of zeros: fewer to queue for one word)
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (middle(key[e])) atomicAdd(sm.hist[0] + (key[e] >> 21), 1u);
      }
    });
    find_digit(counts(0));
    uint32_t prefix = sm.bin;
    const uint32_t inside = sm.inside;
    if (inside == need) {  // the whole digit is kept
      mark(prefix << 21, kAlways);
    } else {
      const bool listed = inside <= kList;  // (the same for the whole cluster)
      if (listed) {
        mark((prefix + 1) << 21, prefix << 21);
        sync();
      }
      uint32_t last = 0;
#pragma unroll 1
      for (int p = 1; p < 3; ++p) {
        const int shift = p == 1 ? 10 : 0, above_shift = p == 1 ? 21 : 10;
        const uint32_t mask = p == 1 ? 2047u : 1023u;
        auto count = [&](uint32_t k) {
          if ((k >> above_shift) == prefix) atomicAdd(sm.hist[p] + ((k >> shift) & mask), 1u);
        };
        if (listed) {  // every CTA counts the whole list
          for (int q = 0; q < ctas; ++q) {
            const uint32_t len = kCluster ? ld_cluster(cluster_addr(smem_u32(&sm.listed), static_cast<uint32_t>(q))) : sm.listed;
            for (uint32_t i = tid; i < len; i += kThreads)
              count(kCluster ? ld_cluster(cluster_addr(smem_u32(sm.list + i), static_cast<uint32_t>(q))) : sm.list[i]);
          }
          __syncthreads();
          find_digit(*reinterpret_cast<const uint4*>(sm.hist[p] + at));
        } else {
          quads([&](int, const uint32_t(&key)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (middle(key[e])) count(key[e]);
          });
          find_digit(counts(p));
        }
        prefix = (prefix << (p == 1 ? 11 : 10)) | sm.bin;
        last = prefix;
      }
      ties = need;
      if (listed) {
        for (uint32_t i = tid; i < sm.listed; i += kThreads) {
          const uint32_t k = sm.list[i], t = sm.token[i];
          if (k < last) continue;
          const uint32_t bit = ((t >> 2) & 3u) * 8 + (t & 3u) + (k == last ? 4 : 0);
          atomicOr(reinterpret_cast<uint32_t*>(map) + (t >> 4), 1u << bit);
        }
      } else {
        quads([&](int t, const uint32_t(&key)[4]) {
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (key[e] > last) m |= 1u << e;
            if (key[e] == last) m |= 16u << e;
          }
          map[(t - begin) >> 2] = static_cast<uint8_t>(m);
        });
      }
    }
  }
  __syncthreads();

  // ---- the tokens marked, in ascending order -------------------------------------------------
  const uint32_t* words = reinterpret_cast<const uint32_t*>(map);  // of 16 tokens
  const int nwords = (end16 - begin) / 16;
  auto both = [](uint32_t x) { return __popc(x & 0x0f0f0f0fu) | __popc(x & 0xf0f0f0f0u) << 16; };
  uint32_t greater = 0, equal = 0;  // before this CTA's tokens, later before the round's
  if (kCluster) {
    uint32_t g = 0, q = 0;
    for (int i = tid; i < nwords; i += kThreads) {
      const uint32_t x = both(words[i]);
      g += x & 0xffffu;
      q += x >> 16;
    }
    g = __reduce_add_sync(0xffffffffu, g);
    q = __reduce_add_sync(0xffffffffu, q);
    if (lane == 0) {
      atomicAdd(&sm.total.x, g);
      atomicAdd(&sm.total.y, q);
    }
    cluster_sync();
    for (int c = 0; c < rank; ++c) {
      const uint2 t = ld_cluster2(cluster_addr(smem_u32(&sm.total), static_cast<uint32_t>(c)));
      greater += t.x;
      equal += t.y;
    }
  }
#pragma unroll 1
  for (int i0 = 0; i0 < nwords; i0 += kThreads) {
    const uint32_t x = i0 + tid < nwords ? words[i0 + tid] : 0u;
    const uint32_t own = both(x);  // (a round: at most 8,192 of either)
    uint32_t before = own;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, before, sh);
      if (lane >= sh) before += y;
    }
    __syncthreads();  // (the sums of the round before, or of a digit, have been read)
    if (lane == 31) sm.sum[warp] = before;
    __syncthreads();
    before -= own;
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t c = sm.sum[w];
      if (w < warp) before += c;
      all += c;
    }
    uint32_t g = greater + (before & 0xffffu), q = equal + (before >> 16);
    const int t0 = begin + (i0 + tid) * 16;
    for (uint32_t todo = (x | x >> 4) & 0x0f0f0f0fu; todo != 0u; todo &= todo - 1u) {
      const int bit = __ffs(todo) - 1;
      const bool tie = !(x >> bit & 1u);
      if (!tie || q < ties) keep[g + min(q, ties)] = t0 + (bit >> 3) * 4 + (bit & 3);
      g += !tie;
      q += tie;
    }
    greater += all & 0xffffu;
    equal += all >> 16;
  }
  if (bad && a.err_word) atomicOr(a.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
  if (kCluster) cluster_sync();  // the others have read this CTA's lists and counts
}

}  // namespace

int launch_kv_select(const SelectArgs& a, cudaStream_t st) {
  // One CTA per row where there are rows enough for the device; else as many as give it
  // two to a multiprocessor, with 1,024 tokens each at least.  (The host knows the longest
  // context that the table can hold, not the contexts.)
  const int64_t most = a.max_pages * a.page_tokens, rows = static_cast<int64_t>(a.B) * a.Hkv;
  int64_t ctas = 1;
  while (ctas < kMaxCluster && ((rows * ctas < 2 * sm_count() && ctas * 1024 < most) || most > ctas * kSelectTokens)) ctas *= 2;
  if (rows * ctas > INT32_MAX || most > ctas * kSelectTokens) return -1;
  const int64_t tokens = (most + ctas - 1) / ctas + 15;
  const size_t smem = sizeof(Shared) + static_cast<size_t>(tokens / 16 + 1) * 4;
  const void* kernel = ctas > 1 ? reinterpret_cast<const void*>(kv_select_kernel<true>)
                                : reinterpret_cast<const void*>(kv_select_kernel<false>);
  if (!allow_smem(kernel)) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return (ctas > 1 ? cudaLaunchKernelEx(&cfg, kv_select_kernel<true>, a, static_cast<int>(ctas))
                   : cudaLaunchKernelEx(&cfg, kv_select_kernel<false>, a, static_cast<int>(ctas))) == cudaSuccess
             ? 0 : -1;
}

}  // namespace sa
