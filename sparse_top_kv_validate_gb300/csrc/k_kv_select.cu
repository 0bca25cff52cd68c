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
// ascending order.  (Weights that change meanwhile give some list of tokens: no count of
// one pass is an index of another unchecked.)
//
// Bound by issue slots, and by the way of a row's loads.  A row has one CTA where there
// are enough rows, of 256 threads, so that few warps do what is done once per row (2.16 M
// tokens in 8 heads: 68 us; 512 threads, 72; rows that clusters of four CTAs keep in
// registers, 178), the longest contexts first (in the order given, 5 us more).  Where there
// are few rows a cluster of up to 8 CTAs takes one, its histograms, lists and counts
// shared through distributed shared memory (2 contexts of 118,000 and 144,000 tokens, 4 heads: 29 us).
// The list holds tokens, not keys: the few keys come once more from L1 (keys written by the
// second pass itself, each token's place from an atomic of its own: 83 us).
#include "cluster.cuh"
#include "weights.h"

#include <type_traits>

namespace sa {

namespace {

constexpr int kQuads = 4;                          // of four tokens, that a thread has in flight
constexpr int kMaxCluster = 8;
constexpr int kFirst = 2048, kSecond = 2048, kThird = 1024;  // bins of the key's three digits
constexpr int kShift1 = 21, kShift2 = 10;          // the first digit's place, the second's
constexpr int kList = 2048;                        // tokens that share the first digit found
constexpr uint32_t kLowest = 0x007fffffu;          // the key of -inf
constexpr uint32_t kNoKey = 0xffffffffu;           // above every weight's

// A larger key for a larger weight.  (fmaxf: NaN becomes -inf; the sum: -0 becomes 0.)
__device__ __forceinline__ uint32_t key_of(float w) {
  const int32_t u = __float_as_int(fmaxf(w, SA_NEG_INF) + 0.0f);
  return static_cast<uint32_t>(u ^ ((u >> 31) | static_cast<int32_t>(0x80000000)));
}
// The weight of which w >= it says that w's key is at least k (NaN, so never, above +inf's).
__device__ __forceinline__ float weight_of(uint32_t k) {
  k = max(k, kLowest);
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// A row's CTA, or a cluster's.
template <bool kCluster>
struct Cfg {
  static constexpr int kThreads = kCluster ? 512 : 256;
  static constexpr int kCtas = kCluster ? 2 : 5;  // to a multiprocessor, at least
};

template <bool kCluster>
struct Shared {
  static constexpr int kWarps = Cfg<kCluster>::kThreads / 32;
  uint32_t hist[kFirst + kSecond + kThird];
  uint32_t list[kList], token[kList];  // (the keys are filled in when the list is complete)
  uint32_t listed;                  // tokens in the list
  uint32_t sum[kWarps];             // of a block-wide scan
  uint32_t bin, above, inside;      // the digit found, the keys above it, its own
  uint2 marked[kWarps];             // greater and equal keys of a warp's words
  int seq;                          // the sequence of this CTA's row
  uint2 total;                      // greater and equal keys of the CTA
};

// Sum of the lanes up to and with this one.
__device__ __forceinline__ uint32_t scan_warp(uint32_t v, int lane, int width = 32) {
  for (int sh = 1; sh < width; sh <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, sh);
    if (lane >= sh) v += x;
  }
  return v;
}

// Dynamic shared memory: Shared, then a byte per four tokens of the CTA: greater in the
// low half, equal in the high one.
template <bool kCluster>
__global__ void __launch_bounds__(Cfg<kCluster>::kThreads, Cfg<kCluster>::kCtas)
    kv_select_kernel(const __grid_constant__ SelectArgs a, int ctas, int order) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  using S = Shared<kCluster>;
  constexpr int kThreads = Cfg<kCluster>::kThreads, kWarps = S::kWarps;
  S& sm = *reinterpret_cast<S*>(smem_raw);
  uint8_t* map = smem_raw + sizeof(S);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  int row = static_cast<int>(blockIdx.x / static_cast<uint32_t>(ctas));
  const int rank = kCluster ? static_cast<int>(cluster_rank()) : 0;
  int b = row / a.Hkv;
  const int h = row - b * a.Hkv;
  if (!kCluster && order) {  // the b-th longest context (as many threads as sequences, at least)
    int32_t* len = reinterpret_cast<int32_t*>(sm.list);
    const int own = tid < a.B ? max(__ldg(a.ctx_len + tid), 0) : -1;
    len[tid] = own;
    __syncthreads();
    int longer = 0;
    if (tid < a.B) {
      for (int i = 0; i < a.B; i += 4) {  // (places behind the last sequence hold -1)
        const int4 v = *reinterpret_cast<const int4*>(len + i);
        longer += (v.x > own || (v.x == own && i < tid)) + (v.y > own || (v.y == own && i + 1 < tid)) +
                  (v.z > own || (v.z == own && i + 2 < tid)) + (v.w > own || (v.w == own && i + 3 < tid));
      }
      if (longer == b) sm.seq = tid;
    }
    __syncthreads();
    b = sm.seq;
    row = b * a.Hkv + h;
  }
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
  const int sink = a.sink, stop = min(n - a.recent, end);  // the middle: [sink, stop)
  bool bad = false;
  const int32_t* table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  const uint32_t pt = static_cast<uint32_t>(a.page_tokens);
  const float* pool = a.weights + static_cast<int64_t>(h) * pt;
  const int64_t page_stride = static_cast<int64_t>(a.Hkv) * pt;
  const uint32_t pages = static_cast<uint32_t>(a.num_pages);  // (below 2^31)
  auto weight_at = [&](uint32_t t) -> const float* {
    const uint32_t pi = a.shift >= 0 ? t >> a.shift : t / pt;
    const uint32_t p = static_cast<uint32_t>(__ldg(table + pi));
    if (p >= pages) {
      bad = true;
      return nullptr;
    }
    return pool + p * page_stride + (t - pi * pt);
  };
  // f(t0, weights): this thread's quads at t0 + 4 * kThreads * r, for all tokens of the CTA;
  // whole warps, so also quads behind the last.
  auto quads = [&](auto&& f) {
#pragma unroll 1
    for (int t1 = begin + 128 * warp; t1 < end16; t1 += 4 * kThreads * kQuads) {
      const int t0 = t1 + 4 * lane;
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
      f(t0, w);
    }
  };
  // of four tokens: a bit for each of the middle
  auto middle = [&](int t) {
    uint32_t m = 15u;
    if (t < sink || t + 4 > stop) {  // (few: the row's ends)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t + e < sink || t + e >= stop) m &= ~(1u << e);
    }
    return m;
  };
  // and for each that is kept whatever its weight
  auto always = [&](int t, uint32_t mid) {
    uint32_t m = 0u;
    if (mid != 15u) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t + e < end && !(mid >> e & 1u)) m |= 1u << e;
    }
    return m;
  };

  for (int i = tid; i < static_cast<int>(sizeof(sm.hist) / 4); i += kThreads) sm.hist[i] = 0;
  if (tid == 0) {
    sm.listed = 0;
    sm.total = make_uint2(0u, 0u);
  }
  __syncthreads();

  // The digit whose keys hold the last one kept: c the counts of this thread's bins (the
  // largest bins with the first threads).
  auto find_digit = [&](const auto& c, int bins) {
    constexpr int kPer = sizeof(c) / sizeof(c[0]);
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += c[i];
    uint32_t before = scan_warp(sum, lane);
    if (lane == 31) sm.sum[warp] = before;
    __syncthreads();
    const uint32_t of = scan_warp(sm.sum[lane & (kWarps - 1)], lane, kWarps);
    before -= sum;
    const uint32_t up0 = __shfl_sync(0xffffffffu, of, max(warp - 1, 0));
    if (warp > 0) before += up0;
    if (before < need && need <= before + sum) {  // one thread
      uint32_t up = before;
      bool found = false;
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) {
        if (found) continue;
        if (up + c[i] >= need) {
          found = true;
          sm.bin = static_cast<uint32_t>(bins - kPer * (tid + 1) + i);
          sm.above = up;
          sm.inside = c[i];
        }
        up += c[i];
      }
    }
    __syncthreads();
    need -= sm.above;
  };
  // this thread's bins, over the CTAs `of` the cluster (or of its own alone)
  auto counts = [&](const uint32_t* hist, auto& c, int bins, int of) {
    constexpr int kPer = sizeof(c) / sizeof(c[0]);
    const uint32_t* from = hist + bins - kPer * (tid + 1);
    if (!kCluster || of == 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPer; ++i) c[i] = from[i];
      return;
    }
    cluster_sync();
#pragma unroll
    for (int i = 0; i < kPer; ++i) c[i] = 0;
#pragma unroll
    for (int q = 0; q < kMaxCluster; ++q) {
      if (q >= of) break;
      const uint32_t at = cluster_addr(smem_u32(from), static_cast<uint32_t>(q));
      if constexpr (kPer % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kPer; i += 4) {
          const uint4 v = ld_cluster4(at + i * 4);
          c[i] += v.x;
          c[i + 1] += v.y;
          c[i + 2] += v.z;
          c[i + 3] += v.w;
        }
      } else {
        const uint2 v = ld_cluster2(at);
        c[0] += v.x;
        c[1] += v.y;
      }
    }
  };

  // ---- the key of the last one kept, and the marks -------------------------------------------
  uint32_t ties = 0;
  // tokens of at least `from` are greater; those of `to` .. from - 1 go to the list
  auto mark = [&](uint32_t from, uint32_t to) {
    const float lo = weight_of(to), hi = weight_of(from);
    quads([&](int t0, const float(&w)[kQuads][4]) {
      uint32_t found = 0;
      uint8_t* to = map + ((t0 - begin) >> 2);
#pragma unroll
      for (int r = 0; r < kQuads; ++r) {
        const int t = t0 + 4 * kThreads * r;
        const uint32_t mid = middle(t);
        uint32_t m = 0, l = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = fmaxf(w[r][e], SA_NEG_INF);
          if (x >= hi) m |= 1u << e;
          if (x >= lo) l |= 1u << e;
        }
        found |= (l & ~m & mid) << (4 * r);
        if (t < end16) to[kThreads * r] = static_cast<uint8_t>((m & mid) | always(t, mid));
      }
      if (!__any_sync(0xffffffffu, found != 0u)) return;
      const uint32_t own = __popc(found);
      uint32_t at = scan_warp(own, lane);
      uint32_t base = 0;
      if (lane == 31) base = atomicAdd(&sm.listed, at);
      at += __shfl_sync(0xffffffffu, base, 31) - own;
      for (; found != 0u; found &= found - 1u) {
        const int bit = __ffs(found) - 1;
        if (at < kList) sm.token[at++] = static_cast<uint32_t>(t0 + 4 * kThreads * (bit >> 2) + (bit & 3) - begin);
      }
    });
  };
  if (need == 0) {
    mark(kNoKey, kNoKey);
  } else {
    quads([&](int t0, const float(&w)[kQuads][4]) {
#pragma unroll
      for (int r = 0; r < kQuads; ++r) {
        const uint32_t mid = middle(t0 + 4 * kThreads * r);
        uint32_t d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = key_of(w[r][e]) >> kShift1;
        if (mid == 15u && d[1] == d[0] && d[2] == d[0] && d[3] == d[0]) {
          atomicAdd(sm.hist + d[0], 4u);  // (a pool of zeros: fewer to queue for one word)
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (mid >> e & 1u) atomicAdd(sm.hist + d[e], 1u);
        }
      }
    });
    {
      uint32_t c[kFirst / kThreads];
      counts(sm.hist, c, kFirst, ctas);
      find_digit(c, kFirst);
    }
    uint32_t prefix = sm.bin;
    const uint32_t inside = sm.inside;
    if (inside == need) {  // the whole digit is kept
      mark(prefix << kShift1, kNoKey);
    } else {
      const bool listed = inside <= kList;  // (the same for the whole cluster)
      if (listed) {
        mark((prefix + 1) << kShift1, prefix << kShift1);
        __syncthreads();
        if (tid == 0) sm.listed = min(sm.listed, static_cast<uint32_t>(kList));
        __syncthreads();
        for (uint32_t i = tid; i < sm.listed; i += kThreads) {
          const float* x = weight_at(static_cast<uint32_t>(begin) + sm.token[i]);
          sm.list[i] = x ? key_of(__ldg(x)) : kLowest;
        }
        if (kCluster) cluster_sync();
      }
      auto later = [&](auto digit) {  // the next digit, from the list or from all tokens
        constexpr bool kLast = decltype(digit)::value;
        constexpr int kShift = kLast ? 0 : kShift2, kAbove = kLast ? kShift2 : kShift1, kBins = kLast ? kThird : kSecond;
        uint32_t* hist = sm.hist + kFirst + (kLast ? kSecond : 0);
        auto count = [&](uint32_t k) {
          if ((k >> kAbove) == prefix) atomicAdd(hist + ((k >> kShift) & (kBins - 1)), 1u);
        };
        if (listed) {  // every CTA counts the whole list
          for (int q = 0; q < ctas; ++q) {
            const uint32_t len = kCluster ? ld_cluster(cluster_addr(smem_u32(&sm.listed), static_cast<uint32_t>(q))) : sm.listed;
            for (uint32_t i = tid; i < len; i += kThreads)
              count(kCluster ? ld_cluster(cluster_addr(smem_u32(sm.list + i), static_cast<uint32_t>(q))) : sm.list[i]);
          }
        } else {
          quads([&](int t0, const float(&w)[kQuads][4]) {
#pragma unroll
            for (int r = 0; r < kQuads; ++r) {
              const uint32_t mid = middle(t0 + 4 * kThreads * r);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (mid >> e & 1u) count(key_of(w[r][e]));
            }
          });
        }
        uint32_t c[kBins / kThreads];
        counts(hist, c, kBins, listed ? 1 : ctas);
        find_digit(c, kBins);
        prefix = prefix * kBins + sm.bin;
      };
      later(std::false_type{});
      later(std::true_type{});
      const uint32_t last = prefix;
      ties = need;
      if (listed) {
        for (uint32_t i = tid; i < sm.listed; i += kThreads) {
          const uint32_t k = sm.list[i], t = sm.token[i];
          if (k < last) continue;
          const uint32_t bit = ((t >> 2) & 3u) * 8 + (t & 3u) + (k == last ? 4 : 0);
          atomicOr(reinterpret_cast<uint32_t*>(map) + (t >> 4), 1u << bit);
        }
      } else {
        const float lo = weight_of(last);
        quads([&](int t0, const float(&w)[kQuads][4]) {
#pragma unroll
          for (int r = 0; r < kQuads; ++r) {
            const int t = t0 + 4 * kThreads * r;
            if (t >= end16) break;
            const uint32_t mid = middle(t);
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = fmaxf(w[r][e], SA_NEG_INF);
              if (x > lo) m |= 1u << e;
              if (x == lo) m |= 16u << e;
            }
            map[(t - begin) >> 2] = static_cast<uint8_t>((m & mid * 17u) | always(t, mid));
          }
        });
      }
    }
  }
  __syncthreads();

  // ---- the tokens marked, in ascending order -------------------------------------------------
  const uint32_t* words = reinterpret_cast<const uint32_t*>(map);  // of 16 tokens
  const int nwords = (end16 - begin) / 16;
  auto both = [](uint32_t x) { return __popc(x & 0x0f0f0f0fu) | __popc(x & 0xf0f0f0f0u) << 16; };
  auto sync = [&]() {
    if (kCluster) cluster_sync();
    else __syncthreads();
  };
  // a warp's words: [first, last), and what is marked before them
  const int per = (nwords + kWarps - 1) / kWarps, first = min(warp * per, nwords), last = min(first + per, nwords);
  uint32_t greater = 0, equal = 0;
  for (int i = first + lane; i < last; i += 32) {
    const uint32_t x = both(words[i]);
    greater += x & 0xffffu;
    equal += x >> 16;
  }
  greater = __reduce_add_sync(0xffffffffu, greater);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    sm.marked[warp] = make_uint2(greater, equal);
    if (kCluster) {
      atomicAdd(&sm.total.x, greater);
      atomicAdd(&sm.total.y, equal);
    }
  }
  sync();
  const uint2 w0 = lane < warp ? sm.marked[lane] : make_uint2(0u, 0u);
  greater = __reduce_add_sync(0xffffffffu, w0.x);
  equal = __reduce_add_sync(0xffffffffu, w0.y);
  for (int c = 0; kCluster && c < rank; ++c) {
    const uint2 t = ld_cluster2(cluster_addr(smem_u32(&sm.total), static_cast<uint32_t>(c)));
    greater += t.x;
    equal += t.y;
  }
#pragma unroll 1
  for (int i0 = first; i0 < last; i0 += 32) {
    const uint32_t x = i0 + lane < last ? words[i0 + lane] : 0u;
    const uint32_t own = both(x), with = scan_warp(own, lane), all = __shfl_sync(0xffffffffu, with, 31);
    const uint32_t before = with - own;
    uint32_t g = greater + (before & 0xffffu), q = equal + (before >> 16);
    const int t0 = begin + (i0 + lane) * 16;
    for (uint32_t todo = (x | x >> 4) & 0x0f0f0f0fu; todo != 0u; todo &= todo - 1u) {
      const int bit = __ffs(todo) - 1;
      const bool tie = !(x >> bit & 1u);
      const uint32_t at = g + min(q, ties);
      if ((!tie || q < ties) && at < static_cast<uint32_t>(a.budget)) keep[at] = t0 + (bit >> 3) * 4 + (bit & 3);
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
  const int threads = ctas > 1 ? Cfg<true>::kThreads : Cfg<false>::kThreads;
  const size_t smem = (ctas > 1 ? sizeof(Shared<true>) : sizeof(Shared<false>)) + static_cast<size_t>(tokens / 16 + 1) * 4;
  // Where they come one after the other, the longest contexts go first.
  const int order = ctas == 1 && a.B <= threads && rows > Cfg<false>::kCtas * sm_count() ? 1 : 0;
  const void* kernel = ctas > 1 ? reinterpret_cast<const void*>(kv_select_kernel<true>)
                                : reinterpret_cast<const void*>(kv_select_kernel<false>);
  if (!allow_smem(kernel)) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * ctas));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return (ctas > 1 ? cudaLaunchKernelEx(&cfg, kv_select_kernel<true>, a, static_cast<int>(ctas), order)
                   : cudaLaunchKernelEx(&cfg, kv_select_kernel<false>, a, static_cast<int>(ctas), order)) == cudaSuccess
             ? 0 : -1;
}

}  // namespace sa
