// k_kv_select.cu -- the tokens that a head keeps of a context that has outgrown its
// budget: the first `sink`, the last `recent`, and of those between them the ones
// whose accumulated attention weight is largest (ties: the lower token).
//
// A row is a (sequence, KV head) with n tokens.  The weights are compared as unsigned
// keys (sign and exponent turned so that a larger weight is a larger key; NaN like
// -inf, -0 like 0).  The key T of the last token kept is found digit by digit: a
// histogram of the upper 11 bits, of the 11 below them among the keys that share the
// upper digit, of the last 10; then token t is kept when key > T, or key == T and
// fewer than `ties` equal keys lie before it.  The number kept before a token is
// G + min(E, ties), with G the greater and E the equal keys before it, so one scan of
// the pair (G, E) places every token in ascending order.
//
// Every weight is read once and held in registers (16 keys a thread); what is left
// is issue slots, so a row gets as many CTAs (a cluster, up to 8) as make it 8,192 tokens
// each, and a multiprocessor several of them: their barriers and the loads' latency
// overlap.  Longer rows read their weights again, from L2, for each pass.  The CTAs of a cluster
// read one another's histograms through distributed shared memory; every pass has a
// buffer of its own, so that one barrier per pass is enough.
#include "cluster.cuh"
#include "weights.h"

namespace sa {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kQuads = 4;                          // of tokens, per thread and chunk
constexpr int kChunk = kThreads * kQuads * 4;      // tokens of a CTA's chunk
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;                        // of the first two digits (the third: 1,024)
constexpr uint32_t kLowest = 0x007fffffu;          // the key of -inf
constexpr int kPasses = 3;
__host__ __device__ constexpr int pass_shift(int p) { return p == 0 ? 21 : p == 1 ? 10 : 0; }

__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 becomes 0
  if (w != w) return kLowest;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct Shared {
  uint32_t hist[kPasses][kBins];
  uint2 part[kWarps];               // of a block-wide sum
  uint2 count[kQuads][kWarps];      // (greater, equal) keys of a warp's quads
  uint2 total;                      // of the CTA
  uint32_t bin, above, inside;      // the digit found, the keys above it, its own
};

template <bool kCluster>
__global__ void __launch_bounds__(kThreads, 2)
    kv_select_kernel(const __grid_constant__ SelectArgs a, int ctas) {
  __shared__ __align__(16) Shared sm;
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

  const int sink = a.sink, late = n - a.recent;      // the middle: sink .. late - 1
  uint32_t need = static_cast<uint32_t>(a.budget - a.sink - a.recent);
  const int seg = ((n + ctas - 1) / ctas + 3) & ~3;
  const int begin = min(rank * seg, n), end = min(begin + seg, n);
  const uint32_t pt = static_cast<uint32_t>(a.page_tokens);
  const int32_t* table = a.block_table + static_cast<int64_t>(b) * a.max_pages;

  // The keys of a chunk's quad of tokens; 0, which no weight has, where there is no token
  // of the middle.
  bool bad = false;
  auto page_of = [&](uint32_t pi) {
    const int32_t p = __ldg(table + pi);
    if (p >= 0 && p < a.num_pages) return static_cast<int64_t>(p);
    bad = true;
    return int64_t(-1);
  };
  auto load = [&](int base, uint32_t (&key)[kQuads][4]) {
    float w[kQuads][4];
#pragma unroll
    for (int r = 0; r < kQuads; ++r) {
      const int t = base + (r * kThreads + tid) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[r][e] = SA_NEG_INF;
      if (t >= end) continue;
      if (a.vec) {
        const uint32_t pi = static_cast<uint32_t>(t) / pt;
        const int64_t p = page_of(pi);
        if (p >= 0) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(
              a.weights + (p * a.Hkv + h) * pt + (static_cast<uint32_t>(t) - pi * pt)));
          w[r][0] = v.x;
          w[r][1] = v.y;
          w[r][2] = v.z;
          w[r][3] = v.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (t + e >= end) continue;
          const uint32_t pi = static_cast<uint32_t>(t + e) / pt;
          const int64_t p = page_of(pi);
          if (p >= 0) w[r][e] = __ldg(a.weights + (p * a.Hkv + h) * pt + (static_cast<uint32_t>(t + e) - pi * pt));
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kQuads; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = base + (r * kThreads + tid) * 4 + e;
        key[r][e] = t >= sink && t < late && t < end ? key_of(w[r][e]) : 0u;
      }
  };

  for (int i = tid; i < kPasses * kBins; i += kThreads) (&sm.hist[0][0])[i] = 0;
  uint32_t key[kQuads][4];
  load(begin, key);
  const bool one = end - begin <= kChunk;  // the keys stay where they are
  __syncthreads();

  // ---- the key of the last one kept --------------------------------------------------------
  uint32_t prefix = 0, last = 0xffffffffu, ties = 0;  // (need 0: none of the middle)
#pragma unroll 1
  for (int p = 0; p < kPasses && need > 0; ++p) {
    const int shift = pass_shift(p), above_shift = p == 0 ? 31 : pass_shift(p - 1);
    uint32_t* hist = sm.hist[p];
    const uint32_t mask = p == 2 ? 1023u : 2047u;
    auto count = [&]() {
#pragma unroll
      for (int r = 0; r < kQuads; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t k = key[r][e];
          const bool in = k != 0u && (p == 0 || (k >> above_shift) == prefix);
          const uint32_t bin = in ? (k >> shift) & mask : kBins;
          // keys that are all alike (a fresh pool's zeros) would queue for one word
          if (__all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0))) {
            if (in && lane == 0) atomicAdd(hist + bin, 32u);
          } else if (in) {
            atomicAdd(hist + bin, 1u);
          }
        }
    };
    count();
    if (!one)
      for (int base = begin + kChunk; base < end; base += kChunk) {
        load(base, key);
        count();
      }
    // four bins a thread, the largest first; over the cluster
    uint4 c;
    const int at = kBins - 4 - 4 * tid;
    if (kCluster) {
      cluster_sync();
      const uint32_t addr = smem_u32(hist + at);
      c = make_uint4(0u, 0u, 0u, 0u);
      for (int q = 0; q < ctas; ++q) {
        const uint4 v = ld_cluster4(cluster_addr(addr, static_cast<uint32_t>(q)));
        c.x += v.x;
        c.y += v.y;
        c.z += v.z;
        c.w += v.w;
      }
    } else {
      __syncthreads();
      c = *reinterpret_cast<const uint4*>(hist + at);
    }
    const uint32_t sum = c.x + c.y + c.z + c.w;
    uint32_t before = sum;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, before, sh);
      if (lane >= sh) before += x;
    }
    if (lane == 31) sm.part[warp].x = before;
    __syncthreads();
    before -= sum;
    for (int w = 0; w < warp; ++w) before += sm.part[w].x;
    if (before < need && need <= before + sum) {  // one thread
      const uint32_t v[4] = {c.w, c.z, c.y, c.x};
      uint32_t up = before;
      int i = 0;
      while (up + v[i] < need) up += v[i++];
      sm.bin = static_cast<uint32_t>(at + 3 - i);
      sm.above = up;
      sm.inside = v[i];
    }
    __syncthreads();
    prefix = p == 0 ? sm.bin : (prefix << (p == 2 ? 10 : 11)) | sm.bin;
    need -= sm.above;
    if (p == kPasses - 1) {
      last = prefix;
      ties = need;
    } else if (sm.inside == need) {  // the whole digit is kept
      last = (prefix << shift) - 1u;
      ties = 0;
      break;
    }
    if (!one) load(begin, key);  // (the first chunk again)
  }
  if (!one && need > 0) load(begin, key);

  // ---- their tokens, in ascending order ----------------------------------------------------
  // A chunk at a time; `done`: (greater, equal) before the chunk, over the whole row.
  auto tell = [&](int r, uint32_t& greater, uint32_t& equal) {  // a bit per token of quad r
    greater = equal = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (key[r][e] > last) greater |= 1u << e;
      if (key[r][e] == last) equal |= 1u << e;
    }
  };
  auto guarded = [&](int base, int r, uint32_t& greater) {  // the tokens kept whatever their weight
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = base + (r * kThreads + tid) * 4 + e;
      if (t < end && (t < sink || t >= late)) greater |= 1u << e;
    }
  };
  auto add = [](uint2 x, uint2 y) { return make_uint2(x.x + y.x, x.y + y.y); };
  uint2 done = make_uint2(0u, 0u);
  if (kCluster) {
    // what the CTAs before this one keep
    uint2 mine = make_uint2(0u, 0u);
    for (int base = begin; base < end; base += kChunk) {
      if (base != begin) load(base, key);
#pragma unroll
      for (int r = 0; r < kQuads; ++r) {
        uint32_t g, q;
        tell(r, g, q);
        guarded(base, r, g);
        mine = add(mine, make_uint2(__popc(g), __popc(q)));
      }
    }
    if (!one) load(begin, key);
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1)
      mine = add(mine, make_uint2(__shfl_xor_sync(0xffffffffu, mine.x, sh), __shfl_xor_sync(0xffffffffu, mine.y, sh)));
    if (lane == 0) sm.part[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      uint2 t = make_uint2(0u, 0u);
      for (int w = 0; w < kWarps; ++w) t = add(t, sm.part[w]);
      sm.total = t;
    }
    cluster_sync();
    const uint32_t addr = smem_u32(&sm.total);
    for (int q = 0; q < rank; ++q) done = add(done, ld_cluster2(cluster_addr(addr, static_cast<uint32_t>(q))));
  }
#pragma unroll 1
  for (int base = begin; base < end; base += kChunk) {
    if (base != begin) {
      load(base, key);
      __syncthreads();  // the counts of the chunk before have been read
    }
    uint2 in[kQuads];  // (greater, equal) of this warp's quads r before this thread's
#pragma unroll
    for (int r = 0; r < kQuads; ++r) {
      uint32_t g, q;
      tell(r, g, q);
      guarded(base, r, g);
      // both counts in one word: at most 128 of either in a warp
      const uint32_t own = __popc(g) | __popc(q) << 16;
      uint32_t x = own;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, sh);
        if (lane >= sh) x += y;
      }
      if (lane == 31) sm.count[r][warp] = make_uint2(x & 0xffffu, x >> 16);
      x -= own;
      in[r] = make_uint2(x & 0xffffu, x >> 16);
    }
    __syncthreads();
    uint2 all = done;
#pragma unroll
    for (int r = 0; r < kQuads; ++r) {
      uint2 at = add(all, in[r]);
      for (int w = 0; w < kWarps; ++w) {
        const uint2 c = sm.count[r][w];
        if (w < warp) at = add(at, c);
        all = add(all, c);
      }
      uint32_t g, q;
      tell(r, g, q);
      guarded(base, r, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool greater = (g >> e) & 1u, equal = (q >> e) & 1u;
        if (greater || (equal && at.y < ties))
          keep[at.x + min(at.y, ties)] = base + (r * kThreads + tid) * 4 + e;
        at.x += greater;
        at.y += equal;
      }
    }
    done = all;
  }
  if (bad && a.err_word) atomicOr(a.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
  if (kCluster) cluster_sync();  // the others have read this CTA's counts
}

}  // namespace

int launch_kv_select(const SelectArgs& a, cudaStream_t st) {
  // the host knows the longest context that the table can hold
  const int64_t most = a.max_pages * a.page_tokens;
  int ctas = 1;
  while (ctas < kMaxCluster && static_cast<int64_t>(ctas) * kChunk < most) ctas *= 2;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv;
  if (rows * ctas > INT32_MAX) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return (ctas > 1 ? cudaLaunchKernelEx(&cfg, kv_select_kernel<true>, a, ctas)
                   : cudaLaunchKernelEx(&cfg, kv_select_kernel<false>, a, ctas)) == cudaSuccess ? 0 : -1;
}

}  // namespace sa
