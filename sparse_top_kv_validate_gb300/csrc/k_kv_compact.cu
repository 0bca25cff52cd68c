// k_kv_compact.cu -- the kept rows of a sequence moved to the front of its pages, in
// place: for every (sequence, KV head) and i < m, token i's row of K, of V and its
// weight become those of token keep[i], an ascending list of m tokens.
//
// Pure traffic: each moved row is read and written once.  A row may be written where
// another one has yet to be read from, but only downwards: keep[j] >= j, so with the
// list cut into chunks the sources of a chunk lie at or behind its own first place,
// and never where an earlier chunk writes.  Hence a chunk's rows need to have been read
// before they are written, by all that share it (one barrier), while the reads of the
// chunk after it may already be on their way.
//
// A CTA takes one plane of a (sequence, KV head): the rows of K, those of V, or the
// small ones (scale bytes and weights) one after the other.  Where that makes too few
// CTAs for the device, a cluster of up to 8 shares a plane, each chunk cut in as many pieces.
#include "cluster.cuh"
#include "weights.h"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxCluster = 8;

// The loads whose words were folded into x have returned once this has executed.
__device__ __forceinline__ void arrived(uint32_t x) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %0, 0x5bd1e995;\n\t@p nanosleep.u32 0;\n\t}" ::"r"(x) : "memory");
}
__device__ __forceinline__ uint32_t word_of(uint4 v) { return v.x; }
__device__ __forceinline__ uint32_t word_of(uint32_t v) { return v; }
__device__ __forceinline__ uint32_t word_of(uint16_t v) { return v; }
__device__ __forceinline__ uint32_t word_of(uint8_t v) { return v; }

struct Pages {
  const int32_t* table;  // of the sequence
  uint32_t pt;
  int shift;             // log2(pt), or -1
  int64_t num_pages, heads, head;
  __device__ __forceinline__ void find(uint32_t t, int32_t& page, uint32_t& slot) const {
    const uint32_t pi = shift >= 0 ? t >> shift : t / pt;
    slot = t - pi * pt;
    page = __ldg(table + pi);
  }
  __device__ __forceinline__ bool good(int32_t page) const { return page >= 0 && page < num_pages; }
};

// `pieces` pieces of type V per row of one plane: token t's at
// base + (page * heads + head) * head_stride + slot * row_stride (bytes).
template <typename V, int U, bool kCluster>
__device__ void move_plane(char* base, int64_t head_stride, int64_t row_stride, int pieces, const Pages& pg,
                           const int32_t* keep, int m, int rank, int ctas, bool& bad) {
  const int tid = static_cast<int>(threadIdx.x);
#pragma unroll 1
  for (int col0 = 0; col0 < pieces; col0 += kThreads) {  // (columns are independent of one another)
    const int cols = min(pieces - col0, kThreads);
    const int rows = kThreads / cols;                     // of a step
    const int r = tid / cols, c = col0 + tid - r * cols;
    const bool mine = r < rows;
    const int chunk = rows * U;                           // rows of this CTA's piece of a chunk
    char* col = base + static_cast<int64_t>(c) * sizeof(V);
    auto at = [&](int32_t page, uint32_t slot) {
      return reinterpret_cast<V*>(col + (page * pg.heads + pg.head) * head_stride + slot * row_stride);
    };
    // the rows of a chunk, on their way; bit u: there is one to move
    auto load = [&](int64_t first, V (&v)[U]) {
      uint32_t live = 0;
      int32_t src[U], page[U];
      uint32_t slot[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * rows + r;
        src[u] = -1;
        if (mine && i < m) {
          src[u] = __ldg(keep + i);
          if (src[u] == i) src[u] = -1;  // where it belongs
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        page[u] = -1;
        if (src[u] >= 0) pg.find(static_cast<uint32_t>(src[u]), page[u], slot[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (src[u] < 0) continue;
        if (pg.good(page[u])) {
          v[u] = *at(page[u], slot[u]);
          live |= 1u << u;
        } else {
          bad = true;
        }
      }
      return live;
    };
    const int64_t step = static_cast<int64_t>(chunk) * ctas;
    V v[U], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = w[u] = V{};
    uint32_t live = load(static_cast<int64_t>(rank) * chunk, v);
#pragma unroll 1
    for (int64_t first = 0; first < m; first += step) {
      const int64_t own = first + static_cast<int64_t>(rank) * chunk;
      const uint32_t next = load(own + step, w);
      uint32_t x = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) x ^= word_of(v[u]);
      arrived(x);
      if (kCluster) cluster_sync();
      else __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!((live >> u) & 1u)) continue;
        int32_t page;
        uint32_t slot;
        pg.find(static_cast<uint32_t>(own + u * rows + r), page, slot);
        if (pg.good(page)) *at(page, slot) = v[u];
        else bad = true;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = w[u];
      live = next;
    }
  }
}

template <bool kCluster>
__global__ void __launch_bounds__(kThreads)
    kv_compact_kernel(const __grid_constant__ CompactArgs a, int planes, int ctas, int shift) {
  __shared__ int s_end, s_code;
  const int tid = static_cast<int>(threadIdx.x);
  const uint32_t item = blockIdx.x / static_cast<uint32_t>(ctas);
  const int rank = kCluster ? static_cast<int>(cluster_rank()) : 0;
  const uint32_t row = item / static_cast<uint32_t>(planes);
  const int plane = static_cast<int>(item - row * static_cast<uint32_t>(planes));
  const int b = static_cast<int>(row / static_cast<uint32_t>(a.Hkv)), h = static_cast<int>(row) - b * a.Hkv;
  const int32_t* keep = a.keep + static_cast<int64_t>(row) * a.width;
  const int64_t n = __ldg(a.ctx_len + b);
  const bool tells = plane == 0 && rank == 0 && a.err_word;
  if (n < 0 || n > a.max_pages * a.page_tokens) {
    if (tells && tid == 0) atomicOr(a.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
    return;
  }
  // The list's end, and whether it is one: a row whose list is not valid stays as it is.
  if (tid == 0) {
    s_end = a.width;
    s_code = 0;
  }
  __syncthreads();
  {
    int end = a.width, code = 0;
#pragma unroll 4
    for (int i = tid; i < a.width; i += kThreads) {
      const int32_t v = __ldg(keep + i), before = i > 0 ? __ldg(keep + i - 1) : -2;
      if (v == -1) end = min(end, i);
      else if (v < -1) code |= SA_IDX_BELOW_SENTINEL;
      else if (before == -1) code |= SA_IDX_AFTER_PADDING;
      else if (v >= n) code |= SA_IDX_OUT_OF_RANGE;
      else if (v == before) code |= SA_IDX_DUPLICATE;
      else if (v < before) code |= SA_IDX_NOT_INCREASING;
    }
    end = __reduce_min_sync(0xffffffffu, end);
    code = __reduce_or_sync(0xffffffffu, code);
    if ((tid & 31) == 0) {
      atomicMin(&s_end, end);
      if (code) atomicOr(&s_code, code);
    }
  }
  __syncthreads();
  const int m = s_end, code = s_code;
  if (code) {
    if (tells && tid == 0) atomicOr(a.err_word, static_cast<uint32_t>(code));
    return;
  }
  const Pages pg{a.block_table + static_cast<int64_t>(b) * a.max_pages, static_cast<uint32_t>(a.page_tokens), shift,
                 a.num_pages, a.Hkv, h};
  bool bad = false;
  const int64_t head = static_cast<int64_t>(a.page_tokens) * (a.row_bytes + (a.fp8 ? 1 : 0));
  if (plane < 2) {
    char* base = static_cast<char*>(a.pool[plane]);
    if (a.align == 16)
      move_plane<uint4, 8, kCluster>(base, head, a.row_bytes, a.row_bytes / 16, pg, keep, m, rank, ctas, bad);
    else if (a.align == 4)
      move_plane<uint32_t, 8, kCluster>(base, head, a.row_bytes, a.row_bytes / 4, pg, keep, m, rank, ctas, bad);
    else
      move_plane<uint16_t, 8, kCluster>(base, head, a.row_bytes, a.row_bytes / 2, pg, keep, m, rank, ctas, bad);
  } else {
    if (a.fp8)
      for (int t = 0; t < 2; ++t)
        move_plane<uint8_t, 8, kCluster>(static_cast<char*>(a.pool[t]) + static_cast<int64_t>(a.page_tokens) * a.row_bytes,
                                         head, 1, 1, pg, keep, m, rank, ctas, bad);
    if (a.weights)
      move_plane<uint32_t, 8, kCluster>(reinterpret_cast<char*>(a.weights), static_cast<int64_t>(a.page_tokens) * 4, 4, 1,
                                        pg, keep, m, rank, ctas, bad);
  }
  if (bad && a.err_word) atomicOr(a.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
}

}  // namespace

int launch_kv_compact(const CompactArgs& a, cudaStream_t st) {
  const int planes = a.fp8 || a.weights ? 3 : 2;
  const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * planes;
  // about two CTAs to a multiprocessor, each with a few chunks to move
  const int64_t pieces = a.row_bytes / a.align, rows = pieces >= kThreads ? 1 : kThreads / pieces;
  int ctas = 1;
  while (ctas < kMaxCluster && items * ctas < 2 * sm_count() && rows * 8 * ctas * 2 < a.width) ctas *= 2;
  if (items * ctas > INT32_MAX) return -1;
  int shift = -1;
  for (int s = 0; s < 31; ++s)
    if (a.page_tokens == 1 << s) shift = s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return (ctas > 1 ? cudaLaunchKernelEx(&cfg, kv_compact_kernel<true>, a, planes, ctas, shift)
                   : cudaLaunchKernelEx(&cfg, kv_compact_kernel<false>, a, planes, ctas, shift)) == cudaSuccess
             ? 0 : -1;
}

}  // namespace sa
