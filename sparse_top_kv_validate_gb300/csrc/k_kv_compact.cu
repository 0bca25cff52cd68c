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
// A CTA takes the rows of K, or of V, of a (sequence, KV head).  A chunk's rows are found
// once, a thread to a row (list entry, then page, then place, each a chunk ahead of the
// next), and their places put into shared memory; the rows themselves pass through a ring there,
// each thread storing the pieces of 16 bytes that it has loaded.  (With the places worked
// out for every piece, 160 instructions of it, that was the bound: 128 contexts to 2,048
// tokens, 8 heads of 128, FP8 pages, 289 us; now 245, 66% of the copy bandwidth.)  Scale bytes and weights are moved by the threads that find the
// rows, as soon as they have.  Where there are too few (sequence, KV head)s for the device, a
// cluster of up to 8 larger CTAs shares one, each chunk cut in as many pieces (2 contexts of
// 66,000 and 69,000 tokens to 16,384, 4 heads of 128, 16-bit elements: 54 us; a cluster of 16, 68).
#include "cluster.cuh"
#include "weights.h"

namespace sa {

namespace {

constexpr int kMaxCluster = 8;

// Where a row comes from (-1: there is none) and goes to, in bytes from the start of its plane,
// and where its scale byte and its weight go (an element of theirs).
struct __align__(16) Place {
  int64_t from, to, scale, weight;
};

// A thread moves up to kRows rows of a chunk, two pieces of each at a time; chunks in the ring; the
// chunks whose places are kept: those in the ring and the one behind them.  A cluster's chunks
// are larger, as its barrier costs more; its ring has two, for clusters whose CTAs fill their
// multiprocessors wait for one another (the long contexts with 256 threads of 4 rows and
// three chunks, 67 us; 512 threads of 2, 55; with four chunks, 80).
constexpr int kPieces = 2;
template <bool kCluster>
struct Shape {
  static constexpr int kThreads = kCluster ? 512 : 128;
  static constexpr int kRows = 2;
  static constexpr int kStages = kCluster ? 2 : 4;
  static constexpr int kPlaces = kStages + 1;
  static constexpr int kRing = kStages * kRows * kPieces * kThreads * 16;

  // Rows of a CTA's part of a chunk, for rows of `pieces` pieces (at most kPieces * kThreads).
  static __host__ __device__ constexpr int chunk(int pieces) {
    const int n = kRows * (kThreads / ((pieces + kPieces - 1) / kPieces));
    return n < kThreads ? n : kThreads;  // (a thread finds one row)
  }
  static int bytes(int pieces) {  // of shared memory
    // (a row of more pieces takes several passes, the last of fewer: room for any chunk)
    const int rows = pieces > kPieces * kThreads ? kThreads : chunk(pieces);
    return kRing + kPlaces * rows * static_cast<int>(sizeof(Place));
  }
  static constexpr int kMost = kRing + kPlaces * kThreads * static_cast<int>(sizeof(Place));
};

// The loads whose words were folded into x have returned once this has executed.
__device__ __forceinline__ void arrived(uint32_t x) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %0, 0x5bd1e995;\n\t@p nanosleep.u32 0;\n\t}" ::"r"(x) : "memory");
}
// Every thread of the cluster passes wait() after every one has passed arrive().  No memory is
// ordered by it: what it stands for are reads whose values have come back.  (An arrival that
// releases waits for the stores of the chunk before to reach L2.)
template <bool kCluster>
__device__ __forceinline__ void arrive() {
  __syncthreads();  // (and what this CTA wrote to shared memory is seen)
  if (kCluster) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
template <bool kCluster>
__device__ __forceinline__ void wait() {
  if (kCluster) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename V>
__device__ __forceinline__ void copy_async(V* dst, const V* src) {
  if constexpr (sizeof(V) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else if constexpr (sizeof(V) == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else *dst = *src;
}

// The planes of a (sequence, KV head): rows, and beside them scale bytes and weights
// (nullable).  Row `slot` of unit (page * heads + head) lies at rows + unit * head_stride +
// slot * row_bytes, its scale at scales + unit * head_stride + slot.
struct Planes {
  char* rows;
  uint8_t* scales;
  float* weights;
  int64_t head_stride;
};

// V: the pieces that a row is moved in.
template <typename V, bool kCluster>
__device__ void move_rows(const CompactArgs& a, const Planes& pl, const int32_t* table, const int32_t* keep, int head,
                          int m, int rank, int ctas, uint8_t* smem, bool& bad) {
  using H = Shape<kCluster>;
  constexpr int S = H::kStages, R = H::kPlaces, kThreads = H::kThreads, kRows = H::kRows;
  const int tid = static_cast<int>(threadIdx.x);
  const uint32_t pt = static_cast<uint32_t>(a.page_tokens);
  const int all = a.row_bytes / static_cast<int>(sizeof(V));
  V* ring = reinterpret_cast<V*>(smem) + tid;  // piece q of row u of stage s: ring[((s * kRows + u) * kPieces + q) * kThreads]
  Place* places = reinterpret_cast<Place*>(smem + H::kRing);
#pragma unroll 1
  for (int col0 = 0; col0 < all; col0 += kPieces * kThreads) {  // (columns are independent of one another)
    const int pieces = min(all - col0, kPieces * kThreads), lanes = (pieces + kPieces - 1) / kPieces;
    const int rows = kThreads / lanes, chunk = H::chunk(pieces);
    const int r = tid / lanes, c = tid - r * lanes;  // this thread's first row of a chunk, and piece of it
    const int64_t step = static_cast<int64_t>(chunk) * ctas, own = static_cast<int64_t>(rank) * chunk;
    char* col = pl.rows + static_cast<int64_t>(col0 + c) * sizeof(V);

    // ---- finding a chunk's rows, one to a thread
    auto list = [&](int64_t first) {
      const int64_t i = first + own + tid;
      return tid < chunk && i < m ? __ldg(keep + i) : -1;  // (looked at by pages(), a chunk on)
    };
    struct Found {
      int32_t from, to;  // pages
      uint32_t from_slot, to_slot;
      bool moving;
    };
    auto pages = [&](int64_t first, int32_t src) {
      const uint32_t x = static_cast<uint32_t>(src), y = static_cast<uint32_t>(first + own) + tid;
      Found f{0, 0, 0, 0, src >= 0 && x != y};
      if (!f.moving) return f;
      const uint32_t px = a.shift >= 0 ? x >> a.shift : x / pt, py = a.shift >= 0 ? y >> a.shift : y / pt;
      f.from = __ldg(table + px);
      f.to = __ldg(table + py);
      f.from_slot = x - px * pt;
      f.to_slot = y - py * pt;
      return f;
    };
    // Writes the places down; the row's scale byte and weight are on their way.
    auto place = [&](const Found& f, int at, uint32_t& scale, uint32_t& weight) {
      Place now{-1, -1, -1, -1};
      scale = weight = 0;
      const bool good = f.from >= 0 && f.from < a.num_pages && f.to >= 0 && f.to < a.num_pages;
      if (f.moving && good) {
        const int64_t from = f.from * a.Hkv + head, to = f.to * a.Hkv + head;
        now.from = from * pl.head_stride + f.from_slot * static_cast<int64_t>(a.row_bytes);
        now.to = to * pl.head_stride + f.to_slot * static_cast<int64_t>(a.row_bytes);
        if (pl.scales && col0 == 0) {
          now.scale = to * pl.head_stride + f.to_slot;
          scale = pl.scales[from * pl.head_stride + f.from_slot];
        }
        if (pl.weights && col0 == 0) {
          now.weight = to * static_cast<int64_t>(pt) + f.to_slot;
          weight = reinterpret_cast<const uint32_t*>(pl.weights)[from * static_cast<int64_t>(pt) + f.from_slot];
        }
      }
      bad = bad || (f.moving && !good);
      if (tid < chunk) places[at * chunk + tid] = now;
    };

    // ---- moving them
    uint32_t live = 0;  // a bit per stage and row of this thread: it is to be stored
    auto copy = [&](int stage, int at) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const uint32_t bit = 1u << (stage * kRows + u);
        live &= ~bit;
        const int x = u * rows + r;
        if (r >= rows || x >= chunk) continue;
        const int64_t from = places[at * chunk + x].from;
        if (from < 0) continue;
        live |= bit;
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
          if (c + q * lanes < pieces)
            copy_async(ring + ((stage * kRows + u) * kPieces + q) * kThreads,
                       reinterpret_cast<const V*>(col + from + q * lanes * static_cast<int>(sizeof(V))));
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto store = [&](int stage, int at, uint32_t scale, uint32_t weight) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (!(live >> (stage * kRows + u) & 1u)) continue;
        const int64_t to = places[at * chunk + u * rows + r].to;
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
          if (c + q * lanes < pieces)
            *reinterpret_cast<V*>(col + to + q * lanes * static_cast<int>(sizeof(V))) =
                ring[((stage * kRows + u) * kPieces + q) * kThreads];
      }
      if (tid < chunk) {
        const Place& p = places[at * chunk + tid];
        if (p.scale >= 0) pl.scales[p.scale] = static_cast<uint8_t>(scale);
        if (p.weight >= 0) reinterpret_cast<uint32_t*>(pl.weights)[p.weight] = weight;
      }
    };

    // Chunk k: stage k % S of the ring, places k % R; its small values in scale / weight[k % S].
    // (The loop goes S chunks at a time, so that a value on its way stays in its register.)
    uint32_t scale[S], weight[S];
    Found found[S];
#pragma unroll
    for (int s = 0; s < S; ++s) found[s] = pages(s * step, list(s * step));
#pragma unroll
    for (int s = 0; s < S; ++s) place(found[s], s, scale[s], weight[s]);
    Found ahead = pages(S * step, list(S * step));
    int32_t src = list((S + 1) * step);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) copy(s, s);
    int at = 0;
#pragma unroll 1
    for (int64_t first = 0; first < m; first += S * step) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int64_t now = first + s * step;
        if (now >= m) break;
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");  // this chunk's are there
        const uint32_t now_scale = scale[s], now_weight = weight[s];
        arrived(now_scale ^ now_weight);
        arrive<kCluster>();
        copy((s + S - 1) % S, at + S - 1 < R ? at + S - 1 : at + S - 1 - R);
        place(ahead, at + S < R ? at + S : at + S - R, scale[s], weight[s]);
        ahead = pages(now + (S + 1) * step, src);
        src = list(now + (S + 2) * step);
        wait<kCluster>();
        store(s, at, now_scale, now_weight);
        if (++at == R) at = 0;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the places have been read
  }
}

template <bool kCluster>
__global__ void __launch_bounds__(Shape<kCluster>::kThreads)
    kv_compact_kernel(const __grid_constant__ CompactArgs a, int ctas) {
  constexpr int kThreads = Shape<kCluster>::kThreads;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ int s_end, s_code;
  const int tid = static_cast<int>(threadIdx.x);
  const uint32_t item = blockIdx.x / static_cast<uint32_t>(ctas);
  const int rank = kCluster ? static_cast<int>(cluster_rank()) : 0;
  const uint32_t row = item >> 1;
  const int plane = static_cast<int>(item & 1u);  // K or V
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
  bool bad = false;
  Planes pl;
  pl.rows = static_cast<char*>(a.pool[plane]);
  pl.head_stride = static_cast<int64_t>(a.page_tokens) * (a.row_bytes + (a.fp8 ? 1 : 0));
  pl.scales = a.fp8 ? reinterpret_cast<uint8_t*>(pl.rows) + static_cast<int64_t>(a.page_tokens) * a.row_bytes : nullptr;
  pl.weights = plane == 0 ? a.weights : nullptr;
  const int32_t* table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  if (a.align == 16) move_rows<uint4, kCluster>(a, pl, table, keep, h, m, rank, ctas, ring, bad);
  else if (a.align == 4) move_rows<uint32_t, kCluster>(a, pl, table, keep, h, m, rank, ctas, ring, bad);
  else move_rows<uint16_t, kCluster>(a, pl, table, keep, h, m, rank, ctas, ring, bad);
  if (bad && a.err_word) atomicOr(a.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
}

}  // namespace

int launch_kv_compact(const CompactArgs& a, cudaStream_t st) {
  const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * 2;
  // clusters where a CTA per item would leave half of the multiprocessors idle and there is more
  // than one chunk to move
  const int pieces = a.row_bytes / a.align;
  int ctas = 1;
  const int64_t chunk = pieces > kPieces * Shape<true>::kThreads ? 1 : Shape<true>::chunk(pieces);
  while (ctas < kMaxCluster && items * ctas * 2 <= sm_count() && chunk * ctas / 2 < a.width) ctas *= 2;
  if (items * ctas > INT32_MAX) return -1;
  const void* kernel = ctas > 1 ? reinterpret_cast<const void*>(kv_compact_kernel<true>)
                                : reinterpret_cast<const void*>(kv_compact_kernel<false>);
  if (!allow_smem(kernel, ctas > 1 ? Shape<true>::kMost : Shape<false>::kMost)) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(ctas > 1 ? Shape<true>::kThreads : Shape<false>::kThreads));
  cfg.dynamicSmemBytes = static_cast<size_t>(ctas > 1 ? Shape<true>::bytes(pieces) : Shape<false>::bytes(pieces));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return (ctas > 1 ? cudaLaunchKernelEx(&cfg, kv_compact_kernel<true>, a, ctas)
                   : cudaLaunchKernelEx(&cfg, kv_compact_kernel<false>, a, ctas)) == cudaSuccess
             ? 0 : -1;
}

}  // namespace sa
