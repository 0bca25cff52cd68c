// k_weights.cu -- the attention weight that each key receives from packed queries, on
// the fifth-generation tensor cores (tcgen05.mma, accumulators in tensor memory,
// operands staged by TMA).
//
// w_j = sum over queries i and heads of 2^(c s_ij - L_i) with s = q . k, c = scale
// log2(e) and L_i = log2 sum_j 2^(c s_ij): the row sums have to be known before a
// column can be added up, so the product is formed twice, by one kernel in two forms:
//   kSums 0  outer tiles of query rows, inner tiles of keys: -L of every row;
//   kSums 1  outer tiles of keys, inner tiles of query rows: w of every key.
// Both times a thread owns an outer row, so that its sum runs along the columns of the
// score tile that it reads from tensor memory: no reduction between threads, no
// second operand, no probabilities to be passed on.  Bound by the exponentials (one
// per visible pair, query head and form), then by the tensor cores.
//
// A query row is a (token, head of the group): a tile is 128 / g tokens times the g
// heads of one KV head.  An item is two outer tiles of 128 rows that share every inner
// tile (with one, the inner tiles' way from L2 would be the bound: 32 KB per 700
// cycles and multiprocessor).
//
// The work is the pairs (item, inner tile) that the causal mask leaves, laid end to end
// by sequence, KV head, item; each CTA (one per multiprocessor) takes one
// contiguous range, whatever the lengths.  An item's place has a closed form (sums of
// floor((a x + b) / m)), so no table of items is built.  An item cut between CTAs
// leaves partial sums, merged in order by merge_kernel.
//
// Warps: 0 loads (outer tiles through two buffers, inner ones through a ring), 1 issues
// the MMAs, 4-7 and 8-11 take the scores of one outer tile each, from two buffers of
// tensor memory.  Every mbarrier wait is bounded; a stalled pipeline sets
// SA_ERRBIT_TIMEOUT, stops every role, and still frees the tensor memory.
#include <cuda.h>

#include <cstring>
#include <type_traits>

#include "packed.cuh"
#include "pool_add.cuh"
#include "tc05.cuh"
#include "weights.h"

namespace sa {

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;               // rows of a tile
constexpr int kSlabBytes = kTile * 128;  // 128 rows x 64 sixteen-bit columns
constexpr int kMaxSeqs = 1024;           // sequences per launch
constexpr int kLStages = 3;              // slots of the ring of row statistics
constexpr float kRaiseLog2 = 8.0f;       // the offset of a row's sum is raised beyond 2^8

template <int D>
struct Geo {
  static constexpr int kSlabs = D / 64;
  static constexpr int kTileBytes = kSlabs * kSlabBytes;  // 16 or 32 KB
  static constexpr int kStages = D == 128 ? 3 : 6;        // inner tiles in the ring
  static constexpr int kOffOuter = 0;                     // two buffers of two tiles
  static constexpr int kOffInner = 4 * kTileBytes;
  static constexpr int kOffL = kOffInner + kStages * kTileBytes;  // float [kLStages][128]
  static constexpr int kOffBar = kOffL + kLStages * kTile * 4;
  static constexpr int kBarOFull = 0, kBarOEmpty = 2, kBarIFull = 4, kBarIEmpty = kBarIFull + kStages,
                       kBarLFull = kBarIEmpty + kStages, kBarLEmpty = kBarLFull + kLStages,
                       kBarSFull = kBarLEmpty + kLStages, kBarSEmpty = kBarSFull + 4,  // [warpgroup][buffer]
                       kBarDone = kBarSEmpty + 4, kNumBars = kBarDone + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tensor memory, abort flag
  static constexpr int kBytes = 1024 + kOffMisc + 8;
  static_assert(kBytes <= 227 * 1024, "a CTA's shared memory");
  static_assert(kStages * kTileBytes >= (kMaxSeqs + 1) * 8 + 64, "the ring serves as scratch");
};

struct Params {
  const int32_t* q_start;
  const int32_t* k_start;
  const int32_t* block_table;
  float* weights;
  uint32_t* err_word;
  float* nlse;        // [query tiles][128]: -L of the rows
  float2* part;       // [CTAs][2][256]: (m, l), or (w, -), of items cut at the range's begin, end
  int4* cut;          // [CTAs]: the item cut at the range's end that begins in it, last CTA
  int B, Tq, Tk, Hkv, g;
  int tpt;            // tokens per query tile: 128 / g
  int b0;             // sequences before these
  int accumulate;
  int64_t page_tokens, max_pages, num_pages;
  float c_log2;       // scale * log2(e)
};

// ---- items and their places ------------------------------------------------------------

// sum_{i < n} floor((a i + b) / m), the Euclidean recurrence.  (Tokens stay below 2^30, so
// that a n + b, with a and b reduced, fits 32 bits.)
__device__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t s = 0;
  while (n > 0) {
    if (a >= m) {
      const uint32_t q = a / m;
      s += (static_cast<int64_t>(n) - 1) * n / 2 * q;
      a -= q * m;
    }
    if (b >= m) {
      const uint32_t q = b / m;
      s += static_cast<int64_t>(n) * q;
      b -= q * m;
    }
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return s;
}

struct Seq {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ Seq seq_of(const Params& p, int b) {
  const Span q = span_of(p.q_start, b, p.Tq), k = span_of(p.k_start, b, p.Tk);
  return Seq{q.first, q.n, k.first, k.n};
}

// The items (outer tile pairs) of one sequence and KV head.
template <bool kSums>
struct Items {
  int off;       // nk - nq: query i sees the keys up to i + off
  int nq, nk;
  int tpt, span; // tokens of a query tile; of an item
  int count;     // items

  __device__ __forceinline__ Items(const Params& p, const Seq& s)
      : off(s.nk - s.nq), nq(s.nq), nk(s.nk), tpt(p.tpt), span(kSums ? 2 * kTile : 2 * p.tpt) {
    const int n = kSums ? nk : nq;
    count = nq == 0 || nk == 0 ? 0 : (n + span - 1) / span;
  }
  // Inner tiles of item o: [first, first + size).
  __device__ __forceinline__ int first(int o) const {
    if (!kSums) return 0;
    const int i = o * span - off;  // the first token that sees the item's first key
    return i > 0 ? i / tpt : 0;
  }
  __device__ __forceinline__ int size(int o) const {
    if (kSums) return (nq + tpt - 1) / tpt - first(o);
    const int lim = min(nk - 1, min((o + 1) * span, nq) - 1 + off);
    return lim < 0 ? 0 : lim / kTile + 1;
  }
  // Pairs of the items before o.
  __device__ int64_t before(int o) const {
    if (o == 0) return 0;
    if (kSums) {  // size(x) = all query tiles less floor(max(0, x span - off) / tpt)
      const int x0 = off > 0 ? (off + span - 1) / span : 0;
      int64_t s = static_cast<int64_t>(o) * ((nq + tpt - 1) / tpt);
      if (o > x0) s -= floor_sum(o - x0, tpt, span, x0 * span - off);
      return s;
    }
    // all but the last item: max(0, floor((x span + c) / 128)) with c = span - 1 + off + 128
    const int n = min(o, count - 1), c = span - 1 + off + kTile;
    const int x0 = c < 0 ? (-c + span - 1) / span : 0;
    int64_t s = n > x0 ? floor_sum(n - x0, kTile, span, x0 * span + c) : 0;
    if (o == count) s += size(count - 1);
    return s;
  }
};

// Where a walk over items stands; every role walks on its own from the same start.
template <bool kSums>
struct Walk {
  int b, h, o;
  int64_t off;   // place of the item's first pair
  int size, first;
  Seq s;

  __device__ __forceinline__ void fill(const Params& p) {
    const Items<kSums> it(p, s);
    size = it.size(o);
    first = it.first(o);
  }
  // The next item with a pair (there is one, unless b reaches p.B).
  __device__ __forceinline__ void next(const Params& p) {
    off += size;
    Items<kSums> it(p, s);
    ++o;
    for (;;) {
      while (o < it.count && it.size(o) == 0) ++o;
      if (o < it.count) break;
      o = 0;
      if (++h < p.Hkv) continue;
      h = 0;
      do {
        if (++b >= p.B) {
          size = 0;
          return;
        }
        s = seq_of(p, b);
        it = Items<kSums>(p, s);
      } while (it.count == 0);
    }
    size = it.size(o);
    first = it.first(o);
  }
};

// A query tile's place among the rows' statistics, of Hkv (Tq / tpt + B + 1): each tile's own.
__device__ __forceinline__ int64_t tile_id(const Params& p, int b, int q0, int tile, int h) {
  return (q0 / p.tpt + p.b0 + b + tile) * static_cast<int64_t>(p.Hkv) + h;
}

// ---- what a row ends with ------------------------------------------------------------------

// kSums 0: -L of query row `row` of the item's tile w, from the row's offset and sum.
// -inf, so that its keys get nothing, for a row that sees nothing but -inf and for one
// that holds no query.
__device__ __forceinline__ void put_row(const Params& p, const Walk<false>& wk, int w, int row, float m, float l) {
  const int tile = 2 * wk.o + w, rt = row / p.g;
  if (tile * p.tpt >= wk.s.nq) return;
  const bool live = rt < p.tpt && tile * p.tpt + rt < wk.s.nq;
  p.nlse[tile_id(p, wk.b, wk.s.q0, tile, wk.h) * kTile + row] =
      !live || m == SA_NEG_INF ? SA_NEG_INF : -(m + log2f(l));
}

// kSums 1: the weight of the item's key `row` of tile w.
__device__ __forceinline__ void put_key(const Params& p, const Walk<true>& wk, int w, int row, float sum) {
  const int j = wk.o * 2 * kTile + w * kTile + row;
  if (j >= wk.s.nk) return;
  const uint32_t pi = static_cast<uint32_t>(j) / static_cast<uint32_t>(p.page_tokens);
  int32_t page = -1;
  if (pi < p.max_pages) page = __ldg(p.block_table + wk.b * p.max_pages + pi);
  if (page < 0 || page >= p.num_pages) {
    if (p.err_word) atomicOr(p.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
    return;
  }
  const int64_t slot = j - static_cast<int64_t>(pi) * p.page_tokens;
  pool_put(p.weights + (page * static_cast<int64_t>(p.Hkv) + wk.h) * p.page_tokens + slot, sum,
           p.accumulate && j < wk.s.nk - wk.s.nq);
}

// ---- roles -----------------------------------------------------------------------------------

// This CTA's range of pairs.
struct Range {
  int64_t begin, end;
};

template <int D, bool kSums>
__device__ void producer(const CUtensorMap* tq, const CUtensorMap* tk, const Params& p, Walk<kSums> wk, Range rg,
                         uint8_t* sm, uint64_t* bars, volatile int* abort_flag) {
  using G = Geo<D>;
  const uint32_t q_bytes = static_cast<uint32_t>(G::kSlabs * p.g * p.tpt * 128);
  uint32_t items = 0, inner = 0;
  bool ok = true;
  auto load = [&](uint8_t* dst, bool query, int h, int token, uint64_t* bar) {
#pragma unroll
    for (int s = 0; s < G::kSlabs; ++s)
      if (query) tc05::tma_load3(dst + s * kSlabBytes, tq, s * 64, h * p.g, token, bar);
      else tc05::tma_load3(dst + s * kSlabBytes, tk, s * 64, h, token, bar);
  };
  for (; ok && wk.b < p.B && wk.off < rg.end; wk.next(p), ++items) {
    const uint32_t ob = items & 1;
    if (items >= 2 && !wait_or_abort(&bars[G::kBarOEmpty + ob], ((items >> 1) - 1) & 1, abort_flag, p.err_word)) break;
    uint8_t* outer = sm + G::kOffOuter + ob * 2 * G::kTileBytes;
    if (kSums) {
      const int j = wk.o * 2 * kTile;
      const bool two = j + kTile < wk.s.nk;
      mbar_arrive_expect_tx(&bars[G::kBarOFull + ob], (two ? 2 : 1) * G::kTileBytes);
      load(outer, false, wk.h, wk.s.k0 + j, &bars[G::kBarOFull + ob]);
      if (two) load(outer + G::kTileBytes, false, wk.h, wk.s.k0 + j + kTile, &bars[G::kBarOFull + ob]);
    } else {
      const int i = wk.o * 2 * p.tpt;
      const bool two = i + p.tpt < wk.s.nq;
      mbar_arrive_expect_tx(&bars[G::kBarOFull + ob], (two ? 2 : 1) * q_bytes);
      load(outer, true, wk.h, wk.s.q0 + i, &bars[G::kBarOFull + ob]);
      if (two) load(outer + G::kTileBytes, true, wk.h, wk.s.q0 + i + p.tpt, &bars[G::kBarOFull + ob]);
    }
    const int lo = static_cast<int>(max(rg.begin - wk.off, int64_t(0)));
    const int hi = static_cast<int>(min(rg.end - wk.off, static_cast<int64_t>(wk.size)));
    for (int x = lo; ok && x < hi; ++x, ++inner) {
      const int t = wk.first + x;
      const uint32_t slot = inner % G::kStages, use = inner / G::kStages;
      ok = use == 0 || wait_or_abort(&bars[G::kBarIEmpty + slot], (use - 1) & 1, abort_flag, p.err_word);
      if (!ok) break;
      uint8_t* dst = sm + G::kOffInner + slot * G::kTileBytes;
      if (kSums) {
        const uint32_t ls = inner % kLStages, lu = inner / kLStages;
        ok = lu == 0 || wait_or_abort(&bars[G::kBarLEmpty + ls], (lu - 1) & 1, abort_flag, p.err_word);
        if (!ok) break;
        mbar_arrive_expect_tx(&bars[G::kBarLFull + ls], kTile * 4);
        bulk_g2s(sm + G::kOffL + ls * kTile * 4, p.nlse + tile_id(p, wk.b, wk.s.q0, t, wk.h) * kTile, kTile * 4,
                 &bars[G::kBarLFull + ls]);
        mbar_arrive_expect_tx(&bars[G::kBarIFull + slot], q_bytes);
        load(dst, true, wk.h, wk.s.q0 + t * p.tpt, &bars[G::kBarIFull + slot]);
      } else {
        mbar_arrive_expect_tx(&bars[G::kBarIFull + slot], G::kTileBytes);
        load(dst, false, wk.h, wk.s.k0 + t * kTile, &bars[G::kBarIFull + slot]);
      }
    }
  }
  if (*abort_flag) {
    // Every copy already issued lands before the CTA can exit.
    for (uint32_t b = 0; b < 2; ++b)
      if (items > b) mbar_wait(&bars[G::kBarOFull + b], ((items - b + 1) / 2 - 1) & 1);
    for (uint32_t s = 0; s < G::kStages; ++s)
      if (inner > s) mbar_wait(&bars[G::kBarIFull + s], ((inner - s + G::kStages - 1) / G::kStages - 1) & 1);
    for (uint32_t s = 0; kSums && s < kLStages; ++s)
      if (inner > s) mbar_wait(&bars[G::kBarLFull + s], ((inner - s + kLStages - 1) / kLStages - 1) & 1);
  }
}

// Whether the item's tile w has a visible score in inner tile t (the MMA lane and the
// warpgroups decide alike).
template <bool kSums>
__device__ __forceinline__ bool wanted(const Params& p, const Walk<kSums>& wk, int w, int t) {
  const int off = wk.s.nk - wk.s.nq;
  if (kSums) {
    const int j = (wk.o * 2 + w) * kTile;  // its first key
    return j < wk.s.nk && j <= min((t + 1) * p.tpt, wk.s.nq) - 1 + off;
  }
  const int i = (wk.o * 2 + w) * p.tpt;    // its first token
  return i < wk.s.nq && t * kTile <= min(i + p.tpt, wk.s.nq) - 1 + off;
}

template <int D, bool kBf16, bool kSums>
__device__ void mma_lane(const Params& p, Walk<kSums> wk, Range rg, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                         volatile int* abort_flag) {
  using G = Geo<D>;
  constexpr uint32_t id = tc05::idesc_f16(kTile, kTile, kBf16, false, false);
  const uint64_t dO = tc05::sw128_desc(smem_u32(sm + G::kOffOuter), 16, 1024);
  const uint64_t dI = tc05::sw128_desc(smem_u32(sm + G::kOffInner), 16, 1024);
  uint32_t items = 0, inner = 0, cnt[2] = {0, 0};
  bool ok = true;
  for (; ok && wk.b < p.B && wk.off < rg.end; wk.next(p), ++items) {
    const uint32_t ob = items & 1;
    ok = wait_or_abort(&bars[G::kBarOFull + ob], (items >> 1) & 1, abort_flag, p.err_word);
    const int lo = static_cast<int>(max(rg.begin - wk.off, int64_t(0)));
    const int hi = static_cast<int>(min(rg.end - wk.off, static_cast<int64_t>(wk.size)));
    for (int x = lo; ok && x < hi; ++x, ++inner) {
      const uint32_t slot = inner % G::kStages;
      ok = wait_or_abort(&bars[G::kBarIFull + slot], (inner / G::kStages) & 1, abort_flag, p.err_word);
      if (!ok) break;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!ok || !wanted<kSums>(p, wk, w, wk.first + x)) continue;
        const uint32_t buf = cnt[w] & 1, use = cnt[w] >> 1;
        ok = use == 0 || wait_or_abort(&bars[G::kBarSEmpty + 2 * w + buf], (use - 1) & 1, abort_flag, p.err_word);
        if (!ok) continue;
        tc05::fence_after_sync();
        const uint64_t a0 = dO + (((ob * 2 + w) * G::kTileBytes) >> 4), b0 = dI + ((slot * G::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk / 4) * kSlabBytes + (kk % 4) * 32) >> 4;
          tc05::mma_ss(tmem + (2 * w + buf) * kTile, a0 + o, b0 + o, id, kk > 0 ? 1u : 0u);
        }
        tc05::commit(&bars[G::kBarSFull + 2 * w + buf]);
        ++cnt[w];
      }
      tc05::commit(&bars[G::kBarIEmpty + slot]);
    }
    tc05::commit(&bars[G::kBarOEmpty + ob]);
  }
  // Every MMA this lane issued completes before the tensor memory is released.
  tc05::commit(&bars[G::kBarDone]);
  mbar_wait(&bars[G::kBarDone], 0);
}

__device__ __forceinline__ void lds_f2x2(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}

// 32 scores of a key's row: 2^(c s - L) of the columns from lo to hi - 1, added to s2.
template <bool kMask>
__device__ __forceinline__ void add_columns(const uint32_t (&r)[32], uint64_t c2, uint32_t nl, int lo, int hi,
                                            uint64_t (&s2)[2]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint64_t l[2];
    lds_f2x2(nl + i * 16, l[0], l[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int x = 4 * i + 2 * e;
      float a, b;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(r[x]), __uint_as_float(r[x + 1])), c2, l[e]), a, b);
      a = ex2(a);
      b = ex2(b);
      if (kMask) {
        if (x < lo || x >= hi) a = 0.f;
        if (x + 1 < lo || x + 1 >= hi) b = 0.f;
      }
      s2[e] = f2_add(s2[e], f2_pack(a, b));
    }
  }
}

template <int D, bool kSums>
__device__ void rows(const Params& p, Walk<kSums> wk, Range rg, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                     volatile int* abort_flag) {
  using G = Geo<D>;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int w = (warp - 4) >> 2;
  const int row = ((warp & 3) << 5) | lane;
  const uint32_t tS0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 2 * w * kTile;
  const uint32_t nl0 = smem_u32(sm + G::kOffL);
  const float c = p.c_log2;
  const uint64_t c2 = f2_pack(c, c);
  const int rt = row / p.g;  // token of its tile that a query row belongs to
  uint32_t inner = 0, cnt = 0;
  if (w == 0 && row == 0) p.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  for (; wk.b < p.B && wk.off < rg.end; wk.next(p)) {
    const int lo = static_cast<int>(max(rg.begin - wk.off, int64_t(0)));
    const int hi = static_cast<int>(min(rg.end - wk.off, static_cast<int64_t>(wk.size)));
    const int off = wk.s.nk - wk.s.nq;
    float m = SA_NEG_INF, total = 0.f;  // a query row's offset; the sum
    for (int x = lo; x < hi; ++x, ++inner) {
      const int t = wk.first + x;
      const uint32_t ls = inner % kLStages;
      // (for a tile that is not wanted too: its slot is passed on once, in its turn)
      if (kSums && !wait_or_abort_warp(&bars[G::kBarLFull + ls], (inner / kLStages) & 1, abort_flag, p.err_word)) return;
      if (wanted<kSums>(p, wk, w, t)) {
        const uint32_t buf = cnt & 1, tS = tS0 + buf * kTile;
        if (!wait_or_abort_warp(&bars[G::kBarSFull + 2 * w + buf], (cnt >> 1) & 1, abort_flag, p.err_word)) return;
        ++cnt;
        tc05::fence_after_sync();
        uint32_t r[2][32];
        tc05::tmem_ld32(tS, r[0]);
        uint64_t s2[2] = {0, 0};
        if (kSums) {
          // visible columns: queries that see this key, of this sequence
          const int tok = t * p.tpt;
          const int end = min(p.tpt, wk.s.nq - tok) * p.g;
          const int key = (wk.o * 2 + w) * kTile + row;
          const int from = max(key - off - tok, 0) * p.g;
          // (rows that no query fills hold zeros, and -inf for -L)
          const bool plain = tok + p.tpt <= wk.s.nq && __all_sync(0xffffffffu, from == 0);
          const uint32_t nl = nl0 + ls * kTile * 4;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tc05::tmem_ld_wait();
            if (q < 3) tc05::tmem_ld32(tS + 32 * (q + 1), r[(q + 1) & 1]);
            if (plain) add_columns<false>(r[q & 1], c2, nl + q * 128, 0, 0, s2);
            else if (32 * q < end) add_columns<true>(r[q & 1], c2, nl + q * 128, from - 32 * q, end - 32 * q, s2);
          }
        } else {
          const int tok = (wk.o * 2 + w) * p.tpt + rt;
          const bool live = rt < p.tpt && tok < wk.s.nq;
          // the last visible column (rows that hold no query do not mask)
          const int last = live ? min(wk.s.nk - 1, tok + off) - t * kTile : kTile;
          const bool plain = __all_sync(0xffffffffu, last >= kTile - 1);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t(&v)[32] = r[q & 1];
            tc05::tmem_ld_wait();
            if (q < 3) tc05::tmem_ld32(tS + 32 * (q + 1), r[(q + 1) & 1]);
            float mx[2] = {SA_NEG_INF, SA_NEG_INF};
            if (!plain) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * q + i > last) v[i] = __float_as_uint(SA_NEG_INF);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              mx[i & 1] = max3(mx[i & 1], __uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            const float top = fmaxf(mx[0], mx[1]) * c;
            const bool up = live && (top > m + kRaiseLog2 || (m == SA_NEG_INF && top > m));
            if (__any_sync(0xffffffffu, up)) {
              if (up) {
                const float f = ex2(m - top);
                const uint64_t f2 = f2_pack(f, f);
                total *= f;
                s2[0] = f2_mul(s2[0], f2);
                s2[1] = f2_mul(s2[1], f2);
                m = top;
              }
            }
            // a row of nothing but NaN scores keeps the offset -inf, and 0 in its place
            const float n = m == SA_NEG_INF ? 0.f : -m;
            const uint64_t n2 = f2_pack(n, n);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float a, b;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), c2, n2), a, b);
              s2[i & 1] = f2_add(s2[i & 1], f2_pack(ex2(a), ex2(b)));
            }
          }
        }
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[G::kBarSEmpty + 2 * w + buf]);
        float a, b;
        f2_unpack(f2_add(s2[0], s2[1]), a, b);
        total += a + b;
      }
      if (kSums) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[G::kBarLEmpty + ls]);
      }
    }
    if (!kSums && m == SA_NEG_INF && total != total) m = 0.f;  // NaN scores alone
    if (lo == 0 && hi == wk.size) {
      if constexpr (kSums) put_key(p, wk, w, row, total);
      else put_row(p, wk, w, row, m, total);
    } else {
      p.part[(static_cast<int64_t>(blockIdx.x) * 2 + (lo > 0 ? 0 : 1)) * 256 + w * kTile + row] = make_float2(total, m);
      // begun here and ended by another CTA: for merge_kernel
      if (lo == 0 && w == 0 && row == 0)
        p.cut[blockIdx.x] = make_int4(wk.b, wk.h, wk.o, static_cast<int>((wk.off + wk.size - 1) / (rg.end - rg.begin)));
    }
  }
}

// ---- kernels --------------------------------------------------------------------------------

template <int D, typename T, bool kSums>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ Params p) {
  using G = Geo<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + G::kOffBar);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + G::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + G::kOffMisc) + 1;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[G::kBarOFull + i], 1);
      mbar_init(&bars[G::kBarOEmpty + i], 1);
    }
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&bars[G::kBarIFull + s], 1);
      mbar_init(&bars[G::kBarIEmpty + s], 1);
    }
    for (int s = 0; s < kLStages; ++s) {
      mbar_init(&bars[G::kBarLFull + s], 1);
      mbar_init(&bars[G::kBarLEmpty + s], 8);  // both warpgroups
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars[G::kBarSFull + i], 1);
      mbar_init(&bars[G::kBarSEmpty + i], 4);
    }
    mbar_init(&bars[G::kBarDone], 1);
    *abort_flag = 0;
    fence_mbar_init();
    tc05::prefetch_tmap(&tq);
    tc05::prefetch_tmap(&tk);
  }
  if (warp == 1) {
    tc05::tmem_alloc(tslot, 512);
    tc05::tmem_relinquish();
  }
  tc05::fence_before_sync();

  // ---- the sequences' pairs, and this CTA's range (the ring is scratch until then)
  int64_t* pref = reinterpret_cast<int64_t*>(sm + G::kOffInner);
  bool bad = false;
  for (int b = tid; b < p.B; b += kThreads) {
    const Items<kSums> it(p, seq_of(p, b));
    pref[b + 1] = p.Hkv * it.before(it.count);
    bad = bad || bad_span(p.q_start, b, p.Tq) || bad_span(p.k_start, b, p.Tk);
  }
  if (bad && blockIdx.x == 0 && p.err_word) atomicOr(p.err_word, static_cast<uint32_t>(SA_ERRBIT_SEQ));
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    int64_t carry = 0;
    if (lane == 0) pref[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int64_t v = b0 + lane < p.B ? pref[b0 + lane + 1] : 0;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, sh);
        if (lane >= sh) v += x;
      }
      if (b0 + lane < p.B) pref[b0 + lane + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  const int64_t pairs = bad ? 0 : pref[p.B];
  const int64_t R = (pairs + gridDim.x - 1) / gridDim.x;
  Range rg{static_cast<int64_t>(blockIdx.x) * R, 0};
  rg.end = min(rg.begin + R, pairs);
  Walk<kSums> wk{};
  wk.b = p.B;
  if (rg.begin < rg.end) {  // (every warp alike)
    // the last of n ascending places, the first of them 0, that is not past x
    auto find = [&](int n, int64_t x, auto&& place) {
      int lo = 0, hi = n;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const int k = __popc(__ballot_sync(0xffffffffu, at < hi && place(at) <= x));
        lo += (k - 1) * step;
        hi = min(lo + step, hi);
      }
      return lo;
    };
    wk.b = find(p.B, rg.begin, [&](int b) { return pref[b]; });
    wk.s = seq_of(p, wk.b);
    const Items<kSums> it(p, wk.s);
    const int64_t head = (pref[wk.b + 1] - pref[wk.b]) / p.Hkv;
    int64_t rest = rg.begin - pref[wk.b];
    wk.h = static_cast<int>(rest / head);
    rest -= wk.h * head;
    wk.o = find(it.count, rest, [&](int o) { return it.before(o); });
    wk.off = pref[wk.b] + wk.h * head + it.before(wk.o);
    wk.fill(p);
  }
  if (kSums && p.g * p.tpt < kTile) {
    // rows of a query tile that no head fills: nothing is loaded there, and nothing that
    // is not finite may lie there
    __syncthreads();  // the prefix has been read
    constexpr int kWords = G::kTileBytes / 16;
    for (int i = tid; i < G::kStages * kWords; i += kThreads)
      reinterpret_cast<uint4*>(sm + G::kOffInner)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();  // the scratch becomes a target of TMA
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = *tslot;
  if (kSums) pdl_wait();  // the rows' statistics
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) producer<D, kSums>(&tq, &tk, p, wk, rg, sm, bars, abort_flag);
  } else if (warp == 1) {
    if (lane == 0) mma_lane<D, kBf16, kSums>(p, wk, rg, sm, bars, tmem, abort_flag);
  } else if (warp >= 4) {
    rows<D, kSums>(p, wk, rg, sm, bars, tmem, abort_flag);
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc05::fence_after_sync();
    tc05::tmem_dealloc(tmem, 512);
  }
}

// Items cut between CTAs: a block for each CTA, which does something where an item
// begins in the CTA's range and goes on in the next.
template <bool kSums>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int4 c = p.cut[blockIdx.x];
  if (c.x < 0) return;
  Walk<kSums> wk{};
  wk.b = c.x;
  wk.h = c.y;
  wk.o = c.z;
  wk.s = seq_of(p, c.x);
  const int x = static_cast<int>(threadIdx.x);
  auto part = [&](int cta) { return __ldg(p.part + (static_cast<int64_t>(cta) * 2 + (cta == static_cast<int>(blockIdx.x) ? 1 : 0)) * 256 + x); };
  if constexpr (kSums) {
    float sum = 0.f;
    for (int i = blockIdx.x; i <= c.w; ++i) sum += part(i).x;
    put_key(p, wk, x / kTile, x % kTile, sum);
  } else {
    float m = SA_NEG_INF, l = 0.f;
    for (int i = blockIdx.x; i <= c.w; ++i) {
      const float2 e = part(i);
      if (e.y == SA_NEG_INF) continue;
      const float up = fmaxf(m, e.y);
      l = l * ex2(m - up) + e.x * ex2(e.y - up);
      m = up;
    }
    put_row(p, wk, x / kTile, x % kTile, m, l);
  }
}

// ---- host side -----------------------------------------------------------------------------

// [tokens, heads, D] sixteen-bit rows with the given strides, boxes of 64 columns x
// `heads` heads x `tokens` tokens in the 128-byte swizzle; tokens past the end read as
// zero.
bool rows_map(CUtensorMap* m, const void* base, int dtype, int64_t D, int64_t H, int64_t T,
              const int64_t (&st)[2], int heads, int tokens) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(T)};
  // an axis of one element may have any stride; the map wants a multiple of 16 bytes
  const int64_t hs = H > 1 ? st[1] * 2 : D * 2, ts = T > 1 ? st[0] * 2 : D * H * 2;
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hs), static_cast<cuuint64_t>(ts)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, dtype == SA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

template <typename... Args>
int launch_after(void (*kernel)(Args...), int grid, int block, size_t smem, cudaStream_t st, bool dependent,
                 const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? 0 : -1;
}

template <int D, typename T>
int launch_t(const WeightsArgs& a, cudaStream_t st) {
  using G = Geo<D>;
  const int64_t g = a.Hq / a.Hkv, tpt = kTile / g;
  CUtensorMap tq, tk;
  if (!rows_map(&tq, a.q, a.dtype, D, a.Hq, a.Tq, a.qs, static_cast<int>(g), static_cast<int>(tpt)) ||
      !rows_map(&tk, a.k, a.dtype, D, a.Hkv, a.Tk, a.ks, 1, kTile))
    return -1;
  const int sms = sm_count();
  Params p;
  memset(&p, 0, sizeof(p));
  char* ws = static_cast<char*>(a.workspace);
  p.part = reinterpret_cast<float2*>(ws);
  ws += up256(static_cast<size_t>(sms) * 2 * 256 * sizeof(float2));
  p.cut = reinterpret_cast<int4*>(ws);
  ws += up256(static_cast<size_t>(sms) * sizeof(int4));
  p.nlse = reinterpret_cast<float*>(ws);
  p.weights = a.weights;
  p.err_word = a.err_word;
  p.Tq = static_cast<int>(a.Tq);
  p.Tk = static_cast<int>(a.Tk);
  p.Hkv = static_cast<int>(a.Hkv);
  p.g = static_cast<int>(g);
  p.tpt = static_cast<int>(tpt);
  p.accumulate = a.accumulate;
  p.page_tokens = a.page_tokens;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.c_log2 = a.scale * 1.4426950408889634f;
  auto stats = weights_kernel<D, T, false>;
  auto sums = weights_kernel<D, T, true>;
  if (!allow_smem(reinterpret_cast<const void*>(stats)) || !allow_smem(reinterpret_cast<const void*>(sums))) return -1;
  for (int64_t b0 = 0; b0 < a.B; b0 += kMaxSeqs) {
    p.q_start = a.q_start + b0;
    p.k_start = a.k_start + b0;
    p.block_table = a.block_table + b0 * a.max_pages;
    p.B = static_cast<int>(a.B - b0 < kMaxSeqs ? a.B - b0 : kMaxSeqs);
    p.b0 = static_cast<int>(b0);
    if (launch_after(stats, sms, kThreads, G::kBytes, st, false, tq, tk, p) != 0 ||
        launch_after(merge_kernel<false>, sms, 256, 0, st, true, p) != 0 ||
        launch_after(sums, sms, kThreads, G::kBytes, st, true, tq, tk, p) != 0 ||
        launch_after(merge_kernel<true>, sms, 256, 0, st, true, p) != 0)
      return -1;
  }
  return 0;
}

}  // namespace

bool weights_tc_supported(const WeightsArgs& a) {
  if (a.dtype != SA_BF16 && a.dtype != SA_F16) return false;
  if (a.D != 64 && a.D != 128) return false;
  return a.scale > 0.0f && a.Hq / a.Hkv <= kTile && a.Hkv < 65536 && a.Tq > 0 && a.Tk > 0 && encode_tiled() != nullptr;
}

size_t weights_tc_workspace(const WeightsArgs& a) {
  const size_t sms = static_cast<size_t>(sm_count());
  const int64_t tpt = kTile / (a.Hq / a.Hkv);
  return up256(sms * 2 * 256 * sizeof(float2)) + up256(sms * sizeof(int4)) +
         static_cast<size_t>(a.Tq / tpt + a.B + 1) * static_cast<size_t>(a.Hkv) * kTile * sizeof(float);
}

int launch_weights_tc(const WeightsArgs& a, cudaStream_t st) {
  if (a.dtype == SA_BF16)
    return a.D == 128 ? launch_t<128, __nv_bfloat16>(a, st) : launch_t<64, __nv_bfloat16>(a, st);
  return a.D == 128 ? launch_t<128, __half>(a, st) : launch_t<64, __half>(a, st);
}

}  // namespace sa
