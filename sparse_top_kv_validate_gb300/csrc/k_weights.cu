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
// second operand, no probabilities to be passed on.  8 prompts of 299 to 3,338 tokens, 16,384
// in all, 32 / 8 heads of 128: 348 us, 55% of the bf16 peak for both products (of 2,048
// tokens each, 267 us in f16, 54%); an inner tile takes 1,450 to
// 1,750 cycles, of which its MMAs take 1,090 and its exponentials (one per visible pair,
// query head and form) 1,024: bound by what the lanes that issue the MMAs do besides.
// Groups that leave rows of a query tile unfilled mask their columns in every tile: 5 heads to
// the group, 361 us (masked at a sequence's end alone, 349).
// The last 32 queries of 8 contexts, 112,700 keys: 111 us, 43 for the statistics (K at 80% of
// the copy bandwidth) and 65 for the sums, whose items have one inner tile each.
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
// Warps: 0 loads (outer tiles through two buffers, inner ones through a ring), 1 and 3
// issue the MMAs of one outer tile each, 2 works out the items, 4-11 and 12-19 take the
// scores of one outer tile each, from two buffers of tensor memory, a warpgroup half of
// the columns: a thread reads 64 scores at once, gives the buffer back and then works on
// them, four warps to a scheduler (the prompts with two, and whole rows to a thread: 432 us).
// A row's two halves meet in the item's own outer tile, which its MMAs have read.  Every
// mbarrier wait is bounded; a stalled pipeline sets SA_ERRBIT_TIMEOUT, stops every role,
// and still frees the tensor memory.
#include <cuda.h>

#include <cstring>
#include <type_traits>

#include "packed.cuh"
#include "pool_add.cuh"
#include "tc05.cuh"
#include "weights.h"

namespace sa {

namespace {

constexpr int kThreads = 640;           // 4 service warps, 4 warpgroups
constexpr int kTile = 128;               // rows of a tile
constexpr int kSlabBytes = kTile * 128;  // 128 rows x 64 sixteen-bit columns
constexpr int kMaxSeqs = 1024;           // sequences per launch
constexpr int kItemCost = 1;             // (the prompts: 0 385 us, 1 and 2 349, 5 360)
constexpr int kItems = 3;                // items worked out ahead
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
                       kBarSFull = kBarLEmpty + kLStages, kBarSEmpty = kBarSFull + 4,  // [outer tile][buffer]
                       kBarXFull = kBarSEmpty + 4, kBarXEmpty = kBarXFull + 2, kBarWFull = kBarXEmpty + 2,
                       kBarWEmpty = kBarWFull + kItems, kBarDone = kBarWEmpty + kItems, kNumBars = kBarDone + 2;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tensor memory, abort flag
  static constexpr int kOffItems = (kOffMisc + 8 + 15) / 16 * 16;
  static constexpr int kBytes = 1024 + kOffItems + kItems * 64;
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
  int* bad;           // nullable [CTAs]: whether any start of the call, beyond this launch's too, is malformed
  int B, Tq, Tk, Hkv, g;
  int tpt;            // tokens per query tile: 128 / g
  int b0;             // sequences before these
  int accumulate;
  int64_t page_tokens, max_pages, num_pages;
  int shift;          // log2(page_tokens), or -1
  float c_log2;       // scale * log2(e)
};

// ---- items and their places ------------------------------------------------------------

// sum_{i < n} floor((a i + b) / m) by Euclid's algorithm on (a, m): the quotients leave the sum,
// and the points under the line that is left are counted along the other axis (Graham, Knuth,
// Patashnik, Concrete Mathematics, 3.5).  (Tokens stay below 2^30, so that a n + b, with a
// and b reduced, fits 32 bits.)
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
  // Places of the items before o: their pairs, and kItemCost for each that has any.
  __device__ int64_t before(int o) const {
    if (o == 0) return 0;
    if (kSums) {  // size(x) = all query tiles less floor(max(0, x span - off) / tpt)
      const int x0 = off > 0 ? (off + span - 1) / span : 0;
      int64_t s = static_cast<int64_t>(o) * ((nq + tpt - 1) / tpt + kItemCost);
      if (o > x0) s -= floor_sum(o - x0, tpt, span, x0 * span - off);
      return s;
    }
    // all but the last item: max(0, floor((x span + c) / 128)) with c = span - 1 + off + 128
    const int n = min(o, count - 1), c = span - 1 + off + kTile;
    const int x0 = c < kTile ? (kTile - c + span - 1) / span : 0;  // the first that has any
    int64_t s = n > x0 ? floor_sum(n - x0, kTile, span, x0 * span + c) + static_cast<int64_t>(n - x0) * kItemCost : 0;
    if (o == count) s += size(count - 1) + kItemCost;
    return s;
  }
};

// Where the walk over this CTA's items stands.
template <bool kSums>
struct Walk {
  int b, h, o;
  int64_t off;   // the item's first place; its pairs begin kItemCost further
  int size, first;
  Seq s;

  __device__ __forceinline__ void fill(const Params& p) {
    const Items<kSums> it(p, s);
    size = it.size(o);
    first = it.first(o);
  }
  // The next item with a pair (there is one, unless b reaches p.B).
  __device__ __forceinline__ void next(const Params& p) {
    off += size + kItemCost;
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

// An item as the roles take it: inner tiles [t0, t1), and those that its tile w has a visible
// score in, [from[w], to[w]).
struct __align__(16) Item {
  int b, h, o;               // sequence (-1: no more items), KV head, item
  int q0, nq, k0, nk;
  int t0, t1, from[2], to[2];
  int cut;                   // 0: whole; 1: begun by another CTA; 2: begun here, ended by another
  int id;                    // the sequence's first query tile among the rows' statistics
  int spare;
};
static_assert(sizeof(Item) == 64, "");

// A query tile's place among the rows' statistics: of Hkv (Tq / tpt + B + 1), each tile's own.
__device__ __forceinline__ int64_t tile_id(const Params& p, const Item& it, int tile) {
  return (it.id + tile) * static_cast<int64_t>(p.Hkv) + it.h;
}

template <bool kSums>
__device__ __forceinline__ Item item_of(const Params& p, const Walk<kSums>& wk, int64_t begin, int64_t end) {
  Item it;
  it.b = wk.b;
  it.h = wk.h;
  it.o = wk.o;
  it.q0 = wk.s.q0;
  it.nq = wk.s.nq;
  it.k0 = wk.s.k0;
  it.nk = wk.s.nk;
  const int64_t first = wk.off + kItemCost, size = wk.size;
  const int lo = static_cast<int>(min(max(begin - first, int64_t(0)), size));
  const int hi = static_cast<int>(min(max(end - first, int64_t(0)), size));
  it.t0 = wk.first + lo;
  it.t1 = wk.first + hi;
  it.cut = lo > 0 ? 1 : hi < wk.size ? 2 : 0;
  it.id = wk.s.q0 / p.tpt + p.b0 + wk.b;
  it.spare = 0;
  const int off = it.nk - it.nq;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (kSums) {
      const int j = (it.o * 2 + w) * kTile, i = j - off;  // its first key; the first token that sees it
      it.from[w] = max(it.t0, i > 0 ? i / p.tpt : 0);
      it.to[w] = j < it.nk ? it.t1 : it.t0;
    } else {
      const int i = (it.o * 2 + w) * p.tpt;               // its first token; the last key that its last sees
      const int last = min(i + p.tpt, it.nq) - 1 + off;
      it.from[w] = it.t0;
      it.to[w] = i < it.nq && last >= 0 ? min(it.t1, last / kTile + 1) : it.t0;
    }
  }
  return it;
}

// ---- what a row ends with ------------------------------------------------------------------

// kSums 0: -L of query row `row` of the item's tile w, from the row's offset and sum.
// -inf, so that its keys get nothing, for a row that sees nothing but -inf and for one
// that holds no query.
__device__ __forceinline__ void put_row(const Params& p, const Item& it, int w, int row, float m, float l) {
  const int tile = 2 * it.o + w, rt = row / p.g;
  if (tile * p.tpt >= it.nq) return;
  const bool live = rt < p.tpt && tile * p.tpt + rt < it.nq;
  p.nlse[tile_id(p, it, tile) * kTile + row] = !live || m == SA_NEG_INF ? SA_NEG_INF : -(m + log2f(l));
}

__device__ __forceinline__ uint32_t page_index(const Params& p, int j) {
  return p.shift >= 0 ? static_cast<uint32_t>(j) >> p.shift : static_cast<uint32_t>(j) / static_cast<uint32_t>(p.page_tokens);
}

// kSums 1: the weight of the item's key `row` of tile w.
__device__ __forceinline__ void put_key(const Params& p, const Item& it, int w, int row, float sum) {
  const int j = it.o * 2 * kTile + w * kTile + row;
  if (j >= it.nk) return;
  const uint32_t pi = page_index(p, j);
  int32_t page = -1;
  if (pi < p.max_pages) page = __ldg(p.block_table + it.b * p.max_pages + pi);
  if (page < 0 || page >= p.num_pages) {
    if (p.err_word) atomicOr(p.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
    return;
  }
  const int64_t slot = j - static_cast<int64_t>(pi) * p.page_tokens;
  pool_put(p.weights + (page * static_cast<int64_t>(p.Hkv) + it.h) * p.page_tokens + slot, sum,
           p.accumulate && j < it.nk - it.nq);
}

// ---- roles -----------------------------------------------------------------------------------

// This CTA's range of places.
struct Range {
  int64_t begin, end;
};

// Works the items out ahead of the other roles (a walk's divisions between two items would
// hold up the lanes that issue the copies and the MMAs).
template <int D, bool kSums>
__device__ void walker(const Params& p, Walk<kSums> wk, Range rg, uint8_t* sm, uint64_t* bars, volatile int* abort_flag) {
  using G = Geo<D>;
  int4 cut = make_int4(-1, 0, 0, 0);  // the item that this range begins and does not end, for merge_kernel
  for (uint32_t n = 0;;) {
    const bool more = wk.b < p.B && wk.off < rg.end;
    Item it;
    if (more) it = item_of(p, wk, rg.begin, rg.end);
    else it.b = -1;
    if (more && it.t0 == it.t1) {  // (of this item the range has what its change costs, no pair)
      wk.next(p);
      continue;
    }
    if (more && it.cut == 2)
      cut = make_int4(it.b, it.h, it.o, static_cast<int>((wk.off + kItemCost + wk.size - 1) / (rg.end - rg.begin)));
    const uint32_t slot = n % kItems, use = n / kItems;
    if (use > 0 && !wait_or_abort(&bars[G::kBarWEmpty + slot], (use - 1) & 1, abort_flag, p.err_word)) break;
    *reinterpret_cast<Item*>(sm + G::kOffItems + slot * 64) = it;
    mbar_arrive(&bars[G::kBarWFull + slot]);
    if (!more) break;
    wk.next(p);
    ++n;
  }
  p.cut[blockIdx.x] = cut;
}

template <int D, bool kSums>
__device__ void producer(const CUtensorMap* tq, const CUtensorMap* tk, const Params& p, uint8_t* sm, uint64_t* bars,
                         volatile int* abort_flag) {
  using G = Geo<D>;
  const uint32_t q_bytes = static_cast<uint32_t>(G::kSlabs * p.g * p.tpt * 128);
  uint32_t items = 0, inner = 0, slot = 0, use = 0, ls = 0, lu = 0;
  auto load = [&](uint8_t* dst, bool query, int h, int token, uint64_t* bar) {
#pragma unroll
    for (int s = 0; s < G::kSlabs; ++s)
      if (query) tc05::tma_load3(dst + s * kSlabBytes, tq, s * 64, h * p.g, token, bar);
      else tc05::tma_load3(dst + s * kSlabBytes, tk, s * 64, h, token, bar);
  };
  bool ok = true;
  for (uint32_t n = 0; ok; ++n) {
    if (!wait_or_abort(&bars[G::kBarWFull + n % kItems], (n / kItems) & 1, abort_flag, p.err_word)) break;
    const Item it = *reinterpret_cast<const Item*>(sm + G::kOffItems + (n % kItems) * 64);
    mbar_arrive(&bars[G::kBarWEmpty + n % kItems]);
    if (it.b < 0) break;
    const uint32_t ob = items & 1;
    if (items >= 2 && !wait_or_abort(&bars[G::kBarOEmpty + ob], ((items >> 1) - 1) & 1, abort_flag, p.err_word)) break;
    uint8_t* outer = sm + G::kOffOuter + ob * 2 * G::kTileBytes;
    const int first = kSums ? it.o * 2 * kTile : it.o * 2 * p.tpt, next = kSums ? kTile : p.tpt;
    const bool two = first + next < (kSums ? it.nk : it.nq);
    const int row0 = (kSums ? it.k0 : it.q0) + first;
    mbar_arrive_expect_tx(&bars[G::kBarOFull + ob], (two ? 2 : 1) * (kSums ? G::kTileBytes : q_bytes));
    load(outer, !kSums, it.h, row0, &bars[G::kBarOFull + ob]);
    if (two) load(outer + G::kTileBytes, !kSums, it.h, row0 + next, &bars[G::kBarOFull + ob]);
    ++items;
    const float* nlse = p.nlse + tile_id(p, it, it.t0) * kTile;
    int token = kSums ? it.q0 + it.t0 * p.tpt : it.k0 + it.t0 * kTile;
    for (int t = it.t0; t < it.t1; ++t) {
      ok = use == 0 || wait_or_abort(&bars[G::kBarIEmpty + slot], (use - 1) & 1, abort_flag, p.err_word);
      if (ok && kSums) ok = lu == 0 || wait_or_abort(&bars[G::kBarLEmpty + ls], (lu - 1) & 1, abort_flag, p.err_word);
      if (!ok) break;
      mbar_arrive_expect_tx(&bars[G::kBarIFull + slot], kSums ? q_bytes : G::kTileBytes);
      load(sm + G::kOffInner + slot * G::kTileBytes, kSums, it.h, token, &bars[G::kBarIFull + slot]);
      if (kSums) {
        mbar_arrive_expect_tx(&bars[G::kBarLFull + ls], kTile * 4);
        bulk_g2s(sm + G::kOffL + ls * kTile * 4, nlse, kTile * 4, &bars[G::kBarLFull + ls]);
        nlse += static_cast<int64_t>(p.Hkv) * kTile;
        if (++ls == kLStages) ls = 0, ++lu;
      }
      token += kSums ? p.tpt : kTile;
      ++inner;
      if (++slot == G::kStages) slot = 0, ++use;
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

// The MMAs of outer tile w.  (A lane each: with one for both, its own instructions, 1,950
// cycles of them for the 1,090 that the MMAs of an inner tile take, were the bound.)
template <int D, bool kBf16>
__device__ void mma_lane(const Params& p, int w, uint8_t* sm, uint64_t* bars, uint32_t tmem, volatile int* abort_flag) {
  using G = Geo<D>;
  constexpr uint32_t id = tc05::idesc_f16(kTile, kTile, kBf16, false, false);
  const uint64_t dO = tc05::sw128_desc(smem_u32(sm + G::kOffOuter), 16, 1024);
  const uint64_t dI = tc05::sw128_desc(smem_u32(sm + G::kOffInner), 16, 1024);
  const uint32_t tS = tmem + 2 * w * kTile;
  uint32_t items = 0, slot = 0, parity = 0, cnt = 0;
  bool ok = true;
  for (uint32_t n = 0; ok; ++n, ++items) {
    if (!wait_or_abort(&bars[G::kBarWFull + n % kItems], (n / kItems) & 1, abort_flag, p.err_word)) break;
    const Item& it = *reinterpret_cast<const Item*>(sm + G::kOffItems + (n % kItems) * 64);
    const int b = it.b, first = it.t0, end = it.t1, from = it.from[w], to = it.to[w];
    mbar_arrive(&bars[G::kBarWEmpty + n % kItems]);
    if (b < 0) break;
    const uint32_t ob = items & 1;
    ok = wait_or_abort(&bars[G::kBarOFull + ob], (items >> 1) & 1, abort_flag, p.err_word);
    const uint64_t a0 = dO + (((ob * 2 + w) * G::kTileBytes) >> 4);
    for (int t = first; ok && t < end; ++t) {
      ok = wait_or_abort(&bars[G::kBarIFull + slot], parity, abort_flag, p.err_word);
      if (!ok) break;
      if (t >= from && t < to) {
        const uint64_t b0 = dI + ((slot * G::kTileBytes) >> 4);
        const uint32_t buf = cnt & 1, use = cnt >> 1;
        ok = use == 0 || wait_or_abort(&bars[G::kBarSEmpty + 2 * w + buf], (use - 1) & 1, abort_flag, p.err_word);
        if (!ok) break;
        tc05::fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk / 4) * kSlabBytes + (kk % 4) * 32) >> 4;
          tc05::mma_ss(tS + buf * kTile, a0 + o, b0 + o, id, kk > 0 ? 1u : 0u);
        }
        tc05::commit(&bars[G::kBarSFull + 2 * w + buf]);
        tc05::commit(&bars[G::kBarIEmpty + slot]);
        ++cnt;
      } else {
        mbar_arrive(&bars[G::kBarIEmpty + slot]);
      }
      if (++slot == G::kStages) slot = 0, parity ^= 1;
    }
    tc05::commit(&bars[G::kBarOEmpty + ob]);
  }
  // Every MMA this lane issued completes before the tensor memory is released.
  tc05::commit(&bars[G::kBarDone + w]);
  mbar_wait(&bars[G::kBarDone + w], 0);
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
__device__ void rows(const Params& p, uint8_t* sm, uint64_t* bars, uint32_t tmem, volatile int* abort_flag) {
  using G = Geo<D>;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int w = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;
  const int row = ((warp & 3) << 5) | lane, col0 = half * 64;
  const uint32_t tS0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 2 * w * kTile + col0;
  const uint32_t nl0 = smem_u32(sm + G::kOffL) + col0 * 4;
  const float c = p.c_log2;
  const uint64_t c2 = f2_pack(c, c);
  const int rt = row / p.g;  // token of its tile that a query row belongs to
  uint32_t cnt = 0, ls = 0, lp = 0;
  for (uint32_t items = 0;; ++items) {
    const uint32_t ws = items % kItems;
    if (!wait_or_abort_warp(&bars[G::kBarWFull + ws], (items / kItems) & 1, abort_flag, p.err_word)) return;
    const Item& it = *reinterpret_cast<const Item*>(sm + G::kOffItems + ws * 64);  // (ours until the item's end)
    if (it.b < 0) return;
    const int nq = it.nq, nk = it.nk, off = nk - nq, t1 = it.t1, from_t = it.from[w], to_t = it.to[w];
    const int tile = 2 * it.o + w;
    float m = SA_NEG_INF, total = 0.f;  // a query row's offset; the sum
    for (int t = it.t0; t < t1; ++t) {
      // (for a tile that is not wanted too: its slot is passed on once, in its turn)
      if (kSums && !wait_or_abort_warp(&bars[G::kBarLFull + ls], lp, abort_flag, p.err_word)) return;
      if (t >= from_t && t < to_t) {
        const uint32_t buf = cnt & 1, tS = tS0 + buf * kTile;
        if (!wait_or_abort_warp(&bars[G::kBarSFull + 2 * w + buf], (cnt >> 1) & 1, abort_flag, p.err_word)) return;
        ++cnt;
        tc05::fence_after_sync();
        uint32_t r[2][32];
        float mx[2];
        if (kSums) {
          tc05::tmem_ld32(tS, r[0]);
          tc05::tmem_ld32(tS + 32, r[1]);
        } else {
          tc05::tmem_ld32_max<false>(tS, r[0], mx[0]);
          tc05::tmem_ld32_max<false>(tS + 32, r[1], mx[1]);
        }
        tc05::tmem_ld_wait();
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[G::kBarSEmpty + 2 * w + buf]);
        uint64_t s2[2] = {0, 0};
        if (kSums) {
          // visible columns: queries that see this key, of this sequence
          const int tok = t * p.tpt;
          const int end = min(p.tpt, nq - tok) * p.g - col0;
          const int key = tile * kTile + row;
          const int from = max(key - off - tok, 0) * p.g - col0;
          // (the columns that no head of the group fills, where 128 is no multiple of it, lie behind
          // `end` in every tile: what their rows hold is anything's)
          const bool all = __all_sync(0xffffffffu, from <= 0);
          const uint32_t nl = nl0 + ls * kTile * 4;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (all && 32 * q + 32 <= end) add_columns<false>(r[q], c2, nl + q * 128, 0, 0, s2);
            else if (32 * q < end) add_columns<true>(r[q], c2, nl + q * 128, from - 32 * q, end - 32 * q, s2);
          }
        } else {
          const int tok = tile * p.tpt + rt;
          const bool live = rt < p.tpt && tok < nq;
          // the last visible column (rows that hold no query do not mask)
          const int last = live ? min(nk - 1, tok + off) - t * kTile - col0 : kTile;
          float top;
          if (__all_sync(0xffffffffu, last >= 63)) {
            top = fmaxf(tc05::arrived(mx[0]), tc05::arrived(mx[1])) * c;
          } else {
            top = SA_NEG_INF;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if (32 * q + i > last) r[q][i] = __float_as_uint(SA_NEG_INF);
                top = fmaxf(top, __uint_as_float(r[q][i]));
              }
            top *= c;
          }
          const bool up = live && (top > m + kRaiseLog2 || (m == SA_NEG_INF && top > m));
          if (up) {
            total *= ex2(m - top);
            m = top;
          }
          // a row of nothing but NaN scores keeps the offset -inf, and 0 in its place
          const float n = m == SA_NEG_INF ? 0.f : -m;
          const uint64_t n2 = f2_pack(n, n);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float a, b;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(r[q][2 * i]), __uint_as_float(r[q][2 * i + 1])), c2, n2), a, b);
              s2[i & 1] = f2_add(s2[i & 1], f2_pack(ex2(a), ex2(b)));
            }
        }
        float a, b;
        f2_unpack(f2_add(s2[0], s2[1]), a, b);
        total += a + b;
      }
      if (kSums) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[G::kBarLEmpty + ls]);
        if (++ls == kLStages) ls = 0, lp ^= 1;
      }
    }
    if (!kSums && m == SA_NEG_INF && total != total) m = 0.f;  // NaN scores alone

    // the two halves, in the item's outer tile: its copy has landed and its MMAs have read it
    const uint32_t ob = items & 1;
    float2* meet = reinterpret_cast<float2*>(sm + G::kOffOuter + (ob * 2 + w) * G::kTileBytes) + row;
    if (half == 1) {
      if (!wait_or_abort_warp(&bars[G::kBarOFull + ob], (items >> 1) & 1, abort_flag, p.err_word)) return;
      if (items > 0 && !wait_or_abort_warp(&bars[G::kBarXEmpty + w], (items - 1) & 1, abort_flag, p.err_word)) return;
      *meet = make_float2(total, m);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars[G::kBarXFull + w]);
        mbar_arrive(&bars[G::kBarWEmpty + ws]);
      }
      continue;
    }
    if (!wait_or_abort_warp(&bars[G::kBarXFull + w], items & 1, abort_flag, p.err_word)) return;
    const float2 other = *meet;
    fence_proxy_async_smem();  // the tile becomes a target of TMA again
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bars[G::kBarXEmpty + w]);
      mbar_arrive(&bars[G::kBarOEmpty + ob]);
    }
    if (kSums) {
      total += other.x;
    } else {
      const float top = fmaxf(m, other.y);
      total = top == SA_NEG_INF ? total + other.x : total * ex2(m - top) + other.x * ex2(other.y - top);
      m = top;
    }
    if (it.cut == 0) {
      if constexpr (kSums) put_key(p, it, w, row, total);
      else put_row(p, it, w, row, m, total);
    } else {
      p.part[(static_cast<int64_t>(blockIdx.x) * 2 + it.cut - 1) * 256 + w * kTile + row] = make_float2(total, m);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[G::kBarWEmpty + ws]);
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
      mbar_init(&bars[G::kBarOEmpty + i], 10);  // both lanes' MMAs, and the warps that read the halves
      mbar_init(&bars[G::kBarXFull + i], 4);
      mbar_init(&bars[G::kBarXEmpty + i], 4);
    }
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&bars[G::kBarIFull + s], 1);
      mbar_init(&bars[G::kBarIEmpty + s], 2);  // both lanes
    }
    for (int s = 0; s < kLStages; ++s) {
      mbar_init(&bars[G::kBarLFull + s], 1);
      mbar_init(&bars[G::kBarLEmpty + s], 16);  // all warpgroups
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars[G::kBarSFull + i], 1);
      mbar_init(&bars[G::kBarSEmpty + i], 8);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars[G::kBarWFull + i], 1);
      mbar_init(&bars[G::kBarWEmpty + i], 19);  // the producer, the MMA lanes, 16 warps
    }
    mbar_init(&bars[G::kBarDone], 1);
    mbar_init(&bars[G::kBarDone + 1], 1);
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

  // ---- the sequences' places, and this CTA's range (the ring is scratch until then)
  int64_t* pref = reinterpret_cast<int64_t*>(sm + G::kOffInner);
  bool bad = false;
  for (int b = tid; b < p.B; b += kThreads) {
    const Items<kSums> it(p, seq_of(p, b));
    pref[b + 1] = p.Hkv * it.before(it.count);
    bad = bad || bad_span(p.q_start, b, p.Tq) || bad_span(p.k_start, b, p.Tk);
  }
  for (int i = tid; p.bad && i < static_cast<int>(gridDim.x); i += kThreads) bad = bad || p.bad[i] != 0;
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
  const int64_t places = bad ? 0 : pref[p.B];
  const int64_t R = (places + gridDim.x - 1) / gridDim.x;
  Range rg{static_cast<int64_t>(blockIdx.x) * R, 0};
  rg.end = min(rg.begin + R, places);
  Walk<kSums> wk{};
  wk.b = p.B;
  if (warp == 2 && rg.begin < rg.end) {  // (the walker's)
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
  fence_proxy_async_smem();  // the scratch becomes a target of TMA
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = *tslot;
  if (kSums) pdl_wait();  // the rows' statistics
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) producer<D, kSums>(&tq, &tk, p, sm, bars, abort_flag);
  } else if (warp == 1) {
    if (lane == 0) mma_lane<D, kBf16>(p, 0, sm, bars, tmem, abort_flag);
  } else if (warp == 3) {
    if (lane == 0) mma_lane<D, kBf16>(p, 1, sm, bars, tmem, abort_flag);
  } else if (warp == 2) {
    if (lane == 0) walker<D, kSums>(p, wk, rg, sm, bars, abort_flag);
  } else if (warp >= 4) {
    rows<D, kSums>(p, sm, bars, tmem, abort_flag);
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc05::fence_after_sync();
    tc05::tmem_dealloc(tmem, 512);
  }
}

// Calls of more sequences than a launch takes: every start is looked at before any weight
// is written (4 us of 209 for 3,000 sequences).  B: of the whole call.
__global__ void __launch_bounds__(256) starts_kernel(const __grid_constant__ Params p, int B) {
  bool bad = false;
  for (int b = blockIdx.x * 256 + static_cast<int>(threadIdx.x); b < B; b += static_cast<int>(gridDim.x) * 256)
    bad = bad || bad_span(p.q_start, b, p.Tq) || bad_span(p.k_start, b, p.Tk);
  bad = __syncthreads_or(bad);
  if (threadIdx.x != 0) return;
  p.bad[blockIdx.x] = bad;
  if (bad && p.err_word) atomicOr(p.err_word, static_cast<uint32_t>(SA_ERRBIT_SEQ));
}

// Items cut between CTAs: a block for each CTA, which does something where an item
// begins in the CTA's range and goes on in the next.
template <bool kSums>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int4 c = __ldcg(p.cut + blockIdx.x);
  if (c.x < 0) return;
  const Seq q = seq_of(p, c.x);
  Item it;
  it.b = c.x;
  it.h = c.y;
  it.o = c.z;
  it.nq = q.nq;
  it.nk = q.nk;
  it.id = q.q0 / p.tpt + p.b0 + c.x;
  const int x = static_cast<int>(threadIdx.x);
  // (from L2: the read-only path promises nothing for what is written while this kernel is
  // already resident, as it may be while the kernel before it still works)
  auto part = [&](int cta) { return __ldcg(p.part + (static_cast<int64_t>(cta) * 2 + (cta == static_cast<int>(blockIdx.x) ? 1 : 0)) * 256 + x); };
  if constexpr (kSums) {
    float sum = 0.f;
    for (int i = blockIdx.x; i <= c.w; ++i) sum += part(i).x;
    put_key(p, it, x / kTile, x % kTile, sum);
  } else {
    float m = SA_NEG_INF, l = 0.f;
    for (int i = blockIdx.x; i <= c.w; ++i) {
      const float2 e = part(i);
      if (e.y == SA_NEG_INF) continue;
      const float up = fmaxf(m, e.y);
      l = l * ex2(m - up) + e.x * ex2(e.y - up);
      m = up;
    }
    put_row(p, it, x / kTile, x % kTile, m, l);
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
  int* bad = reinterpret_cast<int*>(ws);
  ws += up256(static_cast<size_t>(sms) * sizeof(int));
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
  p.shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_tokens == int64_t(1) << i) p.shift = i;
  auto stats = weights_kernel<D, T, false>;
  auto sums = weights_kernel<D, T, true>;
  if (!allow_smem(reinterpret_cast<const void*>(stats)) || !allow_smem(reinterpret_cast<const void*>(sums))) return -1;
  if (a.B > kMaxSeqs) {
    p.q_start = a.q_start;
    p.k_start = a.k_start;
    p.bad = bad;
    if (launch_after(starts_kernel, sms, 256, 0, st, false, p, static_cast<int>(a.B)) != 0) return -1;
  }
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
  return up256(sms * 2 * 256 * sizeof(float2)) + up256(sms * sizeof(int4)) + up256(sms * sizeof(int)) +
         static_cast<size_t>(a.Tq / tpt + a.B + 1) * static_cast<size_t>(a.Hkv) * kTile * sizeof(float);
}

int launch_weights_tc(const WeightsArgs& a, cudaStream_t st) {
  if (a.dtype == SA_BF16)
    return a.D == 128 ? launch_t<128, __nv_bfloat16>(a, st) : launch_t<64, __nv_bfloat16>(a, st);
  return a.D == 128 ? launch_t<128, __half>(a, st) : launch_t<64, __half>(a, st);
}

}  // namespace sa
