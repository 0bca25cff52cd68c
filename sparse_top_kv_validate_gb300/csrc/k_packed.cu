// k_packed.cu -- packed prefill attention on the fifth-generation tensor cores
// (tcgen05.mma, accumulators in tensor memory, operands staged by TMA).
//
// y_i = sum_j softmax_j(c s_ij) v_j over the keys j <= i + nk - nq (causal) of
// the query's own sequence; sequences of any lengths lie one after the other.
// Bound by the tensor cores for long sequences (4 D flops per visible pair and
// query head), by the softmax's issue slots next to them, and by latency for
// short ones.
//
// GB300 design (one persistent CTA per SM; warps 0-3 service, 4-11 softmax):
//  * A work item is a query tile of 128 rows: 128 / g tokens times the g query
//    heads of one KV head, so that a short sequence fills its tiles and the
//    heads share every K/V tile.
//  * Tensor memory holds three score buffers and O.  Key tile t of the CTA (the
//    count runs on across its items) goes to buffer t % 3 and to softmax
//    warpgroup t % 2, whose threads own a row each.  A tile's way (scores,
//    softmax, PV, buffer free) takes about four times as long as its MMAs: three
//    tiles on the way at once, two of them in softmax, keep the tensor cores
//    about half busy.  Measured, 4 x 4,096 tokens, 32 / 8 heads of 128, causal,
//    bf16: 425 us, 1,295 TFLOP/s (softcap 50: 475 us).  Other orders tried, at
//    463 us for this one: two row tiles per item that share K and V, a score
//    buffer and a warpgroup each, 500 us; the same with two MMA lanes that
//    interleave, so that both tiles' softmax runs at the same time, 625 us; with
//    two warpgroups per row tile, half the columns each, 646 us.
//  * P is passed on in halves: the PV of the first 64 keys runs while the other
//    64 probabilities are still being formed (463 -> 453 us).
//  * A thread reads its 128 scores from tensor memory twice (once where the
//    offset is fixed, below), in a loop over chunks of 32 columns.  Kept in
//    registers they spill, and local memory shares its path with the MMAs'
//    shared-memory operands; unrolled, the roles' loops no longer fit the
//    instruction cache together (both measured: 575 us).  The first pass's
//    maximum comes with the load (tcgen05.ld.red; 453 -> 434 us), one chunk at a
//    time: with two on their way the plain variant spills (520 us).
//  * The two threads of a row agree on its offset tile by tile: a thread posts
//    the offset after its tile (the old one unless the tile's maximum exceeds it
//    by more than 2^8), the other one's next tile starts from it.  The raise
//    rescales O in tensor memory, after the previous PV.  With a softcap that bounds
//    2^logit to the normal numbers of P's type (up to 67 in bf16, 9.7 in f16) the
//    offset is 0 and nothing is posted (softcap 50: bf16 475 us, f16, with an
//    offset, 618).
//  * P enters the second product in q's type, as the MMA takes it: each probability
//    is off by up to half a step of it (2^-8 bf16, 2^-11 f16 of itself; in f16 also
//    by 2^-25 of the row's largest), while the row's sum adds them in fp32.  Against
//    64 bits the outputs are 1.2 to 1.4 times as far off as with fp32 probabilities.
//    (P in two parts would be a second PV per tile.)
//  * Warp 0 loads Q (box: 64 dims x g heads x 128 / g tokens; two buffers) and the
//    K and V tiles through two rings; warp 1's lane issues S = Q K^T and warp 3's
//    O += P V (P over the first half of its scores), so that a barrier wait or a
//    commit of one leaves the other's MMAs running.
//  * Warp 2 passes every V tile on: where keys end inside a tile it zeroes the
//    rows behind them (0 times another sequence's NaN is NaN), and where some of
//    a tile's keys are hidden from some rows it looks for values that are not
//    finite: these are zeroed too, and the rows that do see them add them in the
//    epilogue.
//  * Items go to CTAs in a snake order of falling cost.  The lengths are on
//    the device, so every CTA works out the order itself: the rank of an item
//    among all has a closed form per sequence (an item's number of key tiles
//    grows along its sequence), and a CTA keeps only its own items.
//  * Every mbarrier wait is bounded; a stalled pipeline sets
//    SA_ERRBIT_TIMEOUT, stops every role, and still frees the tensor memory.
#include <cuda.h>

#include <cmath>
#include <cstring>
#include <type_traits>
#include <utility>

#include "packed.cuh"
#include "serving.h"
#include "tc05.cuh"

namespace sa {

namespace {

constexpr int kThreads = 384;            // 4 service warps, 2 softmax warpgroups
constexpr int kSBufs = 3;                // score buffers in tensor memory
constexpr int kLead = 2;                 // K tiles loaded ahead of the V tiles
constexpr int kTile = 128;               // rows of a query tile; keys of a K/V tile
constexpr int kSlabBytes = kTile * 128;  // 128 rows x 64 sixteen-bit columns
constexpr float kRescaleLog2 = 8.0f;     // lazy-maximum slack (factor 256)
// tanh(x) ~= x * sum_k c_k (x^2)^k: the terms and the |x| range of two fits, of an
// absolute error of 1e-7 both
constexpr int kTanhTerms = 5, kTanhShortTerms = 3;
constexpr float kTanhBound = 0.625f, kTanhShortBound = 0.25f;
// softcap * log2(e) up to which 2^logit needs no offset: the logits lie within that on
// either side, and every 2^logit is a normal number of the type that P is held in (the
// row sums, fp32, hold 2^30 of them).  f16 ends at 2^16 and its normal numbers at 2^-14.
template <typename T>
constexpr float fixed_offset_max_log2() {
  return std::is_same<T, __half>::value ? 14.0f : 97.0f;
}
constexpr float kFarMax = 67.0f;         // softcap up to which 2^-20 of it is a small error of a logit
constexpr int kMaxSeqs = 1024;           // sequences per launch
constexpr int kSmemLimit = 227 * 1024;

template <int D>
struct Geo {
  static constexpr int kSlabs = D / 64;
  static constexpr int kTileBytes = kSlabs * kSlabBytes;   // 16 or 32 KB
  static constexpr int kStages = D == 128 ? 2 : 4;         // slots of the K ring, and of the V ring
  static constexpr int kOffQ = 0;                          // two buffers
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffBar = kOffV + kStages * kTileBytes;
  // barriers: per Q buffer q_full, q_empty; per ring slot k_full, k_empty, v_full,
  // v_ready (past warp 2), v_empty; per score buffer s_full, p_full (two halves), pv_done; o_full,
  // o_read; per warpgroup and turn posted (offsets), sums; per MMA lane done.  (A
  // warpgroup may be one post ahead of the other's wait, never two.)
  static constexpr int kBarQFull = 0, kBarQEmpty = 2, kBarKFull = 4, kBarKEmpty = kBarKFull + kStages,
                       kBarVFull = kBarKEmpty + kStages, kBarVReady = kBarVFull + kStages,
                       kBarVEmpty = kBarVReady + kStages, kBarS = kBarVEmpty + kStages,
                       kBarP = kBarS + kSBufs, kBarPv = kBarP + 2 * kSBufs, kBarO = kBarPv + kSBufs,
                       kBarORead = kBarO + 1, kBarPost = kBarORead + 1, kBarSum = kBarPost + 4,
                       kBarDone = kBarSum + 4, kNumBars = kBarDone + 2;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffFlags = kOffTmemSlot + 4;       // abort, hidden values found
  // float [2 warpgroups][2 turns][128] posted offsets; [2 turns][2 warpgroups][2][128] offsets
  // and sums at the end of an item
  static constexpr int kOffXch = (kOffFlags + 8 + 15) / 16 * 16;
  static constexpr int kOffSeq = kOffXch + 12 * kTile * 4;  // int4 [B]; int [B + 1]; uint2 [items]
  static constexpr uint32_t kColS = 0, kColO = kSBufs * kTile;
  static constexpr uint32_t kTmemCols = 512;
};

struct Params {
  void* y;
  int64_t ys0, ys1;        // token and head strides of y (elements)
  const void* v;           // for the rows that add values that are not finite
  int64_t vs0, vs1;
  const int32_t* q_start;
  const int32_t* k_start;
  uint32_t* err_word;
  int B, Tq, Tk, Hkv, g;
  int tpt;                 // tokens per query tile: 128 / g
  int causal;
  int cap_items;           // places in the item list
  float k1;                // x = score * k1 (scale / softcap)
  float c_log2;            // log2-domain multiplier of tanh(x) (softcap * log2e) or of the score (scale * log2e)
  // c_log2 tanh(k1 s) as polynomials in the score s, and the |s| up to which they hold
  float tq[kTanhTerms], tq_bound;
  float ts[kTanhShortTerms], ts_bound;
};

// ---- work items -----------------------------------------------------------------------

// Key tiles that queries up to token `last` of a sequence read (at least one:
// rows that see nothing still have to come out as 0).
__device__ __forceinline__ int last_key(int causal, int nq, int nk, int token) {
  return causal ? min(nk - 1, token + nk - nq) : nk - 1;
}
__device__ __forceinline__ int tiles_of(int causal, int nq, int nk, int last) {
  const int lim = last_key(causal, nq, nk, last);
  return lim < 0 ? 1 : lim / kTile + 1;
}

// Query tiles of a sequence with at least x key tiles.
__device__ __forceinline__ int tiles_with(const Params& p, int nq, int nk, int x) {
  const int tiles = (nq + p.tpt - 1) / p.tpt;
  if (x <= 1) return tiles;
  const int thr = (x - 1) * kTile;      // the tile's last key must reach thr
  if (nk - 1 < thr) return 0;
  if (!p.causal) return tiles;
  const int need = thr - (nk - nq);     // and so its last token
  if (need <= 0) return tiles;
  if (nq - 1 < need) return 0;
  return tiles - need / p.tpt;          // tiles from the one that holds token `need` on
}

struct Item {
  int q0, nq, k0, nk, kvh;
  int tok;      // first token
  int n;        // key tiles
  int seen;     // the last key that every row of the item sees
};

// Snake assignment: round k gives CTA c item k * G + c (even k) or
// k * G + G - 1 - c (odd k).
__device__ __forceinline__ int item_index(int k, int G) {
  const int c = static_cast<int>(blockIdx.x);
  return k * G + ((k & 1) ? G - 1 - c : c);
}

struct Work {
  const int4* seq;      // first query row, queries, first key row, keys
  const uint2* list;    // this CTA's items: sequence << 16 | KV head, query tile
  int n_items, G, cap;

  __device__ __forceinline__ bool get(int k, const Params& p, Item& it) const {
    if (item_index(k, G) >= n_items || k >= cap) return false;
    const uint2 e = list[k];
    const int4 s = seq[e.x >> 16];
    it.q0 = s.x;
    it.nq = s.y;
    it.k0 = s.z;
    it.nk = s.w;
    it.kvh = e.x & 0xffff;
    it.tok = static_cast<int>(e.y) * p.tpt;
    it.n = tiles_of(p.causal, it.nq, it.nk, min(it.tok + p.tpt, it.nq) - 1);
    it.seen = last_key(p.causal, it.nq, it.nk, it.tok);
    return true;
  }
};

// Every CTA: the sequences' extents, the number of items, and this CTA's items
// in the order of falling cost (all threads; ends with a barrier).  `scratch`:
// kOrderBytes, free until then.
//
// Up to kRankSeqs sequences a tile's rank is the sum of a closed form over all
// sequences; with more that sum is the longer way, and the tiles are counted by their
// cost instead: each warp counts its run of tiles, the counts are summed from the
// largest cost on and over the warps, and the warps pass over their runs again, in
// order, as every CTA has to come to the same ranks.  Measured, whole calls, 32 / 8
// heads of 128, sums against counts: 2 prompts of 64 tokens 10.3 and 12.3 us, 32 of 128
// 42.9 and 43.0, 64 of 128 87 and 84, 1,024 of 128 2,124 and 1,134.
constexpr int kRankSeqs = 32;
constexpr int kCosts = 1024;  // (key tiles; larger ones count as that many)
constexpr int kOrderBytes = (kThreads / 32 + 1) * kCosts * 4;
__device__ __forceinline__ Work lay_out_work(const Params& p, uint8_t* area, uint8_t* scratch) {
  int4* seq = reinterpret_cast<int4*>(area);
  int* pref = reinterpret_cast<int*>(seq + p.B);
  uint2* list = reinterpret_cast<uint2*>(pref + ((p.B + 2) & ~1));
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const int step = p.tpt;
  bool bad = false;
  for (int b = tid; b < p.B; b += kThreads) {
    const Span q = span_of(p.q_start, b, p.Tq), k = span_of(p.k_start, b, p.Tk);
    seq[b] = make_int4(q.first, q.n, k.first, k.n);
    bad = bad || bad_span(p.q_start, b, p.Tq) || bad_span(p.k_start, b, p.Tk);
  }
  if (bad && blockIdx.x == 0 && p.err_word) atomicOr(p.err_word, static_cast<uint32_t>(SA_ERRBIT_SEQ));
  // starts in disorder could name more items than the list holds: no work then
  if (__syncthreads_or(bad)) return Work{seq, list, 0, static_cast<int>(gridDim.x), p.cap_items};
  if (tid < 32) {
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int v = b0 + lane < p.B ? (seq[b0 + lane].y + step - 1) / step : 0;
      const int mine = v;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, sh);
        if (lane >= sh) v += x;
      }
      if (b0 + lane < p.B) pref[b0 + lane] = carry + v - mine;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) pref[p.B] = carry;
  }
  __syncthreads();
  const int tiles = pref[p.B];
  const int G = static_cast<int>(gridDim.x);
  Work w{seq, list, tiles * p.Hkv, G, p.cap_items};
  struct Tile {
    int b, qt, n;
  };
  auto tile_at = [&](int i) {
    int lo = 0, hi = p.B;  // the last sequence with pref <= i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pref[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int4 s = seq[lo];
    const int qt = i - pref[lo];
    return Tile{lo, qt, tiles_of(p.causal, s.y, s.w, min((qt + 1) * step, s.y) - 1)};
  };
  auto place = [&](const Tile& t, int rank) {
    for (int h = 0; h < p.Hkv; ++h) {
      const int x = rank * p.Hkv + h, k = x / G, r = x - k * G;
      if (((k & 1) ? G - 1 - r : r) == static_cast<int>(blockIdx.x) && k < p.cap_items)
        list[k] = make_uint2(static_cast<uint32_t>(t.b) << 16 | static_cast<uint32_t>(h), static_cast<uint32_t>(t.qt));
    }
  };
  if (p.B <= kRankSeqs) {
    for (int i = tid; i < tiles; i += kThreads) {
      const Tile t = tile_at(i);
      const int4 s = seq[t.b];
      // items with more key tiles, then those with as many of earlier sequences
      // and of this one
      int rank = t.qt - (pref[t.b + 1] - pref[t.b] - tiles_with(p, s.y, s.w, t.n));
      for (int o = 0; o < p.B; ++o) {
        const int4 u = seq[o];
        rank += o < t.b ? tiles_with(p, u.y, u.w, t.n) : tiles_with(p, u.y, u.w, t.n + 1);
      }
      place(t, rank);
    }
  } else {
    constexpr int kW = kThreads / 32;
    int* count = reinterpret_cast<int*>(scratch);  // [kW][kCosts], largest cost first
    int* total = count + kW * kCosts;              // [kCosts]
    int* own = count + (tid >> 5) * kCosts;
    auto slot_of = [](const Tile& t) { return kCosts - min(t.n, kCosts); };
    for (int x = tid; x < kW * kCosts; x += kThreads) count[x] = 0;
    __syncthreads();
    const int run = (tiles + kW - 1) / kW, from = min((tid >> 5) * run, tiles), to = min(from + run, tiles);
    for (int i = from + lane; i < to; i += 32) atomicAdd(own + slot_of(tile_at(i)), 1);
    __syncthreads();
    for (int c = tid; c < kCosts; c += kThreads) {
      int sum = 0;
#pragma unroll
      for (int v = 0; v < kW; ++v) sum += count[v * kCosts + c];
      total[c] = sum;
    }
    __syncthreads();
    if (tid < 32) {
      int carry = 0;
      for (int c0 = 0; c0 < kCosts; c0 += 32) {
        const int mine = total[c0 + lane];
        int v = mine;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, v, sh);
          if (lane >= sh) v += x;
        }
        total[c0 + lane] = carry + v - mine;
        carry += __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
    for (int c = tid; c < kCosts; c += kThreads) {
      int at = total[c];
      for (int v = 0; v < kW; ++v) {
        const int n = count[v * kCosts + c];
        count[v * kCosts + c] = at;
        at += n;
      }
    }
    __syncthreads();
    for (int i0 = from; i0 < to; i0 += 32) {
      const bool live = i0 + lane < to;
      const Tile t = tile_at(live ? i0 + lane : from);
      const int c = live ? slot_of(t) : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, c);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int rank = live ? own[c] + before : 0;
      __syncwarp();
      if (live && before == 0) own[c] += __popc(same);
      __syncwarp();
      if (live) place(t, rank);
    }
    fence_proxy_async_smem();  // the scratch becomes a target of TMA
  }
  __syncthreads();
  return w;
}

// ---- role: TMA producer (one lane) ------------------------------------------------------

template <int D>
__device__ void producer(const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv,
                         const Params& p, const Work& work, uint8_t* sm, uint64_t* bars,
                         volatile int* abort_flag) {
  using G = Geo<D>;
  tc05::prefetch_tmap(tq);
  tc05::prefetch_tmap(tk);
  tc05::prefetch_tmap(tv);
  const uint32_t q_bytes = static_cast<uint32_t>(G::kSlabs * p.g * p.tpt * 128);
  uint32_t k_cnt = 0, v_cnt = 0, q_cnt = 0;
  Item it;
  auto load_tile = [&](const CUtensorMap* map, int off, int full, int empty, uint32_t& cnt, int t) {
    const uint32_t slot = cnt % G::kStages, use = cnt / G::kStages;
    if (use > 0 && !wait_or_abort(&bars[empty + slot], (use - 1) & 1, abort_flag, p.err_word)) return false;
    mbar_arrive_expect_tx(&bars[full + slot], G::kTileBytes);
#pragma unroll
    for (int s = 0; s < G::kSlabs; ++s)
      tc05::tma_load3(sm + off + slot * G::kTileBytes + s * kSlabBytes, map, s * 64, it.kvh, it.k0 + t * kTile,
                      &bars[full + slot]);
    ++cnt;
    return true;
  };
  bool ok = true;
  for (int k = 0; ok && work.get(k, p, it); ++k) {
    // the buffer is free once the item before the last has stored its rows through it
    const uint32_t qb = q_cnt & 1;
    if (q_cnt >= 2 && !wait_or_abort(&bars[G::kBarQEmpty + qb], ((q_cnt >> 1) - 1) & 1, abort_flag, p.err_word)) break;
    mbar_arrive_expect_tx(&bars[G::kBarQFull + qb], q_bytes);
#pragma unroll
    for (int s = 0; s < G::kSlabs; ++s)
      tc05::tma_load3(sm + G::kOffQ + qb * G::kTileBytes + s * kSlabBytes, tq, s * 64, it.kvh * p.g, it.q0 + it.tok,
                      &bars[G::kBarQFull + qb]);
    ++q_cnt;
    for (int j = -kLead; ok && j < it.n; ++j) {  // K_0, K_1, then K_(j + 2), V_j
      if (j + kLead < it.n) ok = load_tile(tk, G::kOffK, G::kBarKFull, G::kBarKEmpty, k_cnt, j + kLead);
      if (ok && j >= 0) ok = load_tile(tv, G::kOffV, G::kBarVFull, G::kBarVEmpty, v_cnt, j);
    }
  }
  if (*abort_flag) {
    // Let every copy already issued land before the CTA can exit.
    for (uint32_t b = 0; b < 2; ++b)
      if (q_cnt > b) mbar_wait(&bars[G::kBarQFull + b], ((q_cnt - b + 1) / 2 - 1) & 1);
    for (uint32_t s = 0; s < G::kStages; ++s) {
      if (k_cnt > s) mbar_wait(&bars[G::kBarKFull + s], ((k_cnt - s + G::kStages - 1) / G::kStages - 1) & 1);
      if (v_cnt > s) mbar_wait(&bars[G::kBarVFull + s], ((v_cnt - s + G::kStages - 1) / G::kStages - 1) & 1);
    }
  }
}

// ---- role: V gate (one warp) --------------------------------------------------------------

// Largest magnitude of two 16-bit pairs, NaN kept.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x, __half) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<__half2*>(&m), __habs2(*reinterpret_cast<__half2*>(&x)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x, __nv_bfloat16) {
  const __nv_bfloat162 r =
      __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&m), __habs2(*reinterpret_cast<__nv_bfloat162*>(&x)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ bool odd16(uint32_t bits) {  // infinity or NaN
  const uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  return (bits & e) == e;
}

template <int D, typename T>
__device__ void v_gate(const Params& p, const Work& work, uint8_t* sm, uint64_t* bars,
                       volatile int* abort_flag, volatile int* found) {
  using G = Geo<D>;
  const int lane = static_cast<int>(threadIdx.x & 31);
  uint32_t cnt = 0;
  Item it;
  for (int k = 0; work.get(k, p, it); ++k) {
    for (int j = 0; j < it.n; ++j, ++cnt) {
      const uint32_t slot = cnt % G::kStages;
      if (!wait_or_abort_warp(&bars[G::kBarVFull + slot], (cnt / G::kStages) & 1, abort_flag, p.err_word))
        return;
      const int first = j * kTile;
      if (first + kTile - 1 > it.seen) {  // (rows behind the last key are past `seen` too)
        uint8_t* tile = sm + G::kOffV + slot * G::kTileBytes;
        const int end = min(max(it.nk - first, 0), kTile);      // rows behind: nobody's keys
        for (int e = lane; e < (kTile - end) * 8 * G::kSlabs; e += 32) {
          const int r = end + e / (8 * G::kSlabs), c = e % (8 * G::kSlabs);
          *reinterpret_cast<uint4*>(tile + (c >> 3) * kSlabBytes + r * 128 + (c & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        const int begin = min(max(it.seen + 1 - first, 0), end);  // hidden from some rows: begin .. end - 1
        const int chunks = (end - begin) * 8 * G::kSlabs;
        uint32_t m = 0;
#pragma unroll 4
        for (int e = lane; e < chunks; e += 32) {
          const int r = begin + e / (8 * G::kSlabs), c = e % (8 * G::kSlabs);
          const uint4 x = *reinterpret_cast<const uint4*>(tile + (c >> 3) * kSlabBytes + r * 128 + (c & 7) * 16);
          m = max_abs2(m, x.x, T());
          m = max_abs2(m, x.y, T());
          m = max_abs2(m, x.z, T());
          m = max_abs2(m, x.w, T());
        }
        if (__any_sync(0xffffffffu, odd16<T>(m) || odd16<T>(m >> 16))) {
          if (lane == 0) *found = 1;
          for (int e = lane; e < chunks * 8; e += 32) {  // one 16-bit value each
            const int r = begin + e / (64 * G::kSlabs), c = e % (64 * G::kSlabs);
            uint16_t* x = reinterpret_cast<uint16_t*>(tile + (c >> 6) * kSlabBytes + r * 128) + (c & 63);
            if (odd16<T>(*x)) *x = 0;
          }
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[G::kBarVReady + slot]);
    }
  }
}

// ---- role: MMA issuers (one lane each) ----------------------------------------------------------

// S(t) = Q . K^T into score buffer t % 3, once the buffer's previous P has been
// read by its PV.
template <int D, bool kBf16>
__device__ void score_lane(const Params& p, const Work& work, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                           volatile int* abort_flag) {
  using G = Geo<D>;
  constexpr uint32_t id_s = tc05::idesc_f16(kTile, kTile, kBf16, false, false);
  const uint64_t dQ = tc05::sw128_desc(smem_u32(sm + G::kOffQ), 16, 1024);
  const uint64_t dK = tc05::sw128_desc(smem_u32(sm + G::kOffK), 16, 1024);
  uint32_t t = 0, q_cnt = 0, buf = 0, buf_use = 0;
  Item it;
  bool ok = true;
  for (int k = 0; ok && work.get(k, p, it); ++k, ++q_cnt) {
    ok = wait_or_abort(&bars[G::kBarQFull + (q_cnt & 1)], (q_cnt >> 1) & 1, abort_flag, p.err_word);
    for (int j = 0; ok && j < it.n; ++j, ++t) {
      const uint32_t slot = t % G::kStages;
      ok = (buf_use == 0 || wait_or_abort(&bars[G::kBarPv + buf], (buf_use - 1) & 1, abort_flag, p.err_word)) &&
           wait_or_abort(&bars[G::kBarKFull + slot], (t / G::kStages) & 1, abort_flag, p.err_word);
      if (!ok) break;
      tc05::fence_after_sync();
      const uint64_t a0 = dQ + (((q_cnt & 1) * G::kTileBytes) >> 4), b0 = dK + ((slot * G::kTileBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * kSlabBytes + (kk % 4) * 32) >> 4;
        tc05::mma_ss(tmem + G::kColS + buf * kTile, a0 + off, b0 + off, id_s, kk > 0 ? 1u : 0u);
      }
      tc05::commit(&bars[G::kBarS + buf]);
      tc05::commit(&bars[G::kBarKEmpty + slot]);
      if (++buf == kSBufs) {
        buf = 0;
        ++buf_use;
      }
    }
  }
  // Every MMA this lane issued completes before the tensor memory is released.
  tc05::commit(&bars[G::kBarDone]);
  mbar_wait(&bars[G::kBarDone], 0);
}

// O (+)= P(t) . V; the first PV of an item waits until the previous O has been read.
template <int D, bool kBf16>
__device__ void value_lane(const Params& p, const Work& work, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                           volatile int* abort_flag) {
  using G = Geo<D>;
  constexpr uint32_t id_o = tc05::idesc_f16(kTile, D, kBf16, false, true);
  const uint64_t dV = tc05::sw128_desc(smem_u32(sm + G::kOffV), kSlabBytes, 1024);
  uint32_t t = 0, buf = 0, buf_use = 0;
  Item it;
  bool ok = true;
  for (int k = 0; ok && work.get(k, p, it); ++k) {
    if (k > 0) ok = wait_or_abort(&bars[G::kBarORead], (k - 1) & 1, abort_flag, p.err_word);
    for (int j = 0; ok && j < it.n; ++j, ++t) {
      const uint32_t slot = t % G::kStages;
      ok = wait_or_abort(&bars[G::kBarVReady + slot], (t / G::kStages) & 1, abort_flag, p.err_word) &&
           wait_or_abort(&bars[G::kBarP + 2 * buf], buf_use & 1, abort_flag, p.err_word);
      if (!ok) break;
      tc05::fence_after_sync();
      const uint64_t v0 = dV + ((slot * G::kTileBytes) >> 4);
      const uint32_t tP = tmem + G::kColS + buf * kTile;
#pragma unroll
      for (int kk = 0; kk < kTile / 32; ++kk)
        tc05::mma_ts(tmem + G::kColO, tP + kk * 8, v0 + ((kk * 2048) >> 4), id_o, (j > 0 || kk > 0) ? 1u : 0u);
      ok = wait_or_abort(&bars[G::kBarP + 2 * buf + 1], buf_use & 1, abort_flag, p.err_word);
      if (!ok) break;
      tc05::fence_after_sync();
#pragma unroll
      for (int kk = kTile / 32; kk < kTile / 16; ++kk)
        tc05::mma_ts(tmem + G::kColO, tP + kk * 8, v0 + ((kk * 2048) >> 4), id_o, 1u);
      tc05::commit(&bars[G::kBarPv + buf]);
      tc05::commit(&bars[G::kBarVEmpty + slot]);
      if (j == it.n - 1) tc05::commit(&bars[G::kBarO]);
      if (++buf == kSBufs) {
        buf = 0;
        ++buf_use;
      }
    }
  }
  tc05::commit(&bars[G::kBarDone + 1]);
  mbar_wait(&bars[G::kBarDone + 1], 0);
}

// ---- role: softmax (tile t belongs to warpgroup t % 2, a row to a thread) -----------------------

// kCols columns of this thread's O row *= alpha, in tensor memory (warp-collective).
template <int kCols>
__device__ __forceinline__ void rescale_o(uint32_t tO, float alpha) {
  const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll
  for (int c = 0; c < kCols / 16; ++c) {
    uint32_t o[16];
    tc05::tmem_ld16(tO + c * 16, o);
    tc05::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), a2), lo, hi);
      o[2 * i] = __float_as_uint(lo);
      o[2 * i + 1] = __float_as_uint(hi);
    }
    tc05::tmem_st16(tO + c * 16, o);
  }
  tc05::tmem_st_wait();
}

// How the log2-domain logit of a score s is formed: c_log2 s (no softcap), or
// c_log2 tanh(k1 s) by the fitted polynomials (kShort, kPoly) or, where a score of the
// warp lies outside their ranges or is hidden, from the hardware exponential and
// reciprocal (kFar: off by 2^-20 of the softcap).  Above a softcap of 67 that is too
// much: there each score in the first polynomial's range takes that one (kEach; for
// every softcap 257 -> 273 us at 256 prompts of 128 tokens).
enum ScoreMode { kPlain = 0, kShort = 1, kPoly = 2, kFar = 3, kEach = 4 };

// The constants of that: c2 = c_log2, k1 and the polynomials.
struct Logits {
  float c2, k1;
  float tq[kTanhTerms], ts[kTanhShortTerms];
  float ts_bound;
};

__device__ __forceinline__ float tanh_far(float x) {
  // 1 - 2 / (e^2x + 1), absolute error below 2^-20; saturates cleanly
  return 1.0f - 2.0f * rcp(ex2(x * (2.0f * kLog2e)) + 1.0f);
}

template <int N>
__device__ __forceinline__ float poly_logit(float x, const float (&tq)[N]) {
  const float y = x * x;
  float q = tq[N - 1];
#pragma unroll
  for (int k = N - 2; k >= 0; --k) q = fmaf(q, y, tq[k]);
  return x * q;
}
template <int N>
__device__ __forceinline__ uint64_t poly_logit2(uint64_t x, const float (&tq)[N], uint64_t add) {
  const uint64_t y = f2_mul(x, x);
  uint64_t q = f2_pack(tq[N - 1], tq[N - 1]);
#pragma unroll
  for (int k = N - 2; k >= 0; --k) q = f2_fma(q, y, f2_pack(tq[k], tq[k]));
  return f2_fma(x, q, add);
}

// 32 columns of a thread's row and the largest of them (kAbs: of their magnitudes),
// found by the load itself.  Valid after tmem_ld_wait, m through arrived().
template <bool kAbs>
__device__ __forceinline__ void tmem_ld32_max(uint32_t addr, uint32_t (&r)[32], float& m) {
#define SA_LD32_MAX(op)                                                                         \
  asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x32." op                                      \
               ".f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20," \
               "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"                       \
               : SA_TC05_R32(r), "=f"(m)                                                         \
               : "r"(addr))
  if (kAbs) SA_LD32_MAX("max.abs");
  else SA_LD32_MAX("max");
#undef SA_LD32_MAX
}
__device__ __forceinline__ float arrived(float& m) {
  asm volatile("" : "+f"(m));
  return m;
}

// The largest magnitude of 32 scores.
__device__ __forceinline__ float largest(const uint32_t (&r)[32]) {
  float ax[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    ax[i & 1] = max3(ax[i & 1], fabsf(__uint_as_float(r[2 * i])), fabsf(__uint_as_float(r[2 * i + 1])));
  return fmaxf(ax[0], ax[1]);
}

// Maximum of the chunk; kMask: its columns above rel become -inf first.
template <bool kMask>
__device__ __forceinline__ float max_chunk(uint32_t (&r)[32], int rel, float m) {
  float mx[2] = {m, SA_NEG_INF};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (kMask) {
      if (2 * i > rel) r[2 * i] = __float_as_uint(SA_NEG_INF);
      if (2 * i + 1 > rel) r[2 * i + 1] = __float_as_uint(SA_NEG_INF);
    }
    mx[i & 1] = max3(mx[i & 1], __uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
  }
  return fmaxf(mx[0], mx[1]);
}

// p = 2^(logit - m) of 32 columns, masked ones 0, as 16 packed pairs; added to
// the two partial sums.
template <int kMode, bool kMask, typename T>
__device__ __forceinline__ void exp_chunk(const uint32_t (&r)[32], uint32_t (&pk)[16], const Logits& lg, float neg_m,
                                          int rel, uint64_t (&ls)[2]) {
  const uint64_t c2x2 = f2_pack(lg.c2, lg.c2), nm2 = f2_pack(neg_m, neg_m);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float x0 = __uint_as_float(r[2 * i]), x1 = __uint_as_float(r[2 * i + 1]);
    uint64_t v;
    if (kMode == kPlain) v = f2_fma(f2_pack(x0, x1), c2x2, nm2);
    else if (kMode == kFar || kMode == kEach) v = f2_fma(f2_pack(tanh_far(x0 * lg.k1), tanh_far(x1 * lg.k1)), c2x2, nm2);
    else if (kMode == kPoly) v = poly_logit2(f2_pack(x0, x1), lg.tq, nm2);
    else v = poly_logit2(f2_pack(x0, x1), lg.ts, nm2);
    float a, b;
    f2_unpack(v, a, b);
    if (kMode == kEach) {
      float n0, n1;
      f2_unpack(poly_logit2(f2_pack(x0, x1), lg.ts, nm2), n0, n1);
      if (fabsf(x0) <= lg.ts_bound) a = n0;
      if (fabsf(x1) <= lg.ts_bound) b = n1;
    }
    if (kMask) {
      if (2 * i > rel) a = SA_NEG_INF;
      if (2 * i + 1 > rel) b = SA_NEG_INF;
    }
    a = ex2(a);
    b = ex2(b);
    ls[i & 1] = f2_add(ls[i & 1], f2_pack(a, b));
    pk[i] = pack2<T>(a, b);
  }
}

// Without a softcap; with one and offsets; offset 0; a softcap above kFarMax, with offsets.
enum Variant { kVarPlain = 0, kVarCapMax = 1, kVarCapFixed = 2, kVarCapLarge = 3 };

// What a thread keeps of an item until its epilogue: the item, and the offset and
// sum of the row over the warpgroup's own tiles.
struct Finished {
  int k;
  uint32_t last;  // the item's last tile
  float m, l;
};

template <int D, typename T, int kVariant>
__device__ void softmax_rows(const Params& p, const Work& work, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                             volatile int* abort_flag, volatile int* found) {
  using G = Geo<D>;
  constexpr bool kCap = kVariant != kVarPlain, kFixed = kVariant == kVarCapFixed;
  constexpr int kAnyScore = kVariant == kVarCapLarge ? kEach : kFar;  // the form that holds for all
  constexpr int kOCols = D / 2;  // O columns that this warpgroup stores
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int wg = (warp - 4) >> 2;
  const int row = ((warp & 3) << 5) | lane;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t tS0 = tmem + lanes + G::kColS, tO = tmem + lanes + G::kColO;
  volatile float* xch = reinterpret_cast<volatile float*>(sm + G::kOffXch) + row;
  const int rt = row / p.g;  // token of the tile that this row belongs to
  const int inv_g = (65536 + p.g - 1) / p.g;
  Logits lg;
  lg.c2 = p.c_log2;
  lg.k1 = p.k1;
  lg.ts_bound = p.ts_bound;
#pragma unroll
  for (int i = 0; i < kTanhTerms; ++i) lg.tq[i] = p.tq[i];
#pragma unroll
  for (int i = 0; i < kTanhShortTerms; ++i) lg.ts[i] = p.ts[i];
  // The other warpgroup's post after its tile u (every one is waited for, in order).
  auto posted = [&](uint32_t u) {
    return wait_or_abort_warp(&bars[G::kBarPost + 2 * (wg ^ 1) + ((u >> 1) & 1)], (u >> 2) & 1, abort_flag, p.err_word);
  };

  int k = 0;             // current item
  uint32_t t = 0;        // tiles before it
  Item it;
  bool more = work.get(k, p, it);
  int j = wg;            // this warpgroup's next tile of it
  float m = SA_NEG_INF;  // this row's offset after the tiles so far
  uint64_t ls[2] = {0, 0};
  Finished done{0, 0, 0.f, 0.f};
  bool pending = false;  // an item whose epilogue waits until after the next tile
  while (more || pending) {
    if (more && j < it.n) {
      const uint32_t u = t + j, buf = u % kSBufs;
      const uint32_t tS = tS0 + buf * kTile;
      if (!wait_or_abort_warp(&bars[G::kBarS + buf], (u / kSBufs) & 1, abort_flag, p.err_word)) return;
      tc05::fence_after_sync();
      uint32_t r[2][32];
      float mr[2];
      tmem_ld32_max<kFixed>(tS + (kFixed ? 0 : 96), r[0], mr[0]);  // (the first pass goes backwards)
      const int tok = it.tok + rt;
      // A row of no query is no reason to mask: nothing of it is kept, and it has no say in what
      // the warp does.  (As a row that sees nothing it sent every tile of a sequence's last item
      // the longer way: chunks after 24,000 tokens 175 us, softcap 50 206, now 155 and 175.)
      const bool live = rt < p.tpt && tok < it.nq;
      const int lim = live ? last_key(p.causal, it.nq, it.nk, tok) : 0x7fffffff;  // last visible key
      const int rel = lim - j * kTile;  // columns above rel are masked
      const bool masked = __any_sync(0xffffffffu, rel < kTile - 1);
      if (!kFixed && j > 0) {
        // the offset after the previous tile, the other warpgroup's
        if (!posted(u - 1)) return;
        const float o = xch[(2 * (wg ^ 1) + (((u - 1) >> 1) & 1)) * kTile];
        if (__any_sync(0xffffffffu, o != m)) {
          const float f = m == o ? 1.0f : ex2(m - o);  // (0 from no offset at all)
          ls[0] = f2_mul(ls[0], f2_pack(f, f));
          ls[1] = f2_mul(ls[1], f2_pack(f, f));
          m = o;
        }
      }
      auto mode_of = [&](float most) {  // the cheapest form that holds for the warp's scores
        most = live ? most : 0.f;
        return !__any_sync(0xffffffffu, !(most <= p.ts_bound))   ? kShort
               : !__any_sync(0xffffffffu, !(most <= p.tq_bound)) ? kPoly
                                                                 : kFar;
      };
      // Whether chunk c holds scores that some row of the warp does not see.  They may be anything
      // and must not choose the form of the others, so such a chunk takes the one that holds for
      // all, and no form at all where no row sees any of it.  (bf16, softcap 50, 4 x 4,096 tokens
      // and 256 x 128: 475 and 257 us; the form chosen by the scores that are seen, the others
      // cleared, 525 and 276: the loops outgrow the instruction cache; kFar for every chunk of a
      // tile with hidden scores 450 and 292.)
      auto partial = [&](int c) { return masked && __any_sync(0xffffffffu, rel - 32 * c < 31); };
      int mode = kPlain;
      float mx = SA_NEG_INF;
      if (!kCap && !masked) {  // the loads find the maximum
        tc05::tmem_ld_wait();
        mx = arrived(mr[0]);
#pragma unroll 1
        for (int c = 2; c >= 0; --c) {
          tmem_ld32_max<false>(tS + 32 * c, r[0], mr[0]);
          tc05::tmem_ld_wait();
          mx = fmaxf(mx, arrived(mr[0]));
        }
      } else if (!kFixed) {
        float ax = 0.f;
        auto look = [&](uint32_t (&x)[32], int c) {
          if (kCap && !partial(c)) ax = fmaxf(ax, largest(x));
          mx = masked ? max_chunk<true>(x, rel - 32 * c, mx) : max_chunk<false>(x, 0, mx);
        };
        tc05::tmem_ld_wait();
#pragma unroll 1
        for (int c = 3;; --c) {
          look(r[0], c);
          if (c == 0) break;
          tc05::tmem_ld32(tS + 32 * (c - 1), r[0]);
          tc05::tmem_ld_wait();
        }
        if (kCap) mode = mode_of(ax);
      }
      if (!kFixed) {
        float mt = SA_NEG_INF;
        if (live && mx != SA_NEG_INF)
          mt = !kCap                       ? mx * lg.c2
               : fabsf(mx) <= lg.ts_bound  ? poly_logit(mx, lg.ts)
                                           : tanh_far(mx * lg.k1) * lg.c2;
        const bool up = mt > m + kRescaleLog2 || (m == SA_NEG_INF && mt > m);
        xch[(2 * wg + ((u >> 1) & 1)) * kTile] = up ? mt : m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[G::kBarPost + 2 * wg + ((u >> 1) & 1)]);
        if (__any_sync(0xffffffffu, up)) {
          float alpha = 1.0f;
          if (up) {
            alpha = ex2(m - mt);
            m = mt;
            ls[0] = f2_mul(ls[0], f2_pack(alpha, alpha));
            ls[1] = f2_mul(ls[1], f2_pack(alpha, alpha));
          }
          if (j > 0) {
            // O follows once PV(u - 1) has completed.  (S(u - 1) was issued after
            // PV(u - 4) completed, so no other phase of that barrier is outstanding.)
            const uint32_t pb = (u - 1) % kSBufs;
            if (!wait_or_abort_warp(&bars[G::kBarPv + pb], ((u - 1) / kSBufs) & 1, abort_flag, p.err_word)) return;
            tc05::fence_after_sync();
            rescale_o<D>(tO, alpha);
          }
        }
      }
      const float neg_m = (kFixed || m == SA_NEG_INF) ? 0.0f : -m;
      auto load = [](uint32_t at, uint32_t (&x)[32], float& most) {
        if (kFixed) tmem_ld32_max<true>(at, x, most);
        else tc05::tmem_ld32(at, x);
      };
      auto exps = [&](uint32_t (&x)[32], int c, float& most) {
        const int rc = rel - 32 * c;
        uint32_t pk[16];
        const bool part = kCap && partial(c);
        if (kFixed) mode = mode_of(arrived(most));
        if (!kCap && masked) exp_chunk<kPlain, true, T>(x, pk, lg, neg_m, rc, ls);
        else if (!kCap) exp_chunk<kPlain, false, T>(x, pk, lg, neg_m, 0, ls);
        else if (part && !__any_sync(0xffffffffu, live && rc >= 0)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 0u;
        } else if (part || mode == kFar) exp_chunk<kAnyScore, true, T>(x, pk, lg, neg_m, part ? rc : kTile, ls);
        else if (mode == kPoly) exp_chunk<kPoly, false, T>(x, pk, lg, neg_m, 0, ls);
        else exp_chunk<kShort, false, T>(x, pk, lg, neg_m, 0, ls);
        tc05::tmem_st16(tS + c * 16, pk);
      };
#pragma unroll 1
      for (int c = 0; c < 4; c += 2) {
        tc05::tmem_ld_wait();
        load(tS + 32 * (c + 1), r[1], mr[1]);
        exps(r[0], c, mr[0]);
        tc05::tmem_ld_wait();
        if (c == 0) load(tS + 64, r[0], mr[0]);
        exps(r[1], c + 1, mr[1]);
        // half of P is there: its PV need not wait for the other half
        tc05::tmem_st_wait();
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[G::kBarP + 2 * buf + c / 2]);
      }
      j += 2;
    }

    // The end of an item: its last tile is L's; the other warpgroup, which also
    // has the next item's first tile, takes that one before the epilogue, so that
    // the tensor cores find work when O has been read.
    bool epilogue = pending;
    pending = false;
    if (more && j >= it.n && !epilogue) {
      float a, b;
      f2_unpack(f2_add(ls[0], ls[1]), a, b);
      done = Finished{k, t + it.n - 1, m, a + b};
      volatile float* mine = xch + (4 + 4 * (k & 1) + 2 * wg) * kTile;
      mine[0] = m;
      mine[kTile] = a + b;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[G::kBarSum + 2 * wg + (k & 1)]);
      const bool owner = (done.last & 1) == static_cast<uint32_t>(wg);
      t += it.n;
      more = work.get(++k, p, it);
      j = static_cast<int>((t ^ wg) & 1);
      m = SA_NEG_INF;
      ls[0] = ls[1] = 0;
      epilogue = owner || !more;
      pending = !epilogue;
    }
    if (!epilogue) continue;

    // ---- O / l of the rows, half of the columns per warpgroup
    Item e;
    work.get(done.k, p, e);
    const uint32_t turn = done.k & 1;
    const int tok = e.tok + rt;
    const int lim = rt < p.tpt && tok < e.nq ? last_key(p.causal, e.nq, e.nk, tok) : -1;
    if (!wait_or_abort_warp(&bars[G::kBarSum + 2 * (wg ^ 1) + turn], (done.k >> 1) & 1, abort_flag, p.err_word) ||
        (!kFixed && (done.last & 1) != static_cast<uint32_t>(wg) && !posted(done.last)) ||
        !wait_or_abort_warp(&bars[G::kBarO], turn, abort_flag, p.err_word))
      return;
    tc05::fence_after_sync();
    float l = done.l;
    {
      volatile float* others = xch + (4 + 4 * turn + 2 * (wg ^ 1)) * kTile;
      const float mo = others[0], lo = others[kTile];
      // O carries the last tile's offset
      const float mf = (done.last & 1) == static_cast<uint32_t>(wg) ? done.m : mo;
      l = (kFixed || done.m == mf ? l : l * ex2(done.m - mf)) + (kFixed || mo == mf ? lo : lo * ex2(mo - mf));
    }
    const float inv_l = l != 0.0f ? 1.0f / l : 0.0f;  // no key: 0; a NaN sum stays NaN
    // The rows leave through the item's Q tile (its last S has completed): 16-byte
    // pieces, the piece number XORed with the row, so that neither side meets a
    // bank conflict and a store covers whole lines of 4 (or 8) rows.
    constexpr int kPieces = kOCols / 8;
    uint4* stage = reinterpret_cast<uint4*>(sm + G::kOffQ + turn * G::kTileBytes) + (wg * 4 + (warp & 3)) * 32 * kPieces;
    const bool add = *found != 0;
#pragma unroll 1
    for (int c = 0; c < kOCols / 16; ++c) {
      uint32_t o[16];
      tc05::tmem_ld16(tO + wg * kOCols + c * 16, o);
      tc05::tmem_ld_wait();
      if (add) {
        // values that are not finite were zeroed in the tiles that hide keys from
        // some rows; this row adds those of the keys it sees (rare: read again)
        const T* v = static_cast<const T*>(p.v) + e.kvh * p.vs1 + wg * kOCols + c * 16;
        for (int key = max(e.seen + 1, 0); key <= lim; ++key)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = to_f32<T>(v[(e.k0 + key) * p.vs0 + i]);
            if (!isfinite(x)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
          }
      }
      uint32_t pk[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        pk[i] = pack2<T>(__uint_as_float(o[2 * i]) * inv_l, __uint_as_float(o[2 * i + 1]) * inv_l);
      stage[lane * kPieces + ((2 * c) ^ (lane & (kPieces - 1)))] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      stage[lane * kPieces + ((2 * c + 1) ^ (lane & (kPieces - 1)))] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
    }
    tc05::fence_before_sync();  // these reads precede the next item's first PV
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[G::kBarORead]);
    // four loads before the first store (one by one, 434 -> 425 us at 4 x 4,096 tokens);
    // one piece of 32 / kPieces rows each
    T* y = static_cast<T*>(p.y) + (e.q0 + e.tok) * p.ys0 + e.kvh * p.g * p.ys1 + wg * kOCols + (lane % kPieces) * 8;
    constexpr int kAtOnce = 4;
#pragma unroll 1
    for (int i = 0; i < kPieces; i += kAtOnce) {
      uint4 v[kAtOnce];
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const int rl = (i + x) * (32 / kPieces) + lane / kPieces;  // row of this warp's 32
        v[x] = stage[rl * kPieces + ((lane % kPieces) ^ (rl & (kPieces - 1)))];
      }
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const int rr = (warp & 3) * 32 + (i + x) * (32 / kPieces) + lane / kPieces;
        const int r_t = (rr * inv_g) >> 16, r_h = rr - r_t * p.g;  // rr / g: exact below 128
        if (r_t < p.tpt && e.tok + r_t < e.nq) *reinterpret_cast<uint4*>(y + r_t * p.ys0 + r_h * p.ys1) = v[x];
      }
    }
    fence_proxy_async_smem();  // these reads precede the buffer's next load
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[G::kBarQEmpty + turn]);
  }
}

// ---- kernel -------------------------------------------------------------------------------

template <int D, typename T, int kVariant>
__global__ void __launch_bounds__(kThreads, 1)
    packed_tc05_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ Params p) {
  using G = Geo<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + G::kOffBar);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + G::kOffTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + G::kOffFlags);
  volatile int* found = abort_flag + 1;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[G::kBarQFull + i], 1);
      mbar_init(&bars[G::kBarQEmpty + i], 8);  // every softmax warp
      mbar_init(&bars[G::kBarDone + i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars[G::kBarPost + i], 4);  // the warps of a warpgroup
      mbar_init(&bars[G::kBarSum + i], 4);
    }
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&bars[G::kBarKFull + s], 1);
      mbar_init(&bars[G::kBarKEmpty + s], 1);
      mbar_init(&bars[G::kBarVFull + s], 1);
      mbar_init(&bars[G::kBarVReady + s], 1);
      mbar_init(&bars[G::kBarVEmpty + s], 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&bars[G::kBarS + i], 1);
      mbar_init(&bars[G::kBarP + 2 * i], 4);
      mbar_init(&bars[G::kBarP + 2 * i + 1], 4);
      mbar_init(&bars[G::kBarPv + i], 1);
    }
    mbar_init(&bars[G::kBarO], 1);
    mbar_init(&bars[G::kBarORead], 8);  // every softmax warp
    *abort_flag = 0;
    *found = 0;
    fence_mbar_init();
  }
  // (Rows of a query tile that no head fills, where g does not divide 128, hold whatever the
  // shared memory held.)
  if (warp == 1) {
    tc05::tmem_alloc(tslot, G::kTmemCols);
    tc05::tmem_relinquish();
  }
  tc05::fence_before_sync();
  static_assert(G::kOffBar - G::kOffK >= kOrderBytes, "the rings serve as scratch");
  const Work work = lay_out_work(p, sm + G::kOffSeq, sm + G::kOffK);  // (barriers inside)
  tc05::fence_after_sync();
  const uint32_t tmem = *tslot;

  if (warp == 0) {
    if (lane == 0) producer<D>(&tq, &tk, &tv, p, work, sm, bars, abort_flag);
  } else if (warp == 1) {
    if (lane == 0) score_lane<D, kBf16>(p, work, sm, bars, tmem, abort_flag);
  } else if (warp == 2) {
    v_gate<D, T>(p, work, sm, bars, abort_flag, found);
  } else if (warp == 3) {
    if (lane == 0) value_lane<D, kBf16>(p, work, sm, bars, tmem, abort_flag);
  } else {
    softmax_rows<D, T, kVariant>(p, work, sm, bars, tmem, abort_flag, found);
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc05::fence_after_sync();
    tc05::tmem_dealloc(tmem, G::kTmemCols);
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

// Least-squares fit of tanh(x) / x = sum_k c_k (x^2)^k over 0 < x <= B (Chebyshev
// nodes in x; normal equations in u = x^2 / B^2, solved in double by Gaussian
// elimination with partial pivoting).
template <int N>
void fit_tanh(double B, double (&c)[N]) {
  constexpr int kNodes = 2048;
  const double pi = 3.14159265358979323846;
  double A[N][N + 1] = {};
  for (int i = 0; i < kNodes; ++i) {
    const double x = B * std::cos(pi * (i + 0.5) / (2.0 * kNodes));
    const double u = x * x / (B * B), f = std::tanh(x) / x;
    double pw[N];
    pw[0] = 1.0;
    for (int k = 1; k < N; ++k) pw[k] = pw[k - 1] * u;
    for (int r = 0; r < N; ++r) {
      for (int q = 0; q < N; ++q) A[r][q] += pw[r] * pw[q];
      A[r][N] += pw[r] * f;
    }
  }
  for (int col = 0; col < N; ++col) {
    int piv = col;
    for (int r = col + 1; r < N; ++r)
      if (std::fabs(A[r][col]) > std::fabs(A[piv][col])) piv = r;
    for (int q = 0; q <= N; ++q) std::swap(A[col][q], A[piv][q]);
    for (int r = 0; r < N; ++r) {
      if (r == col) continue;
      const double f = A[r][col] / A[col][col];
      for (int q = col; q <= N; ++q) A[r][q] -= f * A[col][q];
    }
  }
  double scale = 1.0;  // 1 / B^(2k): back from u to x^2
  for (int k = 0; k < N; ++k) {
    c[k] = A[k][N] / A[k][k] * scale;
    scale /= B * B;
  }
}

struct TanhFits {
  double full[kTanhTerms], brief[kTanhShortTerms];
  TanhFits() {
    fit_tanh(kTanhBound, full);
    fit_tanh(kTanhShortBound, brief);
  }
};

// c_log2 tanh(k1 s) as a polynomial in s: coefficient k is c_log2 c_k k1^(2k + 1).
// The largest |s| of the fit's range; less where a coefficient is below fp32's normal
// range (a softcap far above the scale), as far as its rounding, 2^-149 |s|^(2k + 1),
// stays below 1e-4; -1, so that no score is in it, where one leaves the range above.
template <int N>
float score_polynomial(const double (&c)[N], double bound, double softcap, double k1, float (&out)[N]) {
  double f = softcap * 1.4426950408889634 * k1, most = bound / k1;
  bool ok = true;
  for (int k = 0; k < N; ++k) {
    out[k] = static_cast<float>(c[k] * f);
    ok = ok && std::isfinite(out[k]) && (k > 0 || std::isnormal(out[k]));
    if (!std::isnormal(out[k])) most = std::fmin(most, std::pow(1e-4 * std::ldexp(1.0, 149), 1.0 / (2 * k + 1)));
    f *= k1 * k1;
  }
  return ok && most < 1e18 ? static_cast<float>(most) : -1.0f;  // (s^2 is a finite fp32)
}

// Shared memory with `seqs` sequences and `items` places in the item list.
template <int D>
int64_t smem_bytes(int64_t seqs, int64_t items) {
  return 1024 + Geo<D>::kOffSeq + seqs * 16 + ((seqs + 2) & ~int64_t(1)) * 4 + items * 8;
}

// Items of one launch over `seqs` sequences, at most.
int64_t items_bound(const PackedArgs& a, int64_t seqs) {
  const int64_t g = a.Hq / a.Hkv, step = kTile / g;
  return (a.Tq / step + seqs) * a.Hkv;
}

template <int D, typename T>
int launch_t(const PackedArgs& a, cudaStream_t st) {
  const int64_t g = a.Hq / a.Hkv, tpt = kTile / g;
  CUtensorMap tq, tk, tv;
  if (!rows_map(&tq, a.q, a.dtype, D, a.Hq, a.Tq, a.qs, static_cast<int>(g), static_cast<int>(tpt)) ||
      !rows_map(&tk, a.k, a.dtype, D, a.Hkv, a.Tk, a.ks, 1, kTile) ||
      !rows_map(&tv, a.v, a.dtype, D, a.Hkv, a.Tk, a.vs, 1, kTile))
    return -1;
  Params p;
  memset(&p, 0, sizeof(p));
  p.y = a.y;
  p.ys0 = a.ys[0];
  p.ys1 = a.ys[1];
  p.v = a.v;
  p.vs0 = a.vs[0];
  p.vs1 = a.vs[1];
  p.err_word = a.err_word;
  p.Tq = static_cast<int>(a.Tq);
  p.Tk = static_cast<int>(a.Tk);
  p.Hkv = static_cast<int>(a.Hkv);
  p.g = static_cast<int>(g);
  p.tpt = static_cast<int>(tpt);
  p.causal = a.causal;
  const float log2e = 1.4426950408889634f;
  int variant = kVarPlain;
  p.k1 = a.softcap != 0.0f ? a.scale / a.softcap : 0.0f;
  if (p.k1 > kNoCapMax) {
    p.c_log2 = a.softcap * log2e;
    variant = p.c_log2 <= fixed_offset_max_log2<T>() ? kVarCapFixed
              : a.softcap <= kFarMax                 ? kVarCapMax
                                                     : kVarCapLarge;
    static const TanhFits fits;
    p.tq_bound = score_polynomial(fits.full, kTanhBound, a.softcap, p.k1, p.tq);
    p.ts_bound = score_polynomial(fits.brief, kTanhShortBound, a.softcap, p.k1, p.ts);
  } else {
    p.c_log2 = a.scale * log2e;
  }
  const int sms = sm_count();
  if (sms <= 0) return -1;
  // (in bf16 every softcap up to kFarMax has the offset 0)
  constexpr Variant kSmallCap = std::is_same<T, __half>::value ? kVarCapMax : kVarCapLarge;
  auto kern = variant == kVarPlain      ? packed_tc05_kernel<D, T, kVarPlain>
              : variant == kVarCapFixed ? packed_tc05_kernel<D, T, kVarCapFixed>
              : variant == kVarCapMax   ? packed_tc05_kernel<D, T, kSmallCap>
                                        : packed_tc05_kernel<D, T, kVarCapLarge>;
  if (!allow_smem(reinterpret_cast<const void*>(kern))) return -1;
  for (int64_t b0 = 0; b0 < a.B; b0 += kMaxSeqs) {
    const int64_t seqs = a.B - b0 < kMaxSeqs ? a.B - b0 : kMaxSeqs;
    const int64_t items = items_bound(a, seqs);
    const int64_t grid = items < sms ? items : sms;
    p.q_start = a.q_start + b0;
    p.k_start = a.k_start + b0;
    p.B = static_cast<int>(seqs);
    p.cap_items = static_cast<int>((items + grid - 1) / grid);
    kern<<<static_cast<unsigned>(grid), kThreads, static_cast<size_t>(smem_bytes<D>(seqs, p.cap_items)), st>>>(tq, tk, tv, p);
    if (cudaGetLastError() != cudaSuccess) return -1;
  }
  return 0;
}

}  // namespace

bool packed_tc_supported(const PackedArgs& a) {
  if (a.dtype != SA_BF16 && a.dtype != SA_F16) return false;
  if (a.D != 64 && a.D != 128) return false;
  if (!(a.scale > 0.0f) || a.Hq / a.Hkv > kTile || a.Hkv >= 65536 || a.Tk == 0) return false;
  const int64_t seqs = a.B < kMaxSeqs ? a.B : kMaxSeqs;
  const int64_t items = items_bound(a, seqs), sms = sm_count();
  if (sms <= 0 || items >= (int64_t(1) << 30)) return false;
  const int64_t grid = items < sms ? items : sms, cap = (items + grid - 1) / grid;
  // (beyond the list's room, millions of tokens times heads, the other kernel serves)
  const int64_t bytes = a.D == 128 ? smem_bytes<128>(seqs, cap) : smem_bytes<64>(seqs, cap);
  return bytes <= kSmemLimit && encode_tiled() != nullptr;
}

int launch_packed_tc(const PackedArgs& a, cudaStream_t st) {
  if (a.dtype == SA_BF16)
    return a.D == 128 ? launch_t<128, __nv_bfloat16>(a, st) : launch_t<64, __nv_bfloat16>(a, st);
  return a.D == 128 ? launch_t<128, __half>(a, st) : launch_t<64, __half>(a, st);
}

}  // namespace sa
