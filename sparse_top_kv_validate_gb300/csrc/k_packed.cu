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
//  * A query tile is 128 rows: 128 / g tokens times the g query heads of one
//    KV head, so that a short sequence fills its tiles and the heads share
//    every K/V tile.  A work item is a pair of neighbouring tiles, the two
//    "sides": each has its own scores, probabilities and outputs in tensor
//    memory (S0 S1 O0 O1, 128 columns each at D 128), its own MMA lane and its
//    own softmax warpgroup of 128 threads, one row per thread.  While one side's
//    softmax runs, the tensor cores work for the other; a row's maximum and sum
//    never leave its thread.
//  * P (16 bits) overwrites the first half of its own scores.  An MMA lane
//    issues PV(j) and then S(j + 1) into the same columns: the tensor cores take
//    one thread's MMAs in order.
//  * Warp 0 loads Q (box: 64 dims x g heads x 128 / g tokens) and the K and V
//    tiles through a ring of slots; warps 1 and 3 are the MMA lanes; warp 2
//    passes every V tile on: where keys end inside a tile it zeroes the rows
//    behind them (0 times another sequence's NaN is NaN), and where some of a
//    tile's keys are hidden from some rows it looks for values that are not
//    finite: these are zeroed too, and the rows that do see them add them in
//    the epilogue.
//  * Items go to CTAs in a snake order of falling cost.  The lengths are on
//    the device, so every CTA works out the order itself: the rank of an item
//    among all has a closed form per sequence (an item's number of key tiles
//    grows along its sequence), and a CTA keeps only its own items.
//  * Without a softcap, or with a large one, the row's offset is a maximum that
//    is raised only by more than 2^8 (O is then rescaled in tensor memory);
//    with a softcap up to 67 the logits are bounded and the offset is 0.
//  * Every mbarrier wait is bounded; a stalled pipeline sets
//    SA_ERRBIT_TIMEOUT, stops every role, and still frees the tensor memory.
#include <cuda.h>

#include <cmath>
#include <cstring>
#include <mutex>
#include <type_traits>
#include <utility>

#include "packed.cuh"
#include "serving.h"
#include "tc05.cuh"

namespace sa {

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;               // rows of a query tile; keys of a K/V tile
constexpr int kSlabBytes = kTile * 128;  // 128 rows x 64 sixteen-bit columns
constexpr float kRescaleLog2 = 8.0f;     // lazy-maximum slack (factor 256)
constexpr int kTanhTerms = 5;            // tanh(x) ~= x * sum_k c_k (x^2)^k
constexpr float kTanhPolyBound = 0.625f; // |x| range of the fit (abs error ~1e-7)
constexpr float kFixedOffsetMaxLog2 = 97.0f;  // softcap * log2(e) up to which 2^logit needs no offset
constexpr int kMaxSeqs = 1024;           // sequences per launch
constexpr int kSmemLimit = 227 * 1024;

template <int D>
struct Geo {
  static constexpr int kSlabs = D / 64;
  static constexpr int kTileBytes = kSlabs * kSlabBytes;   // 16 or 32 KB
  static constexpr int kStages = D == 128 ? 4 : 8;         // ring slots: K tiles even, V tiles odd
  static constexpr int kOffQ = 0;                          // two sides
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kOffBar = kOffRing + kStages * kTileBytes;
  // barriers: per side q_full, q_empty, s_full, p_full, o_full, done; per slot
  // kv_full, kv_empty, v_ready (V slots)
  static constexpr int kBarQFull = 0, kBarQEmpty = 2, kBarS = 4, kBarP = 6, kBarO = 8, kBarDone = 10,
                       kBarKvFull = 12, kBarKvEmpty = kBarKvFull + kStages,
                       kBarV = kBarKvEmpty + kStages, kNumBars = kBarV + kStages;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffFlags = kOffTmemSlot + 4;       // abort, hidden values found
  static constexpr int kOffSeq = (kOffFlags + 8 + 15) / 16 * 16;  // int4 [B]; int [B + 1]; uint2 [items]
  static constexpr uint32_t kColS = 0, kColO = 2 * kTile;  // + side * 128, + side * D
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
  float k1;                // x = score * k1 (scale / softcap), or the raw score
  float c_log2;            // log2-domain multiplier of tanh(x) (softcap * log2e) or of x (scale * log2e)
  float tq[kTanhTerms];    // c_log2 * c_k: the tanh polynomial already in log2 units
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

// Pairs of a sequence with at least x key tiles.
__device__ __forceinline__ int pairs_with(const Params& p, int nq, int nk, int x) {
  const int step = 2 * p.tpt, pairs = (nq + step - 1) / step;
  if (x <= 1) return pairs;
  const int thr = (x - 1) * kTile;      // the pair's last key must reach thr
  if (nk - 1 < thr) return 0;
  if (!p.causal) return pairs;
  const int need = thr - (nk - nq);     // and so its last token
  if (need <= 0) return pairs;
  if (nq - 1 < need) return 0;
  return pairs - need / step;           // pairs from the one that holds token `need` on
}

struct Item {
  int q0, nq, k0, nk, kvh;
  int tok;      // first token of side 0
  int ns[2];    // key tiles of each side (0: the side has no rows)
  int n;        // of both
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
  const uint2* list;    // this CTA's items: sequence << 16 | KV head, pair
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
    it.tok = static_cast<int>(e.y) * 2 * p.tpt;
    it.ns[0] = tiles_of(p.causal, it.nq, it.nk, min(it.tok + p.tpt, it.nq) - 1);
    it.ns[1] = it.tok + p.tpt < it.nq
                   ? tiles_of(p.causal, it.nq, it.nk, min(it.tok + 2 * p.tpt, it.nq) - 1)
                   : 0;
    it.n = max(it.ns[0], it.ns[1]);
    it.seen = last_key(p.causal, it.nq, it.nk, it.tok);
    return true;
  }
};

// Every CTA: the sequences' extents, the number of items, and this CTA's items
// in the order of falling cost (all threads; ends with a barrier).
__device__ __forceinline__ Work lay_out_work(const Params& p, uint8_t* area) {
  int4* seq = reinterpret_cast<int4*>(area);
  int* pref = reinterpret_cast<int*>(seq + p.B);
  uint2* list = reinterpret_cast<uint2*>(pref + ((p.B + 2) & ~1));
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const int step = 2 * p.tpt;
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
  const int pairs = pref[p.B];
  const int G = static_cast<int>(gridDim.x);
  Work w{seq, list, pairs * p.Hkv, G, p.cap_items};
  for (int i = tid; i < pairs; i += kThreads) {
    int lo = 0, hi = p.B;  // the last sequence with pref <= i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pref[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int b = lo, pr = i - pref[b];
    const int4 s = seq[b];
    const int n = tiles_of(p.causal, s.y, s.w, min((pr + 1) * step, s.y) - 1);
    // items with more key tiles, then those with as many of earlier sequences
    // and of this one
    int rank = pr - (pref[b + 1] - pref[b] - pairs_with(p, s.y, s.w, n));
    for (int o = 0; o < p.B; ++o) {
      const int4 t = seq[o];
      rank += o < b ? pairs_with(p, t.y, t.w, n) : pairs_with(p, t.y, t.w, n + 1);
    }
    for (int h = 0; h < p.Hkv; ++h) {
      const int x = rank * p.Hkv + h, k = x / G, r = x - k * G;
      if (((k & 1) ? G - 1 - r : r) == static_cast<int>(blockIdx.x) && k < p.cap_items)
        list[k] = make_uint2(static_cast<uint32_t>(b) << 16 | static_cast<uint32_t>(h), static_cast<uint32_t>(pr));
    }
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
  uint32_t kv_cnt = 0, q_cnt[2] = {0, 0};
  bool stop = false;
  Item it;
  for (int k = 0; !stop && work.get(k, p, it); ++k) {
    for (int side = 0; side < 2 && !stop; ++side) {
      if (it.ns[side] == 0) continue;
      // the side's Q is free once the last S MMA of its previous item has completed
      if (q_cnt[side] > 0 &&
          !wait_or_abort(&bars[G::kBarQEmpty + side], (q_cnt[side] - 1) & 1, abort_flag, p.err_word)) {
        stop = true;
        break;
      }
      mbar_arrive_expect_tx(&bars[G::kBarQFull + side], q_bytes);
#pragma unroll
      for (int s = 0; s < G::kSlabs; ++s)
        tc05::tma_load3(sm + G::kOffQ + side * G::kTileBytes + s * kSlabBytes, tq, s * 64, it.kvh * p.g,
                        it.q0 + it.tok + side * p.tpt, &bars[G::kBarQFull + side]);
      ++q_cnt[side];
    }
    for (int e = 0; e < 2 * it.n && !stop; ++e) {  // K_0, V_0, K_1, V_1, ...
      const uint32_t slot = kv_cnt % G::kStages, use = kv_cnt / G::kStages;
      if (use > 0 && !wait_or_abort(&bars[G::kBarKvEmpty + slot], (use - 1) & 1, abort_flag, p.err_word)) {
        stop = true;
        break;
      }
      mbar_arrive_expect_tx(&bars[G::kBarKvFull + slot], G::kTileBytes);
#pragma unroll
      for (int s = 0; s < G::kSlabs; ++s)
        tc05::tma_load3(sm + G::kOffRing + slot * G::kTileBytes + s * kSlabBytes, (e & 1) ? tv : tk, s * 64,
                        it.kvh, it.k0 + (e >> 1) * kTile, &bars[G::kBarKvFull + slot]);
      ++kv_cnt;
    }
  }
  if (*abort_flag) {
    // Let every copy already issued land before the CTA can exit.
    for (int side = 0; side < 2; ++side)
      if (q_cnt[side] > 0) mbar_wait(&bars[G::kBarQFull + side], (q_cnt[side] - 1) & 1);
    for (uint32_t s = 0; s < G::kStages; ++s) {
      if (kv_cnt <= s) break;
      const uint32_t issued = (kv_cnt - s + G::kStages - 1) / G::kStages;
      mbar_wait(&bars[G::kBarKvFull + s], (issued - 1) & 1);
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
  uint32_t kv_cnt = 0;
  Item it;
  for (int k = 0; work.get(k, p, it); ++k) {
    for (int j = 0; j < it.n; ++j, kv_cnt += 2) {
      const uint32_t idx = kv_cnt + 1, slot = idx % G::kStages;
      if (!wait_or_abort_warp(&bars[G::kBarKvFull + slot], (idx / G::kStages) & 1, abort_flag, p.err_word))
        return;
      const int first = j * kTile;
      if (first + kTile - 1 > it.seen) {  // (rows behind the last key are past `seen` too)
        uint8_t* tile = sm + G::kOffRing + slot * G::kTileBytes;
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
      if (lane == 0) mbar_arrive(&bars[G::kBarV + slot]);
    }
  }
}

// ---- role: MMA issuer of one side (one lane) ------------------------------------------------

template <int D, bool kBf16>
__device__ void mma_lane(int side, const Params& p, const Work& work, uint8_t* sm, uint64_t* bars,
                         uint32_t tmem, volatile int* abort_flag) {
  using G = Geo<D>;
  constexpr uint32_t id_s = tc05::idesc_f16(kTile, kTile, kBf16, false, false);
  constexpr uint32_t id_o = tc05::idesc_f16(kTile, D, kBf16, false, true);
  const uint64_t dQ = tc05::sw128_desc(smem_u32(sm + G::kOffQ + side * G::kTileBytes), 16, 1024);
  const uint64_t dK = tc05::sw128_desc(smem_u32(sm + G::kOffRing), 16, 1024);
  const uint64_t dV = tc05::sw128_desc(smem_u32(sm + G::kOffRing), kSlabBytes, 1024);
  const uint32_t tS = tmem + G::kColS + side * kTile, tO = tmem + G::kColO + side * D;

  auto issue_s = [&](uint32_t slot) {  // S = Q . K^T
    const uint64_t b0 = dK + ((slot * G::kTileBytes) >> 4);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = ((kk / 4) * kSlabBytes + (kk % 4) * 32) >> 4;
      tc05::mma_ss(tS, dQ + off, b0 + off, id_s, kk > 0 ? 1u : 0u);
    }
  };
  auto issue_pv = [&](uint32_t slot, bool acc) {  // O (+)= P . V
    const uint64_t v0 = dV + ((slot * G::kTileBytes) >> 4);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk)
      tc05::mma_ts(tO, tS + kk * 8, v0 + ((kk * 2048) >> 4), id_o, (acc || kk > 0) ? 1u : 0u);
  };

  uint32_t kv_cnt = 0, q_cnt = 0, p_cnt = 0;
  bool stop = false;
  Item it;
  for (int k = 0; !stop && work.get(k, p, it); ++k) {
    const int n = it.ns[side];
    const uint32_t base = kv_cnt;
    kv_cnt += 2 * it.n;
    auto wait_k = [&](int j) {
      const uint32_t i = base + 2 * j;
      return wait_or_abort(&bars[G::kBarKvFull + i % G::kStages], (i / G::kStages) & 1, abort_flag, p.err_word);
    };
    auto wait_v = [&](int j) {
      const uint32_t i = base + 2 * j + 1;
      return wait_or_abort(&bars[G::kBarV + i % G::kStages], (i / G::kStages) & 1, abort_flag, p.err_word);
    };
    auto score = [&](int j) {
      if (!wait_k(j)) return false;
      const uint32_t slot = (base + 2 * j) % G::kStages;
      tc05::fence_after_sync();
      issue_s(slot);
      tc05::commit(&bars[G::kBarS + side]);
      tc05::commit(&bars[G::kBarKvEmpty + slot]);
      if (j == n - 1) tc05::commit(&bars[G::kBarQEmpty + side]);
      return true;
    };
    if (n > 0) {
      if (!wait_or_abort(&bars[G::kBarQFull + side], q_cnt & 1, abort_flag, p.err_word) || !score(0)) break;
      ++q_cnt;
    }
    for (int j = 0; j < n; ++j) {
      if (!wait_v(j) || !wait_or_abort(&bars[G::kBarP + side], p_cnt & 1, abort_flag, p.err_word)) {
        stop = true;
        break;
      }
      ++p_cnt;
      const uint32_t slot = (base + 2 * j + 1) % G::kStages;
      tc05::fence_after_sync();
      issue_pv(slot, j > 0);
      tc05::commit(&bars[G::kBarKvEmpty + slot]);
      if (j == n - 1) tc05::commit(&bars[G::kBarO + side]);
      if (j + 1 < n && !score(j + 1)) {
        stop = true;
        break;
      }
    }
    // tiles that only the other side reads
    for (int j = n; j < it.n && !stop; ++j) {
      if (!wait_k(j)) {
        stop = true;
        break;
      }
      mbar_arrive(&bars[G::kBarKvEmpty + (base + 2 * j) % G::kStages]);
      if (!wait_v(j)) {
        stop = true;
        break;
      }
      mbar_arrive(&bars[G::kBarKvEmpty + (base + 2 * j + 1) % G::kStages]);
    }
  }
  // Every MMA this lane issued completes before the tensor memory is released.
  uint64_t* done = &bars[G::kBarDone + side];
  tc05::commit(done);
  mbar_wait(done, 0);
}

// ---- role: softmax (one warpgroup per side, one row per thread) ------------------------------

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

// How the log2-domain logit of x is formed: c_log2 * x (no softcap), or
// c_log2 * tanh(x) by the fitted polynomial (kPoly) or, where a score of the
// warp lies outside its range, from the hardware exponential and reciprocal.
enum ScoreMode { kPlain = 0, kPoly = 1, kFar = 2 };

__device__ __forceinline__ float tanh_far(float x) {
  // 1 - 2 / (e^2x + 1), absolute error below 2^-20; saturates cleanly
  return 1.0f - 2.0f * rcp(ex2(x * (2.0f * kLog2e)) + 1.0f);
}

__device__ __forceinline__ float poly_logit(float x, const float (&tq)[kTanhTerms]) {
  const float y = x * x;
  float q = tq[kTanhTerms - 1];
#pragma unroll
  for (int k = kTanhTerms - 2; k >= 0; --k) q = fmaf(q, y, tq[k]);
  return x * q;
}

// x = s * k1 of 32 scores in place (softcap), and their largest magnitude.
__device__ __forceinline__ float scale_chunk(uint32_t (&r)[32], float k1) {
  const uint64_t k2 = f2_pack(k1, k1);
  float ax[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a, b;
    f2_unpack(f2_mul(f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), k2), a, b);
    r[2 * i] = __float_as_uint(a);
    r[2 * i + 1] = __float_as_uint(b);
    ax[i & 1] = max3(ax[i & 1], fabsf(a), fabsf(b));
  }
  return fmaxf(ax[0], ax[1]);
}

// Maximum of the chunk's columns <= rel.
template <bool kMask>
__device__ __forceinline__ float max_chunk(const uint32_t (&r)[32], int rel, float m) {
  float mx[2] = {m, SA_NEG_INF};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a = __uint_as_float(r[2 * i]), b = __uint_as_float(r[2 * i + 1]);
    if (kMask) {
      if (2 * i > rel) a = SA_NEG_INF;
      if (2 * i + 1 > rel) b = SA_NEG_INF;
    }
    mx[i & 1] = max3(mx[i & 1], a, b);
  }
  return fmaxf(mx[0], mx[1]);
}

// p = 2^(logit(x) - m) of 32 columns, masked ones 0, written to tensor memory at
// tP as 16 columns of 16-bit pairs and added to the two partial sums.
template <int kMode, bool kMask, typename T>
__device__ __forceinline__ void exp_chunk(const uint32_t (&r)[32], uint32_t tP, float c2, float neg_m,
                                          const float (&tq)[kTanhTerms], int rel, uint64_t (&ls)[2]) {
  const uint64_t c2x2 = f2_pack(c2, c2), nm2 = f2_pack(neg_m, neg_m);
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float x0 = __uint_as_float(r[2 * i]), x1 = __uint_as_float(r[2 * i + 1]);
    uint64_t v;
    if (kMode == kPlain) {
      v = f2_fma(f2_pack(x0, x1), c2x2, nm2);
    } else if (kMode == kFar) {
      v = f2_fma(f2_pack(tanh_far(x0), tanh_far(x1)), c2x2, nm2);
    } else {
      const uint64_t xx = f2_pack(x0, x1);
      const uint64_t y = f2_mul(xx, xx);
      uint64_t q = f2_fma(f2_pack(tq[4], tq[4]), y, f2_pack(tq[3], tq[3]));
      q = f2_fma(q, y, f2_pack(tq[2], tq[2]));
      q = f2_fma(q, y, f2_pack(tq[1], tq[1]));
      q = f2_fma(q, y, f2_pack(tq[0], tq[0]));
      v = f2_fma(xx, q, nm2);
    }
    float a, b;
    f2_unpack(v, a, b);
    if (kMask) {
      if (2 * i > rel) a = SA_NEG_INF;
      if (2 * i + 1 > rel) b = SA_NEG_INF;
    }
    a = ex2(a);
    b = ex2(b);
    ls[i & 1] = f2_add(ls[i & 1], f2_pack(a, b));
    pk[i] = pack2<T>(a, b);
  }
  tc05::tmem_st16(tP, pk);
}

enum Variant { kVarPlain = 0, kVarCapMax = 1, kVarCapFixed = 2 };

template <int D, typename T, int kVariant>
__device__ void softmax_rows(const Params& p, const Work& work, uint64_t* bars, uint32_t tmem,
                             volatile int* abort_flag, volatile int* found) {
  using G = Geo<D>;
  constexpr bool kCap = kVariant != kVarPlain, kFixed = kVariant == kVarCapFixed;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int side = (warp - 4) >> 2;
  const int row = ((warp & 3) << 5) | lane;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t tS = tmem + lanes + G::kColS + side * kTile, tO = tmem + lanes + G::kColO + side * D;
  const int rt = row / p.g, rh = row - rt * p.g;  // token of the tile, head of the group
  const float c2 = p.c_log2, k1 = p.k1;
  float tq[kTanhTerms];
#pragma unroll
  for (int k = 0; k < kTanhTerms; ++k) tq[k] = p.tq[k];
  uint32_t s_cnt = 0, o_cnt = 0;
  Item it;
  for (int k = 0; work.get(k, p, it); ++k) {
    const int n = it.ns[side];
    if (n == 0) continue;
    const int tok = it.tok + side * p.tpt + rt;
    const bool live = rt < p.tpt && tok < it.nq;
    const int lim = live ? last_key(p.causal, it.nq, it.nk, tok) : -1;  // last visible key
    float m = SA_NEG_INF;
    uint64_t ls[2] = {0, 0};
    for (int j = 0; j < n; ++j) {
      if (!wait_or_abort_warp(&bars[G::kBarS + side], s_cnt & 1, abort_flag, p.err_word)) return;
      ++s_cnt;
      tc05::fence_after_sync();
      const int rel = lim - j * kTile;  // columns above rel are masked
      const bool masked = __any_sync(0xffffffffu, rel < kTile - 1);
      uint32_t r[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc05::tmem_ld32(tS + c * 32, r[c]);
      tc05::tmem_ld_wait();
      int mode = kPlain;
      if (kCap) {
        float ax = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) ax = fmaxf(ax, scale_chunk(r[c], k1));
        mode = __any_sync(0xffffffffu, ax > kTanhPolyBound) ? kFar : kPoly;
      }
      float alpha = 1.0f;
      bool any_raise = false;
      if (!kFixed) {
        float mx = SA_NEG_INF;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mx = masked ? max_chunk<true>(r[c], rel - 32 * c, mx) : max_chunk<false>(r[c], 0, mx);
        float mt = SA_NEG_INF;
        if (mx != SA_NEG_INF)
          mt = mode == kPlain ? mx * c2 : mode == kPoly ? poly_logit(mx, tq) : tanh_far(mx) * c2;
        const bool raise = mt > m + kRescaleLog2 || (m == SA_NEG_INF && mt > m);
        any_raise = __any_sync(0xffffffffu, raise);
        if (raise) {
          alpha = ex2(m - mt);
          m = mt;
          ls[0] = f2_mul(ls[0], f2_pack(alpha, alpha));
          ls[1] = f2_mul(ls[1], f2_pack(alpha, alpha));
        }
      }
      const float neg_m = (kFixed || m == SA_NEG_INF) ? 0.0f : -m;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t tP = tS + c * 16;
        const int rc = rel - 32 * c;
        if (!kCap) {
          if (masked) exp_chunk<kPlain, true, T>(r[c], tP, c2, neg_m, tq, rc, ls);
          else exp_chunk<kPlain, false, T>(r[c], tP, c2, neg_m, tq, rc, ls);
        } else if (mode == kPoly) {
          if (masked) exp_chunk<kPoly, true, T>(r[c], tP, c2, neg_m, tq, rc, ls);
          else exp_chunk<kPoly, false, T>(r[c], tP, c2, neg_m, tq, rc, ls);
        } else {
          exp_chunk<kFar, true, T>(r[c], tP, c2, neg_m, tq, masked ? rc : kTile, ls);
        }
      }
      // PV(j - 1) was issued before S(j) by the same lane, so it has completed
      // with it: O may follow the new maximum
      if (!kFixed && any_raise && j > 0) rescale_o<D>(tO, alpha);
      tc05::tmem_st_wait();
      tc05::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[G::kBarP + side]);
    }

    // epilogue: O / l of this row
    float l;
    {
      float a, b;
      f2_unpack(f2_add(ls[0], ls[1]), a, b);
      l = a + b;
    }
    if (!wait_or_abort_warp(&bars[G::kBarO + side], o_cnt & 1, abort_flag, p.err_word)) return;
    ++o_cnt;
    tc05::fence_after_sync();
    const float inv_l = l != 0.0f ? 1.0f / l : 0.0f;  // no key: 0; a NaN sum stays NaN
    T* yrow = static_cast<T*>(p.y) + (it.q0 + tok) * p.ys0 + (it.kvh * p.g + rh) * p.ys1;
    const bool add = *found != 0;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t o[16];
      tc05::tmem_ld16(tO + c * 16, o);
      tc05::tmem_ld_wait();
      if (add && live) {
        // values that are not finite were zeroed in the tiles that hide keys from
        // some rows; this row adds those of the keys it sees (rare: read again)
        const T* v = static_cast<const T*>(p.v) + it.kvh * p.vs1 + c * 16;
        for (int key = max(it.seen + 1, 0); key <= lim; ++key)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = to_f32<T>(v[(it.k0 + key) * p.vs0 + i]);
            if (!isfinite(x)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
          }
      }
      if (live) {
        uint32_t pk[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          pk[i] = pack2<T>(__uint_as_float(o[2 * i]) * inv_l, __uint_as_float(o[2 * i + 1]) * inv_l);
        uint4* dst = reinterpret_cast<uint4*>(yrow + c * 16);
        dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
      }
    }
    tc05::fence_before_sync();  // these reads of O precede the next item's first P
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
      mbar_init(&bars[G::kBarQEmpty + i], 1);
      mbar_init(&bars[G::kBarS + i], 1);
      mbar_init(&bars[G::kBarP + i], 4);   // the side's softmax warps
      mbar_init(&bars[G::kBarO + i], 1);
      mbar_init(&bars[G::kBarDone + i], 1);
    }
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&bars[G::kBarKvFull + s], 1);
      mbar_init(&bars[G::kBarKvEmpty + s], 2);  // both MMA lanes
      mbar_init(&bars[G::kBarV + s], 1);
    }
    *abort_flag = 0;
    *found = 0;
    fence_mbar_init();
  }
  // rows of the query tiles that no head fills (g does not divide 128): zeros once
  const int used = p.g * p.tpt;
  for (int e = static_cast<int>(threadIdx.x); e < (kTile - used) * 8 * G::kSlabs * 2; e += kThreads) {
    const int r = used + e / (16 * G::kSlabs), c = e % (16 * G::kSlabs);
    *reinterpret_cast<uint4*>(sm + G::kOffQ + (c >> 3) * kSlabBytes + r * 128 + (c & 7) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (warp == 1) {
    tc05::tmem_alloc(tslot, G::kTmemCols);
    tc05::tmem_relinquish();
  }
  tc05::fence_before_sync();
  const Work work = lay_out_work(p, sm + G::kOffSeq);  // (barriers inside)
  tc05::fence_after_sync();
  const uint32_t tmem = *tslot;

  if (warp == 0) {
    if (lane == 0) producer<D>(&tq, &tk, &tv, p, work, sm, bars, abort_flag);
  } else if (warp == 1) {
    if (lane == 0) mma_lane<D, kBf16>(0, p, work, sm, bars, tmem, abort_flag);
  } else if (warp == 2) {
    v_gate<D, T>(p, work, sm, bars, abort_flag, found);
  } else if (warp == 3) {
    if (lane == 0) mma_lane<D, kBf16>(1, p, work, sm, bars, tmem, abort_flag);
  } else {
    softmax_rows<D, T, kVariant>(p, work, bars, tmem, abort_flag, found);
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
void fit_tanh(double (&c)[kTanhTerms]) {
  constexpr int kNodes = 2048;
  const double B = kTanhPolyBound, pi = 3.14159265358979323846;
  double A[kTanhTerms][kTanhTerms + 1] = {};
  for (int i = 0; i < kNodes; ++i) {
    const double x = B * std::cos(pi * (i + 0.5) / (2.0 * kNodes));
    const double u = x * x / (B * B), f = std::tanh(x) / x;
    double pw[kTanhTerms];
    pw[0] = 1.0;
    for (int k = 1; k < kTanhTerms; ++k) pw[k] = pw[k - 1] * u;
    for (int r = 0; r < kTanhTerms; ++r) {
      for (int q = 0; q < kTanhTerms; ++q) A[r][q] += pw[r] * pw[q];
      A[r][kTanhTerms] += pw[r] * f;
    }
  }
  for (int col = 0; col < kTanhTerms; ++col) {
    int piv = col;
    for (int r = col + 1; r < kTanhTerms; ++r)
      if (std::fabs(A[r][col]) > std::fabs(A[piv][col])) piv = r;
    for (int q = 0; q <= kTanhTerms; ++q) std::swap(A[col][q], A[piv][q]);
    for (int r = 0; r < kTanhTerms; ++r) {
      if (r == col) continue;
      const double f = A[r][col] / A[col][col];
      for (int q = col; q <= kTanhTerms; ++q) A[r][q] -= f * A[col][q];
    }
  }
  double scale = 1.0;  // 1 / B^(2k): back from u to x^2
  for (int k = 0; k < kTanhTerms; ++k) {
    c[k] = A[k][kTanhTerms] / A[k][k] * scale;
    scale /= B * B;
  }
}

const double* tanh_coefficients() {
  static std::once_flag once;
  static double c[kTanhTerms];
  std::call_once(once, [] { fit_tanh(c); });
  return c;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Shared memory with `seqs` sequences and `items` places in the item list.
template <int D>
int64_t smem_bytes(int64_t seqs, int64_t items) {
  return 1024 + Geo<D>::kOffSeq + seqs * 16 + ((seqs + 2) & ~int64_t(1)) * 4 + items * 8;
}

// Items of one launch over `seqs` sequences, at most.
int64_t items_bound(const PackedArgs& a, int64_t seqs) {
  const int64_t g = a.Hq / a.Hkv, step = 2 * (kTile / g);
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
  if (a.softcap != 0.0f) {
    p.k1 = a.scale / a.softcap;
    p.c_log2 = a.softcap * log2e;
    variant = p.c_log2 <= kFixedOffsetMaxLog2 ? kVarCapFixed : kVarCapMax;
    const double* c = tanh_coefficients();
    for (int k = 0; k < kTanhTerms; ++k)
      p.tq[k] = static_cast<float>(c[k] * static_cast<double>(a.softcap) * 1.4426950408889634);
  } else {
    p.k1 = 1.0f;
    p.c_log2 = a.scale * log2e;
  }
  const int sms = sm_count();
  if (sms <= 0) return -1;
  auto kern = variant == kVarPlain    ? packed_tc05_kernel<D, T, kVarPlain>
              : variant == kVarCapMax ? packed_tc05_kernel<D, T, kVarCapMax>
                                      : packed_tc05_kernel<D, T, kVarCapFixed>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess)
    return -1;
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
