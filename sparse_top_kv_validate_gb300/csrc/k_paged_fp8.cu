// k_paged_fp8.cu -- decode attention over FP8 pages (one new query per sequence).
//
// Per query head: s_t = scale 2^(ek_t) (q . ck_t) over the codes ck_t of key t
// and its exponent ek_t, y = sum_t softmax(s)_t 2^(ev_t) cv_t.  Each page is
// read once and nothing else is large, so DRAM bandwidth is the bound; what
// must not get in its way is the decoding of two codes per byte pair read.
//
// The work is laid out as in the stream kernel (k_stream.cu): every (sequence,
// KV head)'s context cut into 16-token tiles laid end to end, one contiguous
// range of tiles per warp of a persistent grid, whatever the contexts.
//
//  * Each warp has a ring of tiles that TMA fills (16 rows of codes of K and of
//    V in the 128-byte swizzle, 64-byte for D 64, and their 16 scale bytes each).
//    With keys as M of S^T = K Q^T and dims as M of O^T = V^T P^T, the 16 codes
//    that a lane reads with one shared-memory load are values of its own MMA
//    fragments once the contraction index (for S) and the output dims (for O)
//    are numbered to fit, so no ldmatrix and no exchange is needed; the swizzle
//    keeps those loads free of bank conflicts.  (Codes straight from DRAM to
//    registers, the next tile's loads under this tile's arithmetic, reached
//    2.75 TB/s: too few bytes in flight.)
//  * K: e4m3 -> f16 is exact (one conversion per pair), and q enters as f16
//    after a power of two per head brings its largest element to [2^14, 2^15),
//    so bf16 and f16 queries lose nothing that fp32 sums would keep (an
//    element 2^-39 below the row's largest is rounded).  The key's scale and
//    the head's power of two multiply the fp32 score.
//  * V: the codes become f16 the same way (exact).  The value's scale is folded
//    into the probability: w = p 2^(ev - E), E a power of two per head.  It is raised
//    when w passes 2^15, to put the tile's largest weight into [2^6, 2^7), and lowered
//    by d when the running maximum rises by d (rounded up), as everything that set it
//    has then shrunk by 2^-d; O follows both.  So the largest weight that still
//    counts (rows of zeros do not) is held as 2^6 or more, and f16 holds every weight
//    to 2^-31 of it (half its smallest step of 2^-24); w is split into two f16 (hi + lo,
//    22 bits), so that its rounding stays far below the output's.  (V as bf16, whose
//    range needs no E, costs 96 more integer instructions of 620 per tile.)
//  * The running maximum is raised only when a score exceeds it by 2^8 (one
//    vote per tile instead of a reduction and a rescale).
//  * A unit split across warps is merged in shared memory by its CTA; only one
//    split across CTAs leaves partials, one per CTA, for fp8_combine_kernel.
//    (With a partial per warp the merge of a 131,072-token context, 282 partials
//    per unit, took longer than the attention.)
//  * Where a warp goes from one unit to the next, the unit follows by a step (no
//    search), and its queries were prefetched when its first tile was issued; the
//    partition counts the change as two tiles (unit_place): short contexts, many
//    units per warp, are bound by these changes.
//
// Measured (8 KV heads of 128, pages of 16 or 32; 6.80 TB/s copy): 128 sequences of
// 1,024 to 32,768 tokens, 4.5 GB, 724 us, 91% of the copy bandwidth; one context of
// 131,072 among 23 of some hundred, 290 MB, 70 us (61%; about 20 us are launch, tile
// space, the rings' first fill and the merges); one sequence of 1,500, 15.6 us,
// latency.  64 sequences of 8,192 tokens: 8 heads of 128, groups of 4, 190 us, of 16,
// 275 (two MMA columns to a tile); heads of 64, 138 and 170; 8 heads of 256, groups of 4
// and 8, 357 and 367; 4 of 256, groups of 16, 364 (cut in two, every page read twice).  Twelve warps per CTA with three stages; with the earlier partition (727
// and 90 us) sixteen with two took 800 and 85 us, ten with four 848 and 95.
#include "gather_common.cuh"
#include "serving.h"
#include "tc05.cuh"

namespace sa {

namespace {

constexpr float kRaiseLog2 = 8.0f;
constexpr int kMinWarps = 8;  // per CTA, where there are few tiles
// Of a held value weight: the largest before its head's E is raised (f16 ends at 2^16),
// and the exponent that the tile's largest then gets.
constexpr float kWeightMax = 32768.0f;
constexpr uint32_t kWeightExp = 6;
constexpr uint32_t kDownExpMax = 252;  // biased exponent of 2^-E: its inverse is a normal number too

template <int D, int NT>
struct FGeo {
  // warps per CTA (one CTA per SM) that the registers and the rings allow
  static constexpr int kWarps = D == 64 ? 16 : (D == 128 && NT == 1) ? 12 : 8;
  static constexpr int kStages = D == 64 ? (NT == 1 ? 5 : 4) : D == 128 ? (NT == 1 ? 3 : 4) : 2;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kKs = D / 16;       // contraction steps of S, 16-dim tiles of O
  static constexpr int kSlabs = D == 256 ? 2 : 1;          // TMA boxes of a K or V tile
  static constexpr int kBoxCols = D == 64 ? 64 : 128;
  static constexpr int kTileBytes = 16 * D;                // K, and V
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kHeads = 8 * NT;
  // per CTA: rings | partials | stage scales | barriers | merge lists | tile prefix
  // a partial: o (rows 16 bytes apart in the banks, so that the lanes' stores to
  // different heads do not meet), then m and l per head
  static constexpr int kPartRow = D + 4;
  static constexpr int kPartMl = kHeads * kPartRow;
  static constexpr int kPartFloats = kPartMl + 2 * kHeads;
  static constexpr int kOffPart = kWarps * kStages * kStageBytes;
  static constexpr int kOffScale = kOffPart + kWarps * kPartFloats * 4;
  static constexpr int kOffBar = kOffScale + kWarps * kStages * 32;
  static constexpr int kOffList = kOffBar + kWarps * kStages * 8;
  static constexpr int kOffPref = kOffList + (2 * kWarps + 2) * 16;
  static_assert(kStages * kStageBytes >= kPartFloats * 4, "the last partial reuses the ring");
};

// Two E4M3 codes (low 16 bits) -> two f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two));
  return h;
}

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float e8m0_f32(uint32_t byte) {
  const uint32_t odd = ((byte + 1) & 255u) < 2u ? 0x400000u : 0u;  // 0: 2^-127, subnormal; 255: NaN
  return __uint_as_float((byte << 23) | odd);
}

// (tile indices and places stay below 2^31, checked on the host)
//
// Ranges are cut in a space that gives every unit kFp8UnitCost places before its
// tiles, for what a warp does at a change of unit: tile i of a unit at `place` lies
// at place + kFp8UnitCost + i, and a warp takes the tiles of its R places.  (One
// context of 131,072 among 23 short ones: 70 us, 79 with a cost of 0; 400 contexts of
// 350: 73.4, 72.6 with 0, 75.9 with 8.)
__device__ __forceinline__ int32_t unit_place(const GatherArgs& a, int32_t seq_tiles_before, int32_t b, int32_t grp,
                                              int32_t tu) {
  return static_cast<int32_t>(a.Hkv) * (seq_tiles_before + kFp8UnitCost * b) + grp * (tu + kFp8UnitCost);
}

// Tiles that lie before place x.
__device__ __forceinline__ int32_t tiles_before(const GatherArgs& a, const int32_t* pref, int32_t x) {
  int lo = 0, hi = static_cast<int>(a.B);  // largest b whose first place is <= x
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (unit_place(a, pref[mid], mid, 0, 0) <= x) lo = mid;
    else hi = mid;
  }
  const int32_t heads = static_cast<int32_t>(a.Hkv);
  const int32_t tb = pref[lo + 1] - pref[lo], y = x - unit_place(a, pref[lo], lo, 0, 0);
  const int32_t q = static_cast<int32_t>(static_cast<uint32_t>(y) / static_cast<uint32_t>(tb + kFp8UnitCost));
  const int32_t grp = min(q, heads);  // (heads: past the last sequence)
  const int32_t z = y - grp * (tb + kFp8UnitCost) - kFp8UnitCost;
  return heads * pref[lo] + grp * tb + (grp < heads && z > 0 ? z : 0);
}

struct Unit {
  int32_t off, tu;      // first tile, tiles
  int32_t b, grp;       // sequence, head group
  int32_t ctx;
};

// The unit of tile t.  pref[b]: tiles of the sequences before b, per group.
__device__ __forceinline__ Unit unit_at(const GatherArgs& a, const int32_t* pref, int32_t t) {
  int lo = 0, hi = static_cast<int>(a.B);  // largest b with Hkv * pref[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int32_t>(a.Hkv) * pref[mid] <= t) lo = mid;
    else hi = mid;
  }
  Unit r;
  const int32_t tb = pref[lo + 1] - pref[lo];
  const int32_t base = static_cast<int32_t>(a.Hkv) * pref[lo];
  r.b = lo;
  r.grp = static_cast<int32_t>(static_cast<uint32_t>(t - base) / static_cast<uint32_t>(tb));
  r.off = base + r.grp * tb;
  r.tu = tb;
  r.ctx = __ldg(a.ctx_len + lo);
  return r;
}

// The unit after u (there is one: the caller's range goes on).
__device__ __forceinline__ void next_unit(const GatherArgs& a, const int32_t* pref, Unit& u) {
  u.off += u.tu;
  if (++u.grp < static_cast<int32_t>(a.Hkv)) return;
  u.grp = 0;
  do ++u.b;
  while (pref[u.b + 1] == pref[u.b]);
  u.tu = pref[u.b + 1] - pref[u.b];
  u.ctx = __ldg(a.ctx_len + u.b);
}

// A unit's partial result in shared memory: where, whose, and what of it it covers.
struct Part {
  int32_t unit_off;            // first tile of the unit
  int32_t b, grp;              // sequence, head group
  int32_t where;               // float offset of o from the shared-memory base (-1: none)
};

// kScores: the scores and the rows' statistics are kept for the tokens' weights (a form
// of its own, so that the plain decode keeps its registers).
template <typename T, int D, int NT, bool kScores>
__global__ void __launch_bounds__(FGeo<D, NT>::kThreads, 1)
    fp8_pages_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                     const GatherArgs a, int64_t pool_heads, int64_t min_range) {
  using G = FGeo<D, NT>;
  constexpr int NW = G::kWarps, S = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  int32_t* pref = reinterpret_cast<int32_t*>(sm + G::kOffPref);  // [B + 1]
  Part* parts = reinterpret_cast<Part*>(sm + G::kOffList);       // [2 * NW]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int hpu = static_cast<int>(a.hpu);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + G::kOffBar) + warp * S;
  if (threadIdx.x == 0) {
    tc05::prefetch_tmap(&tk);
    tc05::prefetch_tmap(&tv);
  }
  if (lane < S) mbar_init(&full[lane], 1);
  if (lane < 2) parts[2 * warp + lane].where = -1;
  fence_mbar_init();
  pdl_launch_dependents();  // the combine kernel may start launching (it waits for this grid)

  // ---- tile space (every CTA computes it) ----------------------------------------------
  for (int64_t b = threadIdx.x; b < a.B; b += blockDim.x) {
    const int64_t ctx = a.ctx_len[b];
    const bool ok = ctx >= 1 && ctx <= a.max_pages * a.page_tokens;
    if (!ok && blockIdx.x == 0 && a.err_word) atomicOr(a.err_word, SA_ERRBIT_PAGE);
    pref[b + 1] = ok ? static_cast<int32_t>((ctx + 15) / 16) : 0;
  }
  __syncthreads();
  if (warp == 0) {
    int32_t carry = 0;
    if (lane == 0) pref[0] = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += 32) {
      const int64_t b = b0 + lane;
      int32_t v = (b < a.B) ? pref[b + 1] : 0;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int32_t n = __shfl_up_sync(0xffffffffu, v, sh);
        if (lane >= sh) v += n;
      }
      if (b < a.B) pref[b + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  const int32_t total = unit_place(a, pref[a.B], static_cast<int32_t>(a.B), 0, 0);
  const int64_t gw_total = static_cast<int64_t>(gridDim.x) * NW;
  int64_t R = (total + gw_total - 1) / gw_total;
  int nw = NW;  // warps that get a range
  if (R < min_range) {
    // few tiles: more CTAs with fewer warps each (one context of 1,500: 15.6 us, with
    // all twelve 16.5, with four 15.8)
    R = min_range;
    nw = static_cast<int>(min(static_cast<int64_t>(NW), max((total + gridDim.x * R - 1) / (gridDim.x * R), int64_t(kMinWarps))));
  }
  if (blockIdx.x == 0) {
    // the combine kernel sees the CTAs as its "warps"
    for (int64_t b = threadIdx.x; b <= a.B; b += blockDim.x) a.pref_out[b] = pref[b];
    if (threadIdx.x == 0) a.meta[0] = R * nw;
    // sequences without tiles still need a (zero) output
    for (int b = warp; b < a.B; b += NW)
      if (pref[b + 1] == pref[b])
        for (int64_t e = lane; e < a.Hq * D / 2; e += 32)
          reinterpret_cast<uint32_t*>(a.y)[b * (a.Hq * D / 2) + e] = 0u;
  }
  const int64_t c_first = static_cast<int64_t>(blockIdx.x) * nw * R;
  if (c_first >= total) return;  // the whole CTA
  const int32_t c_place = static_cast<int32_t>(c_first), c_end = c_place + nw * static_cast<int32_t>(R);
  int32_t t_begin, t_end;
  {
    const int32_t t = tiles_before(a, pref, c_place + min(warp + (lane & 1), nw) * static_cast<int32_t>(R));
    t_begin = __shfl_sync(0xffffffffu, t, 0);
    t_end = __shfl_sync(0xffffffffu, t, 1);
  }

  if (t_begin < t_end) {
    uint8_t* ring = sm + warp * S * G::kStageBytes;
    uint8_t* scales = sm + G::kOffScale + warp * S * 32;
    const uint32_t ring_s = smem_u32(ring), scales_s = smem_u32(scales);
    const uint32_t pt = static_cast<uint32_t>(a.page_tokens);
    const int64_t page_bytes = a.page_tokens * (D + 1);
    const uint32_t sub = static_cast<uint32_t>(a.Hkv / pool_heads);
    const uint8_t* kp = static_cast<const uint8_t*>(a.k);
    const uint8_t* vp = static_cast<const uint8_t*>(a.v);

    // The issue side: a tile's table entry is loaded a step before its copies.
    struct Ahead {
      int32_t page, slot, head;
    };
    Unit nxt = unit_at(a, pref, t_begin);
    const int32_t* table;             // next entry to look at
    int32_t n_slot, n_head, n_left;   // slot in its page, head, tiles of the unit to go
    auto enter = [&](int32_t t) {
      const uint32_t tok = static_cast<uint32_t>(t - nxt.off) * 16u, pi = tok / pt;
      n_slot = static_cast<int32_t>(tok - pi * pt);
      n_head = static_cast<int32_t>(static_cast<uint32_t>(nxt.grp) / sub);
      n_left = nxt.off + nxt.tu - t;
      table = a.block_table + nxt.b * a.max_pages + pi;
    };
    enter(t_begin);
    auto look = [&](int32_t t) {
      if (n_left == 0) {
        next_unit(a, pref, nxt);
        enter(t);
        // its queries, wanted in S tiles' time
        const T* qr = static_cast<const T*>(a.q) + (nxt.b * a.Hq + nxt.grp * a.hpu) * D;
        for (int x = lane * 64; x < hpu * D; x += 32 * 64)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(qr + x));
      }
      const Ahead h{__ldg(table), n_slot, n_head};
      n_slot += 16;
      if (n_slot == static_cast<int32_t>(pt)) {
        n_slot = 0;
        ++table;
      }
      --n_left;
      return h;
    };
    uint32_t good = 0;  // bit per stage: its page exists
    auto issue = [&](int stage, const Ahead& h) {
      const bool ok = h.page >= 0 && h.page < a.num_pages;
      good = ok ? good | (1u << stage) : good & ~(1u << stage);
      fence_proxy_async_smem();  // this warp's reads of the stage precede the refill
      __syncwarp();
      if (lane == 0) {
        uint64_t* bar = &full[stage];
        if (ok) {
          const int64_t ph = h.page * pool_heads + h.head;
          uint8_t* dst = ring + stage * G::kStageBytes;
          mbar_arrive_expect_tx(bar, G::kStageBytes + 32);
#pragma unroll
          for (int s = 0; s < G::kSlabs; ++s) {
            tc05::tma_load3(dst + s * 2048, &tk, s * 128, h.slot, static_cast<int>(ph), bar);
            tc05::tma_load3(dst + G::kTileBytes + s * 2048, &tv, s * 128, h.slot, static_cast<int>(ph), bar);
          }
          const int64_t so = ph * page_bytes + a.page_tokens * D + h.slot;
          bulk_g2s(scales + stage * 32, kp + so, 16, bar);
          bulk_g2s(scales + stage * 32 + 16, vp + so, 16, bar);
        } else {
          if (a.err_word) atomicOr(a.err_word, SA_ERRBIT_PAGE);
          mbar_arrive(bar);
        }
      }
    };
    Unit cur = nxt;
    const int32_t first_off = cur.off;
    {
      Ahead h[S];
#pragma unroll
      for (int q = 0; q < S; ++q)
        if (t_begin + q < t_end) h[q] = look(t_begin + q);
#pragma unroll
      for (int q = 0; q < S; ++q)
        if (t_begin + q < t_end) issue(q, h[q]);
    }
    Ahead next{-1, 0, 0};
    if (t_begin + S < t_end) next = look(t_begin + S);

    // ---- per-unit state -------------------------------------------------------------------
    uint32_t qf[NT][G::kKs][2];
    float mult[NT][2];                 // per head: scale * log2(e) * the query's power of two
    float o[G::kKs][NT][4];
    float m_run[NT][2], l_run[NT][2];  // heads 2 tig, 2 tig + 1; l: this lane's tokens
    float down_v[NT][2];               // 2^-E of the value weights (0: none yet)
    int left = 0;                      // tokens of the unit from this tile on
    bool fresh = true;                 // a head has no maximum or no E yet

    // Dims of contraction step kk that this lane holds: 4 of them, consecutive.
    auto q_dim = [&](int kk) {
      return D == 64 ? 16 * tig + 4 * kk : 128 * (kk / 8) + 32 * tig + 4 * (kk % 8);
    };
    auto start_unit = [&]() {
      const T* qp = static_cast<const T*>(a.q);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int hh = nt * 8 + gid;
        const bool live = hh < hpu;
        const T* qr = qp + (cur.b * a.Hq + cur.grp * a.hpu + (live ? hh : 0)) * D;
        // this lane's dims as they lie: two contraction steps per load
#pragma unroll
        for (int kk = 0; kk < G::kKs; kk += 2) {
          const uint4 r = __ldg(reinterpret_cast<const uint4*>(qr + q_dim(kk)));
          qf[nt][kk][0] = r.x;
          qf[nt][kk][1] = r.y;
          qf[nt][kk + 1][0] = r.z;
          qf[nt][kk + 1][1] = r.w;
        }
        float amax = 0.f;
#pragma unroll
        for (int kk = 0; kk < G::kKs; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const T* x = reinterpret_cast<const T*>(&qf[nt][kk][e]);
            amax = fmaxf(amax, fmaxf(fabsf(to_f32<T>(x[0])), fabsf(to_f32<T>(x[1]))));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // a power of two that puts amax into [2^14, 2^15); kept inside fp32's exponents
        int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14;
        if (amax == 0.f || !(amax <= 3.0e38f)) ex = 0;
        ex = max(ex, -126);
        const float down = live ? __uint_as_float(static_cast<uint32_t>(127 - ex) << 23) : 0.f;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
        for (int kk = 0; kk < G::kKs; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const T* x = reinterpret_cast<const T*>(&qf[nt][kk][e]);
            const float lo = to_f32<T>(x[0]), hi = to_f32<T>(x[1]);
            qf[nt][kk][e] = live ? pack2<__half>(lo * down, hi * down) : 0u;
          }
        mult[nt][0] = a.scale_log2 * __shfl_sync(0xffffffffu, up, 8 * tig);
        mult[nt][1] = a.scale_log2 * __shfl_sync(0xffffffffu, up, 8 * tig + 4);
        m_run[nt][0] = m_run[nt][1] = SA_NEG_INF;
        l_run[nt][0] = l_run[nt][1] = 0.f;
        down_v[nt][0] = down_v[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < G::kKs; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
      }
      fresh = true;
    };
    // This lane's dims of O tile mt: 2 of them, consecutive.
    auto dim_of = [&](int mt) {
      return D == 64 ? 8 * gid + 2 * mt : (mt / 8) * 128 + 16 * gid + 2 * (mt % 8);
    };
    // End of a unit's tiles in this warp: y when the whole unit lies in this
    // warp's range, else a partial in shared memory (the first unit's in the
    // area for partials, the last one's, at the end, over the ring).
    auto flush_unit = [&]() {
      const bool whole = cur.off >= t_begin && cur.off + cur.tu <= t_end;
      const int second = cur.off != first_off;
      float* po = second ? reinterpret_cast<float*>(ring)
                         : reinterpret_cast<float*>(sm + G::kOffPart) + warp * G::kPartFloats;
      const int32_t head0 = static_cast<int32_t>(cur.b * a.Hq + cur.grp * a.hpu);
      if (!whole && lane == 0)
        parts[2 * warp + second] = Part{cur.off, cur.b, cur.grp, static_cast<int32_t>(po - reinterpret_cast<float*>(sm))};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float l = l_run[nt][j];
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
          const int hh = nt * 8 + 2 * tig + j;
          if (hh >= hpu) continue;
          const float up_v = down_v[nt][j] == 0.f ? 1.0f : 1.0f / down_v[nt][j];  // 2^E
          if (whole) {
            if (kScores && gid == 0) a.stats[head0 + hh] = row_stat(m_run[nt][j], l);
            const float inv = (m_run[nt][j] == SA_NEG_INF || l == 0.f) ? 0.f : up_v / l;
            T* yp = static_cast<T*>(a.y) + static_cast<int64_t>(head0 + hh) * D;
#pragma unroll
            for (int mt = 0; mt < G::kKs; mt += 4) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack2<T>(o[mt + i][nt][j] * inv, o[mt + i][nt][2 + j] * inv);
              *reinterpret_cast<uint4*>(yp + dim_of(mt)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int mt = 0; mt < G::kKs; mt += 2)
              *reinterpret_cast<float4*>(po + hh * G::kPartRow + dim_of(mt)) =
                  make_float4(o[mt][nt][j] * up_v, o[mt][nt][2 + j] * up_v,
                              o[mt + 1][nt][j] * up_v, o[mt + 1][nt][2 + j] * up_v);
            if (gid == 0)
              *reinterpret_cast<float2*>(po + G::kPartMl + 2 * hh) = make_float2(m_run[nt][j], l);
          }
        }
    };

    // ---- main loop -----------------------------------------------------------------------------
    start_unit();
    left = cur.ctx - (t_begin - cur.off) * 16;
    bool timed_out = false;
    int stage = 0;
    uint32_t parity = 0;
#pragma unroll 1
    for (int32_t t = t_begin; t < t_end; ++t, left -= 16) {
      if (left <= 0) {
        flush_unit();
        next_unit(a, pref, cur);
        left = cur.ctx;
        start_unit();
      }
      if (!mbar_wait(&full[stage], parity)) timed_out = true;
      const bool have = (good >> stage) & 1u;
      const bool lo_ok = have && gid < left, hi_ok = have && gid + 8 < left;
      const uint32_t kt = ring_s + stage * G::kStageBytes, vt = kt + G::kTileBytes;
      const uint32_t sc = scales_s + stage * 32 + gid;
      auto lds16 = [](uint32_t addr) {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
        return v;
      };
      auto lds1 = [](uint32_t addr) {
        uint32_t v;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
        return v;
      };
      const uint32_t kb0 = lds1(sc), kb1 = lds1(sc + 8), vb0 = lds1(sc + 16), vb1 = lds1(sc + 24);

      // S^T = K . Q^T over the codes: rows gid and gid + 8, 16 dims per load
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint32_t at;
        if (D == 64) at = gid * 64 + ((tig ^ ((gid >> 1) & 3)) << 4);
        else at = (i >> 1) * 2048 + gid * 128 + (((2 * tig + (i & 1)) ^ gid) << 4);
        const uint4 r0 = lds16(kt + at), r1 = lds16(kt + at + (D == 64 ? 512 : 1024));
        const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a0 = e4m3x2_f16x2(w0[w]), a2 = e4m3x2_f16x2(w0[w] >> 16);
          const uint32_t a1 = e4m3x2_f16x2(w1[w]), a3 = e4m3x2_f16x2(w1[w] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816<__half>(s[nt], a0, a1, a2, a3, qf[nt][4 * i + w][0], qf[nt][4 * i + w][1]);
        }
      }
      // V's codes of tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9: this lane's dims
      uint32_t vx[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * tig + (i & 1);  // + 8: the same swizzle phase
        if (D == 64) {
          const uint32_t at = vt + ((i >> 1) * 8 + r) * 64 + (((gid >> 1) ^ ((r >> 1) & 3)) << 4) + (gid & 1) * 8;
          asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(vx[i][0]), "=r"(vx[i][1]) : "r"(at));
        } else {
#pragma unroll
          for (int b = 0; b < D / 128; ++b) {
            const uint4 v = lds16(vt + b * 2048 + ((i >> 1) * 8 + r) * 128 + ((gid ^ r) << 4));
            vx[i][4 * b] = v.x;
            vx[i][4 * b + 1] = v.y;
            vx[i][4 * b + 2] = v.z;
            vx[i][4 * b + 3] = v.w;
          }
        }
      }

      if (left < 16) {
        // slots past the context: their codes may be NaN, and 0 times NaN is NaN
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * tig + (i & 1) + (i >> 1) * 8 >= left)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) vx[i][w] = 0u;
      }

      // scores in log2 units less the running maximum; probabilities
      const float ks0 = e8m0_f32(kb0), ks1 = e8m0_f32(kb1);
      const float vs0 = lo_ok ? e8m0_f32(vb0) : 0.f, vs1 = hi_ok ? e8m0_f32(vb1) : 0.f;
      if (kScores) {
        // (a token's scores of 8 heads: sectors of 32 bytes, 8 tokens each)
        float* sp = a.scores + (cur.b * a.Hq + cur.grp * a.hpu + 2 * tig) * a.score_stride + (cur.ctx - left + gid);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (nt * 8 + 2 * tig + j >= hpu) continue;
            float* at = sp + (nt * 8 + j) * a.score_stride;
            if (lo_ok) at[0] = s[nt][j] * (ks0 * mult[nt][j]);
            if (hi_ok) at[8] = s[nt][2 + j] * (ks1 * mult[nt][j]);
          }
      }
      bool raise = fresh;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float mu0 = m_run[nt][0] == SA_NEG_INF ? 0.f : m_run[nt][0];
        const float mu1 = m_run[nt][1] == SA_NEG_INF ? 0.f : m_run[nt][1];
        s[nt][0] = lo_ok ? fmaf(s[nt][0], ks0 * mult[nt][0], -mu0) : SA_NEG_INF;
        s[nt][1] = lo_ok ? fmaf(s[nt][1], ks0 * mult[nt][1], -mu1) : SA_NEG_INF;
        s[nt][2] = hi_ok ? fmaf(s[nt][2], ks1 * mult[nt][0], -mu0) : SA_NEG_INF;
        s[nt][3] = hi_ok ? fmaf(s[nt][3], ks1 * mult[nt][1], -mu1) : SA_NEG_INF;
        // (a NaN score raises nothing and makes its row NaN through p)
        raise = raise || fmaxf(max3(s[nt][0], s[nt][1], s[nt][2]), s[nt][3]) > kRaiseLog2;
      }
      if (__any_sync(0xffffffffu, raise) && have) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float al[2];  // of O
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // a row of nothing but NaN scores still gets a finite maximum, so that its
            // NaN sum is not taken for an empty one
            const float mu = m_run[nt][j] == SA_NEG_INF ? 0.f : m_run[nt][j];
            const float x0 = s[nt][j], x1 = s[nt][2 + j];
            float tm = fmaxf(x0 == x0 ? x0 : 0.f, x1 == x1 ? x1 : 0.f);
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, sh));
            const float mn = fmaxf(m_run[nt][j], tm + mu);
            const float fall = mn == SA_NEG_INF ? 0.f : m_run[nt][j] - mn;  // (-inf: no maximum before)
            // E falls with the weights that set it
            const uint32_t dn = __float_as_uint(down_v[nt][j]);
            const uint32_t by = dn == 0u ? 0u : min(static_cast<uint32_t>(ceilf(fminf(-fall, 256.f))), kDownExpMax - (dn >> 23));
            down_v[nt][j] = __uint_as_float(dn + (by << 23));
            al[j] = ex2(fall + static_cast<float>(by));
            const float d = mn == SA_NEG_INF ? 0.f : mu - mn;
            s[nt][j] += d;
            s[nt][2 + j] += d;
            m_run[nt][j] = mn;
            l_run[nt][j] *= ex2(fall);
          }
#pragma unroll
          for (int mt = 0; mt < G::kKs; ++mt) {
            o[mt][nt][0] *= al[0];
            o[mt][nt][1] *= al[1];
            o[mt][nt][2] *= al[0];
            o[mt][nt][3] *= al[1];
          }
        }
      }
      float wt[NT][4];  // value weights p 2^(ev)
      raise = fresh;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float p0 = ex2(s[nt][0]), p1 = ex2(s[nt][1]), p2 = ex2(s[nt][2]), p3 = ex2(s[nt][3]);
        l_run[nt][0] += p0 + p2;
        l_run[nt][1] += p1 + p3;
        wt[nt][0] = p0 * vs0;
        wt[nt][1] = p1 * vs0;
        wt[nt][2] = p2 * vs1;
        wt[nt][3] = p3 * vs1;
        raise = raise || fmaxf(wt[nt][0], wt[nt][2]) * down_v[nt][0] > kWeightMax ||
                fmaxf(wt[nt][1], wt[nt][3]) * down_v[nt][1] > kWeightMax;
      }
      if (__any_sync(0xffffffffu, raise) && have) {
        fresh = false;
        // A row whose codes are all zero says nothing about the others, whatever its scale
        // (1 where paged_kv_write stored it): it has no weight here, but for a NaN scale.
        uint32_t some[4];  // per token of vx: the lanes that hold a code other than zero
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t any = 0;
#pragma unroll
          for (int w = 0; w < D / 32; ++w) any |= vx[i][w];
          some[i] = __ballot_sync(0xffffffffu, (any & 0x7f7f7f7fu) != 0u);
        }
        const uint32_t quad = 0x11111111u << (gid >> 1);  // the lanes with token gid, and gid + 8
        const bool none0 = vb0 != 255u && !((gid & 1 ? some[1] : some[0]) & quad);
        const bool none1 = vb1 != 255u && !((gid & 1 ? some[3] : some[2]) & quad);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float al[2];
          if (none0) wt[nt][0] = wt[nt][1] = 0.f;
          if (none1) wt[nt][2] = wt[nt][3] = 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float w = fmaxf(wt[nt][j], wt[nt][2 + j]);
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, sh));
            // 2^-E, raised only here; weights of nothing (all zero, or infinite) leave it
            const uint32_t ex = __float_as_uint(w) >> 23;
            float down = down_v[nt][j];
            if (w > 0.f && ex < 255) {
              const float want = __uint_as_float(min(254u + kWeightExp - ex, kDownExpMax) << 23);
              if (down == 0.f || want < down) down = want;
            }
            al[j] = down_v[nt][j] == 0.f ? 1.f : down * (1.0f / down_v[nt][j]);
            down_v[nt][j] = down;
            if (m_run[nt][j] == SA_NEG_INF || down == 0.f) fresh = true;
          }
#pragma unroll
          for (int mt = 0; mt < G::kKs; ++mt) {
            o[mt][nt][0] *= al[0];
            o[mt][nt][1] *= al[1];
            o[mt][nt][2] *= al[0];
            o[mt][nt][3] *= al[1];
          }
        }
      }
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float w0 = wt[nt][0] * down_v[nt][0], w1 = wt[nt][1] * down_v[nt][1];
        const float w2 = wt[nt][2] * down_v[nt][0], w3 = wt[nt][3] * down_v[nt][1];
        const __half2 h01 = __floats2half2_rn(w0, w1), h23 = __floats2half2_rn(w2, w3);
        const float2 f01 = __half22float2(h01), f23 = __half22float2(h23);
        ph[nt][0] = movm_t(*reinterpret_cast<const uint32_t*>(&h01));
        ph[nt][1] = movm_t(*reinterpret_cast<const uint32_t*>(&h23));
        pl[nt][0] = movm_t(pack2<__half>(w0 - f01.x, w1 - f01.y));
        pl[nt][1] = movm_t(pack2<__half>(w2 - f23.x, w3 - f23.y));
      }

      // the stage is free: its refill, S tiles on
      if (t + S < t_end) {
        const Ahead h = next;
        if (t + S + 1 < t_end) next = look(t + S + 1);
        issue(stage, h);
      }

      // O^T += V^T . P^T
      if (have) {
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          // (tokens 2 tig, 2 tig + 1), (2 tig + 8, 2 tig + 9): dims 4w, 4w + 1 | 4w + 2, 4w + 3
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362u : 0x5140u;
            const uint32_t z0 = __byte_perm(vx[0][w], vx[1][w], sel);
            const uint32_t z1 = __byte_perm(vx[2][w], vx[3][w], sel);
            const uint32_t a0 = e4m3x2_f16x2(z0), a1 = e4m3x2_f16x2(z0 >> 16);
            const uint32_t a2 = e4m3x2_f16x2(z1), a3 = e4m3x2_f16x2(z1 >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<__half>(o[2 * w + half][nt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
              mma16816<__half>(o[2 * w + half][nt], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
            }
          }
        }
      }
      if (++stage == S) {
        stage = 0;
        parity ^= 1u;
      }
    }
    if (timed_out && lane == 0 && a.err_word) atomicOr(a.err_word, SA_ERRBIT_TIMEOUT);
    __syncwarp();  // every lane has read the ring before a partial goes over it
    flush_unit();
  }
  __syncthreads();

  // ---- merge of the units that this CTA's warps share ----------------------------------------
  // The partials are in tile order, a unit's next to one another.  The units are
  // dealt out to the warps; where there are few, several warps share one.
  const float* fsm = reinterpret_cast<const float*>(sm);
  static_assert(2 * NW <= 32, "a lane per partial");
  Part mine{0, 0, 0, -1};
  if (lane < 2 * NW) mine = parts[lane];
  const uint32_t valid = __ballot_sync(0xffffffffu, mine.where >= 0);
  const uint32_t before = valid & ((1u << lane) - 1u);
  const int before_off = __shfl_sync(0xffffffffu, mine.unit_off, before ? 31 - __clz(before) : lane);
  uint32_t starts = __ballot_sync(0xffffffffu, mine.where >= 0 && (!before || before_off != mine.unit_off));
  const int units = __popc(starts), share = units > 0 && units < NW ? NW / units : 1;
  const int part0 = warp % share;
  for (int g = 0; starts; ++g) {
    const int e = __ffs(starts) - 1;
    starts &= starts - 1u;
    const int last = starts ? __ffs(starts) - 2 : 2 * NW - 1;
    if (g % (NW / share) != warp / share) continue;
    const Part p = parts[e];
    const int32_t tu = pref[p.b + 1] - pref[p.b], place = unit_place(a, pref[p.b], p.b, p.grp, tu);
    const bool whole = place + kFp8UnitCost >= c_place && place + kFp8UnitCost + tu <= c_end;
    const int64_t head0 = p.b * a.Hq + p.grp * a.hpu;
    // slot 0: the CTA's places begin inside the unit's (or with them), else 1
    const int64_t slot = (static_cast<int64_t>(blockIdx.x) * 2 + (c_place >= place ? 0 : 1)) * a.hpu;
    for (int x = part0 * 32 + lane; x < hpu * (D / 4); x += share * 32) {
      const int hh = x / (D / 4), d = (x - hh * (D / 4)) * 4;
      float M = SA_NEG_INF;
      for (int f = e; f <= last; ++f)
        if (parts[f].where >= 0) M = fmaxf(M, fsm[parts[f].where + G::kPartMl + 2 * hh]);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int f = e; f <= last; ++f) {
        const int w = parts[f].where;
        if (w < 0) continue;
        const float2 ml = *reinterpret_cast<const float2*>(fsm + w + G::kPartMl + 2 * hh);
        if (ml.x == SA_NEG_INF) continue;
        const float c = ex2(ml.x - M);
        const float4 v = *reinterpret_cast<const float4*>(fsm + w + hh * G::kPartRow + d);
        L += ml.y * c;
        acc.x = fmaf(v.x, c, acc.x);
        acc.y = fmaf(v.y, c, acc.y);
        acc.z = fmaf(v.z, c, acc.z);
        acc.w = fmaf(v.w, c, acc.w);
      }
      if (whole) {
        if (kScores && d == 0) a.stats[head0 + hh] = row_stat(M, L);
        const float inv = (M == SA_NEG_INF || L == 0.f) ? 0.f : 1.0f / L;
        *reinterpret_cast<uint2*>(static_cast<T*>(a.y) + (head0 + hh) * D + d) =
            make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot + hh) * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * (slot + hh)) = make_float2(M, L);
      }
    }
  }
}

// Merge of the units split across CTAs: y = sum_w o_w 2^(m_w - M) / sum_w l_w 2^(m_w - M)
// over the CTAs w that share the unit, in order.  A thread takes four dims of one
// head, so that a unit's partials are read by as many threads as it has, eight at a
// time: the loads' latency is all that this takes (a block per unit, 25 us for the 18
// partials of a 65,536-token context, was bound by walking over them).
template <typename T>
__global__ void __launch_bounds__(128) fp8_combine_kernel(const GatherArgs a) {
  pdl_wait();  // the attention kernel's partials and tile space
  const int D4 = static_cast<int>(a.D) / 4;
  const int64_t x = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  const int64_t row = x / D4;  // (unit, head of the group)
  const int d = static_cast<int>(x - row * D4) * 4;
  const int64_t u = row / a.hpu;
  if (u >= a.units) return;
  const int hh = static_cast<int>(row - u * a.hpu);
  const int32_t b = static_cast<int32_t>(u / a.Hkv), grp = static_cast<int32_t>(u - b * a.Hkv);
  const int64_t R = a.meta[0];  // places per CTA
  const int32_t lo = a.pref_out[b], tu = a.pref_out[b + 1] - lo;
  const int32_t place = unit_place(a, lo, b, grp, tu), first = place + kFp8UnitCost;
  if (tu == 0) return;
  const int64_t c0 = first / R, c1 = (first + tu - 1) / R;
  if (c0 == c1) return;  // written by the attention kernel
  auto part = [&](int64_t c) { return (c * 2 + (c * R >= place ? 0 : 1)) * a.hpu + hh; };
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  float M = SA_NEG_INF, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t c = c0; c <= c1; c += 8) {
    float2 e[8];
    float4 v[8];  // (not through the read-only path: written while this kernel may be resident)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = make_float2(SA_NEG_INF, 0.f);
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + i <= c1) {
        e[i] = ml[part(c + i)];
        v[i] = *reinterpret_cast<const float4*>(a.part_o + part(c + i) * a.D + d);
      }
    }
    float mn = M;
#pragma unroll
    for (int i = 0; i < 8; ++i) mn = fmaxf(mn, e[i].x);
    if (mn == SA_NEG_INF) continue;
    const float f0 = ex2(M - mn);
    L *= f0;
    acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
    M = mn;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (e[i].x == SA_NEG_INF) continue;
      const float f = ex2(e[i].x - mn);
      L += e[i].y * f;
      acc.x = fmaf(v[i].x, f, acc.x);
      acc.y = fmaf(v[i].y, f, acc.y);
      acc.z = fmaf(v[i].z, f, acc.z);
      acc.w = fmaf(v[i].w, f, acc.w);
    }
  }
  if (a.stats && d == 0) a.stats[b * a.Hq + grp * a.hpu + hh] = row_stat(M, L);
  const float inv = (M == SA_NEG_INF || L == 0.f) ? 0.f : 1.0f / L;
  *reinterpret_cast<uint2*>(static_cast<T*>(a.y) + (b * a.Hq + grp * a.hpu + hh) * a.D + d) =
      make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
}

// A pool as rows of codes: [pages * heads, page_tokens, D] bytes, the page stride with
// its scale bytes; boxes of 16 rows.
template <int D, int NT>
bool pool_map(CUtensorMap* m, const void* base, const GatherArgs& a, int64_t pool_heads) {
  using G = FGeo<D, NT>;
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.page_tokens),
                              static_cast<cuuint64_t>(a.num_pages * pool_heads)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.page_tokens * (D + 1))};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(G::kBoxCols), 16, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int NT, bool kScores>
int launch_s(const GatherArgs& a, int64_t pool_heads, int sms, cudaStream_t st) {
  using G = FGeo<D, NT>;
  CUtensorMap tk, tv;
  if (!pool_map<D, NT>(&tk, a.k, a, pool_heads) || !pool_map<D, NT>(&tv, a.v, a, pool_heads)) return -1;
  const size_t smem = 1024 + G::kOffPref + static_cast<size_t>(a.B + 1) * sizeof(int32_t);
  if (!allow_smem(reinterpret_cast<const void*>(fp8_pages_kernel<T, D, NT, kScores>))) return -1;
  mark_event(a.ev_before, st);
  // Ranges of at least two tiles: below that a warp's set-up and the merge of its
  // partial cost more than the tiles.
  fp8_pages_kernel<T, D, NT, kScores><<<static_cast<unsigned>(sms), G::kThreads, smem, st>>>(tk, tv, a, pool_heads, 2);
  if (cudaGetLastError() != cudaSuccess) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.units * a.hpu * (D / 4) + 127) / 128));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  mark_event(a.ev_after, st);
  return cudaLaunchKernelEx(&cfg, fp8_combine_kernel<T>, a) == cudaSuccess ? 0 : -1;
}

template <typename T, int D, int NT>
int launch_t(const GatherArgs& a, int64_t pool_heads, int sms, cudaStream_t st) {
  return a.scores ? launch_s<T, D, NT, true>(a, pool_heads, sms, st) : launch_s<T, D, NT, false>(a, pool_heads, sms, st);
}

template <typename T>
int launch_d(const GatherArgs& a, int64_t pool_heads, int sms, cudaStream_t st) {
  const bool two = a.hpu > 8;
  if (a.D == 64) return two ? launch_t<T, 64, 2>(a, pool_heads, sms, st) : launch_t<T, 64, 1>(a, pool_heads, sms, st);
  if (a.D == 128)
    return two ? launch_t<T, 128, 2>(a, pool_heads, sms, st) : launch_t<T, 128, 1>(a, pool_heads, sms, st);
  return launch_t<T, 256, 1>(a, pool_heads, sms, st);
}

}  // namespace

int64_t fp8_pages_max_heads(int D) { return D == 256 ? 8 : 16; }

int launch_fp8_pages(const GatherArgs& a, int64_t pool_heads, int dtype, int sms, cudaStream_t st) {
  if (dtype == SA_F16) return launch_d<__half>(a, pool_heads, sms, st);
  return launch_d<__nv_bfloat16>(a, pool_heads, sms, st);
}

}  // namespace sa
