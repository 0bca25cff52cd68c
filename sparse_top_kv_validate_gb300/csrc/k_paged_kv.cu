// k_paged_kv.cu -- packed K/V rows into their pages (rotated and quantised on
// the way) and a context back out of its pages.
//
// Quantised rows (SA_FP8_E4M3_PAGE): exponent e = the smallest with
// max|x| / 2^e <= 448 (E4M3's largest value), codes = nearest-even E4M3FN of
// x / 2^e.  448 = 1.75 * 2^8, so e follows from the bits of the largest
// magnitude, and x / 2^e is an exact product: a code depends on x alone.
//
// Both directions move every byte once and compute little: DRAM bandwidth is
// the bound for long spans, the chain start -> context -> table entry for a
// decode step's few rows.  The row data do not depend on that chain, so the
// write loads its rows first and resolves the places meanwhile.
//
// Measured (8 heads of 128, pages of 16): read-back of 65,536 rows (403 MB) to
// bf16 67.5 us, 6.0 TB/s, 88% of the copy bandwidth; write of 16,384 rotated fp16
// rows (100 MB) 24.7 us, 4.1 TB/s: two waves of blocks, each of which waits for
// its places and angles before its first row.  Steps of that: a sequence found by
// one load per lane instead of a search and three more loads, 31 -> 28; the angles'
// fractions by ordinary loads, -> 24.7; rows in flight in shared memory instead of
// registers (four blocks to an SM instead of two), keys and values in loops of
// their own, packed fp32 pairs, 50 -> 31.  A decode step's 128 rows take 6.2 us.
// Pages of plain elements, 65,536 rows: write 83 us (bf16, 537 MB, 6.5 TB/s; rotated
// 84; fp32 223, 4.8 TB/s), read-back, a warp per row, 255 us (2.1 TB/s; fp32 263).
#include <type_traits>

#include "rope.cuh"
#include "serving.h"

namespace sa {

namespace {

constexpr int kThreads = kRingThreads;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTok = 16;  // tokens per block

// Sequence b = the largest with start[b] <= r, its rows and context: found by the
// whole warp, 32 probes per step, the last step's bringing all of it at once (one
// load's latency up to 32 sequences).  b < 0 when the row is nobody's.
struct Owner {
  int b, first, next, ctx;
};
__device__ __forceinline__ Owner owner_of(const KvPagesArgs& a, int r, int lane) {
  int lo = 0, hi = a.B;
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < hi && __ldg(a.seq_start + at) <= r;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    if (n > 1) lo += (n - 1) * step;  // starts out of order: still below hi
    hi = min(lo + step, hi);
  }
  const int at = min(lo + lane, hi - 1);
  Owner o{at, __ldg(a.seq_start + at), __ldg(a.seq_start + at + 1), __ldg(a.ctx_len + at)};
  const int n = __popc(__ballot_sync(0xffffffffu, lo + lane < hi && o.first <= r)), from = max(n - 1, 0);
  o.b = __shfl_sync(0xffffffffu, o.b, from);
  o.first = __shfl_sync(0xffffffffu, o.first, from);
  o.next = __shfl_sync(0xffffffffu, o.next, from);
  o.ctx = __shfl_sync(0xffffffffu, o.ctx, from);
  if (!(o.first <= r && r < o.next)) o.b = -1;
  return o;
}

struct Place {
  int64_t page;  // page * Hkv, or -1 (nothing is done)
  int32_t slot, pos;
};

// Where packed row r of a sequence lives.  kWrite: the rows are the last of the
// context; else its first.
template <bool kWrite>
__device__ __forceinline__ Place place_in(const KvPagesArgs& a, const Owner& o, int r) {
  Place p{-1, 0, 0};
  const int64_t pos = (kWrite ? static_cast<int64_t>(o.ctx) - (o.next - o.first) : 0) + (r - o.first);
  int32_t page = -1;
  if (pos >= 0 && pos < o.ctx && o.ctx <= a.max_pages * a.page_tokens) {
    // a context is an int32: 32-bit division
    const uint32_t pi = static_cast<uint32_t>(pos) / static_cast<uint32_t>(a.page_tokens);
    page = __ldg(a.block_table + o.b * a.max_pages + pi);
    p.slot = static_cast<int32_t>(pos - static_cast<int64_t>(pi) * a.page_tokens);
    p.pos = static_cast<int32_t>(pos);
  }
  if (page < 0 || page >= a.num_pages) {
    if (a.err_word) atomicOr(a.err_word, SA_ERRBIT_PAGE);
    return p;
  }
  p.page = static_cast<int64_t>(page) * a.Hkv;
  return p;
}

// Row r's place, by a warp, uniform over it.
template <bool kWrite>
__device__ __forceinline__ Place place_of(const KvPagesArgs& a, int r, int lane) {
  const Owner o = a.seq_start ? owner_of(a, r, lane) : Owner{r, r, r + 1, __ldg(a.ctx_len + r)};
  return o.b < 0 ? Place{-1, 0, 0} : place_in<kWrite>(a, o, r);
}

// The places of a tile's `n` tokens, by the whole block.  A tile inside one
// sequence, as most tiles of long spans are, takes one search and then a lane
// per token; else each warp searches for its tokens.
template <bool kWrite>
__device__ __forceinline__ void tile_places(const KvPagesArgs& a, int t0, int n, Place* place) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (a.seq_start && n > 1) {
    const Owner o = owner_of(a, t0, lane);
    if (o.b >= 0 && t0 + n <= o.next) {
      if (threadIdx.x < n) place[threadIdx.x] = place_in<kWrite>(a, o, t0 + threadIdx.x);
      return;
    }
  }
  for (int k = warp; k < n; k += kWarps) {
    const Place p = place_of<kWrite>(a, t0 + k, lane);
    if (lane == 0) place[k] = p;
  }
}

// Block 0 looks the starts over.
__device__ __forceinline__ void check_starts(const KvPagesArgs& a) {
  if (blockIdx.x != 0 || !a.seq_start || !a.err_word) return;
  bool bad = false;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const int32_t s = __ldg(a.seq_start + b), e = __ldg(a.seq_start + b + 1);
    if (s < 0 || e < s || e > a.T) bad = true;
  }
  if (bad) atomicOr(a.err_word, SA_ERRBIT_SEQ);
}

// An FP8 page of head h: its rows of codes, then a scale byte per row.
__device__ __forceinline__ uint8_t* fp8_page(const KvPagesArgs& a, int w, int64_t page, int h) {
  return static_cast<uint8_t*>(a.pool[w]) + (page + h) * (a.page_tokens * (a.D + 1));
}

// Exponent of a row whose largest magnitude has the fp32 bits m (finite).
__device__ __forceinline__ int row_exponent(uint32_t m) {
  if (m == 0) return 0;
  const int e = static_cast<int>(m >> 23) - 127 - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -127);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

constexpr uint32_t kInfBits = 0x7f800000u;

// The largest magnitude; a NaN among them stays one.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

// A block's threads over a tile of tokens: the low half of them has the keys,
// the high half the values; a half's lane is (chunk c, token k, head hl) with
// the chunk fastest, and takes the heads hl, hl + hs, ...: chunk, token and
// tensor are a thread's own, and a step is an addition.
struct Seat {
  int w, c, k, hl, hs;
};
__device__ __forceinline__ Seat seat_of(int lanes, int tt) {
  const int u = threadIdx.x % (kThreads / 2), slot = u >> (__ffs(lanes) - 1);
  return Seat{threadIdx.x >= kThreads / 2, u & (lanes - 1), slot & (tt - 1),
              slot >> (__ffs(tt) - 1), (kThreads / 2) >> (__ffs(lanes * tt) - 1)};
}

// ---- write, 16 elements per lane ------------------------------------------------------
//
// D / 16 lanes hold a row (two 8-element pieces each, pieces_of), so a pair
// meets in one lane and the row's maximum in log2(D / 16) shuffles.  A block takes `tt` tokens; a thread's first rows are on their way
// (RowRing) before it knows where they go.
template <typename T, bool kFp8, bool kInter>
__global__ void __launch_bounds__(kThreads, 4)
    kv_write_kernel(const __grid_constant__ KvPagesArgs a, int tt) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Place place[kMaxTok];
  RowRing<T> ring(smem);
  float* cs_sm = reinterpret_cast<float*>(smem + RowRing<T>::kBytes);  // [tt][cos, sin][half]
  const int t0 = blockIdx.x * tt, n = min(tt, a.T - t0);
  const int lanes = a.D / 16;
  const Seat st = seat_of(lanes, tt);
  const int rot = a.has_rope ? a.rope.rotary_dim : 0, half = rot / 2;
  const Pieces pc = pieces_of<kInter>(st.c, a.D, st.w ? 0 : rot);
  const int d0 = pc.d[0], d1 = pc.d[1];
  const T* x = static_cast<const T*>(a.x[st.w]) + (t0 + st.k) * a.xs[st.w][0] +
               st.hl * a.xs[st.w][1];
  const int64_t xstep = st.hs * a.xs[st.w][1];
  const int steps = (a.Hkv + st.hs - 1) / st.hs;  // rows of a thread, the last one perhaps nobody's
  const int mine = st.k < n && st.hl < a.Hkv ? (a.Hkv - st.hl + st.hs - 1) / st.hs : 0;
  auto fetch = [&](int i) {
    if (i < mine) {
      ring.fetch(i, 0, x + d0, a.aligned);
      ring.fetch(i, 1, x + d1, a.aligned);
      x += xstep;
    }
    ring.commit();
  };
  TurnTables<kThreads> tables(a.rope);
  for (int i = 0; i < RowRing<T>::kRowsAhead; ++i) fetch(i);
  check_starts(a);
  tile_places<true>(a, t0, n, place);
  __syncthreads();
  if (rot) {
    tables.fill(a.rope, n, [&](int k) { return place[k].pos; }, cs_sm);
    __syncthreads();
  }
  const Place p = st.k < n ? place[st.k] : Place{-1, 0, 0};
  // the pieces in their page, and the way to the next head's
  const int64_t page = a.page_tokens * (kFp8 ? a.D + 1 : a.D * static_cast<int64_t>(sizeof(T)));
  const int64_t ystep = st.hs * page;
  uint8_t* base = static_cast<uint8_t*>(a.pool[st.w]) + (p.page + st.hl) * page;
  uint8_t* y = base + (static_cast<int64_t>(p.slot) * a.D + d0) * (kFp8 ? 1 : sizeof(T));
  uint8_t* scale = base + a.page_tokens * a.D + p.slot;
  const int dd = d1 - d0;
  bool any_bad = false;

  // A row's way; kTurn: a key to be rotated.  The same trips for the whole
  // block, and `put` uniform over a row's lanes: the shuffles stay within them.
  auto rows = [&](auto turn_tag) {
    constexpr bool kTurn = decltype(turn_tag)::value;
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      ring.arrived();
      const bool put = p.page >= 0 && i < mine;
      const Raw8<T> va = ring.get(i, 0), vb = ring.get(i, 1);
      float fa[8], fb[8];
      if (kFp8 || kTurn) {
        unpack8<T>(va, fa);
        unpack8<T>(vb, fb);
      }
      Piece pa = piece_from<kInter>(fa), pb = piece_from<kInter>(fb);
      if (kTurn) {
        rotate_pieces<kInter>(pa, pb, cs_sm + 2 * st.k * half, half, pc);
        piece_to<kInter>(pa, fa);
        piece_to<kInter>(pb, fb);
      }
      if (kFp8) {
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = max_abs(mx, fa[j], fb[j]);
        for (int o = lanes / 2; o > 0; o >>= 1)
          mx = max_abs(mx, __shfl_xor_sync(0xffffffffu, mx, o), 0.f);
        const uint32_t m = __float_as_uint(mx);
        const bool bad = m >= kInfBits;
        const int ex = row_exponent(m);
        const float mul = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        const F2 mul2 = f2(mul, mul);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          pa.x[j] = f2_mul(pa.x[j], mul2);
          pb.x[j] = f2_mul(pb.x[j], mul2);
        }
        piece_to<kInter>(pa, fa);
        piece_to<kInter>(pb, fb);
        uint2 wa = make_uint2(to_e4m3x4(fa[0], fa[1], fa[2], fa[3]),
                              to_e4m3x4(fa[4], fa[5], fa[6], fa[7]));
        uint2 wb = make_uint2(to_e4m3x4(fb[0], fb[1], fb[2], fb[3]),
                              to_e4m3x4(fb[4], fb[5], fb[6], fb[7]));
        if (put) {
          if (bad) wa = wb = make_uint2(0u, 0u);
          any_bad |= bad;
          *reinterpret_cast<uint2*>(y) = wa;
          *reinterpret_cast<uint2*>(y + dd) = wb;
          if (st.c == 0) *scale = static_cast<uint8_t>(bad ? 255 : ex + 127);
        }
      } else if (put) {
        T* o = reinterpret_cast<T*>(y);
        if (kTurn && pc.turn[0]) store8<T>(o, fa);
        else store_raw<T>(o, va);  // an exact copy
        if (kTurn && pc.turn[1]) store8<T>(o + dd, fb);
        else store_raw<T>(o + dd, vb);
      }
      y += ystep;
      scale += ystep;
      fetch(i + RowRing<T>::kRowsAhead);
    }
  };
  if (rot && !st.w) rows(std::true_type{});
  else rows(std::false_type{});
  if (any_bad && st.c == 0 && a.err_word) atomicOr(a.err_word, SA_ERRBIT_NONFINITE);
}

// ---- write, any D and rotary_dim: a warp per row, the row in shared memory ----------------

constexpr int kMaxD = 1024;

template <typename T, bool kFp8>
__global__ void __launch_bounds__(kThreads)
    kv_write_any_kernel(const __grid_constant__ KvPagesArgs a) {
  __shared__ float buf[kWarps][kMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* x = buf[warp];
  check_starts(a);
  const int64_t rows = static_cast<int64_t>(a.T) * 2 * a.Hkv;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + warp; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int t = static_cast<int>(r / (2 * a.Hkv));
    const int e = static_cast<int>(r - static_cast<int64_t>(t) * 2 * a.Hkv);
    const int w = e >= a.Hkv, h = e - (w ? a.Hkv : 0);
    const Place p = place_of<true>(a, t, lane);
    if (p.page < 0) continue;
    const T* src = static_cast<const T*>(a.x[w]) + t * a.xs[w][0] + h * a.xs[w][1];
    const int rot = (a.has_rope && !w) ? a.rope.rotary_dim : 0, half = rot / 2;
    uint32_t m = 0;
    for (int d = lane; d < a.D - half; d += 32) {
      if (d < half) {
        const int i0 = a.rope.interleaved ? 2 * d : d, i1 = a.rope.interleaved ? i0 + 1 : d + half;
        const float2 cs = rope_cos_sin(p.pos, a.rope.turns[d], a.rope.mscale);
        const float u = to_f32<T>(src[i0]), v = to_f32<T>(src[i1]);
        x[i0] = u * cs.x - v * cs.y;
        x[i1] = u * cs.y + v * cs.x;
        m = max(m, max(abs_bits(x[i0]), abs_bits(x[i1])));
      } else {
        const float u = to_f32<T>(src[d + half]);
        x[d + half] = u;
        m = max(m, abs_bits(u));
      }
    }
    __syncwarp();
    if (kFp8) {
      for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const bool bad = m >= kInfBits;
      const int ex = bad ? 0 : row_exponent(m);
      const float mul = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      uint8_t* page = fp8_page(a, w, p.page, h);
      for (int d = lane; d < a.D / 4; d += 32)
        *reinterpret_cast<uint32_t*>(page + static_cast<int64_t>(p.slot) * a.D + 4 * d) =
            bad ? 0u
                : to_e4m3x4(x[4 * d] * mul, x[4 * d + 1] * mul, x[4 * d + 2] * mul,
                            x[4 * d + 3] * mul);
      if (lane == 0) {
        page[a.page_tokens * a.D + p.slot] = static_cast<uint8_t>(bad ? 255 : ex + 127);
        if (bad && a.err_word) atomicOr(a.err_word, SA_ERRBIT_NONFINITE);
      }
    } else {
      T* y = static_cast<T*>(a.pool[w]) + ((p.page + h) * a.page_tokens + p.slot) * a.D;
      for (int d = lane; d < a.D; d += 32) y[d] = d < rot ? from_f32<T>(x[d]) : src[d];
    }
    __syncwarp();
  }
}

// ---- read ------------------------------------------------------------------------------------

// Eight codes times a scale -> eight elements.
template <typename T>
__device__ __forceinline__ void put8(T* y, const uint2& codes, float scale, int aligned) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h2;
    asm("{\n\t.reg .b16 t;\n\tmov.b16 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(h2)
        : "h"(static_cast<uint16_t>((i / 2 ? codes.y : codes.x) >> (16 * (i & 1)))));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    f2_split(f2_mul(f2(v.x, v.y), f2(scale, scale)), f[2 * i], f[2 * i + 1]);
  }
  if (aligned) {
    store8<T>(y, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = from_f32<T>(f[i]);
  }
}

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return byte == 0     ? 0x1p-127f
         : byte == 255 ? __int_as_float(0x7fffffff)
                       : __uint_as_float(byte << 23);
}

// FP8 pages -> rows: 16 codes per lane, eight of each half of the row so that an
// access of a row's lanes is one run; kBatch rows in flight per thread; a block
// takes `tt` rows of every head.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv_read_fp8_kernel(const __grid_constant__ KvPagesArgs a, int tt) {
  constexpr int kBatch = 4;
  __shared__ Place place[kMaxTok];
  const int t0 = blockIdx.x * tt, n = min(tt, a.T - t0);
  const Seat st = seat_of(a.D / 16, tt);
  check_starts(a);
  tile_places<false>(a, t0, n, place);
  __syncthreads();
  const Place p = st.k < n ? place[st.k] : Place{-1, 0, 0};
  if (p.page < 0) return;
  const int64_t page = a.page_tokens * (a.D + 1), xstep = st.hs * page;
  const uint8_t* x = static_cast<const uint8_t*>(a.pool[st.w]) + (p.page + st.hl) * page;
  const int64_t row = static_cast<int64_t>(p.slot) * a.D + 8 * st.c;
  const int64_t scale = a.page_tokens * a.D + p.slot;
  T* y = static_cast<T*>(a.x[st.w]) + (t0 + st.k) * a.xs[st.w][0] + st.hl * a.xs[st.w][1] +
         8 * st.c;
  const int64_t ystep = st.hs * a.xs[st.w][1];
  for (int h = st.hl; h < a.Hkv; h += kBatch * st.hs) {
    uint2 codes[kBatch][2];
    uint32_t sb[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (h + i * st.hs < a.Hkv) {
        codes[i][0] = __ldg(reinterpret_cast<const uint2*>(x + i * xstep + row));
        codes[i][1] = __ldg(reinterpret_cast<const uint2*>(x + i * xstep + row + a.D / 2));
        sb[i] = __ldg(x + i * xstep + scale);
      }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (h + i * st.hs < a.Hkv) {
        const float m = e8m0(sb[i]);
        put8<T>(y + i * ystep, codes[i][0], m, a.aligned);
        put8<T>(y + i * ystep + a.D / 2, codes[i][1], m, a.aligned);
      }
    x += kBatch * xstep;
    y += kBatch * ystep;
  }
}

// Pages of plain elements -> rows: a warp per row.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv_read_plain_kernel(const __grid_constant__ KvPagesArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  check_starts(a);
  const int64_t rows = static_cast<int64_t>(a.T) * 2 * a.Hkv;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + warp; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int t = static_cast<int>(r / (2 * a.Hkv));
    const int e = static_cast<int>(r - static_cast<int64_t>(t) * 2 * a.Hkv);
    const int w = e >= a.Hkv, h = e - (w ? a.Hkv : 0);
    const Place p = place_of<false>(a, t, lane);
    if (p.page < 0) continue;
    const T* x = static_cast<const T*>(a.pool[w]) + ((p.page + h) * a.page_tokens + p.slot) * a.D;
    T* y = static_cast<T*>(a.x[w]) + t * a.xs[w][0] + h * a.xs[w][1];
    constexpr int kV = 16 / sizeof(T);
    if (a.aligned && a.D % kV == 0) {
      for (int d = lane; d < a.D / kV; d += 32)
        reinterpret_cast<uint4*>(y)[d] = __ldg(reinterpret_cast<const uint4*>(x) + d);
    } else {
      for (int d = lane; d < a.D; d += 32) y[d] = x[d];
    }
  }
}

// Tokens per block: up to what a half's threads hold side by side (16 for D 128:
// 30.8 us for 16,384 tokens against 32.9 with 8 and 45 with 4, whose set-up is paid
// more often), as long as the blocks cover the SMs twice (a decode step's 128 tokens
// in 128 blocks, 6.2 us).
int tokens_per_block(const KvPagesArgs& a) {
  const int most = kThreads / 2 / (a.D / 16), sms = sm_count();
  int tt = 1;
  while (2 * tt <= kMaxTok && 2 * tt <= most && a.T / (2 * tt) >= 2 * sms) tt *= 2;
  return tt;
}

unsigned row_blocks(const KvPagesArgs& a) {
  const int64_t blocks = (static_cast<int64_t>(a.T) * 2 * a.Hkv + kWarps - 1) / kWarps;
  const int64_t most = 16 * static_cast<int64_t>(sm_count());
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <typename T>
int write_t(const KvPagesArgs& a, cudaStream_t st) {
  const int rot = a.has_rope ? a.rope.rotary_dim : 0;
  const int L = a.D / 16;
  const bool chunks = a.D % 16 == 0 && rot % 16 == 0 && L <= 32 && (L & (L - 1)) == 0;
  if (chunks && (a.fp8 || a.aligned)) {
    const int tt = tokens_per_block(a);
    const unsigned grid = static_cast<unsigned>((a.T + tt - 1) / tt);
    const size_t smem = RowRing<T>::kBytes + static_cast<size_t>(tt) * rot * sizeof(float);
    const bool inter = a.has_rope && a.rope.interleaved;
    auto kernel = a.fp8 ? (inter ? kv_write_kernel<T, true, true> : kv_write_kernel<T, true, false>)
                        : (inter ? kv_write_kernel<T, false, true> : kv_write_kernel<T, false, false>);
    kernel<<<grid, kThreads, smem, st>>>(a, tt);
  } else if (a.fp8) {
    kv_write_any_kernel<T, true><<<row_blocks(a), kThreads, 0, st>>>(a);
  } else {
    kv_write_any_kernel<T, false><<<row_blocks(a), kThreads, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <typename T>
int read_t(const KvPagesArgs& a, cudaStream_t st) {
  if (a.fp8) {
    const int tt = tokens_per_block(a);
    const unsigned grid = static_cast<unsigned>((a.T + tt - 1) / tt);
    kv_read_fp8_kernel<T><<<grid, kThreads, 0, st>>>(a, tt);
  } else {
    kv_read_plain_kernel<T><<<row_blocks(a), kThreads, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_kv_write(const KvPagesArgs& a, int dtype, cudaStream_t st) {
  if (a.T == 0) return 0;
  if (dtype == SA_F32) return write_t<float>(a, st);
  if (dtype == SA_F16) return write_t<__half>(a, st);
  return write_t<__nv_bfloat16>(a, st);
}

int launch_kv_read(const KvPagesArgs& a, int dtype, cudaStream_t st) {
  if (a.T == 0) return 0;
  if (dtype == SA_F32) return read_t<float>(a, st);
  if (dtype == SA_F16) return read_t<__half>(a, st);
  return read_t<__nv_bfloat16>(a, st);
}

}  // namespace sa
