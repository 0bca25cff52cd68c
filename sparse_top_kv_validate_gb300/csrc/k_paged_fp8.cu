// k_paged_fp8.cu -- decode attention over FP8 pages (one new query per sequence).
//
// Per query head: s_t = scale 2^(ek_t) (q . ck_t) over the codes ck_t of key t
// and its exponent ek_t, y = sum_t softmax(s)_t 2^(ev_t) cv_t.  Each page is
// read once and nothing else is large, so DRAM bandwidth is the bound; what
// must not get in its way is the decoding of two codes per byte pair read.
//
// The work is laid out as in the stream kernel (k_stream.cu): every (sequence,
// KV head)'s context cut into 16-token tiles laid end to end, one contiguous
// range of tiles per warp of a persistent grid, whatever the contexts; a unit
// split across warps leaves partials for stream_combine_kernel.
//
//  * A tile's K and V codes go from DRAM straight to registers, 16 bytes per
//    lane and load: with keys as M of S^T = K Q^T and dims as M of
//    O^T = V^T P^T, the 16 codes a lane loads are exactly values of its own
//    MMA fragments once the contraction index (for S) and the output dims (for
//    O) are numbered to fit.  So no shared memory, barrier or ldmatrix is
//    needed; the next tile's loads are issued as soon as a register is free
//    and stay in flight during the arithmetic.
//  * K: e4m3 -> f16 is exact (one conversion per pair), and q enters as f16
//    after a power of two per head brings its largest element to [2^14, 2^15),
//    so bf16 and f16 queries lose nothing that fp32 sums would keep (an
//    element 2^-39 below the row's largest is rounded).  The key's scale and
//    the head's power of two multiply the fp32 score.
//  * V: codes become bf16 by moving their bits (exponent and mantissa shifted
//    into place give value * 2^-120; one multiplication by 2^120, exact).  The
//    value's scale is folded into the probability, p 2^(ev), which bf16's range
//    always holds; it is split into two bf16 (hi + lo, 16 bits), so that the
//    probability's rounding stays far below the output's.
//  * The running maximum is raised only when a score exceeds it by 2^8 (one
//    vote per tile instead of a reduction and a rescale).
#include "gather_common.cuh"
#include "serving.h"

namespace sa {

namespace {

constexpr int kCtaWarps = 4;
constexpr float kRaiseLog2 = 8.0f;

template <int D, int NT>
struct FGeo {
  // CTAs per SM that the registers allow
  static constexpr int kCtas = D == 64 ? (NT == 1 ? 5 : 4) : D == 128 ? (NT == 1 ? 4 : 2) : 2;
  static constexpr int kKs = D / 16;      // contraction steps of S, 16-dim tiles of O
  static constexpr int kKv = D / 64;      // 16-byte pieces of a K row per lane
  static constexpr int kVw = D / 32;      // 4-byte words of a V row per lane
};

__device__ __forceinline__ uint4 ld_stream16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_stream8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

// Two E4M3 codes (low 16 bits) -> two f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two));
  return h;
}

// The codes in the high bytes of the two halves of z -> two bf16 of value * 2^-120.
__device__ __forceinline__ uint32_t high_codes_bf16x2(uint32_t z) {
  return (z & 0x80008000u) | ((z >> 4) & 0x07F007F0u);
}

__device__ __forceinline__ uint32_t times_2p120(uint32_t v) {
  const uint32_t c = 0x7B807B80u;  // bf16 2^120, twice
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                             *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ float e8m0_f32(uint32_t byte) {
  return byte == 0     ? 0x1p-127f
         : byte == 255 ? __int_as_float(0x7fffffff)
                       : __uint_as_float(byte << 23);
}

// (tile indices stay below 2^31, checked on the host)
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

// One tile's codes and scale bytes in registers (raw), as loaded ahead.
template <int D>
struct KTile {
  uint4 x[2][D / 64];     // rows gid and gid + 8
  uint32_t s[2];          // their scale bytes
};
template <int D>
struct VTile {
  uint32_t x[4][D / 32];  // tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9: this lane's dims
  uint32_t s[2];          // scale bytes of tokens gid and gid + 8
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kCtaWarps * 32, FGeo<D, NT>::kCtas)
    fp8_pages_kernel(GatherArgs a, int64_t pool_heads, int64_t min_range) {
  using G = FGeo<D, NT>;
  extern __shared__ int32_t pref[];  // [B + 1]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
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
  const int64_t total = a.Hkv * static_cast<int64_t>(pref[a.B]);
  const int64_t gw_total = static_cast<int64_t>(gridDim.x) * kCtaWarps;
  int64_t R = (total + gw_total - 1) / gw_total;
  if (R < min_range) R = min_range;
  if (blockIdx.x == 0) {
    for (int64_t b = threadIdx.x; b <= a.B; b += blockDim.x) a.pref_out[b] = pref[b];
    if (threadIdx.x == 0) a.meta[0] = R;
    // sequences without tiles still need a (zero) output
    for (int64_t e = threadIdx.x; e < a.B * a.Hq * D; e += blockDim.x) {
      const int64_t b = e / (a.Hq * D);
      if (pref[b + 1] == pref[b]) static_cast<T*>(a.y)[e] = from_f32<T>(0.f);
    }
  }
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kCtaWarps + warp;
  if (gw * R >= total) return;
  const int32_t t_begin = static_cast<int32_t>(gw * R);
  const int32_t t_end = static_cast<int32_t>(min(gw * R + R, total));

  const int pt = static_cast<int>(a.page_tokens);
  const int64_t page_bytes = a.page_tokens * (D + 1);
  const uint32_t sub = static_cast<uint32_t>(a.Hkv / pool_heads);
  const uint8_t* kp = static_cast<const uint8_t*>(a.k);
  const uint8_t* vp = static_cast<const uint8_t*>(a.v);

  // Byte offset of tile t's page (of its head), and its first slot; negative
  // when the table entry is bad.
  auto page_of = [&](const Unit& un, int32_t t, int& slot) -> int64_t {
    const uint32_t tok = static_cast<uint32_t>(t - un.off) * 16u;
    const uint32_t pi = tok / static_cast<uint32_t>(pt);
    slot = static_cast<int>(tok - pi * static_cast<uint32_t>(pt));
    const int32_t page = __ldg(a.block_table + un.b * a.max_pages + pi);
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0 && a.err_word) atomicOr(a.err_word, SA_ERRBIT_PAGE);
      return -1;
    }
    return (page * pool_heads + static_cast<uint32_t>(un.grp) / sub) * page_bytes;
  };
  auto load_k = [&](int64_t off, int slot, KTile<D>& k) {
    const uint8_t* row = kp + off + (slot + gid) * D + 16 * tig;
#pragma unroll
    for (int i = 0; i < G::kKv; ++i) {
      k.x[0][i] = ld_stream16(row + 64 * i);
      k.x[1][i] = ld_stream16(row + 8 * D + 64 * i);
    }
    const uint8_t* sc = kp + off + pt * D + slot + gid;
    k.s[0] = __ldg(sc);
    k.s[1] = __ldg(sc + 8);
  };
  auto load_v = [&](int64_t off, int slot, VTile<D>& v) {
    const uint8_t* row = vp + off + (slot + 2 * tig) * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* r = row + ((i & 1) + (i >> 1) * 8) * D;
      if (D == 64) {
        const uint2 w = ld_stream8(r + 8 * gid);
        v.x[i][0] = w.x;
        v.x[i][1] = w.y;
      } else {
#pragma unroll
        for (int p = 0; p < D / 128; ++p) {
          const uint4 w = ld_stream16(r + 128 * p + 16 * gid);
          v.x[i][4 * p] = w.x;
          v.x[i][4 * p + 1] = w.y;
          v.x[i][4 * p + 2] = w.z;
          v.x[i][4 * p + 3] = w.w;
        }
      }
    }
    const uint8_t* sc = vp + off + pt * D + slot + gid;
    v.s[0] = __ldg(sc);
    v.s[1] = __ldg(sc + 8);
  };

  // ---- per-unit state ---------------------------------------------------------------------
  uint32_t qf[NT][G::kKs][2];
  float mult[NT][2];                 // per head: scale * log2(e) * the query's power of two
  float o[G::kKs][NT][4];
  float m_run[NT][2], l_run[NT][2];  // heads 2 tig, 2 tig + 1; l: this lane's tokens
  Unit cur = unit_at(a, pref, t_begin);
  const int32_t first_off = cur.off;

  auto start_unit = [&]() {
    const T* qp = static_cast<const T*>(a.q);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int hh = nt * 8 + gid;
      const bool live = hh < a.hpu;
      const T* qr = qp + (cur.b * a.Hq + cur.grp * a.hpu + (live ? hh : 0)) * D;
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < G::kKv; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(to_f32<T>(qr[64 * i + 16 * tig + e])));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // a power of two that puts amax into [2^14, 2^15); kept inside fp32's exponents
      int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14;
      if (amax == 0.f || !(amax <= 3.0e38f)) ex = 0;
      ex = max(ex, -126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
      for (int kk = 0; kk < G::kKs; ++kk) {
        // contraction step kk covers dims 64 (kk / 4) + 16 tig + 4 (kk % 4) + 0 .. 3 of this lane
        const T* q4 = qr + 64 * (kk / 4) + 16 * tig + 4 * (kk % 4);
        const float f0 = live ? to_f32<T>(q4[0]) * down : 0.f, f1 = live ? to_f32<T>(q4[1]) * down : 0.f;
        const float f2 = live ? to_f32<T>(q4[2]) * down : 0.f, f3 = live ? to_f32<T>(q4[3]) * down : 0.f;
        qf[nt][kk][0] = pack2<__half>(f0, f1);
        qf[nt][kk][1] = pack2<__half>(f2, f3);
      }
      mult[nt][0] = a.scale_log2 * __shfl_sync(0xffffffffu, up, 8 * tig);
      mult[nt][1] = a.scale_log2 * __shfl_sync(0xffffffffu, up, 8 * tig + 4);
      m_run[nt][0] = m_run[nt][1] = SA_NEG_INF;
      l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < G::kKs; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    }
  };

  // This lane's dims of O tile mt: 2 of them, consecutive.
  auto dim_of = [&](int mt) {
    return D == 64 ? 8 * gid + 2 * mt : (mt / 8) * 128 + 16 * gid + 2 * (mt % 8);
  };

  auto flush_unit = [&]() {
    const bool whole = cur.off >= t_begin && cur.off + cur.tu <= t_end;
    const int64_t pbase = (gw * 2 + ((cur.off == first_off) ? 0 : 1)) * a.hpu;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float l = l_run[nt][j];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
        const int hh = nt * 8 + 2 * tig + j;
        if (hh >= a.hpu) continue;
        if (whole) {
          const float inv = (m_run[nt][j] == SA_NEG_INF || l == 0.f) ? 0.f : 1.0f / l;
          T* yp = static_cast<T*>(a.y) + (cur.b * a.Hq + cur.grp * a.hpu + hh) * D;
#pragma unroll
          for (int mt = 0; mt < G::kKs; ++mt)
            *reinterpret_cast<uint32_t*>(yp + dim_of(mt)) =
                pack2<T>(o[mt][nt][j] * inv, o[mt][nt][2 + j] * inv);
        } else {
          float* po = a.part_o + (pbase + hh) * D;
#pragma unroll
          for (int mt = 0; mt < G::kKs; ++mt)
            *reinterpret_cast<float2*>(po + dim_of(mt)) = make_float2(o[mt][nt][j], o[mt][nt][2 + j]);
          if (gid == 0) {
            a.part_ml[2 * (pbase + hh)] = m_run[nt][j];
            a.part_ml[2 * (pbase + hh) + 1] = l;
          }
        }
      }
  };

  // ---- main loop -----------------------------------------------------------------------------
  KTile<D> kt;
  VTile<D> vt;
  Unit nxt = cur;
  int slot = 0;
  int64_t off = page_of(cur, t_begin, slot);
  if (off >= 0) {
    load_k(off, slot, kt);
    load_v(off, slot, vt);
  }
  start_unit();
  for (int32_t t = t_begin; t < t_end; ++t) {
    if (t >= cur.off + cur.tu) {
      flush_unit();
      cur = nxt;
      start_unit();
    }
    const bool have = off >= 0;
    // the next tile's place (its table entry is on its way during S)
    int64_t off_n = -1;
    int slot_n = 0;
    const bool more = t + 1 < t_end;
    if (more) {
      if (t + 1 >= nxt.off + nxt.tu) nxt = unit_at(a, pref, t + 1);
      off_n = page_of(nxt, t + 1, slot_n);
    }
    const int left = cur.ctx - (t - cur.off) * 16;  // tokens from this tile on
    const bool lo_ok = have && gid < left, hi_ok = have && gid + 8 < left;

    // S^T = K . Q^T over the codes
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
    for (int i = 0; i < G::kKv; ++i) {
      const uint32_t w0[4] = {kt.x[0][i].x, kt.x[0][i].y, kt.x[0][i].z, kt.x[0][i].w};
      const uint32_t w1[4] = {kt.x[1][i].x, kt.x[1][i].y, kt.x[1][i].z, kt.x[1][i].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a0 = e4m3x2_f16x2(w0[w]), a2 = e4m3x2_f16x2(w0[w] >> 16);
        const uint32_t a1 = e4m3x2_f16x2(w1[w]), a3 = e4m3x2_f16x2(w1[w] >> 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816<__half>(s[nt], a0, a1, a2, a3, qf[nt][4 * i + w][0], qf[nt][4 * i + w][1]);
      }
    }
    const float ks0 = e8m0_f32(kt.s[0]), ks1 = e8m0_f32(kt.s[1]);
    if (more && off_n >= 0) load_k(off_n, slot_n, kt);

    // scores in log2 units; probabilities against the running maximum
    const float vs0 = lo_ok ? e8m0_f32(vt.s[0]) : 0.f, vs1 = hi_ok ? e8m0_f32(vt.s[1]) : 0.f;
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = s[nt][e] * ((e < 2) ? ks0 : ks1) * mult[nt][e & 1];
        s[nt][e] = ((e < 2) ? lo_ok : hi_ok) ? x : SA_NEG_INF;
      }
      // (a NaN score raises nothing and makes its row NaN through p)
      const bool raise = fmaxf(s[nt][0], s[nt][2]) > m_run[nt][0] + kRaiseLog2 ||
                         fmaxf(s[nt][1], s[nt][3]) > m_run[nt][1] + kRaiseLog2 ||
                         m_run[nt][0] == SA_NEG_INF || m_run[nt][1] == SA_NEG_INF;
      if (__any_sync(0xffffffffu, raise)) {
        float al[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // a row of nothing but NaN scores still gets a finite maximum, so that its
          // NaN sum is not taken for an empty one
          const float x0 = s[nt][j], x1 = s[nt][2 + j];
          float tm = fmaxf(x0 == x0 ? x0 : 0.f, x1 == x1 ? x1 : 0.f);
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, sh));
          const float mn = fmaxf(m_run[nt][j], tm);
          al[j] = mn == SA_NEG_INF ? 1.f : ex2(m_run[nt][j] - mn);
          m_run[nt][j] = mn;
          l_run[nt][j] *= al[j];
        }
#pragma unroll
        for (int mt = 0; mt < G::kKs; ++mt) {
          o[mt][nt][0] *= al[0];
          o[mt][nt][1] *= al[1];
          o[mt][nt][2] *= al[0];
          o[mt][nt][3] *= al[1];
        }
      }
      const float mu0 = m_run[nt][0] == SA_NEG_INF ? 0.f : m_run[nt][0];
      const float mu1 = m_run[nt][1] == SA_NEG_INF ? 0.f : m_run[nt][1];
      const float p0 = ex2(s[nt][0] - mu0), p1 = ex2(s[nt][1] - mu1);
      const float p2 = ex2(s[nt][2] - mu0), p3 = ex2(s[nt][3] - mu1);
      l_run[nt][0] += p0 + p2;
      l_run[nt][1] += p1 + p3;
      const float w0 = p0 * vs0, w1 = p1 * vs0, w2 = p2 * vs1, w3 = p3 * vs1;
      const uint32_t h01 = pack2<__nv_bfloat16>(w0, w1), h23 = pack2<__nv_bfloat16>(w2, w3);
      ph[nt][0] = movm_t(h01);
      ph[nt][1] = movm_t(h23);
      pl[nt][0] = movm_t(pack2<__nv_bfloat16>(w0 - __uint_as_float(h01 << 16),
                                              w1 - __uint_as_float(h01 & 0xffff0000u)));
      pl[nt][1] = movm_t(pack2<__nv_bfloat16>(w2 - __uint_as_float(h23 << 16),
                                              w3 - __uint_as_float(h23 & 0xffff0000u)));
    }

    // O^T += V^T . P^T
    if (have) {
#pragma unroll
      for (int w = 0; w < G::kVw; ++w) {
        // (tokens 2 tig, 2 tig + 1), (2 tig + 8, 2 tig + 9): dims 4w, 4w + 1 | 4w + 2, 4w + 3
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7632u : 0x5410u;
          const uint32_t z0 = __byte_perm(vt.x[0][w], vt.x[1][w], sel);
          const uint32_t z1 = __byte_perm(vt.x[2][w], vt.x[3][w], sel);
          const uint32_t a0 = times_2p120(high_codes_bf16x2(z0 << 8));
          const uint32_t a1 = times_2p120(high_codes_bf16x2(z0));
          const uint32_t a2 = times_2p120(high_codes_bf16x2(z1 << 8));
          const uint32_t a3 = times_2p120(high_codes_bf16x2(z1));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816<__nv_bfloat16>(o[2 * w + half][nt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
            mma16816<__nv_bfloat16>(o[2 * w + half][nt], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
          }
        }
      }
    }
    if (more && off_n >= 0) load_v(off_n, slot_n, vt);
    off = off_n;
    slot = slot_n;
  }
  flush_unit();
}

template <typename T, int D, int NT>
int launch_t(const GatherArgs& a, int64_t pool_heads, int sms, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(a.B + 1) * sizeof(int32_t);
  // Ranges of at least four tiles: below that a warp's set-up and the merge of
  // its partial cost more than the tiles.
  fp8_pages_kernel<T, D, NT><<<static_cast<unsigned>(sms * FGeo<D, NT>::kCtas), kCtaWarps * 32, smem,
                              st>>>(a, pool_heads, 4);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
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

int64_t fp8_pages_grid_warps(int D, int64_t hpu, int sms) {
  const bool two = hpu > 8;
  const int ctas = D == 64    ? (two ? FGeo<64, 2>::kCtas : FGeo<64, 1>::kCtas)
                   : D == 128 ? (two ? FGeo<128, 2>::kCtas : FGeo<128, 1>::kCtas)
                              : FGeo<256, 1>::kCtas;
  return static_cast<int64_t>(sms) * ctas * kCtaWarps;
}

int launch_fp8_pages(const GatherArgs& a, int64_t pool_heads, int dtype, int sms, cudaStream_t st) {
  if (dtype == SA_F16) return launch_d<__half>(a, pool_heads, sms, st);
  return launch_d<__nv_bfloat16>(a, pool_heads, sms, st);
}

}  // namespace sa
