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
#include "rope.cuh"
#include "serving.h"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTok = 16;  // tokens per block

// Sequence that owns packed row r: the largest b with start[b] <= r, found by
// the whole warp, 32 probes per step (two dependent loads for 1,024
// sequences).  Negative when the row is nobody's.
__device__ __forceinline__ int owner_of(const int32_t* start, int B, int r, int lane) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < hi && __ldg(start + at) <= r;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    if (n > 1) lo += (n - 1) * step;  // starts out of order: still below hi
    hi = min(lo + step, hi);
  }
  return (__ldg(start + lo) <= r && r < __ldg(start + lo + 1)) ? lo : -1;
}

struct Place {
  int64_t page;  // page * Hkv, or -1 (nothing is done)
  int32_t slot, pos;
};

// Where packed row r lives.  kWrite: the rows are the last of the context;
// else its first.  Uniform over the warp.
template <bool kWrite>
__device__ __forceinline__ Place place_of(const KvPagesArgs& a, int r, int lane) {
  Place p{-1, 0, 0};
  int b = r, first = r, n = 1;
  if (a.seq_start) {
    b = owner_of(a.seq_start, a.B, r, lane);
    if (b < 0) return p;
    first = __ldg(a.seq_start + b);
    n = __ldg(a.seq_start + b + 1) - first;
  }
  const int64_t ctx = __ldg(a.ctx_len + b);
  const int64_t pos = (kWrite ? ctx - n : 0) + (r - first);
  int32_t page = -1;
  if (pos >= 0 && pos < ctx && ctx <= a.max_pages * a.page_tokens) {
    // a context is an int32: 32-bit division
    const uint32_t pi = static_cast<uint32_t>(pos) / static_cast<uint32_t>(a.page_tokens);
    page = __ldg(a.block_table + b * a.max_pages + pi);
    p.slot = static_cast<int32_t>(pos - static_cast<int64_t>(pi) * a.page_tokens);
    p.pos = static_cast<int32_t>(pos);
  }
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0 && a.err_word) atomicOr(a.err_word, SA_ERRBIT_PAGE);
    return p;
  }
  p.page = static_cast<int64_t>(page) * a.Hkv;
  return p;
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

template <typename T>
__device__ __forceinline__ void load8_any(const T* p, int aligned, Raw8<T>& v) {
  if (aligned) {
    v = load8<T>(p);
  } else {
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i];
  }
}

// ---- write, 16 elements per lane ------------------------------------------------------
//
// D / 16 lanes hold a row (two 8-element pieces each, chunk_dims), so a pair of
// the half layout meets in one lane and the row's maximum in log2(D / 16)
// shuffles.  A block takes `tt` tokens; a thread has up to kBatch rows in
// flight.
template <typename T, bool kFp8>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(const __grid_constant__ KvPagesArgs a, int tt) {
  constexpr int kBatch = sizeof(T) == 4 ? 2 : 4;
  extern __shared__ float2 cs_sm[];  // [tt][half] when the keys are rotated
  __shared__ Place place[kMaxTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * tt;
  const int lanes = a.D / 16, c = tid % lanes, q0 = tid / lanes, rp = kThreads / lanes;
  const int per_tok = 2 * a.Hkv, rows = min(tt, a.T - t0) * per_tok;
  const int rot = a.has_rope ? a.rope.rotary_dim : 0, half = rot / 2;
  const int inter = a.has_rope ? a.rope.interleaved : 1;
  int d0, d1;
  chunk_dims(c, rot, inter, d0, d1);
  check_starts(a);

  for (int rb = 0; rb < rows; rb += kBatch * rp) {  // the same trips for the whole block
    Raw8<T> va[kBatch], vb[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = rb + q0 + i * rp;
      if (r < rows) {
        const int k = r / per_tok, e = r - k * per_tok, w = e >= a.Hkv, h = e - (w ? a.Hkv : 0);
        const T* x = static_cast<const T*>(a.x[w]) + (t0 + k) * a.xs[w][0] + h * a.xs[w][1];
        load8_any<T>(x + d0, a.aligned, va[i]);
        load8_any<T>(x + d1, a.aligned, vb[i]);
      }
    }
    if (rb == 0) {  // the first batch's loads are on their way
      for (int k = warp; k < tt; k += kWarps) {
        Place p{-1, 0, 0};
        if (t0 + k < a.T) p = place_of<true>(a, t0 + k, lane);
        if (lane == 0) place[k] = p;
      }
      __syncthreads();
      if (rot) {
        for (int e = tid; e < tt * half; e += kThreads) {
          const int k = e / half, i = e - k * half;
          cs_sm[e] = rope_cos_sin(place[k].pos, a.rope.turns[i], a.rope.mscale);
        }
        __syncthreads();
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = rb + q0 + i * rp;
      const bool live = r < rows;  // uniform over a row's lanes; the shuffles stay within them
      const int k = live ? r / per_tok : 0, e = live ? r - k * per_tok : 0, w = e >= a.Hkv;
      const int h = e - (w ? a.Hkv : 0);
      const Place p = place[k];
      const bool put = live && p.page >= 0;
      float fa[8], fb[8];
      unpack8<T>(va[i], fa);
      unpack8<T>(vb[i], fb);
      const bool turn = live && !w && 16 * c < rot;
      if (turn) {
        float2 cs[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) cs[j] = cs_sm[k * half + 8 * c + j];
        rotate_chunk(fa, fb, cs, inter);
      }
      if (kFp8) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, max(abs_bits(fa[j]), abs_bits(fb[j])));
        for (int o = lanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (!put) continue;
        const bool bad = m >= kInfBits;
        const int ex = bad ? 0 : row_exponent(m);
        const float mul = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          fa[j] = bad ? 0.f : fa[j] * mul;
          fb[j] = bad ? 0.f : fb[j] * mul;
        }
        uint8_t* page = fp8_page(a, w, p.page, h);
        uint8_t* codes = page + p.slot * a.D;
        *reinterpret_cast<uint2*>(codes + d0) =
            make_uint2(to_e4m3x4(fa[0], fa[1], fa[2], fa[3]), to_e4m3x4(fa[4], fa[5], fa[6], fa[7]));
        *reinterpret_cast<uint2*>(codes + d1) =
            make_uint2(to_e4m3x4(fb[0], fb[1], fb[2], fb[3]), to_e4m3x4(fb[4], fb[5], fb[6], fb[7]));
        if (c == 0) {
          page[a.page_tokens * a.D + p.slot] = static_cast<uint8_t>(bad ? 255 : ex + 127);
          if (bad && a.err_word) atomicOr(a.err_word, SA_ERRBIT_NONFINITE);
        }
      } else if (put) {
        T* y = static_cast<T*>(a.pool[w]) + ((p.page + h) * a.page_tokens + p.slot) * a.D;
        if (turn) {
          store8<T>(y + d0, fa);
          store8<T>(y + d1, fb);
        } else {  // an exact copy
#pragma unroll
          for (int j = 0; j < static_cast<int>(sizeof(T) / 2); ++j) {
            *(reinterpret_cast<uint4*>(y + d0) + j) = va[i].r[j];
            *(reinterpret_cast<uint4*>(y + d1) + j) = vb[i].r[j];
          }
        }
      }
    }
  }
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
        *reinterpret_cast<uint32_t*>(page + p.slot * a.D + 4 * d) =
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

// Sixteen codes times a scale -> sixteen elements.
template <typename T>
__device__ __forceinline__ void store16(T* y, const uint4& codes, float scale, int aligned) {
  const uint32_t wd[4] = {codes.x, codes.y, codes.z, codes.w};
  float f[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t h2;
    asm("{\n\t.reg .b16 t;\n\tmov.b16 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(h2)
        : "h"(static_cast<uint16_t>(wd[i / 2] >> (16 * (i & 1)))));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    f[i / 4][2 * (i % 4)] = v.x * scale;
    f[i / 4][2 * (i % 4) + 1] = v.y * scale;
  }
  if (aligned) {
    store8<T>(y, f[0]);
    store8<T>(y + 8, f[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = from_f32<T>(f[i / 8][i % 8]);
  }
}

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return byte == 0     ? 0x1p-127f
         : byte == 255 ? __int_as_float(0x7fffffff)
                       : __uint_as_float(byte << 23);
}

// FP8 pages -> rows: 16 codes per lane; a block takes `tt` rows of every head.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv_read_fp8_kernel(const __grid_constant__ KvPagesArgs a, int tt) {
  constexpr int kBatch = 4;
  __shared__ Place place[kMaxTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * tt;
  const int lanes = a.D / 16, c = tid % lanes, q0 = tid / lanes, rp = kThreads / lanes;
  const int n = min(tt, a.T - t0), rows = n * 2 * a.Hkv;
  check_starts(a);
  for (int k = warp; k < n; k += kWarps) {
    const Place p = place_of<false>(a, t0 + k, lane);
    if (lane == 0) place[k] = p;
  }
  __syncthreads();
  // rows in the order (K or V, head, token): neighbours in a page are neighbours here
  for (int r0 = q0; r0 < rows; r0 += kBatch * rp) {
    uint4 codes[kBatch];
    uint32_t sb[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * rp;
      if (r < rows) {
        const int e = r / n, k = r - e * n, w = e >= a.Hkv, h = e - (w ? a.Hkv : 0);
        const Place p = place[k];
        if (p.page >= 0) {
          const uint8_t* page = fp8_page(a, w, p.page, h);
          codes[i] = __ldg(reinterpret_cast<const uint4*>(page + p.slot * a.D) + c);
          sb[i] = __ldg(page + a.page_tokens * a.D + p.slot);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * rp;
      if (r < rows) {
        const int e = r / n, k = r - e * n, w = e >= a.Hkv, h = e - (w ? a.Hkv : 0);
        if (place[k].page >= 0) {
          T* y = static_cast<T*>(a.x[w]) + (t0 + k) * a.xs[w][0] + h * a.xs[w][1] + 16 * c;
          store16<T>(y, codes[i], e8m0(sb[i]), a.aligned);
        }
      }
    }
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

// Tokens per block: as many as give every thread a full batch of rows, once
// the blocks still cover the SMs twice.
int tokens_per_block(const KvPagesArgs& a, int batch) {
  const int rp = kThreads / (a.D / 16);
  int tt = 1;
  while (tt < kMaxTok && 2 * tt * 2 * a.Hkv <= batch * rp && a.T / (2 * tt) >= 2 * 152) tt *= 2;
  return tt;
}

unsigned row_blocks(const KvPagesArgs& a) {
  const int64_t blocks = (static_cast<int64_t>(a.T) * 2 * a.Hkv + kWarps - 1) / kWarps;
  return static_cast<unsigned>(blocks < 152 * 16 ? blocks : 152 * 16);
}

template <typename T>
int write_t(const KvPagesArgs& a, cudaStream_t st) {
  const int rot = a.has_rope ? a.rope.rotary_dim : 0;
  const int L = a.D / 16;
  const bool chunks = a.D % 16 == 0 && rot % 16 == 0 && L <= 32 && (L & (L - 1)) == 0;
  if (chunks && (a.fp8 || a.aligned)) {
    const int tt = tokens_per_block(a, sizeof(T) == 4 ? 2 : 4);
    const unsigned grid = static_cast<unsigned>((a.T + tt - 1) / tt);
    const size_t smem = static_cast<size_t>(tt) * (rot / 2) * sizeof(float2);
    if (a.fp8) kv_write_kernel<T, true><<<grid, kThreads, smem, st>>>(a, tt);
    else kv_write_kernel<T, false><<<grid, kThreads, smem, st>>>(a, tt);
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
    const int tt = tokens_per_block(a, 4);
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
