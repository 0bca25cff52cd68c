// k_weights_simt.cu -- the attention weight that each key receives from packed queries,
// on the fp32 pipes: every element type and head size.  The tensor-core kernel
// (k_weights.cu) takes the 16-bit types with D 64 or 128.
//
// The same two forms: -L of every query row (L the base-2 logarithm of the row's sum),
// then w_j = sum 2^(c s_ij - L_i) of every key, each with 128 outer rows against tiles of
// 64 inner ones, 8 x 4 scores a thread, a product's operands passing through shared
// memory 32 dims at a time.  Bound by the FMAs and the shared-memory reads that feed
// them (three of 16 bytes to 32 FMAs): 8 prompts of 2,048 tokens, 32 / 8 heads of 128 in
// fp32, 10.0 ms, 27 TFLOP/s (with each element's place worked out on its own, 18.6).
#include "packed.cuh"
#include "pool_add.cuh"
#include "weights.h"

namespace sa {

namespace {

constexpr int kOuter = 128, kInner = 64, kDims = 32, kThreads = 256;
constexpr int kRows = 8, kCols = 4;

// Rows that may be read four elements at a time.
template <typename T>
__device__ __forceinline__ bool four_at_once(const void* p, const int64_t (&st)[2]) {
  return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && (st[0] | st[1]) % 4 == 0;
}
template <typename T>
__device__ __forceinline__ void load4(const T* row, int d, bool there, bool vec, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = 0.f;
  if (!row || !there) return;
  if (vec) {
    struct __align__(4 * sizeof(T)) Four { T x[4]; };
    const Four f = *reinterpret_cast<const Four*>(row + d);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_f32<T>(f.x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_f32<T>(row[d + i]);
  }
}

template <typename T, bool kSums>
__global__ void __launch_bounds__(kThreads, 2)
    weights_simt_kernel(const __grid_constant__ WeightsArgs a, float* nlse, float c_log2) {
  __shared__ __align__(16) float so[kDims][kOuter + 4], si[kDims][kInner + 4];
  __shared__ int s_b, s_tile;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const int B = static_cast<int>(a.B), Tq = static_cast<int>(a.Tq), Tk = static_cast<int>(a.Tk);
  const int g = static_cast<int>(a.Hq / a.Hkv), D = static_cast<int>(a.D), h = static_cast<int>(blockIdx.y);

  bool bad = false;
  for (int b = tid; b < B; b += kThreads) bad = bad || bad_span(a.q_start, b, Tq) || bad_span(a.k_start, b, Tk);
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && h == 0 && tid == 0 && a.err_word) atomicOr(a.err_word, static_cast<uint32_t>(SA_ERRBIT_SEQ));
    return;
  }
  // sequence and outer tile of this block: the tiles of the sequences end to end
  if (tid < 32) {
    int64_t before = 0;
    int fb = -1, ft = 0;
    const int64_t want = blockIdx.x;
    for (int b0 = 0; b0 < B && fb < 0; b0 += 32) {
      const int b = min(b0 + lane, B - 1);
      const int64_t n = kSums ? span_of(a.k_start, b, Tk).n : static_cast<int64_t>(span_of(a.q_start, b, Tq).n) * g;
      int64_t v = b0 + lane < B ? (n + kOuter - 1) / kOuter : 0;
      const int64_t mine = v;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, sh);
        if (lane >= sh) v += x;
      }
      const int64_t lo = before + v - mine;
      const unsigned hit = __ballot_sync(0xffffffffu, want >= lo && want < lo + mine);
      if (hit) {
        const int l = __ffs(hit) - 1;
        fb = b0 + l;
        ft = static_cast<int>(want - __shfl_sync(0xffffffffu, lo, l));
      }
      before += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) {
      s_b = fb;
      s_tile = ft;
    }
  }
  __syncthreads();
  const int b = s_b;
  if (b < 0) return;
  const Span q = span_of(a.q_start, b, Tq), k = span_of(a.k_start, b, Tk);
  const int off = k.n - q.n;  // query i sees the keys up to i + off
  const int64_t qrows = static_cast<int64_t>(q.n) * g;
  if (q.n == 0) return;
  const int64_t o0 = static_cast<int64_t>(s_tile) * kOuter;
  // inner rows from i0 on, below i1
  int64_t i0 = 0, i1;
  if (kSums) {
    i0 = max(o0 - off, int64_t(0)) * g / kInner * kInner;
    i1 = qrows;
  } else {
    i1 = min(static_cast<int64_t>(k.n), min((o0 + kOuter - 1) / g, static_cast<int64_t>(q.n) - 1) + off + 1);
  }
  auto row_of = [&](bool query, int64_t row) -> const T* {  // (null: holds none)
    if (query) {
      if (row >= qrows) return nullptr;
      const int64_t t = row / g;
      return static_cast<const T*>(a.q) + (q.first + t) * a.qs[0] + (h * static_cast<int64_t>(g) + (row - t * g)) * a.qs[1];
    }
    return row < k.n ? static_cast<const T*>(a.k) + (k.first + row) * a.ks[0] + h * a.ks[1] : nullptr;
  };
  // A thread brings the same row of a tile each time, lanes one row each (neighbouring dims of a
  // row come from L1), so that what it stores for a dim lies side by side.
  const int ro = tid & (kOuter - 1), ri = tid & (kInner - 1);
  const T* outer = row_of(!kSums, o0 + ro);
  const bool vq = four_at_once<T>(a.q, a.qs), vk = four_at_once<T>(a.k, a.ks);
  float* rows = nlse + static_cast<int64_t>(h) * Tq * g + static_cast<int64_t>(q.first) * g;
  const int ty = tid >> 4, tx = tid & 15;
  float m[kRows], total[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    m[r] = SA_NEG_INF;
    total[r] = 0.f;
  }
  for (int64_t x0 = i0; x0 < i1; x0 += kInner) {
    float s[kRows][kCols];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int c = 0; c < kCols; ++c) s[r][c] = 0.f;
    const T* inner = row_of(kSums, x0 + ri);
    for (int d0 = 0; d0 < D; d0 += kDims) {
      const int n = min(kDims, D - d0);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kDims / 4; e += kThreads / kOuter) {
        const int d = 4 * (e + tid / kOuter);
        float v[4];
        load4(outer, d0 + d, d < n, kSums ? vk : vq, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) so[d + i][ro] = v[i];
      }
#pragma unroll
      for (int e = 0; e < kDims / 4; e += kThreads / kInner) {
        const int d = 4 * (e + tid / kInner);
        float v[4];
        load4(inner, d0 + d, d < n, kSums ? vq : vk, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) si[d + i][ri] = v[i];
      }
      __syncthreads();
#pragma unroll 8
      for (int d = 0; d < kDims; ++d) {
        const float4 a0 = *reinterpret_cast<const float4*>(&so[d][ty * kRows]);
        const float4 a1 = *reinterpret_cast<const float4*>(&so[d][ty * kRows + 4]);
        const float4 b0 = *reinterpret_cast<const float4*>(&si[d][tx * kCols]);
        const float av[kRows] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
        const float bv[kCols] = {b0.x, b0.y, b0.z, b0.w};
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int c = 0; c < kCols; ++c) s[r][c] = fmaf(av[r], bv[c], s[r][c]);
      }
    }
    float nl[kCols];
    int64_t tok[kCols];
    if (kSums) {
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const int64_t x = x0 + tx * kCols + c;
        nl[c] = x < i1 ? __ldg(rows + x) : SA_NEG_INF;
        tok[c] = x / g;
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t o = o0 + ty * kRows + r;
      if (kSums) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const bool see = x0 + tx * kCols + c < i1 && o <= tok[c] + off;
          const float p = exp2f(fmaf(s[r][c], c_log2, nl[c]));
          total[r] += see ? p : 0.f;
        }
      } else {
        const int64_t last = o < qrows ? min(o / g + off, static_cast<int64_t>(k.n) - 1) : -1;
        float top = SA_NEG_INF;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          s[r][c] = x0 + tx * kCols + c <= last ? s[r][c] * c_log2 : SA_NEG_INF;
          top = fmaxf(top, s[r][c]);
        }
        if (top > m[r]) {
          total[r] *= exp2f(m[r] - top);
          m[r] = top;
        }
        const float mu = m[r] == SA_NEG_INF ? 0.f : m[r];
#pragma unroll
        for (int c = 0; c < kCols; ++c) total[r] += exp2f(s[r][c] - mu);
      }
    }
  }
  // the 16 lanes that share a row
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t o = o0 + ty * kRows + r;
    if (kSums) {
      float sum = total[r];
#pragma unroll
      for (int sh = 1; sh < 16; sh <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
      if (tx != 0 || o >= k.n) continue;
      const int64_t pi = o / a.page_tokens;
      int32_t page = -1;
      if (pi < a.max_pages) page = __ldg(a.block_table + b * a.max_pages + pi);
      if (page < 0 || page >= a.num_pages) {
        if (a.err_word) atomicOr(a.err_word, static_cast<uint32_t>(SA_ERRBIT_PAGE));
        continue;
      }
      pool_put(a.weights + (page * a.Hkv + h) * a.page_tokens + (o - pi * a.page_tokens), sum, a.accumulate && o < off);
    } else {
      float top = m[r];
#pragma unroll
      for (int sh = 1; sh < 16; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
      // (a lane of nothing but NaN scores has the offset -inf and a NaN sum)
      float sum = total[r] != total[r] ? total[r] : m[r] == SA_NEG_INF ? 0.f : total[r] * exp2f(m[r] - top);
#pragma unroll
      for (int sh = 1; sh < 16; sh <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
      if (tx == 0 && o < qrows) rows[o] = sum != sum ? sum : top == SA_NEG_INF ? SA_NEG_INF : -(top + log2f(sum));
    }
  }
}

template <typename T>
int launch_t(const WeightsArgs& a, cudaStream_t st) {
  float* nlse = static_cast<float*>(a.workspace);
  const float c = a.scale * 1.4426950408889634f;
  const int64_t g = a.Hq / a.Hkv;
  const int64_t qt = a.Tq * g / kOuter + a.B, kt = a.Tk / kOuter + a.B;  // at least the sequences' own
  if (qt > INT32_MAX || kt > INT32_MAX || a.Hkv > 65535) return -1;
  const unsigned hkv = static_cast<unsigned>(a.Hkv);
  weights_simt_kernel<T, false><<<dim3(static_cast<unsigned>(qt), hkv), kThreads, 0, st>>>(a, nlse, c);
  if (cudaGetLastError() != cudaSuccess) return -1;
  weights_simt_kernel<T, true><<<dim3(static_cast<unsigned>(kt), hkv), kThreads, 0, st>>>(a, nlse, c);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

size_t weights_simt_workspace(const WeightsArgs& a) {
  return static_cast<size_t>(a.Tq) * static_cast<size_t>(a.Hq) * sizeof(float);
}

int launch_weights_simt(const WeightsArgs& a, cudaStream_t st) {
  if (a.dtype == SA_F32) return launch_t<float>(a, st);
  if (a.dtype == SA_F16) return launch_t<__half>(a, st);
  return launch_t<__nv_bfloat16>(a, st);
}

}  // namespace sa
