// k_rope.cu -- rotary positions of queries and keys.
//
// (u, v) of pair i becomes m (u cos a - v sin a, u sin a + v cos a) with
// a = position * f_i (include/sa.h: the frequencies, their scalings and the
// pairing).  Every row is read and written once and little is computed, so
// the operator is bound by DRAM bandwidth (or, for a few tokens, by latency).
//
// One launch takes queries and keys.  A block takes `tt` tokens (a power of
// two) and all their heads: its threads first fill shared memory with the
// tokens' (cos, sin) -- once per token and pair instead of once per head --,
// then each thread owns one chunk of 16 elements of one token, holds the
// chunk's eight (cos, sin) in registers and walks down the heads, four rows
// loaded before the first is used.
#include "rope.cuh"
#include "serving.h"

namespace sa {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t position_of(const RotaryArgs& a, int b, int s) {
  return load_index(a.positions, b * a.pos_stride + s, a.pos_is_i64);
}

// Element offset of (token, head 0) in tensor w of the inputs or outputs.
__device__ __forceinline__ int64_t token_off(const int64_t (&st)[3], int b, int s) {
  return b * st[0] + s * st[1];
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(const __grid_constant__ RotaryArgs a, int tt, int lanes) {
  extern __shared__ float2 cs_sm[];  // [tt][half]
  const int half = a.rope.rotary_dim / 2;
  const int t0 = blockIdx.x * tt;
  const int tid = threadIdx.x;
  // (cos, sin): a thread keeps one pair where the block holds whole rows of pairs
  for (int e = tid; e < tt * half; e += kThreads) {
    const int k = e / half, i = e - k * half, t = t0 + k;
    if (t < a.T) {
      const int b = t / a.S;
      cs_sm[e] = rope_cos_sin(position_of(a, b, t - b * a.S), a.rope.turns[i], a.rope.mscale);
    }
  }
  __syncthreads();
  const int c = tid % lanes, qd = tid / lanes;
  const int k = qd % tt, hl = qd / tt, hstep = kThreads / (lanes * tt);
  const int t = t0 + k;
  if (hl >= hstep || t >= a.T) return;
  const int b = t / a.S, s = t - b * a.S;
  const int heads = a.H[0] + a.H[1];
  const int64_t xo[2] = {token_off(a.xs[0], b, s), token_off(a.xs[1], b, s)};
  const int64_t yo[2] = {token_off(a.ys[0], b, s), token_off(a.ys[1], b, s)};

  if (kVec) {
    constexpr int kRows = sizeof(T) == 4 ? 2 : 4;  // rows in flight per thread
    int d0, d1;
    chunk_dims(c, a.rope.rotary_dim, a.rope.interleaved, d0, d1);
    const bool turn = 16 * c < a.rope.rotary_dim;
    float2 cs[8];
    if (turn) {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = cs_sm[k * half + 8 * c + i];
    }
    for (int h0 = hl; h0 < heads; h0 += kRows * hstep) {
      Raw8<T> va[kRows], vb[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int hh = h0 + r * hstep;
        if (hh < heads) {
          const int w = hh >= a.H[0], h = hh - (w ? a.H[0] : 0);
          if (turn || !a.in_place[w]) {
            const T* x = static_cast<const T*>(a.x[w]) + xo[w] + h * a.xs[w][2];
            va[r] = load8<T>(x + d0);
            vb[r] = load8<T>(x + d1);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int hh = h0 + r * hstep;
        if (hh < heads) {
          const int w = hh >= a.H[0], h = hh - (w ? a.H[0] : 0);
          if (turn || !a.in_place[w]) {
            float fa[8], fb[8];
            unpack8<T>(va[r], fa);
            unpack8<T>(vb[r], fb);
            if (turn) rotate_chunk(fa, fb, cs, a.rope.interleaved);
            T* y = static_cast<T*>(a.y[w]) + yo[w] + h * a.ys[w][2];
            store8<T>(y + d0, fa);
            store8<T>(y + d1, fb);
          }
        }
      }
    }
    return;
  }
  // one pair, or one element past rotary_dim, per lane
  const bool turn = c < half;
  const int d0 = turn ? (a.rope.interleaved ? 2 * c : c) : 2 * half + (c - half);
  const int d1 = a.rope.interleaved ? d0 + 1 : d0 + half;
  const float2 cs = turn ? cs_sm[k * half + c] : make_float2(1.f, 0.f);
  for (int hh = hl; hh < heads; hh += hstep) {
    const int w = hh >= a.H[0], h = hh - (w ? a.H[0] : 0);
    const T* x = static_cast<const T*>(a.x[w]) + xo[w] + h * a.xs[w][2];
    T* y = static_cast<T*>(a.y[w]) + yo[w] + h * a.ys[w][2];
    if (turn) {
      const float u = to_f32<T>(x[d0]), v = to_f32<T>(x[d1]);
      y[d0] = from_f32<T>(u * cs.x - v * cs.y);
      y[d1] = from_f32<T>(u * cs.y + v * cs.x);
    } else if (!a.in_place[w]) {
      y[d0] = x[d0];
    }
  }
}

template <typename T>
int launch_t(const RotaryArgs& a, cudaStream_t st) {
  const int half = a.rope.rotary_dim / 2;
  const int lanes = a.vec ? a.D / 16 : half + (a.D - 2 * half);
  // Up to 8 tokens per block once the blocks still cover the SMs twice: then
  // four tokens' rows share a warp's loads and the set-up is paid once per 8.
  int tt = 8;
  while (tt > 1 && ((a.T + tt - 1) / tt < 2 * 152 || lanes * tt > kThreads)) tt /= 2;
  const unsigned grid = static_cast<unsigned>((a.T + tt - 1) / tt);
  const size_t smem = static_cast<size_t>(tt) * half * sizeof(float2);
  if (a.vec)
    rotary_kernel<T, true><<<grid, kThreads, smem, st>>>(a, tt, lanes);
  else
    rotary_kernel<T, false><<<grid, kThreads, smem, st>>>(a, tt, lanes);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t st) {
  if (a.T == 0) return 0;
  if (dtype == SA_F32) return launch_t<float>(a, st);
  if (dtype == SA_F16) return launch_t<__half>(a, st);
  return launch_t<__nv_bfloat16>(a, st);
}

}  // namespace sa
