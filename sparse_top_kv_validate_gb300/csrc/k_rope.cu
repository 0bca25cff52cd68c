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
// chunk's eight (cos, sin) in registers and walks down the heads, its next
// four rows on their way through shared memory (RowRing).
//
// Measured, 4 x 4,096 tokens, 32 + 8 heads of 128, half of each rotated, fp16,
// head-major (335 MB): 55 us, 6.1 TB/s, 89% of the copy bandwidth; with four rows
// loaded to registers and a lane's pieces side by side (half-filled sectors per
// access) 71 us.  fp32, whole heads rotated (671 MB): 147 us, 4.6 TB/s.  Heads of 96,
// half rotated (252 MB), 54 us; heads of 80, 40 or 20 dims rotated, take the kernel for
// any size, a pair per lane and 2-byte accesses: 127 and 152 us for 210 MB.  A decode
// step (128 tokens) takes 6.2 us, a launch's latency.
#include "rope.cuh"
#include "serving.h"

namespace sa {

namespace {

constexpr int kThreads = kRingThreads;

__device__ __forceinline__ int64_t position_of(const RotaryArgs& a, int b, int s) {
  return load_index(a.positions, b * a.pos_stride + s, a.pos_is_i64);
}

// Element offset of (token, head 0) in tensor w of the inputs or outputs.
__device__ __forceinline__ int64_t token_off(const int64_t (&st)[3], int b, int s) {
  return b * st[0] + s * st[1];
}

// The tokens' tables.
__device__ __forceinline__ void tile_turns(const RotaryArgs& a, TurnTables<kThreads>& tables, int t0, int tt,
                                           float* cs_sm) {
  tables.fill(
      a.rope, min(tt, a.T - t0),
      [&](int k) {
        const int b = (t0 + k) / a.S;
        return position_of(a, b, t0 + k - b * a.S);
      },
      cs_sm);
}

template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads, 3)
    rotary_kernel(const __grid_constant__ RotaryArgs a, int tt, int lanes) {
  extern __shared__ __align__(16) uint8_t smem[];
  RowRing<T> ring(smem);
  float* cs_sm = reinterpret_cast<float*>(smem + RowRing<T>::kBytes);  // [tt][cos, sin][half]
  const int half = a.rope.rotary_dim / 2, t0 = blockIdx.x * tt;
  const int c = threadIdx.x % lanes, slot = threadIdx.x / lanes;
  const int k = slot % tt, hl = slot / tt, step = kThreads / (lanes * tt);
  const int t = t0 + k, b = t / a.S, s = t - b * a.S;
  const Pieces pc = pieces_of<kInter>(c, a.D, a.rope.rotary_dim);
  const int d0 = pc.d[0], d1 = pc.d[1];
  const bool turn = pc.turn[0] || pc.turn[1];
  // this thread's rows: the first tensor's, then the second's
  const T* x[2];
  T* y[2];
  int rows[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    x[w] = static_cast<const T*>(a.x[w]) + token_off(a.xs[w], b, s) + hl * a.xs[w][2];
    y[w] = static_cast<T*>(a.y[w]) + token_off(a.ys[w], b, s) + hl * a.ys[w][2];
    const bool live = hl < step && hl < a.H[w] && t < a.T && (turn || !a.in_place[w]);
    rows[w] = live ? (a.H[w] - hl + step - 1) / step : 0;
  }
  const T* xp = x[0];
  int64_t xstep = step * a.xs[0][2];
  const int total = rows[0] + rows[1];
  auto fetch = [&](int i) {
    if (i < total) {
      if (i == rows[0]) {
        xp = x[1];
        xstep = step * a.xs[1][2];
      }
      ring.fetch(i, 0, xp + d0, true);
      ring.fetch(i, 1, xp + d1, true);
      xp += xstep;
    }
    ring.commit();
  };
  TurnTables<kThreads> tables(a.rope);
  for (int i = 0; i < RowRing<T>::kRowsAhead; ++i) fetch(i);
  tile_turns(a, tables, t0, tt, cs_sm);
  __syncthreads();
  const Turns turns = turns_of<kInter>(cs_sm + 2 * k * half, half, pc);
  T* yp = y[0];
  int64_t ystep = step * a.ys[0][2];
#pragma unroll 1
  for (int i = 0; i < total; ++i) {
    if (i == rows[0]) {
      yp = y[1];
      ystep = step * a.ys[1][2];
    }
    ring.arrived();
    const Raw8<T> va = ring.get(i, 0), vb = ring.get(i, 1);
    float fa[8], fb[8];
    unpack8<T>(va, fa);
    unpack8<T>(vb, fb);
    Piece pa = piece_from<kInter>(fa), pb = piece_from<kInter>(fb);
    rotate_pieces<kInter>(pa, pb, turns, pc);
    piece_to<kInter>(pa, fa);
    piece_to<kInter>(pb, fb);
    if (pc.turn[0]) store8<T>(yp + d0, fa);
    else store_raw<T>(yp + d0, va);
    if (pc.turn[1]) store8<T>(yp + d1, fb);
    else store_raw<T>(yp + d1, vb);
    yp += ystep;
    fetch(i + RowRing<T>::kRowsAhead);
  }
}

// Rows that are no whole chunks or not aligned: one pair, or one element past
// rotary_dim, per lane.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    rotary_any_kernel(const __grid_constant__ RotaryArgs a, int tt, int lanes) {
  extern __shared__ __align__(16) float cs_sm[];
  const int half = a.rope.rotary_dim / 2, t0 = blockIdx.x * tt;
  TurnTables<kThreads> tables(a.rope);
  tile_turns(a, tables, t0, tt, cs_sm);
  __syncthreads();
  const int c = threadIdx.x % lanes, slot = threadIdx.x / lanes;
  const int k = slot % tt, hl = slot / tt, hstep = kThreads / (lanes * tt);
  const int t = t0 + k;
  if (hl >= hstep || t >= a.T) return;
  const int b = t / a.S, s = t - b * a.S;
  const bool turn = c < half;
  const int d0 = turn ? (a.rope.interleaved ? 2 * c : c) : 2 * half + (c - half);
  const int d1 = a.rope.interleaved ? d0 + 1 : d0 + half;
  const float cs = turn ? cs_sm[2 * k * half + c] : 1.f;
  const float sn = turn ? cs_sm[(2 * k + 1) * half + c] : 0.f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const T* x = static_cast<const T*>(a.x[w]) + token_off(a.xs[w], b, s);
    T* y = static_cast<T*>(a.y[w]) + token_off(a.ys[w], b, s);
    for (int h = hl; h < a.H[w]; h += hstep) {
      const T* xh = x + h * a.xs[w][2];
      T* yh = y + h * a.ys[w][2];
      if (turn) {
        const float u = to_f32<T>(xh[d0]), v = to_f32<T>(xh[d1]);
        yh[d0] = from_f32<T>(u * cs - v * sn);
        yh[d1] = from_f32<T>(u * sn + v * cs);
      } else if (!a.in_place[w]) {
        yh[d0] = xh[d0];
      }
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
  const int sms = sm_count();
  while (tt > 1 && ((a.T + tt - 1) / tt < 2 * sms || lanes * tt > kThreads)) tt /= 2;
  const unsigned grid = static_cast<unsigned>((a.T + tt - 1) / tt);
  const size_t smem =
      (a.vec ? RowRing<T>::kBytes : 0) + static_cast<size_t>(tt) * 2 * half * sizeof(float);
  if (a.vec)
    (a.rope.interleaved ? rotary_kernel<T, true> : rotary_kernel<T, false>)<<<grid, kThreads, smem, st>>>(
        a, tt, lanes);
  else
    rotary_any_kernel<T><<<grid, kThreads, smem, st>>>(a, tt, lanes);
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
