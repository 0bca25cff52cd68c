// k_packed_simt.cu -- packed prefill on the fp32 pipes: every element type and
// head size, fp32 products and sums.  The tensor-core kernel (k_packed.cu)
// takes the 16-bit types with D 64 or 128.
//
// y_i = sum_j softmax_j(s_ij) v_j over the keys j <= i + nk - nq (causal) of
// the query's sequence.  A block takes 16 queries of one head and walks over
// the keys in tiles of 32 held in shared memory as fp32; eight lanes share a
// query: four scores each, then D / 8 output dims each, with a running maximum
// and sum.  Bound by shared-memory reads (five of 16 bytes to 16 FMAs): 8 prompts of
// 2,048 tokens, 32 / 8 heads of 128, fp32, 22.6 ms (12 TFLOP/s; the tensor-core kernel
// takes 0.27 ms for the same in 16 bits); bf16, heads of 96 and 80 19.1 and 17.4 ms, of
// 256 72 ms (8 TFLOP/s).
#include "packed.cuh"
#include "serving.h"

namespace sa {

namespace {

constexpr int kRows = 16, kKeys = 32, kThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kThreads)
    packed_simt_kernel(const __grid_constant__ PackedArgs a, float scale_log2, float cap_in,
                       float cap_log2) {
  extern __shared__ float sm[];
  const int D = static_cast<int>(a.D), ld = D + 4;
  float* qs = sm;
  float* ks = qs + kRows * ld;
  float* vs = ks + kKeys * ld;
  float* ps = vs + kKeys * ld;  // [kRows][kKeys + 1]
  __shared__ int s_b, s_tile;
  const int tid = threadIdx.x, lane = tid & 31;
  const int B = static_cast<int>(a.B), Tq = static_cast<int>(a.Tq), Tk = static_cast<int>(a.Tk);

  if (blockIdx.x == 0 && blockIdx.y == 0 && a.err_word) {
    bool bad = false;
    for (int b = tid; b < B; b += kThreads)
      if (bad_span(a.q_start, b, Tq) || bad_span(a.k_start, b, Tk)) bad = true;
    if (bad) atomicOr(a.err_word, SA_ERRBIT_SEQ);
  }
  // sequence and tile of this block: the tiles of the sequences end to end
  if (tid < 32) {
    int before = 0, fb = -1, ft = 0;
    const int want = static_cast<int>(blockIdx.x);
    for (int b0 = 0; b0 < B && fb < 0; b0 += 32) {
      const int n = b0 + lane < B ? span_of(a.q_start, b0 + lane, Tq).n : 0;
      int v = (n + kRows - 1) / kRows;
      const int mine = v;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, sh);
        if (lane >= sh) v += x;
      }
      const int lo = before + v - mine;
      const unsigned hit = __ballot_sync(0xffffffffu, want >= lo && want < lo + mine);
      if (hit) {
        const int l = __ffs(hit) - 1;
        fb = b0 + l;
        ft = want - __shfl_sync(0xffffffffu, lo, l);
      }
      before += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) {
      s_b = fb;
      s_tile = ft;
    }
  }
  __syncthreads();
  if (s_b < 0) return;
  const Span q = span_of(a.q_start, s_b, Tq), k = span_of(a.k_start, s_b, Tk);
  const int h = static_cast<int>(blockIdx.y), kvh = h / static_cast<int>(a.Hq / a.Hkv);
  const int i0 = s_tile * kRows;
  const T* qp = static_cast<const T*>(a.q) + h * a.qs[1];
  const T* kp = static_cast<const T*>(a.k) + kvh * a.ks[1];
  const T* vp = static_cast<const T*>(a.v) + kvh * a.vs[1];
  for (int e = tid; e < kRows * D; e += kThreads) {
    const int r = e / D, d = e - r * D;
    qs[r * ld + d] = i0 + r < q.n ? to_f32<T>(qp[(q.first + i0 + r) * a.qs[0] + d]) : 0.f;
  }
  const int r = tid >> 3, l = tid & 7;
  const int i = i0 + r;
  int lim = k.n - 1;  // the last key this query sees
  if (a.causal) lim = min(lim, i + k.n - q.n);
  if (i >= q.n) lim = -1;
  int last = k.n - 1;  // the last key any query of the block sees
  if (a.causal) last = min(last, min(i0 + kRows, q.n) - 1 + k.n - q.n);
  float m = SA_NEG_INF, sum = 0.f;
  float4 o[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);

  for (int j0 = 0; j0 <= last; j0 += kKeys) {
    __syncthreads();
    for (int e = tid; e < kKeys * D; e += kThreads) {
      const int t = e / D, d = e - t * D;
      const bool in = j0 + t < k.n;
      ks[t * ld + d] = in ? to_f32<T>(kp[(k.first + j0 + t) * a.ks[0] + d]) : 0.f;
      vs[t * ld + d] = in ? to_f32<T>(vp[(k.first + j0 + t) * a.vs[0] + d]) : 0.f;
    }
    __syncthreads();
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int d = 0; d < D; d += 4) {
      const float4 qv = *reinterpret_cast<const float4*>(qs + r * ld + d);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float4 kv = *reinterpret_cast<const float4*>(ks + (l + 8 * x) * ld + d);
        s[x] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[x]))));
      }
    }
    float tm = SA_NEG_INF;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      s[x] = cap_log2 != 0.f ? cap_log2 * tanhf(s[x] * cap_in) : s[x] * scale_log2;
      if (j0 + l + 8 * x > lim) s[x] = SA_NEG_INF;
      tm = fmaxf(tm, s[x]);
    }
#pragma unroll
    for (int sh = 1; sh < 8; sh <<= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, sh));
    const float mn = fmaxf(m, tm), mu = mn == SA_NEG_INF ? 0.f : mn;
    const float al = exp2f(m - mu);
    m = mn;
    float part = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float p = exp2f(s[x] - mu);
      ps[r * (kKeys + 1) + l + 8 * x] = p;
      part += p;
    }
#pragma unroll
    for (int sh = 1; sh < 8; sh <<= 1) part += __shfl_xor_sync(0xffffffffu, part, sh);
    sum = sum * al + part;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      o[x].x *= al;
      o[x].y *= al;
      o[x].z *= al;
      o[x].w *= al;
    }
    __syncwarp();
    const int n = min(kKeys - 1, lim - j0);  // a hidden key's value is never touched
    for (int t = 0; t <= n; ++t) {
      const float p = ps[r * (kKeys + 1) + t];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int d = 4 * l + 32 * x;
        if (d < D) {
          const float4 v = *reinterpret_cast<const float4*>(vs + t * ld + d);
          o[x].x = fmaf(p, v.x, o[x].x);
          o[x].y = fmaf(p, v.y, o[x].y);
          o[x].z = fmaf(p, v.z, o[x].z);
          o[x].w = fmaf(p, v.w, o[x].w);
        }
      }
    }
  }
  if (i >= q.n) return;
  const float inv = sum != 0.f ? 1.0f / sum : 0.f;  // no key: 0; a NaN sum stays NaN
  T* yp = static_cast<T*>(a.y) + (q.first + i) * a.ys[0] + h * a.ys[1];
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int d = 4 * l + 32 * x;
    if (d < D) {
      yp[d] = from_f32<T>(o[x].x * inv);
      yp[d + 1] = from_f32<T>(o[x].y * inv);
      yp[d + 2] = from_f32<T>(o[x].z * inv);
      yp[d + 3] = from_f32<T>(o[x].w * inv);
    }
  }
}

template <typename T>
int launch_t(const PackedArgs& a, cudaStream_t st) {
  const float log2e = 1.4426950408889634f;
  const int64_t tiles = (a.Tq + kRows - 1) / kRows + a.B;  // at least the sequences' own
  const size_t smem = ((kRows + 2 * kKeys) * (a.D + 4) + kRows * (kKeys + 1)) * sizeof(float);
  if (!allow_smem(reinterpret_cast<const void*>(packed_simt_kernel<T>), 96 * 1024)) return -1;
  const float cap = fabsf(a.scale) > kNoCapMax * a.softcap ? a.softcap : 0.f;
  packed_simt_kernel<T><<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(a.Hq)), kThreads,
                          smem, st>>>(a, a.scale * log2e, cap != 0.f ? a.scale / cap : 0.f,
                                      cap * log2e);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_packed_simt(const PackedArgs& a, cudaStream_t st) {
  if (a.Tq == 0) return 0;
  if (a.dtype == SA_F32) return launch_t<float>(a, st);
  if (a.dtype == SA_F16) return launch_t<__half>(a, st);
  return launch_t<__nv_bfloat16>(a, st);
}

}  // namespace sa
