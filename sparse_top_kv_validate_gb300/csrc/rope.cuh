// rope.cuh -- rotary positions: exact angle reduction and the rotation of a
// 16-element chunk, shared by the rotary and the page-write kernels.
#pragma once

#include "common.cuh"

namespace sa {

// cos and sin (times m) of position * f, f given as a 64-bit fraction of a
// turn: the product modulo 2^64 is the fraction of a turn of the angle, exact
// at any position; its top 32 bits as a signed number of half turns go through
// sincospi.  (An fp32 product position * f has lost every fraction bit of the
// angle by position 2^24; this one keeps 32 of them.)
__device__ __forceinline__ float2 rope_cos_sin(int64_t pos, uint64_t turns, float m) {
  const uint64_t phase = static_cast<uint64_t>(pos) * turns;
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * m, s * m);
}

// A lane's two 8-element pieces of a row for chunk c (of D / 16): the first
// elements of the pieces.  Half layout: dims 8c .. and rotary_dim / 2 + 8c ..,
// the two sides of pairs 8c .. 8c + 7; interleaved, or past rotary_dim: 16
// consecutive dims (pairs 8c .. 8c + 7 again when they are rotated).
__device__ __forceinline__ void chunk_dims(int c, int rot, int interleaved, int& d0, int& d1) {
  if (!interleaved && 16 * c < rot) {
    d0 = 8 * c;
    d1 = rot / 2 + 8 * c;
  } else {
    d0 = 16 * c;
    d1 = d0 + 8;
  }
}

// Rotate the two pieces by the chunk's eight (cos, sin).
__device__ __forceinline__ void rotate_chunk(float (&a)[8], float (&b)[8], const float2 (&cs)[8],
                                             int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = a[2 * i], v = a[2 * i + 1];
      a[2 * i] = u * cs[i].x - v * cs[i].y;
      a[2 * i + 1] = u * cs[i].y + v * cs[i].x;
      const float w = b[2 * i], z = b[2 * i + 1];
      b[2 * i] = w * cs[4 + i].x - z * cs[4 + i].y;
      b[2 * i + 1] = w * cs[4 + i].y + z * cs[4 + i].x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = a[i], v = b[i];
      a[i] = u * cs[i].x - v * cs[i].y;
      b[i] = u * cs[i].y + v * cs[i].x;
    }
  }
}

// ---- eight elements of a row as raw registers --------------------------------------------

template <typename T>
struct Raw8 {
  uint4 r[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> v;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    v.r[i] = *(reinterpret_cast<const uint4*>(p) + i);
  return v;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& v, float (&f)[8]) {
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_f32<T>(e[i]);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  Raw8<T> v;
  T* e = reinterpret_cast<T*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(f[i]);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    *(reinterpret_cast<uint4*>(p) + i) = v.r[i];
}

}  // namespace sa
