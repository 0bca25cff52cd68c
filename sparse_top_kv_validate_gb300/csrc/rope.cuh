// rope.cuh -- rotary positions: angle reduction and the rotation of a 16-element
// chunk, shared by the rotary and the page-write kernels.
#pragma once

#include "common.cuh"

namespace sa {

// cos and sin (times m) of position * f, f given as a 64-bit fraction of a
// turn: the product modulo 2^64 is the fraction of a turn of the angle, exact for
// the fraction given; its top 32 bits, as a signed number of half turns rounded to
// fp32 (24 bits: off by at most 2^-25 of a half turn), go through sincospi.  (An
// fp32 product position * f has lost every fraction bit of the angle by position
// 2^24.)  The fraction itself comes from a double: the frequency is off by up to
// about 2^-53 of itself, and the angle by that many times as far as it turned.
__device__ __forceinline__ float2 rope_cos_sin(int64_t pos, uint64_t turns, float m) {
  const uint64_t phase = static_cast<uint64_t>(pos) * turns;
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * m, s * m);
}

// The fraction of pair i, by an ordinary load: the kernel's parameters lie in
// constant memory, which serves a warp one address at a time (read that way, the
// tables took 6 of the page write's 31 us for 16,384 tokens).
__device__ __forceinline__ uint64_t turn_of(const sa_rope& rope, int i) {
  uint64_t f;
  asm volatile("ld.u64 %0, [%1];" : "=l"(f) : "l"(&rope.turns[i]));
  return f;
}

// The tables of a tile's tokens in shared memory, [n][cos, sin][half], by a block of
// kThreads.  Made before the positions are known, so that its load is under way.
template <int kThreads>
struct TurnTables {
  int half, dk, di, k, i;
  uint64_t f;
  __device__ __forceinline__ explicit TurnTables(const sa_rope& rope) {
    half = max(rope.rotary_dim / 2, 1);  // (no rotation: one pair's table, not filled)
    dk = kThreads / half;
    di = kThreads - dk * half;
    k = threadIdx.x / half;
    i = threadIdx.x - k * half;
    f = turn_of(rope, i);
  }
  // pos(k): token k's position, for n tokens.
  template <typename Pos>
  __device__ __forceinline__ void fill(const sa_rope& rope, int n, Pos pos, float* table) {
    while (k < n) {
      const float2 cs = rope_cos_sin(pos(k), f, rope.mscale);
      table[2 * k * half + i] = cs.x;
      table[(2 * k + 1) * half + i] = cs.y;
      k += dk;
      if (di == 0) continue;
      i += di;
      if (i >= half) {
        i -= half;
        ++k;
      }
      f = turn_of(rope, i);
    }
  }
};

// A lane's two 8-element pieces of a row of D elements, chunk c of D / 16:
// neighbouring lanes' pieces are neighbours, so that an access of a row's lanes
// is one run.  Half layout: the two sides of pairs 8c .. 8c + 7, and past
// rotary_dim the two halves of the rest; interleaved: the halves of the row,
// each piece four whole pairs.
struct Pieces {
  int d[2];      // first elements
  bool turn[2];  // below rotary_dim
};
template <bool kInter>
__device__ __forceinline__ Pieces pieces_of(int c, int D, int rot) {
  Pieces p;
  if (kInter) {
    p.d[0] = 8 * c;
    p.d[1] = D / 2 + 8 * c;
    p.turn[0] = p.d[0] < rot;
    p.turn[1] = p.d[1] < rot;
  } else {
    const bool in = 16 * c < rot;
    const int from = in ? 0 : rot, width = in ? rot : D - rot, cc = c - from / 16;
    p.d[0] = from + 8 * cc;
    p.d[1] = p.d[0] + width / 2;
    p.turn[0] = p.turn[1] = in;
  }
  return p;
}

// Two fp32 values side by side: one instruction multiplies both.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_split(F2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// A piece's elements as four F2: neighbours, or for the interleaved layout the
// same side of two neighbouring pairs.
struct Piece {
  F2 x[4];
};
template <bool kInter>
__device__ __forceinline__ Piece piece_from(const float (&f)[8]) {
  if (kInter) return Piece{f2(f[0], f[2]), f2(f[1], f[3]), f2(f[4], f[6]), f2(f[5], f[7])};
  return Piece{f2(f[0], f[1]), f2(f[2], f[3]), f2(f[4], f[5]), f2(f[6], f[7])};
}
template <bool kInter>
__device__ __forceinline__ void piece_to(const Piece& p, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = kInter ? 4 * (i / 2) + i % 2 : 2 * i;
    f2_split(p.x[i], f[at], f[at + (kInter ? 2 : 1)]);
  }
}

// Cosines and sines of a lane's eight pairs, two pairs to an F2; interleaved:
// the first piece's four, then the second's.
struct Turns {
  F2 c[4], s[4];
};

// From a token's table in shared memory: `half` cosines, then `half` sines.
__device__ __forceinline__ void four_turns(const float* at, int half, F2* c, F2* s) {
  const float4 x = *reinterpret_cast<const float4*>(at);
  const float4 y = *reinterpret_cast<const float4*>(at + half);
  c[0] = f2(x.x, x.y);
  c[1] = f2(x.z, x.w);
  s[0] = f2(y.x, y.y);
  s[1] = f2(y.z, y.w);
}
template <bool kInter>
__device__ __forceinline__ Turns turns_of(const float* table, int half, const Pieces& p) {
  Turns t;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!p.turn[i]) {
      t.c[2 * i] = t.c[2 * i + 1] = t.s[2 * i] = t.s[2 * i + 1] = F2{0};
      continue;
    }
    const float* at = table + (kInter ? p.d[i] / 2 : p.d[0] + 4 * i);
    four_turns(at, half, t.c + 2 * i, t.s + 2 * i);
  }
  return t;
}

// (u, v) -> (u c - v s, u s + v c) for two pairs at once.
__device__ __forceinline__ void rotate2(F2& u, F2& v, F2 c, F2 s) {
  const F2 a = f2_mul(u, c), b = f2_mul(v, c);
  const F2 w = f2_fma(f2_mul(v, s), f2(-1.f, -1.f), a);
  v = f2_fma(u, s, b);
  u = w;
}

// Rotate a lane's two pieces.
template <bool kInter>
__device__ __forceinline__ void rotate_pieces(Piece& a, Piece& b, const Turns& t, const Pieces& p) {
  if (kInter) {
    if (p.turn[0]) {
      rotate2(a.x[0], a.x[1], t.c[0], t.s[0]);
      rotate2(a.x[2], a.x[3], t.c[1], t.s[1]);
    }
    if (p.turn[1]) {
      rotate2(b.x[0], b.x[1], t.c[2], t.s[2]);
      rotate2(b.x[2], b.x[3], t.c[3], t.s[3]);
    }
  } else if (p.turn[0]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) rotate2(a.x[i], b.x[i], t.c[i], t.s[i]);
  }
}

// The same with the turns read as they are needed: sixteen registers fewer.
template <bool kInter>
__device__ __forceinline__ void rotate_pieces(Piece& a, Piece& b, const float* table, int half,
                                              const Pieces& p) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!p.turn[i]) continue;
    F2 c[2], s[2];
    four_turns(table + (kInter ? p.d[i] / 2 : p.d[0] + 4 * i), half, c, s);
    if (kInter) {
      Piece& x = i ? b : a;
      rotate2(x.x[0], x.x[1], c[0], s[0]);
      rotate2(x.x[2], x.x[3], c[1], s[1]);
    } else {
      rotate2(a.x[2 * i], b.x[2 * i], c[0], s[0]);
      rotate2(a.x[2 * i + 1], b.x[2 * i + 1], c[1], s[1]);
    }
  }
}

// ---- eight elements of a row as raw registers --------------------------------------------

template <typename T>
struct Raw8 {
  uint4 r[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& v, float (&f)[8]) {
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_f32<T>(e[i]);
}

template <typename T>
__device__ __forceinline__ void store_raw(T* p, const Raw8<T>& v) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    *(reinterpret_cast<uint4*>(p) + i) = v.r[i];
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  Raw8<T> v;
  T* e = reinterpret_cast<T*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(f[i]);
  store_raw<T>(p, v);
}

// ---- a thread's rows on their way through shared memory ------------------------------------
//
// Each thread copies its own two pieces of a row, asynchronously, kRowsAhead
// rows before it needs them, and no other thread reads them: no barrier, no
// registers for loads in flight, and a loop over the rows that is not unrolled.
// (Loads to registers, four rows unrolled, took 104 registers: two blocks to an SM.)
constexpr int kRingThreads = 256;

template <typename T>
struct RowRing {
  static constexpr int kParts = sizeof(T) / 2;                 // 16-byte parts of a piece
  static constexpr int kRowsAhead = sizeof(T) == 4 ? 2 : 4;
  static constexpr int kBytes = kRowsAhead * 2 * kParts * 16 * kRingThreads;
  uint4* own;

  __device__ __forceinline__ explicit RowRing(void* smem)
      : own(static_cast<uint4*>(smem) + threadIdx.x) {}
  __device__ __forceinline__ uint4* part(uint32_t row, int piece, int i) {
    return own + (((row % kRowsAhead) * 2 + piece) * kParts + i) * kRingThreads;
  }
  __device__ __forceinline__ void fetch(int row, int piece, const T* p, bool aligned) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      if (aligned) {
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(part(row, piece, i)));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to),
                     "l"(p + i * (16 / sizeof(T)))
                     : "memory");
      } else {
        T* e = reinterpret_cast<T*>(part(row, piece, i));
#pragma unroll 1
        for (int j = 0; j < static_cast<int>(16 / sizeof(T)); ++j)
          e[j] = p[i * (16 / sizeof(T)) + j];
      }
    }
  }
  // One per row, whether it was fetched or not: `arrived` counts them.
  static __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  static __device__ __forceinline__ void arrived() {  // the oldest of kRowsAhead rows
    asm volatile("cp.async.wait_group %0;" ::"n"(kRowsAhead - 1) : "memory");
  }
  __device__ __forceinline__ Raw8<T> get(int row, int piece) {
    Raw8<T> v;
#pragma unroll
    for (int i = 0; i < kParts; ++i) v.r[i] = *part(row, piece, i);
    return v;
  }
};

}  // namespace sa
