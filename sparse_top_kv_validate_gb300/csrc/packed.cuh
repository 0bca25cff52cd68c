// packed.cuh -- sequences packed one after the other, shared by the packed
// prefill kernels.
#pragma once

#include "common.cuh"

namespace sa {

// |scale| / softcap up to which a softcap does nothing: with k1 that quotient,
// softcap tanh(k1 s) = scale s to fp32's last bit for |s| up to 2^-12 / k1 = 2.4e5.
// (softcap log2(e), which the kernels work with, leaves fp32 at the top of its range.)
constexpr float kNoCapMax = 1e-9f;

// Rows [first, first + n) of sequence b among `total`; starts that decrease or
// leave the tensor are clipped (and reported by whoever checks them).
struct Span {
  int first, n;
};
__device__ __forceinline__ Span span_of(const int32_t* start, int b, int total) {
  const int s = min(max(__ldg(start + b), 0), total);
  const int e = min(max(__ldg(start + b + 1), s), total);
  return Span{s, e - s};
}

__device__ __forceinline__ bool bad_span(const int32_t* start, int b, int total) {
  const int s = __ldg(start + b), e = __ldg(start + b + 1);
  return s < 0 || e < s || e > total;
}

}  // namespace sa
