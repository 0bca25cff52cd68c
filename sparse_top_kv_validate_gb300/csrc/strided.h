// strided.h -- host-side argument checks of the serving-step entry points: tensors
// given by strides, alignment, and whether two of them can share a byte.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/sa.h"

namespace {

constexpr int64_t kMaxInt = int64_t(1) << 31;
// Tokens of a call: the kernels' indexes run past the last token by less than a block.
constexpr int64_t kMaxTokens = kMaxInt - 256;

[[maybe_unused]] size_t dtype_bytes(int dt) { return dt == SA_F32 ? 4 : (dt == SA_F16 || dt == SA_BF16) ? 2 : 0; }

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A tensor [outer..., D] with D contiguous: up to three outer axes (outermost
// first) with element strides.
struct Strided {
  const void* p;
  size_t es;
  int axes;
  int64_t n[3], st[3], D;

  // 16-byte accesses at every row are legal
  bool vec16() const {
    bool ok = aligned(p, 16);
    for (int i = 0; i < axes; ++i) ok = ok && (n[i] <= 1 || st[i] * static_cast<int64_t>(es) % 16 == 0);
    return ok;
  }
  bool strides_ok() const {
    for (int i = 0; i < axes; ++i)  // (no device holds 2^58 elements: extent() stays in 64 bits)
      if (n[i] > 1 && (st[i] < 0 || st[i] >= (int64_t(1) << 40) || st[i] > (int64_t(1) << 58) / n[i])) return false;
    return true;
  }
  // No two elements share an address.
  bool distinct() const {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < axes; ++i)
      for (int j = i + 1; j < axes; ++j)
        if (st[order[j]] < st[order[i]]) {
          const int t = order[i];
          order[i] = order[j];
          order[j] = t;
        }
    int64_t span = D;
    for (int i = 0; i < axes; ++i) {
      const int ax = order[i];
      if (n[ax] <= 1) continue;
      if (st[ax] < span) return false;
      span += (n[ax] - 1) * st[ax];
    }
    return true;
  }
  bool empty() const {
    if (!p) return true;
    for (int i = 0; i < axes; ++i)
      if (n[i] <= 0) return true;
    return false;
  }
  size_t extent() const {  // bytes from the first element's to past the last's
    int64_t e = D;
    for (int i = 0; i < axes; ++i) e += (n[i] - 1) * (n[i] > 1 ? st[i] : 0);
    return static_cast<size_t>(e) * es;
  }
};

bool ranges_meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

// Elements that a tensor takes of every `period` (its axes of smaller strides), or -1
// when it is not a block that repeats with the period.
int64_t block_of(const Strided& t, int64_t period) {
  int64_t e = t.D;
  for (int i = 0; i < t.axes; ++i) {
    if (t.n[i] <= 1) continue;
    if (t.st[i] < period) e += (t.n[i] - 1) * t.st[i];
    else if (t.st[i] % period) return -1;
  }
  return e <= period ? e : -1;
}

// Whether two tensors can share a byte.  Tensors whose rows interleave (heads of one
// projection's output, token-major or head-major, in any number of batches) are told
// apart by their places inside a stride that both repeat with.
[[maybe_unused]] bool overlap(const Strided& a, const Strided& b) {
  if (a.empty() || b.empty()) return false;
  if (!ranges_meet(a.p, a.extent(), b.p, b.extent())) return false;
  if (a.es != b.es) return true;
  const int64_t es = static_cast<int64_t>(a.es);
  for (const Strided* t : {&a, &b})
    for (int i = 0; i < t->axes; ++i) {
      const int64_t period = t->st[i];
      if (t->n[i] <= 1 || period <= 0) continue;
      const int64_t la = block_of(a, period), lb = block_of(b, period);
      if (la < 0 || lb < 0) continue;
      int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) %
                  (period * es);
      if (d < 0) d += period * es;
      if (d >= la * es && d + lb * es <= period * es) return false;
    }
  return true;
}

[[maybe_unused]] bool same(const Strided& a, const Strided& b) {
  if (a.p != b.p) return false;
  for (int i = 0; i < a.axes; ++i)
    if (a.n[i] > 1 && a.st[i] != b.st[i]) return false;
  return true;
}

}  // namespace
