// Host-side checks that the entry points of packed rows share: limits, alignment, and whether buffers
// share a byte.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/seed.h"

namespace seed {

inline constexpr int64_t kMostRows = (int64_t{1} << 31) - 1;  // offsets are int32
inline constexpr int64_t kMostStride = int64_t{1} << 40;      // a row's bytes stay far inside 64 bits
inline constexpr int64_t kMostBytes = int64_t{1} << 56;       // of a buffer, so that its offsets and end stay inside 64 bits

inline bool io_ok(int32_t d) { return d == SEED_F32 || d == SEED_BF16 || d == SEED_F16; }
inline int64_t io_bytes(int32_t d) { return d == SEED_F32 ? 4 : 2; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? SEED_OK : SEED_ERR_HIP; }
inline bool aligned(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(to - 1)) == 0; }
inline bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride <= kMostStride; }

// `rows` rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, stride, width;
  // within the address range that the kernels' and these checks' arithmetic holds
  bool fits() const { return p == nullptr || rows <= 0 || stride <= 0 || (rows <= kMostBytes / stride && lo() <= UINTPTR_MAX - kMostBytes); }
  uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t hi() const { return lo() + static_cast<uintptr_t>((rows - 1) * stride + width); }
};

// Whether two row buffers share a byte. Rows of one stride may interleave (two column ranges of the
// same rows); buffers of different strides whose ranges meet count as sharing.
inline bool overlap(const Rows& a, const Rows& b) {
  if (a.p == nullptr || b.p == nullptr || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  if (a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
  if (a.stride != b.stride) return true;
  const uintptr_t st = static_cast<uintptr_t>(a.stride);
  const uintptr_t d = b.lo() >= a.lo() ? (b.lo() - a.lo()) % st : (st - (a.lo() - b.lo()) % st) % st;
  // row i of b starts d behind some row position of a and ends before the next one
  return !(d >= static_cast<uintptr_t>(a.width) && d + static_cast<uintptr_t>(b.width) <= st);
}
// A buffer of `count` times `bytes` bytes.
inline Rows flat(const void* p, int64_t count, int64_t bytes) { return Rows{p, count, bytes, bytes}; }
inline bool all_fit(std::initializer_list<Rows> all) {
  for (const Rows& r : all)
    if (!r.fits()) return false;
  return true;
}
// Whether one of `outs` shares a byte with one of `ins` or with another of `outs`.
inline bool any_overlap(std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
  for (const Rows* o = outs.begin(); o != outs.end(); ++o) {
    for (const Rows& i : ins)
      if (overlap(*o, i)) return true;
    for (const Rows* p = o + 1; p != outs.end(); ++p)
      if (overlap(*o, *p)) return true;
  }
  return false;
}
// The same rows exactly: reading and writing them in place.
inline bool same(const Rows& a, const Rows& b) { return a.p == b.p && (a.stride == b.stride || a.rows <= 1); }

}  // namespace seed
