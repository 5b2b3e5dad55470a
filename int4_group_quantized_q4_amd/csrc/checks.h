// Host-side checks and small sums shared by the entry points' files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

namespace {

constexpr int kLayerEmpty = 1;   // of a check: nothing to enqueue

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int launch_status() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? W4_OK : W4_ERR_HIP;
}

// (An empty part overlaps nothing.)
inline bool overlap(const void* p, size_t pn, const void* q, size_t qn) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && pn && qn && a < b + qn && b < a + pn;
}

inline int log2_of(int64_t v) {
  int s = 0;
  while (((int64_t)1 << s) < v) ++s;
  return s;
}

// Rows of the caller's k / v / q: 16-byte aligned, `stride` elements apart.
inline int check_rows(const void* p, int64_t rows, int64_t stride, int64_t width) {
  if (!p || !aligned16(p)) return W4_ERR_ARG;
  if (stride < width || stride % 8 != 0) return W4_ERR_ARG;
  return rows > 0 && stride > ((int64_t)1 << 48) / rows ? W4_ERR_SHAPE : W4_OK;
}

inline size_t rows_bytes(int64_t rows, int64_t stride, int64_t width, int64_t element) {
  return (size_t)(((rows - 1) * stride + width) * element);
}

// Two sets of rows (of pw and qw elements) that share memory; rows of one buffer
// side by side, a stride apart, do not.
inline bool rows_overlap(const void* p, int64_t ps, int64_t pw, const void* q, int64_t qs, int64_t qw, int64_t rows,
                         int64_t element) {
  if (!overlap(p, rows_bytes(rows, ps, pw, element), q, rows_bytes(rows, qs, qw, element))) return false;
  if (ps != qs) return true;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  const uintptr_t pitch = (uintptr_t)(ps * element);
  const uintptr_t off = b >= a ? (b - a) % pitch : (pitch - (a - b) % pitch) % pitch;   // of q's row behind p's
  return off < (uintptr_t)(pw * element) || pitch - off < (uintptr_t)(qw * element);
}

}  // namespace
