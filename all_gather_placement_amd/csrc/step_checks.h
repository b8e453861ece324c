// Checks of arguments shared by the entry points of libtide_step.so.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/tide_step.h"

namespace tide_step {

// TIDE_ERR_HIP for a hipError_t that is an error, which it keeps for tide_step_last_hip_error().
tide_status status_of(int hip_error);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool float_type(int t) { return t == TIDE_BF16 || t == TIDE_FP32; }
inline int size_of(int t) { return t == TIDE_BF16 ? 2 : t == TIDE_INT64 ? 8 : 4; }

struct Range {
  uintptr_t lo, hi;
  uintptr_t row = 0, stride = 0;  // bytes of each row and between rows' starts, where rows have gaps between them
};
inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + uintptr_t(bytes)};
}
// `rows` rows of `row` elements, `stride` elements apart
inline Range range_of(const void* p, int64_t rows, int64_t row, int64_t stride, int size) {
  Range r = range_of(p, rows == 0 ? 0 : ((rows - 1) * stride + row) * size);
  if (rows > 1 && stride > row) {
    r.row = uintptr_t(row * size);
    r.stride = uintptr_t(stride * size);
  }
  return r;
}
inline Range opt_range(const void* p, int64_t bytes) { return p == nullptr ? Range{0, 0} : range_of(p, bytes); }
// Blocks of columns of one buffer do not overlap though one's rows lie between the other's: of equal strides,
// or of one whose gaps hold all of the other.  Rows of different strides are taken to meet somewhere.
inline bool overlap(const Range& a, const Range& b) {
  if (!(a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi)) return false;
  const uintptr_t stride = a.stride > b.stride ? a.stride : b.stride;
  if (stride == 0 || (a.stride != b.stride && a.stride != 0 && b.stride != 0)) return true;
  const uintptr_t arow = a.stride != 0 ? a.row : a.hi - a.lo, brow = b.stride != 0 ? b.row : b.hi - b.lo;
  // where a row of a starts, counted from the row of b that starts at or before it
  const uintptr_t from = a.lo >= b.lo ? (a.lo - b.lo) % stride : (stride - (b.lo - a.lo) % stride) % stride;
  return from < brow || from + arow > stride;
}
// Whether any output lies over another output or an input; empty ranges lie over nothing.
template <size_t N, size_t M>
bool outputs_overlap(const Range (&outs)[N], const Range (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (const Range& in : ins)
      if (overlap(outs[i], in)) return true;
  }
  return false;
}

inline bool workspace_ok(const void* p, int64_t have, int64_t need) {
  return need >= 0 && have >= need && (need == 0 || (p != nullptr && aligned(p, 16)));
}

constexpr int64_t kMaxElems = int64_t(1) << 44;

inline bool matrix_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 1 && cols < (int64_t(1) << 31) && rows <= kMaxElems / cols;
}
// A matrix argument: its rows do not lie over each other, and its last element's offset fits.
inline bool strided_ok(const void* p, int64_t rows, int64_t cols, int64_t stride, int dtype) {
  if (rows == 0) return true;
  return p != nullptr && aligned(p, size_of(dtype)) && (rows == 1 || (stride >= cols && stride <= kMaxElems / rows));
}
inline bool vector_ok(const void* p, int dtype) { return aligned(p, size_of(dtype)); }

constexpr int64_t kInt31 = int64_t(1) << 31;

}  // namespace tide_step
