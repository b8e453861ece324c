// Launch shapes, and scans over lanes, shared by the kernels that work on tokens and rows.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace tide_step {

// Workgroups for n items, `per` each: a launch holds less than 2^32 threads, so kernels go on to the
// items a grid further.
constexpr int64_t kMaxGrid = int64_t(1) << 21;
__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline unsigned grid_of(int64_t n, int64_t per) {
  const int64_t g = ceil_div(n, per);
  return unsigned(g < kMaxGrid ? g : kMaxGrid);
}

// The elements of a vector that are left, at most E.
template <int E>
__device__ __forceinline__ int tail(int64_t n) {
  return int(n < E ? n : E);
}

// One step of a scan on the VALU: adds what the lane that kCtrl names has, in the rows of kRows.
template <int kCtrl, int kRows>
__device__ __forceinline__ int dpp_step(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, kCtrl, kRows, 0xf, false);
}
// Inclusive sum over the wave.
__device__ __forceinline__ int wave_scan(int v) {
  v = dpp_step<0x111, 0xf>(v);  // a lane lower, in rows of 16 lanes
  v = dpp_step<0x112, 0xf>(v);  // 2 lanes
  v = dpp_step<0x114, 0xf>(v);  // 4
  v = dpp_step<0x118, 0xf>(v);  // 8
  v = dpp_step<0x142, 0xa>(v);  // the last lane of row 0 to row 1, of row 2 to row 3
  return dpp_step<0x143, 0xc>(v);  // the last lane of row 1 to rows 2 and 3
}

// Lanes of m below this one.
__device__ __forceinline__ int lanes_before(uint64_t m) {
  return int(__builtin_amdgcn_mbcnt_hi(unsigned(m >> 32), __builtin_amdgcn_mbcnt_lo(unsigned(m), 0)));
}

}  // namespace tide_step
