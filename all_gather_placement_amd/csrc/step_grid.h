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

// Inclusive sum over the wave.
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d, 64);
    if (lane >= d) v += u;
  }
  return v;
}

// Lanes of m below this one.
__device__ __forceinline__ int lanes_before(uint64_t m) {
  return int(__builtin_amdgcn_mbcnt_hi(unsigned(m >> 32), __builtin_amdgcn_mbcnt_lo(unsigned(m), 0)));
}

}  // namespace tide_step
