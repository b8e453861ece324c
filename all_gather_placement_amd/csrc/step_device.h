// Device helpers shared by the step kernels: vectors of eight elements, conversions, reductions.
#pragma once

#include <hip/hip_runtime.h>

#include <cstring>

namespace tide_step {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned short bf16_t;  // bit pattern

// 16 bytes at any element boundary: gfx950 reads and writes unaligned vectors in one instruction.
struct __attribute__((packed, aligned(2))) Any16 {
  u32x4 v;
};
__device__ __forceinline__ u32x4 load16(const void* p) {
  return reinterpret_cast<const __attribute__((address_space(1))) Any16*>((uintptr_t)p)->v;
}
__device__ __forceinline__ void store16(void* p, u32x4 v) {
  reinterpret_cast<__attribute__((address_space(1))) Any16*>((uintptr_t)p)->v = v;
}

__device__ __forceinline__ float widen(bf16_t b) { return __uint_as_float(static_cast<unsigned int>(b) << 16); }
__device__ __forceinline__ float widen(float f) { return f; }

// Round to nearest, ties to even; NaN stays NaN.
__device__ __forceinline__ unsigned int round_bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(unsigned int, v);
}
template <typename T>
__device__ __forceinline__ T narrow(float f);
template <>
__device__ __forceinline__ float narrow<float>(float f) { return f; }
template <>
__device__ __forceinline__ bf16_t narrow<bf16_t>(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}

// Eight neighbouring elements as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  u32x4 v;
  __device__ __forceinline__ float get(int i) const {
    const unsigned int w = v[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <>
struct Raw8<float> {
  u32x4 v[2];
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(v[i >> 2][i & 3]); }
};

// The first n (of 8) elements at p, zeros beyond; n <= 0 reads nothing.
__device__ __forceinline__ Raw8<bf16_t> load8(const bf16_t* p, int n) {
  Raw8<bf16_t> r;
  if (n >= 8) {
    r.v = load16(p);
  } else {
    r.v = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) r.v[i >> 1] |= static_cast<unsigned int>(p[i]) << (16 * (i & 1));
  }
  return r;
}
__device__ __forceinline__ Raw8<float> load8(const float* p, int n) {
  Raw8<float> r;
  if (n >= 8) {
    r.v[0] = load16(p);
    r.v[1] = load16(p + 4);
  } else {
    r.v[0] = r.v[1] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) r.v[i >> 2][i & 3] = __float_as_uint(p[i]);
  }
  return r;
}
__device__ __forceinline__ void store8(bf16_t* p, int n, const float f[8]) {
  if (n >= 8) {
    store16(p, u32x4{round_bf16x2(f[0], f[1]), round_bf16x2(f[2], f[3]), round_bf16x2(f[4], f[5]),
                     round_bf16x2(f[6], f[7])});
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = narrow<bf16_t>(f[i]);
  }
}
__device__ __forceinline__ void store8(float* p, int n, const float f[8]) {
  if (n >= 8) {
    store16(p, __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]}));
    store16(p + 4, __builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]}));
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = f[i];
  }
}

// Sum over aligned groups of L lanes (a power of two up to 64), the same in every lane of a group.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace tide_step
