// Device helpers shared by the step kernels: vectors of elements, conversions, reductions.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

namespace tide_step {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned short bf16_t;  // bit pattern

// 16 and 8 bytes at any element boundary: gfx950 reads and writes unaligned vectors in one instruction.
// kOnce marks what is read or written once (non-temporal): it does not push out what is used again.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
#define TIDE_STEP_GLOBAL __attribute__((address_space(1)))
template <bool kOnce = false>
__device__ __forceinline__ u32x4 load16(const void* p) {
  const TIDE_STEP_GLOBAL u32x4_any* g = reinterpret_cast<const TIDE_STEP_GLOBAL u32x4_any*>((uintptr_t)p);
  if constexpr (kOnce) return __builtin_nontemporal_load(g);
  return *g;
}
template <bool kOnce = false>
__device__ __forceinline__ void store16(void* p, u32x4 v) {
  TIDE_STEP_GLOBAL u32x4_any* g = reinterpret_cast<TIDE_STEP_GLOBAL u32x4_any*>((uintptr_t)p);
  if constexpr (kOnce)
    __builtin_nontemporal_store(v, g);
  else
    *g = v;
}
__device__ __forceinline__ u32x2 load8(const void* p) {
  return *reinterpret_cast<const TIDE_STEP_GLOBAL u32x2_any*>((uintptr_t)p);
}

// Keeps the scheduler from putting the use of one load before the next load of a group.
__device__ __forceinline__ void loads_first() { __builtin_amdgcn_sched_barrier(0); }

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

// E neighbouring elements as they lie in memory: 8, 16 or 32 bytes.
template <typename T, int E>
struct Raw {
  static constexpr int kWords = E * int(sizeof(T)) / 4;
  unsigned int w[kWords];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 2) {
      const unsigned int u = w[i >> 1];
      return __uint_as_float((i & 1) ? (u & 0xffff0000u) : (u << 16));
    } else {
      return __uint_as_float(w[i]);
    }
  }
  // Keeps the compiler from holding values made of this vector (twice the registers for bf16) until
  // they are used again: beyond this point they are made again.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int q = 0; q < kWords; ++q) asm volatile("" : "+v"(w[q]));
  }
};

template <typename T, int E, bool kOnce>
__device__ __forceinline__ Raw<T, E> load_whole(const T* p) {
  Raw<T, E> r;
  if constexpr (r.kWords == 2) {
    const u32x2 v = load8(p);
    r.w[0] = v[0];
    r.w[1] = v[1];
  } else {
#pragma unroll
    for (int q = 0; q < r.kWords / 4; ++q) {
      const u32x4 v = load16<kOnce>(reinterpret_cast<const char*>(p) + 16 * q);
#pragma unroll
      for (int k = 0; k < 4; ++k) r.w[4 * q + k] = v[k];
    }
  }
  return r;
}
// Moves elements s, s + 1, ... (s < E) to the front, zeros behind them.
template <typename T, int E>
__device__ __forceinline__ void drop_front(Raw<T, E>& r, int s) {
  constexpr int W = Raw<T, E>::kWords;
  const int words = sizeof(T) == 2 ? s >> 1 : s;
#pragma unroll
  for (int bit = W / 2; bit >= 1; bit >>= 1)
    if (words & bit) {
#pragma unroll
      for (int k = 0; k < W; ++k) r.w[k] = k + bit < W ? r.w[k + bit] : 0;
    }
  if (sizeof(T) == 2 && (s & 1)) {
#pragma unroll
    for (int k = 0; k < W; ++k) r.w[k] = r.w[k] >> 16 | (k + 1 < W ? r.w[k + 1] << 16 : 0);
  }
}
// The first n (of E) elements at p, zeros beyond; n <= 0 reads nothing.  With kWhole rows are of whole
// vectors and n is E or more where it is not 0 or less.  Otherwise, where the row has E elements
// (`wide`), its end is read as the vector that ends there: a load for each element, and their waits,
// would take longer than all the rest of a row.
template <typename T, int E, bool kOnce, bool kWhole>
__device__ __forceinline__ Raw<T, E> load_vec(const T* p, int n, bool wide) {
  Raw<T, E> r;
#pragma unroll
  for (int q = 0; q < r.kWords; ++q) r.w[q] = 0;
  if constexpr (kWhole) {
    if (n > 0) r = load_whole<T, E, kOnce>(p);
  } else if (wide) {
    if (n > 0) r = load_whole<T, E, kOnce>(n < E ? p + (n - E) : p);
    if (n > 0 && n < E) drop_front(r, E - n);
  } else {
    unsigned int e[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      e[i] = 0;
      if (i < n) {
        if constexpr (sizeof(T) == 2)
          e[i] = p[i];
        else
          e[i] = __float_as_uint(p[i]);
      }
    }
#pragma unroll
    for (int q = 0; q < r.kWords; ++q) {
      if constexpr (sizeof(T) == 2)
        r.w[q] = e[2 * q] | e[2 * q + 1] << 16;
      else
        r.w[q] = e[q];
    }
  }
  return r;
}
// N vectors, vector j at p[j] + c, as load_vec: their loads follow each other without a branch or a
// wait.  The addresses p are made before, where all lanes are active: a lane that is not has no value
// to give.
template <typename T, int E, int N, bool kOnce, bool kWhole>
__device__ __forceinline__ void load_vecs(Raw<T, E> (&r)[N], const T* const (&p)[N], int64_t c, int n, bool wide) {
  if (kWhole || wide) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int q = 0; q < Raw<T, E>::kWords; ++q) r[j].w[q] = 0;
    if (n > 0) {
      const int64_t at = !kWhole && n < E ? c + (n - E) : c;
#pragma unroll
      for (int j = 0; j < N; ++j) r[j] = load_whole<T, E, kOnce>(p[j] + at);
      loads_first();
      if (!kWhole && n < E) {
#pragma unroll
        for (int j = 0; j < N; ++j) drop_front(r[j], E - n);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) r[j] = load_vec<T, E, kOnce, false>(p[j] + c, n, false);
  }
}
// The first n (of E) values of f to p, rounded; kWhole as for load_vec.
template <typename T, int E, bool kOnce, bool kWhole>
__device__ __forceinline__ void store_vec(T* p, int n, const float (&f)[E]) {
  if (n >= E) {
    unsigned int w[Raw<T, E>::kWords];
#pragma unroll
    for (int q = 0; q < Raw<T, E>::kWords; ++q) {
      if constexpr (sizeof(T) == 2)
        w[q] = round_bf16x2(f[2 * q], f[2 * q + 1]);
      else
        w[q] = __float_as_uint(f[q]);
    }
    static_assert(Raw<T, E>::kWords % 4 == 0, "stores are of 16 bytes");
#pragma unroll
    for (int q = 0; q < Raw<T, E>::kWords / 4; ++q)
      store16<kOnce>(reinterpret_cast<char*>(p) + 16 * q, u32x4{w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]});
  } else if constexpr (!kWhole) {
#pragma unroll
    for (int i = 0; i < E - 1; ++i)
      if (i < n) p[i] = narrow<T>(f[i]);
  }
}
// The first n (of E) elements of r to p, bit for bit; kWhole as for load_vec.
template <typename T, int E, bool kOnce, bool kWhole>
__device__ __forceinline__ void store_raw(T* p, int n, const Raw<T, E>& r) {
  if (n >= E) {
    static_assert(Raw<T, E>::kWords % 4 == 0, "stores are of 16 bytes");
#pragma unroll
    for (int q = 0; q < Raw<T, E>::kWords / 4; ++q)
      store16<kOnce>(reinterpret_cast<char*>(p) + 16 * q,
                     u32x4{r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]});
  } else if constexpr (!kWhole) {
#pragma unroll
    for (int i = 0; i < E - 1; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2)
          p[i] = T(i & 1 ? r.w[i / 2] >> 16 : r.w[i / 2]);
        else
          p[i] = __uint_as_float(r.w[i]);
      }
  }
}
// f(whole) as a constant: rows of `cols` elements are of whole vectors of E, or not.
template <int E, typename F>
int with_whole(int64_t cols, F&& f) {
  return cols % E == 0 ? f(std::true_type()) : f(std::false_type());
}
// Launches a kernel and returns its own status (a hipError_t): what an earlier call of another library left
// behind is neither reported nor cleared.  A call ends at its first failed launch, since later kernels read
// what earlier ones write.
template <typename T>
struct Same {
  typedef T type;
};
template <typename... P>
int launch(void (*kernel)(P...), dim3 grid, int threads, size_t lds, hipStream_t s,
           const typename Same<P>::type&... args) {
  void* p[] = {const_cast<void*>(static_cast<const void*>(&args))...};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), p, lds, s);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}
// Elements of a 16-byte vector.
template <typename T>
constexpr int kVec = 16 / int(sizeof(T));

// One step of a sum within rows of 16 lanes, on the VALU (no LDS traffic).
template <int kCtrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, true));
}
// Sum over aligned groups of L lanes (a power of two up to 64), the same in every lane of a group.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L >= 2) v = dpp_add<0xb1>(v);   // lane ^ 1
  if constexpr (L >= 4) v = dpp_add<0x4e>(v);   // lane ^ 2
  if constexpr (L >= 8) v = dpp_add<0x141>(v);  // mirrored within 8: the other quad
  if constexpr (L >= 16) v = dpp_add<0x140>(v); // mirrored within 16: the other half
  if constexpr (L >= 32) {  // rows 0 and 1, 2 and 3
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L >= 64) {  // the halves of the wave
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace tide_step
