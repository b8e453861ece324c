// Dropout by a counter-based generator, added to a residual.
//
//   out = x * 65536 / (65536 - t) + residual where the element's 16 bits are at least t, else the residual
//
// Philox4x32 with 10 rounds makes the bits of eight neighbouring elements from the seed and their number, so
// no mask is stored or read: HBM bounds it, each element read and written once (32760 x 5120 bf16 with a residual
// 158 us, 6.4 TB/s).  16 bits an element, not 32: a round's two 64-bit products run at a quarter of the rate of other
// integer operations, and at four elements a call they would take as long as the memory does.
#include "step_device.h"
#include "step_grid.h"
#include "step_internal.h"

namespace tide_step {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 8;  // elements of a call of the generator

__device__ __forceinline__ void philox(uint64_t counter, uint64_t seed, uint32_t (&c)[4]) {
  c[0] = uint32_t(counter), c[1] = uint32_t(counter >> 32), c[2] = 0, c[3] = 0;
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(c[0]) * 0xD2511F53u, b = uint64_t(c[2]) * 0xCD9E8D57u;
    c[0] = uint32_t(b >> 32) ^ c[1] ^ k0;
    c[1] = uint32_t(b);
    c[2] = uint32_t(a >> 32) ^ c[3] ^ k1;
    c[3] = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

__device__ __forceinline__ uint64_t seed_of(const DropoutArgs& a) {
  return a.seed_device != nullptr ? uint64_t(*a.seed_device) : a.seed;
}

// A unit's elements: all of them, or those from lo to hi - 1.  Element k is x[k].
template <typename T, bool kResidual, bool kOnce>
struct Unit {
  int64_t at;  // of element 0 in the row
  int lo, hi;
  Raw<T, kUnit> r, s;
  __device__ __forceinline__ bool whole() const { return lo <= 0 && hi >= kUnit; }
  __device__ __forceinline__ void place(int64_t first, int64_t cols) {
    at = first;
    lo = at < 0 ? int(-at) : 0;
    hi = cols - at < kUnit ? int(cols - at) : kUnit;  // 0 or less: nothing
  }
  __device__ __forceinline__ void load(const T* x, const T* residual) {
    if (hi <= 0) return;
    if (whole()) {
      r = load_whole<T, kUnit, kOnce>(x + at);
      if constexpr (kResidual) s = load_whole<T, kUnit, kOnce>(residual + at);
    } else {
#pragma unroll
      for (int k = 0; k < kUnit; ++k) {
        const bool in = k >= lo && k < hi;
        put(r, k, in ? x[at + k] : T(0));
        if constexpr (kResidual) put(s, k, in ? residual[at + k] : T(0));
      }
    }
  }
  static __device__ __forceinline__ void put(Raw<T, kUnit>& v, int k, T value) {
    if constexpr (sizeof(T) == 2)
      v.w[k / 2] = k & 1 ? v.w[k / 2] | unsigned(value) << 16 : unsigned(value);
    else
      v.w[k] = __float_as_uint(value);
  }
  __device__ __forceinline__ void store(const DropoutArgs& a, uint64_t counter, uint64_t seed, T* out) {
    if (hi <= 0) return;
    uint32_t bits[4];
    philox(counter, seed, bits);
    float v[kUnit];
#pragma unroll
    for (int k = 0; k < kUnit; ++k) {
      const uint32_t u = k & 1 ? bits[k / 2] >> 16 : bits[k / 2] & 0xffff;
      v[k] = u >= a.threshold ? r.get(k) * a.scale : 0.0f;
      if constexpr (kResidual) v[k] += s.get(k);
    }
    if (whole()) {
      store_vec<T, kUnit, kOnce, true>(out + at, kUnit, v);
    } else {
#pragma unroll
      for (int k = 0; k < kUnit; ++k)
        if (k >= lo && k < hi) out[at + k] = narrow<T>(v[k]);
    }
  }
};

// A contiguous tensor, a unit a thread.  Units begin at multiples of eight of the elements' numbers: the first and last
// may be parts.
template <typename T, bool kResidual, bool kOnce>
__global__ __launch_bounds__(kThreads) void dropout_flat_kernel(DropoutArgs a) {
  const uint64_t seed = seed_of(a), counter = uint64_t(a.offset) / kUnit;
  const int skip = int(a.offset & (kUnit - 1));
  const int64_t units = ceil_div(a.cols + skip, kUnit);
  for (int64_t u = int64_t(blockIdx.x) * kThreads + threadIdx.x; u < units; u += int64_t(gridDim.x) * kThreads) {
    Unit<T, kResidual, kOnce> unit;
    unit.place(u * kUnit - skip, a.cols);
    unit.load(static_cast<const T*>(a.x), static_cast<const T*>(a.residual));
    loads_first();
    unit.store(a, counter + uint64_t(u), seed, static_cast<T*>(a.out));
  }
}

// Rows with gaps between them, a row's units to 1 << lshift lanes.
template <typename T, bool kResidual>
__global__ __launch_bounds__(kThreads) void dropout_rows_kernel(DropoutArgs a, int lshift) {
  const uint64_t seed = seed_of(a);
  const int per = kThreads >> lshift, lane = threadIdx.x & ((1 << lshift) - 1);
  for (int64_t row = int64_t(blockIdx.x) * per + (threadIdx.x >> lshift); row < a.rows; row += int64_t(gridDim.x) * per) {
    const int64_t first = a.offset + row * a.cols;
    for (int64_t u = lane;; u += int64_t(1) << lshift) {
      Unit<T, kResidual, false> unit;
      unit.place(u * kUnit - (first & (kUnit - 1)), a.cols);
      if (unit.hi <= 0) break;
      unit.load(static_cast<const T*>(a.x) + row * a.x_stride, static_cast<const T*>(a.residual) + row * a.residual_stride);
      loads_first();
      unit.store(a, uint64_t(first / kUnit + u), seed, static_cast<T*>(a.out) + row * a.out_stride);
    }
  }
}

// More bytes than the last-level cache holds go past the caches where a unit is one vector: 32760 x 5120 bf16 with a
// residual 158 us instead of 169; an eighth of that, whose inputs the cache may hold, 19.5 instead of 22 where it does.  The
// two vectors of a unit of fp32 share cache lines with those of the next lane, which the caches join (half as many rows
// 168 us, past them 187).
constexpr int64_t kPastCaches = int64_t(256) << 20;

template <typename T, bool kResidual>
int dropout(DropoutArgs a, hipStream_t s) {
  const auto dense = [&](int64_t stride) { return a.rows == 1 || stride == a.cols; };
  if (dense(a.x_stride) && dense(a.out_stride) && (!kResidual || dense(a.residual_stride))) {
    a.cols *= a.rows;
    const int64_t units = ceil_div(a.cols + a.offset % kUnit, kUnit);
    const bool once = sizeof(T) == 2 && a.cols * int64_t(sizeof(T)) * (kResidual ? 3 : 2) > kPastCaches;
    return launch(once ? dropout_flat_kernel<T, kResidual, true> : dropout_flat_kernel<T, kResidual, false>,
                  grid_of(units, kThreads), kThreads, 0, s, a);
  }
  int lshift = 0;  // a row's units, one more where its first is a part
  while (lshift < 8 && (int64_t(1) << lshift) < ceil_div(a.cols, kUnit) + 1) ++lshift;
  return launch(dropout_rows_kernel<T, kResidual>, grid_of(a.rows, kThreads >> lshift), kThreads, 0, s, a, lshift);
}

}  // namespace

int launch_dropout(const DropoutArgs& a, int dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.residual != nullptr) return dtype == TIDE_BF16 ? dropout<bf16_t, true>(a, s) : dropout<float, true>(a, s);
  return dtype == TIDE_BF16 ? dropout<bf16_t, false>(a, s) : dropout<float, false>(a, s);
}

}  // namespace tide_step
