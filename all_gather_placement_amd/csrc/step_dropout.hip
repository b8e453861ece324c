// Dropout by a counter-based generator, added to a residual.
//
//   out = x * 65536 / (65536 - t) + residual where the element's 16 bits are at least t, else the residual
//
// Philox4x32 with 10 rounds makes the bits of eight neighbouring elements from the seed and their number, so
// no mask is stored or read: HBM bounds it, each element read and written once.  16 bits an element, not 32:
// a round's two 64-bit products run at a quarter of the rate of other integer operations, and at four
// elements a call they would take as long as the memory does.
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

// Elements lo to hi - 1 of the unit `counter`; element k is x[k].
template <typename T, bool kResidual>
__device__ __forceinline__ void drop(const DropoutArgs& a, uint64_t counter, uint64_t seed, const T* x,
                                     const T* residual, T* out, int lo, int hi) {
  float f[kUnit], add[kUnit];
  const bool whole = lo <= 0 && hi >= kUnit;
  if (whole) {
    const Raw<T, kUnit> r = load_whole<T, kUnit, true>(x);
    Raw<T, kUnit> s;
    if constexpr (kResidual) s = load_whole<T, kUnit, true>(residual);
    loads_first();
#pragma unroll
    for (int k = 0; k < kUnit; ++k) {
      f[k] = r.get(k);
      add[k] = kResidual ? s.get(k) : 0.0f;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kUnit; ++k) {
      f[k] = k >= lo && k < hi ? widen(x[k]) : 0.0f;
      add[k] = kResidual && k >= lo && k < hi ? widen(residual[k]) : 0.0f;
    }
  }
  uint32_t bits[4];
  philox(counter, seed, bits);
#pragma unroll
  for (int k = 0; k < kUnit; ++k) {
    const uint32_t u = k & 1 ? bits[k / 2] >> 16 : bits[k / 2] & 0xffff;
    f[k] = u >= a.threshold ? f[k] * a.scale : 0.0f;
    if constexpr (kResidual) f[k] += add[k];
  }
  if (whole) {
    store_vec<T, kUnit, true, true>(out, kUnit, f);
  } else {
#pragma unroll
    for (int k = 0; k < kUnit; ++k)
      if (k >= lo && k < hi) out[k] = narrow<T>(f[k]);
  }
}

// A row's units to 1 << lshift lanes; a contiguous tensor is one row.  Units begin at multiples of eight of
// the elements' numbers: a row's first and last may be parts.
template <typename T, bool kResidual>
__global__ __launch_bounds__(kThreads) void dropout_kernel(DropoutArgs a, int lshift, int64_t spans) {
  const uint64_t seed = seed_of(a);
  const int per = kThreads >> lshift, group = threadIdx.x >> lshift, lane = threadIdx.x & ((1 << lshift) - 1);
  const int64_t items = ceil_div(a.rows, per) * spans;  // of a workgroup: `per` rows, 1 << lshift units of each
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t block = spans == 1 ? item : item / spans, row = block * per + group;
    if (row >= a.rows) continue;
    const int64_t first = a.offset + row * a.cols;
    const int64_t unit = ((item - block * spans) << lshift) + lane, at = unit * kUnit - (first & (kUnit - 1));
    if (at >= a.cols) continue;
    const int64_t left = a.cols - at;
    drop<T, kResidual>(a, uint64_t(first / kUnit + unit), seed, static_cast<const T*>(a.x) + row * a.x_stride + at,
                       static_cast<const T*>(a.residual) + row * a.residual_stride + at,
                       static_cast<T*>(a.out) + row * a.out_stride + at, at < 0 ? int(-at) : 0,
                       int(left < kUnit ? left : kUnit));
  }
}

template <typename T>
int dropout(DropoutArgs a, hipStream_t s) {
  const auto dense = [&](int64_t stride) { return a.rows == 1 || stride == a.cols; };
  if (dense(a.x_stride) && dense(a.out_stride) && (a.residual == nullptr || dense(a.residual_stride))) {
    a.cols *= a.rows;
    a.rows = 1;
  }
  // a row's units where its first is a part of one
  const int64_t units = a.rows == 1 ? ceil_div(a.cols + a.offset % kUnit, kUnit) : ceil_div(a.cols + kUnit - 1, kUnit);
  int lshift = 0;
  while (lshift < 8 && (int64_t(1) << lshift) < units) ++lshift;
  const int64_t spans = ceil_div(units, int64_t(1) << lshift);
  const unsigned grid = grid_of(ceil_div(a.rows, kThreads >> lshift) * spans, 1);
  return a.residual != nullptr ? launch(dropout_kernel<T, true>, grid, kThreads, 0, s, a, lshift, spans)
                               : launch(dropout_kernel<T, false>, grid, kThreads, 0, s, a, lshift, spans);
}

}  // namespace

int launch_dropout(const DropoutArgs& a, int dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == TIDE_BF16 ? dropout<bf16_t>(a, s) : dropout<float>(a, s);
}

}  // namespace tide_step
