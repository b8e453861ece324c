// Global gradient norm and clipping.
//
//   s = sum over every tensor and element of g^2,  n = sqrt(s),  c = min(1, max_norm / (n + 1e-6)),
//   out = g * c.
//
// Nothing is reused, so HBM bounds both passes; every thread keeps its sum in 64 bits, where no
// finite square overflows or vanishes.  Each workgroup leaves one partial sum, and the partial sums
// are added in order, so the result depends on the sizes alone.
#include "step_device.h"
#include "step_internal.h"

namespace tide_step {
namespace {

constexpr int kWaves = kNormThreads / 64;

// Sum over the workgroup, in every thread; one barrier.  `lds` holds kWaves values and is not
// reused by the caller.
__device__ __forceinline__ double block_sum(double v, double* lds) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += lds[w];
  return s;
}

// Index of the table entry that holds chunk c (entries are in ascending order of `first`).
template <typename Table>
__device__ __forceinline__ int entry_of(const Table& t, uint32_t c) {
  int lo = 0, hi = t.count;  // first[lo] <= c < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].first <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <typename T>
constexpr int kChunk = kNormChunkBytes / int(sizeof(T));
template <typename T>
__device__ __forceinline__ float lane_of(u32x4 v, int i) {
  return Raw<T, kVec<T>>{v[0], v[1], v[2], v[3]}.get(i);
}

template <typename T>
__global__ __launch_bounds__(kNormThreads) void norm_partial_kernel(NormTable t, double* __restrict__ partial) {
  __shared__ double lds[kWaves];
  double acc = 0;
  int i = entry_of(t, blockIdx.x);
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    while (i + 1 < t.count && t.e[i + 1].first <= c) ++i;
    const uint32_t next = i + 1 < t.count ? t.e[i + 1].first : t.chunks;
    const int n = c + 1 == next ? int(t.e[i].last) : kChunk<T>;
    const T* p = static_cast<const T*>(t.e[i].p) + int64_t(c - t.e[i].first) * kChunk<T>;
    if (n == kChunk<T>) {
      u32x4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = load16(p + (k * kNormThreads + threadIdx.x) * kVec<T>);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < kVec<T>; ++j) {
          const double d = lane_of<T>(v[k], j);
          acc += d * d;
        }
    } else {
      for (int k = threadIdx.x; k < n; k += kNormThreads) {
        const double d = widen(p[k]);
        acc += d * d;
      }
    }
  }
  const double s = block_sum(acc, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(kNormThreads) void norm_finish_kernel(const double* __restrict__ partial, int n,
                                                                   double* __restrict__ sumsq,
                                                                   float* __restrict__ norm) {
  __shared__ double lds[kWaves];
  double acc = 0;
  for (int k = threadIdx.x; k < n; k += kNormThreads) acc += partial[k];
  const double s = block_sum(acc, lds);
  if (threadIdx.x == 0) {
    if (sumsq != nullptr) *sumsq = s;
    if (norm != nullptr) *norm = float(sqrt(s));
  }
}

// min(1, max_norm / (n + 1e-6)), NaN kept.
__device__ __forceinline__ float clip_coef(double n, double max_norm) {
  const double c = max_norm / (n + 1e-6);
  return float(c > 1.0 ? 1.0 : c);
}

template <typename T>
__global__ __launch_bounds__(kNormThreads) void clip_kernel(ClipTable t, const double* __restrict__ sumsq,
                                                            double max_norm, float* __restrict__ norm) {
  const double n2 = sqrt(*sumsq);
  const float coef = clip_coef(n2, max_norm);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = float(n2);
  int i = entry_of(t, blockIdx.x);
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    while (i + 1 < t.count && t.e[i + 1].first <= c) ++i;
    const uint32_t next = i + 1 < t.count ? t.e[i + 1].first : t.chunks;
    const int n = c + 1 == next ? int(t.e[i].last) : kChunk<T>;
    const int64_t at = int64_t(c - t.e[i].first) * kChunk<T>;
    const T* p = static_cast<const T*>(t.e[i].p) + at;
    T* o = static_cast<T*>(t.e[i].out) + at;
    if (n == kChunk<T>) {
      u32x4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = load16(p + (k * kNormThreads + threadIdx.x) * kVec<T>);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u32x4 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(T) == 2)
            r[j] = round_bf16x2(lane_of<T>(v[k], 2 * j) * coef, lane_of<T>(v[k], 2 * j + 1) * coef);
          else
            r[j] = __float_as_uint(lane_of<T>(v[k], j) * coef);
        }
        store16(o + (k * kNormThreads + threadIdx.x) * kVec<T>, r);
      }
    } else {
      for (int k = threadIdx.x; k < n; k += kNormThreads) o[k] = narrow<T>(widen(p[k]) * coef);
    }
  }
}

}  // namespace

int launch_norm_partial(const NormTable& t, int dtype, double* partial, int grid, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == TIDE_BF16)
    hipLaunchKernelGGL(norm_partial_kernel<bf16_t>, dim3(grid), dim3(kNormThreads), 0, s, t, partial);
  else
    hipLaunchKernelGGL(norm_partial_kernel<float>, dim3(grid), dim3(kNormThreads), 0, s, t, partial);
  return hipGetLastError();
}

int launch_norm_finish(const double* partial, int n, double* sumsq, float* norm, void* stream) {
  hipLaunchKernelGGL(norm_finish_kernel, dim3(1), dim3(kNormThreads), 0, static_cast<hipStream_t>(stream), partial, n,
                     sumsq, norm);
  return hipGetLastError();
}

int launch_clip(const ClipTable& t, int dtype, const double* sumsq, double max_norm, float* norm, int grid,
                void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == TIDE_BF16)
    hipLaunchKernelGGL(clip_kernel<bf16_t>, dim3(grid), dim3(kNormThreads), 0, s, t, sumsq, max_norm, norm);
  else
    hipLaunchKernelGGL(clip_kernel<float>, dim3(grid), dim3(kNormThreads), 0, s, t, sumsq, max_norm, norm);
  return hipGetLastError();
}

}  // namespace tide_step
