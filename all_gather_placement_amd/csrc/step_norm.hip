// Global gradient norm and clipping.
//
//   s = sum over every tensor and element of g^2,  n = sqrt(s),  c = min(1, max_norm / (n + 1e-6)),
//   out = g * c.
//
// Nothing is reused, so HBM bounds both passes; every thread keeps its sum in 64 bits, where no
// finite square overflows or vanishes (the VALU keeps up: eight squares summed in fp32 first changed
// nothing).  Each workgroup leaves one partial sum, and the partial sums are added in order, so the
// result depends on the sizes alone.
//
// Measured: 391 bf16 tensors of 3 MiB, 1.23 GB, in 186 us with both launches and the finish (6.6 TB/s;
// 7.1 is what reading alone reaches); 64 fp32 tensors, 1.4 GB, summed in 205 us and clipped in 440 to 455 us
// (6.2 to 6.4 TB/s, the rate of a copy).  The sum reads past the caches: with plain loads the call takes 712 us
// instead of 667, and leaving the last 96 or 192 MiB in the caches for the clipping 713 or 734.
#include "step_device.h"
#include "step_internal.h"

namespace tide_step {
namespace {

// Threads of a launch of one workgroup: four times a chunk's.
constexpr int kOneWgThreads = 4 * kNormThreads;

// Sum over a workgroup of kThreads, in every thread; one barrier.  `lds` is not reused by the caller.
template <int kThreads>
__device__ __forceinline__ double block_sum(double v, double (&lds)[kThreads / 64]) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += lds[w];
  return s;
}

// Index of the table entry that holds chunk c (entries are in ascending order of `first`).  Tensors of
// about one size are found at once; a search waits for one entry after another.
template <typename Table>
__device__ __forceinline__ int entry_of(const Table& t, uint32_t c) {
  const int guess = int(uint64_t(c) * uint32_t(t.count) / t.chunks);
  const uint32_t first = t.e[guess].first, next = guess + 1 < t.count ? t.e[guess + 1].first : t.chunks;
  if (first <= c && c < next) return guess;
  int lo = c < first ? 0 : guess + 1, hi = c < first ? guess : t.count;  // first[lo] <= c < first[hi]
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

// What a chunk of a table is: its tensor's entry, its elements and its place there.
struct Chunk {
  int entry, n;
  int64_t at;
};
template <typename T, typename Table>
__device__ __forceinline__ Chunk chunk_of(const Table& t, uint32_t c, int i) {
  const uint32_t first = t.e[i].first, next = i + 1 < t.count ? t.e[i + 1].first : t.chunks;
  return {i, c + 1 == next ? int(t.e[i].last) : kChunk<T>, int64_t(c - first) * kChunk<T>};
}

// This thread's part of a chunk's sum of squares.
template <typename T, bool kOnce>
__device__ __forceinline__ double chunk_squares(const T* p, int n, int thread) {
  double acc = 0;
  if (n == kChunk<T>) {
    u32x4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = load16<kOnce>(p + (k * kNormThreads + thread) * kVec<T>);
    loads_first();
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < kVec<T>; ++j) {
        const double d = lane_of<T>(v[k], j);
        acc += d * d;
      }
  } else {
    for (int k = thread; k < n; k += kNormThreads) {
      const double d = widen(p[k]);
      acc += d * d;
    }
  }
  return acc;
}
// The sum over all of a table's chunks by this workgroup alone.
template <typename T, typename Table>
__device__ __forceinline__ double table_squares(const Table& t, double (&lds)[kOneWgThreads / 64]) {
  double acc = 0;
  for (uint32_t c = threadIdx.x / kNormThreads; c < t.chunks; c += kOneWgThreads / kNormThreads) {
    const Chunk k = chunk_of<T>(t, c, entry_of(t, c));
    acc += chunk_squares<T, false>(static_cast<const T*>(t.e[k.entry].p) + k.at, k.n, threadIdx.x % kNormThreads);
  }
  return block_sum<kOneWgThreads>(acc, lds);
}

template <typename T>
__global__ __launch_bounds__(kNormThreads) void norm_partial_kernel(NormTable t, double* __restrict__ partial) {
  __shared__ double lds[kNormThreads / 64];
  double acc = 0;
  int i = entry_of(t, blockIdx.x);
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    while (i + 1 < t.count && t.e[i + 1].first <= c) ++i;
    const Chunk k = chunk_of<T>(t, c, i);
    acc += chunk_squares<T, true>(static_cast<const T*>(t.e[i].p) + k.at, k.n, threadIdx.x);
  }
  const double s = block_sum<kNormThreads>(acc, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__device__ __forceinline__ void write_norm(double s, double* sumsq, float* norm) {
  if (threadIdx.x != 0) return;
  if (sumsq != nullptr) *sumsq = s;
  if (norm != nullptr) *norm = float(sqrt(s));
}

template <typename T>
__global__ __launch_bounds__(kOneWgThreads) void norm_one_kernel(NormTable t) {
  __shared__ double lds[kOneWgThreads / 64];
  write_norm(table_squares<T>(t, lds), t.sumsq, t.norm);
}

__global__ __launch_bounds__(kOneWgThreads) void norm_finish_kernel(const double* __restrict__ partial, int n,
                                                                    double* __restrict__ sumsq,
                                                                    float* __restrict__ norm) {
  __shared__ double lds[kOneWgThreads / 64];
  double acc = 0;
#pragma unroll 4
  for (int k = threadIdx.x; k < n; k += kOneWgThreads) acc += partial[k];
  write_norm(block_sum<kOneWgThreads>(acc, lds), sumsq, norm);
}

// min(1, max_norm / (n + 1e-6)), NaN kept.
__device__ __forceinline__ float clip_coef(double n, double max_norm) {
  const double c = max_norm / (n + 1e-6);
  return float(c > 1.0 ? 1.0 : c);
}

// kLoads vectors of a thread, kNormThreads apart, or what there is of them.
template <typename T, int kLoads, bool kOnce>
__device__ __forceinline__ void scale_chunk(const T* p, T* o, int n, int thread, float coef) {
  if (n == kLoads * kNormThreads * kVec<T>) {
    u32x4 v[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) v[k] = load16<kOnce>(p + (k * kNormThreads + thread) * kVec<T>);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      u32x4 r;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2)
          r[j] = round_bf16x2(lane_of<T>(v[k], 2 * j) * coef, lane_of<T>(v[k], 2 * j + 1) * coef);
        else
          r[j] = __float_as_uint(lane_of<T>(v[k], j) * coef);
      }
      store16<kOnce>(o + (k * kNormThreads + thread) * kVec<T>, r);
    }
  } else {
    for (int k = thread; k < n; k += kNormThreads) o[k] = narrow<T>(widen(p[k]) * coef);
  }
}

// A workgroup takes a quarter of a chunk, one vector a thread: 440 us where workgroups that stay for
// many chunks of four vectors a thread take 500.
constexpr int kClipParts = 4;
template <typename T>
__global__ __launch_bounds__(kNormThreads) void clip_kernel(ClipTable t, const double* __restrict__ sumsq,
                                                            double max_norm, float* __restrict__ norm) {
  const double n2 = sqrt(*sumsq);
  const float coef = clip_coef(n2, max_norm);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = float(n2);
  constexpr int kPart = kChunk<T> / kClipParts;
  const int from = blockIdx.x % kClipParts * kPart;
  for (uint32_t b = blockIdx.x / kClipParts; b < t.chunks; b += gridDim.x / kClipParts) {
    const Chunk k = chunk_of<T>(t, b, entry_of(t, b));
    const int n = k.n - from < kPart ? k.n - from : kPart;
    scale_chunk<T, 4 / kClipParts, true>(static_cast<const T*>(t.e[k.entry].p) + k.at + from,
                                         static_cast<T*>(t.e[k.entry].out) + k.at + from, n, threadIdx.x, coef);
  }
}

// As norm_finish_kernel, to the bit: a wave adds 64 neighbouring partial sums, the waves' sums follow in
// order.
__device__ __forceinline__ double add_partials(const double* __restrict__ partial, int n) {
  constexpr int kParts = kOneWgThreads / kNormThreads, kWaves = kNormThreads / 64;
  static_assert(kNormWgs <= kOneWgThreads, "one partial sum for each thread of norm_finish_kernel");
  __shared__ double lds[kParts * kWaves];
#pragma unroll
  for (int j = 0; j < kParts; ++j) {
    const int k = j * kNormThreads + int(threadIdx.x);
    const double v = wave_sum(k < n ? partial[k] : 0.0);
    if ((threadIdx.x & 63) == 0) lds[j * kWaves + threadIdx.x / 64] = v;
  }
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int w = 0; w < kParts * kWaves; ++w) s += lds[w];
  return s;
}

// Few chunks: a workgroup for each, which adds up the partial sums itself; a launch less.
template <typename T>
__global__ __launch_bounds__(kNormThreads) void clip_adding_kernel(ClipTable t, double max_norm,
                                                                   float* __restrict__ norm) {
  const double s = add_partials(t.partial, t.partials);
  if (blockIdx.x == 0) write_norm(s, t.sum_to, norm);
  const float coef = clip_coef(sqrt(s), max_norm);
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Chunk k = chunk_of<T>(t, c, entry_of(t, c));
    scale_chunk<T, 4, false>(static_cast<const T*>(t.e[k.entry].p) + k.at, static_cast<T*>(t.e[k.entry].out) + k.at,
                             k.n, threadIdx.x, coef);
  }
}

template <typename T>
__global__ __launch_bounds__(kOneWgThreads) void clip_one_kernel(ClipTable t, double max_norm,
                                                                 float* __restrict__ norm) {
  __shared__ double lds[kOneWgThreads / 64];
  const double s = table_squares<T>(t, lds);
  write_norm(s, t.sum_to, norm);
  const float coef = clip_coef(sqrt(s), max_norm);
  for (uint32_t c = threadIdx.x / kNormThreads; c < t.chunks; c += kOneWgThreads / kNormThreads) {
    const Chunk k = chunk_of<T>(t, c, entry_of(t, c));
    scale_chunk<T, 4, false>(static_cast<const T*>(t.e[k.entry].p) + k.at, static_cast<T*>(t.e[k.entry].out) + k.at,
                             k.n, threadIdx.x % kNormThreads, coef);
  }
}

}  // namespace

template <typename T>
static int norm_partial(const NormTable& t, double* partial, int grid, hipStream_t s) {
  if (t.sumsq != nullptr || t.norm != nullptr) return launch(norm_one_kernel<T>, 1, kOneWgThreads, 0, s, t);
  return launch(norm_partial_kernel<T>, grid, kNormThreads, 0, s, t, partial);
}
int launch_norm_partial(const NormTable& t, int dtype, double* partial, int grid, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == TIDE_BF16 ? norm_partial<bf16_t>(t, partial, grid, s) : norm_partial<float>(t, partial, grid, s);
}

int launch_norm_finish(const double* partial, int n, double* sumsq, float* norm, void* stream) {
  if (sumsq == nullptr && norm == nullptr) return hipSuccess;
  return launch(norm_finish_kernel, 1, kOneWgThreads, 0, static_cast<hipStream_t>(stream), partial, n, sumsq, norm);
}

template <typename T>
static int clip(const ClipTable& t, const double* sumsq, double max_norm, float* norm, int grid, hipStream_t s) {
  if (t.partial != nullptr) return launch(clip_adding_kernel<T>, grid, kNormThreads, 0, s, t, max_norm, norm);
  if (t.sum_to != nullptr) return launch(clip_one_kernel<T>, 1, kOneWgThreads, 0, s, t, max_norm, norm);
  return launch(clip_kernel<T>, grid * kClipParts, kNormThreads, 0, s, t, sumsq, max_norm, norm);
}
int launch_clip(const ClipTable& t, int dtype, const double* sumsq, double max_norm, float* norm, int grid,
                void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == TIDE_BF16 ? clip<bf16_t>(t, sumsq, max_norm, norm, grid, s)
                            : clip<float>(t, sumsq, max_norm, norm, grid, s);
}

}  // namespace tide_step
