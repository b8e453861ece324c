// Tokens sorted by expert and back.
//
//   sort     place[p] = offsets[e] + pairs of e before p;  source = its inverse
//   dispatch out[r]   = x[source[r] / choices]
//   combine  y[t]     = sum over j of w[t, j] x[place[t, j]]
//   gradient dx[r]    = w[source[r]] dy[source[r] / choices],  dw[t, j] = <dy[t], x[place[t, j]]>
//
// The sort is a stable counting sort of whole numbers; the others move rows in 16-byte vectors and are
// bound by HBM.
#include "step_device.h"
#include "step_grid.h"
#include "step_internal.h"

namespace tide_step {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------------------------

// Each wave of a workgroup counts its own pairs of each expert: as many waves as 32 KiB of LDS hold the
// counts of.
constexpr int kCountBytes = 32768;
constexpr int kHeld = 8;  // ids of a lane that stay in registers between counting and placing
inline int sort_waves(int experts) {
  int w = 16;
  while (w > 1 && w * experts * 4 > kCountBytes) w /= 2;
  return w;
}

// Pairs [begin, end) of workgroup `part` of `parts`, a whole number of 64 for each wave.
struct Part {
  int64_t begin, end;
  __device__ Part(int64_t pairs, int part, int parts) {
    const int64_t size = ceil_div(ceil_div(pairs, parts), 64) * 64;
    begin = part * size < pairs ? part * size : pairs;
    end = begin + size < pairs ? begin + size : pairs;
  }
};
template <typename I>
__device__ __forceinline__ int expert_of(I id, int experts) {  // -1: none
  return id >= 0 && id < experts ? int(id) : -1;
}

template <typename I>
__global__ __launch_bounds__(1024) void expert_count_kernel(ExpertSortArgs a) {
  extern __shared__ int count[];  // [experts]
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) count[e] = 0;
  __syncthreads();
  const Part part(a.pairs, blockIdx.x, gridDim.x);
  const I* ids = static_cast<const I*>(a.ids);
  for (int64_t p = part.begin + threadIdx.x; p < part.end; p += blockDim.x) {
    const int e = expert_of(ids[p], a.experts);
    if (e >= 0) atomicAdd(count + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) a.counts[int64_t(blockIdx.x) * a.experts + e] = count[e];
}

// Sum over the workgroup before this thread.  `lds` holds a value for each wave.
__device__ __forceinline__ int block_exclusive(int v, int* lds) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int incl = wave_scan(v);
  if (lane == 63) lds[wave] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += lds[w];
  return before + incl - v;
}

// The lanes of the wave with this lane's expert.
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
  uint64_t same = __ballot(e >= 0);
  for (int k = 0; k < bits; ++k) {
    const uint64_t set = __ballot((e >> k) & 1);
    same &= (e >> k) & 1 ? set : ~set;
  }
  return same;
}

template <typename I>
__global__ __launch_bounds__(1024) void expert_place_kernel(ExpertSortArgs a, int bits) {
  extern __shared__ int lds[];
  const int waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int experts = a.experts, parts = gridDim.x;
  int* count = lds;                         // [waves][experts]: pairs of a wave, then the row of its next
  int* total = count + waves * experts;     // [experts]: pairs of all parts
  int* before = total + experts;            // [experts]: of lower parts
  int* start = before + experts;            // [experts + 1]: offsets
  int* sums = start + experts + 1;          // [waves]
  for (int i = threadIdx.x; i < (waves + 2) * experts; i += blockDim.x) count[i] = 0;
  const Part part(a.pairs, blockIdx.x, parts);
  const int64_t share = ceil_div(ceil_div(part.end - part.begin, waves), 64) * 64;
  const int64_t first = part.begin + wave * share;
  const int n = int(first + share < part.end ? share : part.end > first ? part.end - first : 0);
  const I* ids = static_cast<const I*>(a.ids) + first;
  const bool held = share <= 64 * kHeld;
  int mine[kHeld];
  const auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) mine[j] = i0 + j * 64 + lane < n ? expert_of(ids[i0 + j * 64 + lane], experts) : -1;
  };
  load(0);
  __syncthreads();
  int* own = count + wave * experts;
  for (int i0 = 0; i0 < n; i0 += 64 * kHeld) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (mine[j] >= 0) atomicAdd(own + mine[j], 1);
  }
  if (parts > 1) {
    // each thread adds up some of the parts' counts of an expert, or of several
    const int groups = blockDim.x > unsigned(experts) ? int(blockDim.x) / experts : 1;
    const int g = threadIdx.x / experts;
    if (g < groups)
      for (int e = threadIdx.x - g * experts; e < experts; e += blockDim.x) {
        int all = 0, low = 0;
        for (int b = g; b < parts; b += groups) {
          const int c = a.counts[int64_t(b) * experts + e];
          all += c;
          if (b < int(blockIdx.x)) low += c;
        }
        atomicAdd(total + e, all);
        atomicAdd(before + e, low);
      }
    __syncthreads();
  } else {
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += blockDim.x)
      for (int w = 0; w < waves; ++w) total[e] += count[w * experts + e];
    __syncthreads();
  }
  // offsets: each thread adds up neighbouring experts
  const int per = (experts + int(blockDim.x) - 1) / int(blockDim.x), e0 = threadIdx.x * per;
  const auto padded = [&](int e) { return (total[e] + a.align - 1) / a.align * a.align; };
  int sum = 0;
  for (int e = e0; e < e0 + per && e < experts; ++e) sum += padded(e);
  int at = block_exclusive(sum, sums);
  for (int e = e0; e < e0 + per && e < experts; ++e) {
    start[e] = at;
    at += padded(e);
    if (e == experts - 1) start[experts] = at;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= experts; e += blockDim.x) a.offsets[e] = start[e];
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    int row = start[e] + before[e];
    for (int w = 0; w < waves; ++w) {
      const int c = count[w * experts + e];
      count[w * experts + e] = row;
      row += c;
    }
  }
  __syncthreads();
  // Only this wave uses its row of `count`, and its LDS accesses stay in order.
  for (int i0 = 0; i0 < n; i0 += 64 * kHeld) {
    if (!held) load(i0);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int i = i0 + j * 64 + lane, e = mine[j];
      if (i0 + j * 64 >= n) break;
      const uint64_t same = same_expert(e, bits);
      int row = -1;
      if (e >= 0) {
        row = __hip_atomic_load(own + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) + lanes_before(same);
        a.source[row] = int(first) + i;
        if (lane == 63 - __clzll((long long)same))  // the last of its expert: the next row
          __hip_atomic_store(own + e, row + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      }
      if (i < n) a.place[first + i] = row;
    }
  }
  // rows of no pair: a wave for each expert's, all for those behind the last expert
  for (int e = int(blockIdx.x) * waves + wave; e < experts; e += parts * waves)
    for (int r = start[e] + total[e] + lane; r < start[e + 1]; r += 64) a.source[r] = -1;
  for (int64_t r = start[experts] + int64_t(blockIdx.x) * blockDim.x + threadIdx.x; r < a.rows;
       r += int64_t(parts) * blockDim.x)
    a.source[r] = -1;
}

// ---------------------------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------------------------

// Lanes (a power of two up to the workgroup) that share a row of `vecs` vectors.
inline int lanes_shift(int64_t vecs) {
  int s = 0;
  while (s < 8 && (int64_t(1) << s) < vecs) ++s;
  return s;
}

template <typename T, int E, bool kWhole>
__device__ __forceinline__ void store_raw(T* p, int n, const Raw<T, E>& r) {
  float f[E];
#pragma unroll
  for (int k = 0; k < E; ++k) f[k] = r.get(k);
  store_vec<T, E, true, kWhole>(p, n, f);
}

// A row of the sorted buffer to 1 << lshift lanes.
template <typename T, bool kWhole>
__global__ __launch_bounds__(kThreads) void expert_dispatch_kernel(ExpertRowsArgs a, int lshift) {
  constexpr int E = kVec<T>;
  const int lane = threadIdx.x & ((1 << lshift) - 1), per = kThreads >> lshift;
  int group = threadIdx.x >> lshift;
  if (lshift >= 6) group = __builtin_amdgcn_readfirstlane(group);
  const int64_t pairs = a.tokens * a.choices;
  for (int64_t r = int64_t(blockIdx.x) * per + group; r < a.rows; r += int64_t(gridDim.x) * per) {
    const int s = a.source[r];
    const bool real = s >= 0 && s < pairs;
    const T* from = static_cast<const T*>(a.x) + (real ? s / a.choices * a.x_stride : 0);
    T* to = static_cast<T*>(a.out) + r * a.out_stride;
    for (int64_t c = int64_t(lane) * E; c < a.dim; c += int64_t(E) << lshift) {
      const Raw<T, E> v = load_vec<T, E, false, kWhole>(from + c, real ? tail<E>(a.dim - c) : 0, a.dim >= E);
      store_raw<T, E, kWhole>(to + c, tail<E>(a.dim - c), v);
    }
  }
}

template <typename W>
__device__ __forceinline__ float weight_of(const void* weights, int64_t p) {
  return widen(static_cast<const W*>(weights)[p]);
}

// A token to 1 << lshift lanes; the rows of N choices are in flight at a time and added in order.
template <typename T, typename W, int N, bool kWhole>
__global__ __launch_bounds__(kThreads) void expert_combine_kernel(ExpertRowsArgs a, int lshift) {
  constexpr int E = kVec<T>;
  const int lane = threadIdx.x & ((1 << lshift) - 1), per = kThreads >> lshift;
  int group = threadIdx.x >> lshift;
  if (lshift >= 6) group = __builtin_amdgcn_readfirstlane(group);
  for (int64_t t = int64_t(blockIdx.x) * per + group; t < a.tokens; t += int64_t(gridDim.x) * per) {
    const int32_t* place = a.place + t * a.choices;
    for (int64_t c = int64_t(lane) * E; c < a.dim; c += int64_t(E) << lshift) {
      const int n = tail<E>(a.dim - c);
      float acc[E] = {};
      for (int j0 = 0; j0 < a.choices; j0 += N) {
        const T* from[N];
        float w[N];
        bool real[N];
        bool any = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int row = j0 + j < a.choices ? place[j0 + j] : -1;
          real[j] = row >= 0 && row < a.rows;
          w[j] = real[j] && a.weights != nullptr ? weight_of<W>(a.weights, t * a.choices + j0 + j) : 1.0f;
          from[j] = static_cast<const T*>(a.x) + (real[j] ? row * a.x_stride : 0);
          any |= real[j];
        }
        if (!any) continue;
        Raw<T, E> r[N];
        load_vecs<T, E, N, false, kWhole>(r, from, c, n, a.dim >= E);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (real[j]) {
#pragma unroll
            for (int k = 0; k < E; ++k) acc[k] = fmaf(w[j], r[j].get(k), acc[k]);
          }
      }
      store_vec<T, E, true, kWhole>(static_cast<T*>(a.out) + t * a.out_stride + c, n, acc);
    }
  }
}

// Zeros to the rows of no pair among the rows from r0 on, one a lane looked at; the workgroup's waves share
// the columns.
template <typename T, bool kWhole>
__device__ __forceinline__ void zero_rows(const ExpertRowsArgs& a, int64_t r0, int count) {
  constexpr int E = kVec<T>;
  const int lane = threadIdx.x & 63;
  const int64_t pairs = a.tokens * a.choices;
  bool none = false;
  if (lane < count && r0 + lane < a.rows) {
    const int s = a.source[r0 + lane];
    none = s < 0 || s >= pairs;
  }
  const float zero[E] = {};
  for (uint64_t todo = __ballot(none); todo != 0; todo &= todo - 1) {
    T* to = static_cast<T*>(a.out) + (r0 + __ffsll((unsigned long long)todo) - 1) * a.out_stride;
    for (int64_t c = int64_t(threadIdx.x) * E; c < a.dim; c += kThreads * E)
      store_vec<T, E, true, kWhole>(to + c, tail<E>(a.dim - c), zero);
  }
}

constexpr int kZeroRows = 16;  // a workgroup's

// Workgroups below `summing` take tokens, 1 << lshift lanes each (up to 64); the others write zeros.
template <typename T, typename W, int N, bool kWhole, int kLanes>
__global__ __launch_bounds__(kThreads) void expert_combine_bwd_kernel(ExpertRowsArgs a, unsigned summing) {
  constexpr int E = kVec<T>;
  if (blockIdx.x >= summing) {
    for (int64_t r = int64_t(blockIdx.x - summing) * kZeroRows; r < a.rows; r += int64_t(gridDim.x - summing) * kZeroRows)
      zero_rows<T, kWhole>(a, r, kZeroRows);
    return;
  }
  const int lane = threadIdx.x & (kLanes - 1), per = kThreads / kLanes;
  int group = threadIdx.x / kLanes;
  if (kLanes == 64) group = __builtin_amdgcn_readfirstlane(group);
  for (int64_t t = int64_t(blockIdx.x) * per + group; t < a.tokens; t += int64_t(summing) * per) {
    const T* dy = static_cast<const T*>(a.dy) + t * a.dy_stride;
    for (int j0 = 0; j0 < a.choices; j0 += N) {
      const T* from[N];
      T* to[N];
      float w[N], dot[N];
      bool real[N];
      bool any = false;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int row = j0 + j < a.choices ? a.place[t * a.choices + j0 + j] : -1;
        real[j] = row >= 0 && row < a.rows;
        w[j] = real[j] ? weight_of<W>(a.weights, t * a.choices + j0 + j) : 0.0f;
        from[j] = static_cast<const T*>(a.x) + (real[j] ? row * a.x_stride : 0);
        to[j] = static_cast<T*>(a.out) + (real[j] ? row * a.out_stride : 0);
        dot[j] = 0.0f;
        any |= real[j];
      }
      if (any)
        for (int64_t c = int64_t(lane) * E; c < a.dim; c += kLanes * E) {
          const int n = tail<E>(a.dim - c);
          const Raw<T, E> d = load_vec<T, E, false, kWhole>(dy + c, n, a.dim >= E);
          Raw<T, E> r[N];
          load_vecs<T, E, N, false, kWhole>(r, from, c, n, a.dim >= E);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            if (!real[j]) continue;
            float f[E];
#pragma unroll
            for (int k = 0; k < E; ++k) {
              dot[j] = fmaf(d.get(k), r[j].get(k), dot[j]);
              f[k] = w[j] * d.get(k);
            }
            store_vec<T, E, true, kWhole>(to[j] + c, n, f);
          }
        }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float sum = lanes_sum<kLanes>(dot[j]);
        if (lane == 0 && j0 + j < a.choices) static_cast<W*>(a.dweights)[t * a.choices + j0 + j] = narrow<W>(sum);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------------------------

template <typename I>
int sort(const ExpertSortArgs& a, hipStream_t s) {
  const int parts = expert_parts(a.pairs), waves = sort_waves(a.experts);
  int bits = 0;
  while ((1 << bits) < a.experts) ++bits;
  if (parts > 1)
    if (const int e = launch(expert_count_kernel<I>, unsigned(parts), 1024, size_t(a.experts) * 4, s, a)) return e;
  const size_t lds = (size_t(waves + 3) * a.experts + 1 + waves) * 4;
  return launch(expert_place_kernel<I>, unsigned(parts), waves * 64, lds, s, a, bits);
}

template <typename T>
int dispatch(const ExpertRowsArgs& a, hipStream_t s) {
  return with_whole<kVec<T>>(a.dim, [&](auto whole) {
    const int lshift = lanes_shift(ceil_div(a.dim, kVec<T>));
    return launch(expert_dispatch_kernel<T, decltype(whole)::value>, grid_of(a.rows, kThreads >> lshift), kThreads, 0, s,
                  a, lshift);
  });
}

// f(choices in flight) as a constant.
template <typename F>
int with_choices(int choices, F&& f) {
  if (choices > 4) return f(std::integral_constant<int, 8>());
  if (choices > 2) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 2>());
}

template <typename T, typename W>
int combine(const ExpertRowsArgs& a, hipStream_t s) {
  return with_whole<kVec<T>>(a.dim, [&](auto whole) {
    return with_choices(a.choices, [&](auto n) {
      const int lshift = lanes_shift(ceil_div(a.dim, kVec<T>));
      return launch(expert_combine_kernel<T, W, decltype(n)::value, decltype(whole)::value>,
                    grid_of(a.tokens, kThreads >> lshift), kThreads, 0, s, a, lshift);
    });
  });
}

template <typename F>
int with_lanes(int64_t vecs, F&& f) {
  if (vecs > 16) return f(std::integral_constant<int, 64>());
  if (vecs > 4) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 4>());
}

template <typename T, typename W>
int combine_bwd(const ExpertRowsArgs& a, hipStream_t s) {
  return with_whole<kVec<T>>(a.dim, [&](auto whole) {
    return with_choices(a.choices, [&](auto n) {
      return with_lanes(ceil_div(a.dim, kVec<T>), [&](auto lanes) {
        const unsigned summing = a.tokens > 0 ? grid_of(a.tokens, kThreads / decltype(lanes)::value) : 0;
        const unsigned zeroing = a.rows > 0 ? grid_of(a.rows, kZeroRows) : 0;
        return launch(
            expert_combine_bwd_kernel<T, W, decltype(n)::value, decltype(whole)::value, decltype(lanes)::value>,
            summing + zeroing, kThreads, 0, s, a, summing);
      });
    });
  });
}

}  // namespace

int launch_expert_sort(const ExpertSortArgs& a, int ids_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return ids_dtype == TIDE_INT32 ? sort<int32_t>(a, s) : sort<int64_t>(a, s);
}
int launch_expert_dispatch(const ExpertRowsArgs& a, int dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == TIDE_BF16 ? dispatch<bf16_t>(a, s) : dispatch<float>(a, s);
}
int launch_expert_combine(const ExpertRowsArgs& a, int dtype, int weight_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == TIDE_BF16) return weight_dtype == TIDE_BF16 ? combine<bf16_t, bf16_t>(a, s) : combine<bf16_t, float>(a, s);
  return weight_dtype == TIDE_BF16 ? combine<float, bf16_t>(a, s) : combine<float, float>(a, s);
}
int launch_expert_combine_bwd(const ExpertRowsArgs& a, int dtype, int weight_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == TIDE_BF16)
    return weight_dtype == TIDE_BF16 ? combine_bwd<bf16_t, bf16_t>(a, s) : combine_bwd<bf16_t, float>(a, s);
  return weight_dtype == TIDE_BF16 ? combine_bwd<float, bf16_t>(a, s) : combine_bwd<float, float>(a, s);
}

}  // namespace tide_step
