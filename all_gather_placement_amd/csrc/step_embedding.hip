// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = table[ids[t]] * scale                      (zeros for ids outside the table)
//   dtable[v] = scale * sum of dy[t] over ids[t] = v    (in ascending t)
//
// HBM bounds the lookup: rows are read and written once in 16-byte vectors.
//
// The gradient has to write every row of the table, and most rows have no token.  Its first kernel
// brings tokens of equal id together and writes the zero rows meanwhile.  Each workgroup owns a
// range of rows.  It reads all ids (which stay in the L2), counts those of each of its rows and
// those below its range -- the place where its tokens begin -- and then places its tokens in
// ascending order: a stable counting sort with no traffic between workgroups.  The second kernel
// sums the sorted tokens in pieces of equal length, so a frequent id is shared by many waves, and a
// third adds the partial sums of ids that cross pieces, in order.
#include "step_device.h"
#include "step_internal.h"

namespace tide_step {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------------------------

template <typename T, int E>
__device__ __forceinline__ void store_scaled(T* out, int n, const Raw<T, E>& r, bool inside, float scale) {
  float f[E];
#pragma unroll
  for (int k = 0; k < E; ++k) f[k] = inside ? r.get(k) * scale : 0.0f;
  store_vec<T, E, true>(out, n, f);
}
template <int E>
__device__ __forceinline__ int tail(int64_t n) {
  return int(n < E ? n : E);
}

// Rows of 64 vectors and more: a row goes to 1 << wshift waves of a workgroup of four, a lane holding
// NV vectors at a time.
template <typename T, typename I, int NV>
__global__ __launch_bounds__(kThreads) void embedding_rows_kernel(int64_t tokens, const I* __restrict__ ids,
                                                                  int64_t vocab, int64_t dim,
                                                                  const T* __restrict__ table, float scale,
                                                                  T* __restrict__ out, int wshift) {
  constexpr int E = kVec<T>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t t = (int64_t(blockIdx.x) << (2 - wshift)) + (wave >> wshift);
  if (t >= tokens) return;
  const int64_t id = ids[t];
  const bool inside = id >= 0 && id < vocab;
  const T* row = table + (inside ? id * dim : 0);
  T* o = out + t * dim;
  const int64_t step = int64_t(64 * NV * E) << wshift;
  for (int64_t c0 = int64_t(wave & ((1 << wshift) - 1)) * (64 * NV * E); c0 < dim; c0 += step) {
    Raw<T, E> r[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = c0 + (v * 64 + lane) * E;
      r[v] = load_vec<T, E>(row + c, inside ? tail<E>(dim - c) : 0);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = c0 + (v * 64 + lane) * E;
      if (c < dim) store_scaled<T, E>(o + c, tail<E>(dim - c), r[v], inside, scale);
    }
  }
}

// Narrow rows: a group of 1 << lshift lanes for each of NT tokens in turn.
template <typename T, typename I, int NT>
__global__ __launch_bounds__(kThreads) void embedding_narrow_kernel(int64_t tokens, const I* __restrict__ ids,
                                                                    int64_t vocab, int dim,
                                                                    const T* __restrict__ table, float scale,
                                                                    T* __restrict__ out, int lshift) {
  constexpr int E = kVec<T>;
  const int groups = kThreads >> lshift, c = (threadIdx.x & ((1 << lshift) - 1)) * E;
  const int64_t t0 = int64_t(blockIdx.x) * groups * NT + (threadIdx.x >> lshift);
  int64_t id[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) id[i] = t0 + i * groups < tokens ? int64_t(ids[t0 + i * groups]) : -1;
  Raw<T, E> r[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const bool inside = id[i] >= 0 && id[i] < vocab;
    r[i] = load_vec<T, E>(table + (inside ? id[i] * dim : 0) + c, inside ? dim - c : 0);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t t = t0 + i * groups;
    if (t < tokens && c < dim)
      store_scaled<T, E>(out + t * dim + c, dim - c, r[i], id[i] >= 0 && id[i] < vocab, scale);
  }
}

// ---------------------------------------------------------------------------------------------
// Gradient: sorting tokens by id, and the rows without tokens
// ---------------------------------------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

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

// Sum over the workgroup before this thread, and the total.  `lds` holds kSortWaves values.
__device__ __forceinline__ int block_exclusive(int v, int* lds, int* total) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int incl = wave_scan(v);
  if (lane == 63) lds[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) before += lds[w];
    all += lds[w];
  }
  __syncthreads();
  *total = all;
  return before + incl - v;
}

template <typename T, typename I>
__global__ __launch_bounds__(kSortThreads) void embedding_sort_kernel(EmbeddingBwdArgs a, int rows_per_range) {
  extern __shared__ int count[];  // [kSortWaves][rows_per_range]: tokens of a wave's part, then their places
  __shared__ int lds[kSortWaves];
  const I* __restrict__ ids = static_cast<const I*>(a.ids);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t r0 = int64_t(blockIdx.x) * rows_per_range;
  const int rows = int(a.vocab - r0 < rows_per_range ? a.vocab - r0 : rows_per_range);
  for (int i = threadIdx.x; i < kSortWaves * rows_per_range; i += kSortThreads) count[i] = 0;
  __syncthreads();

  // each wave reads a part of the tokens of its own, in order
  const int64_t part = ((a.tokens + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t begin = wave * part, end = begin + part < a.tokens ? begin + part : a.tokens;
  int* mine = count + wave * rows_per_range;
  int below = 0;
  for (int64_t t = begin + lane; t < end; t += 64) {
    const int64_t id = ids[t];
    below += id >= 0 && id < r0;
    if (id >= r0 && id < r0 + rows) atomicAdd(mine + (id - r0), 1);
  }
  int base;
  block_exclusive(below, lds, &base);  // its barriers also end the counting

  // places: rows in order, a row's tokens by wave
  int of_row = 0;
  if (int(threadIdx.x) < rows)
    for (int w = 0; w < kSortWaves; ++w) of_row += count[w * rows_per_range + threadIdx.x];
  int found;
  int place = base + block_exclusive(of_row, lds, &found);
  if (int(threadIdx.x) < rows)
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = count[w * rows_per_range + threadIdx.x];
      count[w * rows_per_range + threadIdx.x] = place;
      place += n;
    }
  __shared__ unsigned char empty[kSortMaxRows];
  if (int(threadIdx.x) < rows) empty[threadIdx.x] = of_row == 0;
  if (r0 + rows == a.vocab && threadIdx.x == 0) *a.num_sorted = base + found;
  __syncthreads();

  if (found > 0) {
    for (int64_t t0 = begin; t0 < end; t0 += 64) {
      const int64_t t = t0 + lane;
      const int64_t id = t < end ? int64_t(ids[t]) : -1;
      const int row = id >= r0 && id < r0 + rows ? int(id - r0) : -1;
      uint64_t todo = __ballot(row >= 0);
      while (todo != 0) {
        const int leader = __ffsll((unsigned long long)todo) - 1;
        const int r = __shfl(row, leader, 64);
        const uint64_t same = __ballot(row == r);
        // only this wave uses this place, and its LDS accesses stay in order
        const int first = __hip_atomic_load(mine + r, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        if (row == r) {
          const int at = first + __popcll(same & ((uint64_t(1) << lane) - 1));
          a.sorted_token[at] = int(t);
          a.sorted_row[at] = int(r0) + r;
        }
        if (lane == leader)
          __hip_atomic_store(mine + r, first + __popcll(same), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        todo &= ~same;
      }
    }
  }

  if (a.accumulate) return;
  const float zero[8] = {};
  for (int r = wave; r < rows; r += kSortWaves) {
    if (!empty[r]) continue;
    T* out = static_cast<T*>(a.dtable) + (r0 + r) * a.dim;
    for (int64_t c = lane * 8; c < a.dim; c += 512) store_vec<T, 8>(out + c, int(a.dim - c < 8 ? a.dim - c : 8), zero);
  }
}

// ---------------------------------------------------------------------------------------------
// Gradient: sums
// ---------------------------------------------------------------------------------------------

template <typename T>
__device__ __forceinline__ void write_row(const EmbeddingBwdArgs& a, int row, int64_t c, int n, const float (&acc)[8]) {
  T* out = static_cast<T*>(a.dtable) + int64_t(row) * a.dim + c;
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = acc[k] * a.scale;
  if (a.accumulate) {
    const Raw<T, 8> old = load_vec<T, 8>(out, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] += old.get(k);
  }
  store_vec<T, 8>(out, n, f);
}

// blockIdx.x: piece of kPiece sorted tokens; a wave takes 512 columns of it.
template <typename T>
__global__ __launch_bounds__(kThreads) void embedding_sum_kernel(EmbeddingBwdArgs a) {
  const int64_t piece = blockIdx.x;
  const int total = *a.num_sorted;
  const int begin = int(piece * kPiece);
  if (begin >= total) return;
  const int end = begin + kPiece < total ? begin + kPiece : total;
  const int before = begin > 0 ? a.sorted_row[begin - 1] : -1;
  const int after = end < total ? a.sorted_row[end] : -1;
  for (int64_t c = (int64_t(blockIdx.y) * kThreads + threadIdx.x) * 8; c < a.dim; c += int64_t(gridDim.y) * kThreads * 8) {
    const int n = int(a.dim - c < 8 ? a.dim - c : 8);
    float acc[8] = {};
    int row = a.sorted_row[begin];
    bool open = row == before;  // the run began in an earlier piece
    for (int i = begin; i < end; ++i) {
      const Raw<T, 8> r = load_vec<T, 8>(static_cast<const T*>(a.dy) + int64_t(a.sorted_token[i]) * a.dim + c, n);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += r.get(k);
      const int next = i + 1 < end ? a.sorted_row[i + 1] : after;
      if (next == row && i + 1 < end) continue;
      if (open || next == row)
        store_vec<float, 8>(a.partial + (2 * piece + (open ? 0 : 1)) * a.dim + c, n, acc);
      else
        write_row<T>(a, row, c, n, acc);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
      row = next;
      open = false;
    }
  }
}

// blockIdx.x: piece that a run begins in and does not end in.
template <typename T>
__global__ __launch_bounds__(kThreads) void embedding_join_kernel(EmbeddingBwdArgs a) {
  const int64_t piece = blockIdx.x;
  const int total = *a.num_sorted;
  const int64_t border = (piece + 1) * kPiece;
  if (border >= total) return;
  const int row = a.sorted_row[border];
  if (a.sorted_row[border - 1] != row) return;
  const int64_t begin = piece * kPiece;
  if (begin > 0 && a.sorted_row[begin - 1] == row) return;  // begins earlier
  // the last piece of the run: its tokens go on to before `hi`
  int lo = int(border), hi = total;  // sorted_row[lo] == row, sorted_row[hi] != row
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (a.sorted_row[mid] == row)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t last = lo / kPiece;
  for (int64_t c = (int64_t(blockIdx.y) * kThreads + threadIdx.x) * 8; c < a.dim; c += int64_t(gridDim.y) * kThreads * 8) {
    const int n = int(a.dim - c < 8 ? a.dim - c : 8);
    float acc[8] = {};
    for (int64_t q = piece; q <= last; ++q) {
      const Raw<float, 8> r = load_vec<float, 8>(a.partial + (2 * q + (q == piece ? 1 : 0)) * a.dim + c, n);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += r.get(k);
    }
    write_row<T>(a, row, c, n, acc);
  }
}

template <typename T, typename I>
void gradient(const EmbeddingBwdArgs& a, hipStream_t s) {
  const int rows = int(sort_rows(a.vocab));
  const int64_t ranges = (a.vocab + rows - 1) / rows;
  hipLaunchKernelGGL((embedding_sort_kernel<T, I>), dim3(unsigned(ranges)), dim3(kSortThreads),
                     kSortWaves * rows * sizeof(int), s, a, rows);
  const int64_t pieces = (a.tokens + kPiece - 1) / kPiece;
  if (pieces == 0) return;
  int64_t cols = (a.dim + kThreads * 8 - 1) / (kThreads * 8);
  if (cols > 1024) cols = 1024;
  hipLaunchKernelGGL((embedding_sum_kernel<T>), dim3(unsigned(pieces), unsigned(cols)), dim3(kThreads), 0, s, a);
  if (pieces > 1)
    hipLaunchKernelGGL((embedding_join_kernel<T>), dim3(unsigned(pieces - 1), unsigned(cols)), dim3(kThreads), 0, s, a);
}

// Two vectors a lane and up to four waves a row: 65536 rows of 4096 bf16 (20132 distinct of 131072) in
// 129 us, 5.4 TB/s of the bytes that have to move; four vectors 131, eight 134, one wave a row 140.  The
// output is written past the caches, which keep the table's frequent rows: with plain stores 142 us, and
// 18 us against 19 at 8192 rows, where it would fit.
template <typename T, typename I>
void lookup(int64_t tokens, const void* ids, int64_t vocab, int64_t dim, const void* table, float scale, void* out,
            hipStream_t s) {
  constexpr int NV = 2, NT = 4;
  const int64_t vecs = (dim + kVec<T> - 1) / kVec<T>;
  const auto* i = static_cast<const I*>(ids);
  const auto* w = static_cast<const T*>(table);
  auto* o = static_cast<T*>(out);
  if (vecs < 64) {
    int lshift = 0;
    while ((1 << lshift) < vecs) ++lshift;
    const int64_t per = int64_t(kThreads >> lshift) * NT;
    hipLaunchKernelGGL((embedding_narrow_kernel<T, I, NT>), dim3(unsigned((tokens + per - 1) / per)), dim3(kThreads), 0,
                       s, tokens, i, vocab, int(dim), w, scale, o, lshift);
    return;
  }
  const int wshift = vecs <= 64 * NV ? 0 : vecs <= 128 * NV ? 1 : 2;
  const int64_t per = 4 >> wshift;
  hipLaunchKernelGGL((embedding_rows_kernel<T, I, NV>), dim3(unsigned((tokens + per - 1) / per)), dim3(kThreads), 0, s,
                     tokens, i, vocab, dim, w, scale, o, wshift);
}

}  // namespace

int launch_embedding(int64_t tokens, const void* ids, int ids_dtype, int64_t vocab, int64_t dim, const void* table,
                     int dtype, float scale, void* out, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == TIDE_BF16) {
    if (ids_dtype == TIDE_INT32) lookup<bf16_t, int32_t>(tokens, ids, vocab, dim, table, scale, out, s);
    else lookup<bf16_t, int64_t>(tokens, ids, vocab, dim, table, scale, out, s);
  } else {
    if (ids_dtype == TIDE_INT32) lookup<float, int32_t>(tokens, ids, vocab, dim, table, scale, out, s);
    else lookup<float, int64_t>(tokens, ids, vocab, dim, table, scale, out, s);
  }
  return hipGetLastError();
}

int launch_embedding_bwd(const EmbeddingBwdArgs& a, int dtype, int ids_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == TIDE_BF16) {
    if (ids_dtype == TIDE_INT32) gradient<bf16_t, int32_t>(a, s);
    else gradient<bf16_t, int64_t>(a, s);
  } else {
    if (ids_dtype == TIDE_INT32) gradient<float, int32_t>(a, s);
    else gradient<float, int64_t>(a, s);
  }
  return hipGetLastError();
}

}  // namespace tide_step
