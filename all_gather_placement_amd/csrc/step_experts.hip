// Tokens sorted by expert and back.
//
//   sort     place[p] = offsets[e] + pairs of e before p;  source = its inverse
//   dispatch out[r]   = x[source[r] / choices]
//   combine  y[t]     = sum over j of w[t, j] x[place[t, j]]
//   gradient dx[r]    = w[source[r]] dy[source[r] / choices],  dw[t, j] = <dy[t], x[place[t, j]]>
//
// The sort is a stable counting sort of whole numbers: each workgroup counts the pairs of its part by expert, a second
// launch adds up the parts' counts and places each part's pairs, every wave its own in order.  Its memory traffic is
// small; it is bound by its launches and the latencies between its barriers.
//
// The others move rows in 16-byte vectors and are bound by HBM.  A token belongs to one group of lanes, which reads
// its row once and writes all of its rows of the sorted buffer, or has all of those in flight together: 8192 x 2048
// bf16 dispatched to eight experts each 62 us (5.9 TB/s; by rows of the sorted buffer, each reading its token's, 77),
// back 53, the gradients 110 (147 with a wave to a token, which goes on to further columns: loads and stores are
// counted together and in order, so its later loads wait for its stores).
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
constexpr int kWaves = 16;
// Ids of a lane at a time: the code for each is long, so that a wave of few rounds does best with few of them, and one
// of many, where more than 512 experts leave a workgroup fewer waves, with more (in a graph, with 2, 4 and 8: 524288 pairs of
// 128 experts 13.0 us, 13.0, 13.1; of 512 18.0, 17.7, 18.0; of 1024 28.7, 27.5, 27.1; of 2048 72.8, 67.5, 64.8).  In registers 2 do
// best (4: 524288 pairs of 128 experts 13.5, 4096 9.1 instead of 8.4).
constexpr int kHeldIds = 2, kIds = 4, kLongIds = 8;
constexpr int kExpertBits = 11;
static_assert(TIDE_MAX_EXPERTS <= 1 << kExpertBits, "bits of an expert's number");
inline int sort_waves(int experts) {
  int w = kWaves;
  while (w > 1 && w * experts * 4 > kCountBytes) w /= 2;
  return w;
}

// How the pairs are shared: `part` of them to a workgroup, `share` of those to a wave, whole numbers of 64.
struct SortShape {
  int64_t part;
  int32_t share, bits;  // of an expert's number
  __device__ __forceinline__ int64_t begin(int64_t pairs, int wg) const { return wg * part < pairs ? wg * part : pairs; }
};
template <typename I>
__device__ __forceinline__ int expert_of(I id, int experts) {  // -1: none
  return id >= 0 && id < experts ? int(id) : -1;
}

template <typename I>
__global__ __launch_bounds__(1024) void expert_count_kernel(ExpertSortArgs a, SortShape g) {
  extern __shared__ int count[];  // [experts]
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) count[e] = 0;
  __syncthreads();
  const int64_t end = g.begin(a.pairs, blockIdx.x + 1);
  const I* ids = static_cast<const I*>(a.ids);
  for (int64_t p = g.begin(a.pairs, blockIdx.x) + threadIdx.x; p < end; p += blockDim.x) {
    const int e = expert_of(ids[p], a.experts);
    if (e >= 0) atomicAdd(count + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) a.counts[int64_t(blockIdx.x) * a.experts + e] = count[e];
}

// Sum over the workgroup before this thread, of which the first `waves` waves have something to add; in those.
// `lds` holds a value for each.
__device__ __forceinline__ int block_exclusive(int v, int* lds, int waves) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  int incl = 0, before = 0;
  if (wave < waves) {
    incl = wave_scan(v);
    if (lane == 63) lds[wave] = incl;
  }
  __syncthreads();
  if (wave < waves)
    for (int w = 0; w < wave; ++w) before += lds[w];
  return before + incl - v;
}

// The lanes of the wave with this lane's expert (any, without one).
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
  const uint64_t some = __ballot(e >= 0);
  unsigned low = unsigned(some), high = unsigned(some >> 32);
#pragma unroll
  for (int k = 0; k < kExpertBits; ++k)
    if (k < bits) {
      const unsigned mine = unsigned(__builtin_amdgcn_sbfe(e, k, 1));  // all ones or none
      const uint64_t set = __ballot(mine != 0);
      low &= ~(unsigned(set) ^ mine);
      high &= ~(unsigned(set >> 32) ^ mine);
    }
  return uint64_t(high) << 32 | low;
}

// A lane takes kAtOnce ids at a time.  kHeld: these are all of them, and stay in registers with the number of pairs of the same
// expert that the wave has before each (136 pairs 4.6 us in a graph, in the other form 4.9 to 5.1; 65536 8.4 and 8.6 to
// 8.7; 524288 no less).  Otherwise they are read twice, and ranks are found when the wave's first row of each expert is
// known.
template <typename I, int kAtOnce, bool kHeld>
__global__ __launch_bounds__(1024) void expert_place_kernel(ExpertSortArgs a, SortShape g) {
  extern __shared__ int lds[];
  const int waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int experts = a.experts, parts = gridDim.x;
  int* count = lds;                         // [waves][experts]: pairs of a wave, then the row of its next
  int* total = count + waves * experts;     // [experts]: pairs of all parts
  int* before = total + experts;            // [experts]: of lower parts
  int* start = before + experts;            // [experts + 1]: offsets
  int* sums = start + experts + 1;          // [waves]
  const int64_t end = g.begin(a.pairs, blockIdx.x + 1), first = g.begin(a.pairs, blockIdx.x) + wave * int64_t(g.share);
  const int n = int(first + g.share < end ? g.share : end > first ? end - first : 0);
  const I* ids = static_cast<const I*>(a.ids) + first;
  I id[kAtOnce];
  int mine[kAtOnce], rank[kAtOnce];
  const auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) id[j] = i0 + j * 64 + lane < n ? ids[i0 + j * 64 + lane] : I(-1);
  };
  const auto find = [&] {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) mine[j] = expert_of(id[j], experts);
  };
  load(0);  // while the counts are read
  for (int i = threadIdx.x; i < (waves + 2) * experts; i += blockDim.x) count[i] = 0;
  __syncthreads();
  if (parts > 1) {
    // each thread adds up the counts of neighbouring parts for an expert, or for several
    constexpr int kAhead = 16;
    const int groups = blockDim.x > unsigned(experts) ? int(blockDim.x) / experts : 1;
    const int group = int(threadIdx.x) / experts, chunk = (parts + groups - 1) / groups, here = int(blockIdx.x);
    const int b1 = group < groups ? (group * chunk + chunk < parts ? group * chunk + chunk : parts) : 0;
    for (int e = int(threadIdx.x) - group * experts; e < experts; e += blockDim.x) {
      int all = 0, low = 0;
      for (int b0 = group * chunk; b0 < b1; b0 += kAhead) {
        int c[kAhead], sum = 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) c[k] = b0 + k < b1 ? a.counts[int64_t(b0 + k) * experts + e] : 0;
        loads_first();
#pragma unroll
        for (int k = 0; k < kAhead; ++k) sum += c[k];
        all += sum;
        if (b0 + kAhead <= here) {
          low += sum;
        } else if (b0 < here) {
#pragma unroll
          for (int k = 0; k < kAhead; ++k) low += b0 + k < here ? c[k] : 0;
        }
      }
      if (all > 0) atomicAdd(total + e, all);
      if (low > 0) atomicAdd(before + e, low);
    }
  }
  find();
  // Only this wave uses its row of `count` between barriers, and its LDS accesses stay in order.
  int* own = count + wave * experts;
  // the next places of the lanes' experts, in order of the lanes; own[e] goes on behind them
  const auto take = [&](int e) {
    const uint64_t same = same_expert(e, g.bits);
    int at = -1;
    if (e >= 0) {
      at = __hip_atomic_load(own + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) + lanes_before(same);
      if (lane == 63 - __clzll((long long)same))  // the last of its expert
        __hip_atomic_store(own + e, at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    return at;
  };
  if constexpr (kHeld) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (j * 64 >= n) break;
      rank[j] = take(mine[j]);
    }
  } else {
    for (int i0 = 0; i0 < n; i0 += 64 * kAtOnce) {
      if (i0 > 0) {
        load(i0);
        find();
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (mine[j] >= 0) atomicAdd(own + mine[j], 1);
    }
  }
  __syncthreads();
  if (parts == 1) {
    for (int e = threadIdx.x; e < experts; e += blockDim.x) {
      int all = 0;
      for (int w0 = 0; w0 < waves; w0 += 8)
#pragma unroll
        for (int w = 0; w < 8; ++w) all += w0 + w < waves ? count[(w0 + w) * experts + e] : 0;
      total[e] = all;
    }
    __syncthreads();
  }
  // offsets: each thread adds up neighbouring experts
  const int per = (experts + int(blockDim.x) - 1) / int(blockDim.x), e0 = threadIdx.x * per;
  const auto padded = [&](int e) { return int((unsigned(total[e]) + unsigned(a.align) - 1) / unsigned(a.align)) * a.align; };
  int sum = 0;
  for (int e = e0; e < e0 + per && e < experts; ++e) sum += padded(e);
  int at = block_exclusive(sum, sums, (experts + 64 * per - 1) / (64 * per));
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
    for (int w0 = 0; w0 < waves; w0 += 8) {
      int c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = w0 + w < waves ? count[(w0 + w) * experts + e] : 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w0 + w < waves) count[(w0 + w) * experts + e] = row;
        row += c[w];
      }
    }
  }
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += 64 * kAtOnce) {
    if (!kHeld) {
      load(i0);
      find();
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (i0 + j * 64 >= n) break;
      const int i = i0 + j * 64 + lane, e = mine[j];
      int row = -1;
      if constexpr (kHeld) {
        if (e >= 0) row = own[e] + rank[j];
      } else {
        row = take(e);
      }
      if (row >= 0) a.source[row] = int(first) + i;
      if (i < n) a.place[first + i] = row;
    }
    if constexpr (kHeld) break;
  }
  // rows of no pair: 16 lanes for each expert's, all for those behind the last expert
  if (a.align > 1)
    for (int e = int((blockIdx.x * blockDim.x + threadIdx.x) >> 4); e < experts; e += int((gridDim.x * blockDim.x) >> 4))
      // without a sign: the last of 2^31 - 1 rows may be an expert's, or end where another's begin
      for (unsigned r = unsigned(start[e] + total[e]) + (threadIdx.x & 15); r < unsigned(start[e + 1]); r += 16)
        a.source[r] = -1;
  for (int64_t r = start[experts] + int64_t(blockIdx.x) * blockDim.x + threadIdx.x; r < a.rows;
       r += int64_t(parts) * blockDim.x)
    a.source[r] = -1;
}

// ---------------------------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------------------------

// A row's columns in vectors of E, one a lane.  Where a row ends inside a vector, the last one is the vector that
// ends with the row: it shares elements with the one before, which both read, and write alike -- but not over what they
// read, where the one before may be late: another wave's, or an earlier turn's.  Loads and stores of single elements, and
// their waits, would take longer than the rest of a row.  kTiny: rows of less than a vector.
template <typename T, bool kTiny>
struct Columns {
  static constexpr int E = kVec<T>;
  int64_t at;  // first element
  int n;       // elements of a tiny row
  int shared;  // of the first ones, those of the vector before
  __device__ __forceinline__ Columns(int64_t c, int64_t dim) {
    at = kTiny || c + E <= dim ? c : dim - E;
    n = kTiny ? int(dim) : E;
    shared = int(c - at);
  }
  template <bool kOnce>
  __device__ __forceinline__ Raw<T, E> load(const T* row) const {
    if constexpr (kTiny)
      return load_vec<T, E, kOnce, false>(row, n, false);
    else
      return load_whole<T, E, kOnce>(row + at);
  }
  template <bool kOnce>
  __device__ __forceinline__ void store(T* row, const float (&f)[E]) const {
    store_vec<T, E, kOnce, !kTiny>(row + at, n, f);
  }
  // The same without the elements of the vector before.
  __device__ __forceinline__ void store_own(T* row, const float (&f)[E]) const {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k >= shared && k < n) row[at + k] = narrow<T>(f[k]);
  }
  template <bool kOnce>
  __device__ __forceinline__ void store(T* row, const Raw<T, E>& r) const {
    store_raw<T, E, kOnce, !kTiny>(row + at, n, r);
  }
};

// A lane's place: 1 << lshift neighbouring lanes of the workgroup share a row, whole waves of it from 64 on.
struct Lanes {
  int lane, group, per;  // of the row; the row's number and the workgroup's rows
  __device__ __forceinline__ explicit Lanes(int lshift) {
    lane = threadIdx.x & ((1 << lshift) - 1);
    group = threadIdx.x >> lshift;
    per = kThreads >> lshift;
    if (lshift >= 6) group = __builtin_amdgcn_readfirstlane(group);
  }
};
inline int lanes_shift(int64_t vecs) {
  int s = 0;
  while (s < 8 && (int64_t(1) << s) < vecs) ++s;
  return s;
}

// Rows that a wave looks at for those of no pair: zeros of up to 16 KiB (4 rows of 4 KiB for each wave; one for each
// made the gradient of 8192 tokens' rows 5 us slower), and of a row at least.
inline int zero_rows_of(int64_t vecs) { return int(vecs >= 1024 ? 1 : vecs <= 16 ? 64 : 1024 / vecs); }
inline unsigned zeroing_of(const ExpertRowsArgs& a, int64_t vecs) {
  return a.rows > 0 ? grid_of(a.rows, zero_rows_of(vecs) * (kThreads / 64)) : 0;
}

// Workgroups that write zeros among those that take tokens, spread evenly.
struct Mixed {
  unsigned tokens, zeros;
  uint64_t step;  // zeros of all, in 2^-32, rounded up
  Mixed(unsigned t, unsigned z) : tokens(t), zeros(z), step(t + z > 0 ? ((uint64_t(z) << 32) + t + z - 1) / (t + z) : 0) {}
  // The workgroup's number among those of its kind.
  __device__ __forceinline__ unsigned number(bool* zero) const {
    const unsigned before = unsigned(blockIdx.x * step >> 32);
    *zero = unsigned((blockIdx.x + 1) * step >> 32) != before;
    return *zero ? before : blockIdx.x - before;
  }
};

// Zeros to the rows of no pair, `count` rows a wave at a time, far apart: many of those rows lie together behind the
// last expert.
template <typename T, bool kTiny>
__device__ __forceinline__ void zero_rows(const ExpertRowsArgs& a, int count, unsigned wg, unsigned wgs) {
  constexpr int E = kVec<T>, kWaves = kThreads / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t pairs = a.tokens * a.choices;
  const Raw<T, E> zero = {};
  const int64_t apart = int64_t(wgs) * kWaves;
  for (int64_t r0 = int64_t(wg) * kWaves + wave; r0 < a.rows; r0 += apart * count) {
    bool none = false;
    if (lane < count && r0 + lane * apart < a.rows) {
      const int s = a.source[r0 + lane * apart];
      none = s < 0 || s >= pairs;
    }
    for (uint64_t todo = __ballot(none); todo != 0; todo &= todo - 1) {
      T* to = static_cast<T*>(a.out) + (r0 + (__ffsll((unsigned long long)todo) - 1) * apart) * a.out_stride;
      for (int64_t c = int64_t(lane) * E; c < a.dim; c += 64 * E) Columns<T, kTiny>(c, a.dim).template store<false>(to, zero);
    }
  }
}

// A token to 1 << lshift lanes, which write it to its rows.
template <typename T, bool kTiny, bool kOnce>
__global__ __launch_bounds__(kThreads) void expert_dispatch_kernel(ExpertRowsArgs a, Mixed mixed, int lshift,
                                                                   int zero_count) {
  constexpr int E = kVec<T>;
  bool zero;
  const unsigned wg = mixed.number(&zero);
  if (zero) return zero_rows<T, kTiny>(a, zero_count, wg, mixed.zeros);
  const Lanes l(lshift);
  for (int64_t t = int64_t(wg) * l.per + l.group; t < a.tokens; t += int64_t(mixed.tokens) * l.per) {
    const T* from = static_cast<const T*>(a.x) + t * a.x_stride;
    const int32_t* place = a.place + t * a.choices;
    for (int64_t c = int64_t(l.lane) * E; c < a.dim; c += int64_t(E) << lshift) {
      const Columns<T, kTiny> col(c, a.dim);
      const Raw<T, E> v = col.template load<true>(from);
      for (int j = 0; j < a.choices; ++j) {
        const int row = place[j];
        if (row >= 0 && row < a.rows) col.template store<kOnce>(static_cast<T*>(a.out) + row * a.out_stride, v);
      }
    }
  }
}

// Rows of choices j0 to j0 + N - 1 of token t, -1 for none, and their weights.
template <int N>
struct Choices {
  int row[N];
  float w[N];
  bool any;
  __device__ __forceinline__ Choices(const ExpertRowsArgs& a, int64_t t, int j0, bool bf16) {
    any = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      row[j] = j0 + j < a.choices ? a.place[t * a.choices + j0 + j] : -1;
      if (row[j] >= a.rows) row[j] = -1;
      any |= row[j] >= 0;
      w[j] = 1.0f;
    }
    if (a.weights == nullptr) return;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (row[j] >= 0) {
        const int64_t p = t * a.choices + j0 + j;
        w[j] = bf16 ? widen(static_cast<const bf16_t*>(a.weights)[p]) : static_cast<const float*>(a.weights)[p];
      }
  }
};

// A token to 1 << lshift lanes; the rows of N choices are in flight at a time and added in order.
template <typename T, int N, bool kTiny, bool kOnce>
__global__ __launch_bounds__(kThreads) void expert_combine_kernel(ExpertRowsArgs a, bool bf16_weights, int lshift) {
  constexpr int E = kVec<T>;
  const Lanes l(lshift);
  for (int64_t t = int64_t(blockIdx.x) * l.per + l.group; t < a.tokens; t += int64_t(gridDim.x) * l.per) {
    for (int64_t c = int64_t(l.lane) * E; c < a.dim; c += int64_t(E) << lshift) {
      const Columns<T, kTiny> col(c, a.dim);
      float acc[E] = {};
      for (int j0 = 0; j0 < a.choices; j0 += N) {
        const Choices<N> ch(a, t, j0, bf16_weights);
        Raw<T, E> r[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (ch.row[j] >= 0) r[j] = col.template load<kOnce>(static_cast<const T*>(a.x) + ch.row[j] * a.x_stride);
        loads_first();
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (ch.row[j] >= 0) {
#pragma unroll
            for (int k = 0; k < E; ++k) acc[k] = fmaf(ch.w[j], r[j].get(k), acc[k]);
          }
      }
      col.template store<kOnce>(static_cast<T*>(a.out) + t * a.out_stride, acc);
    }
  }
}

// A token belongs to kLanes lanes; with 64, to 1 << wshift waves of the workgroup's four, whose sums meet in LDS.  Rows
// of whole waves are read and written past the caches, beside the zeros, which go through them: 8192 x 2048 bf16 by
// eight experts 110 us, through the caches 129, a quarter of that 38 and 47; rows of 100 columns 19 us, past the
// caches 21.
// kOwn: an element is written by the lane that has it in its dot product, and read by no other for its own.  Rows that end
// inside a vector need that in place; a form of its own, since the other takes 2% longer with a branch for it.
template <typename T, int N, bool kTiny, int kLanes, bool kOwn>
__global__ __launch_bounds__(kThreads) void expert_combine_bwd_kernel(ExpertRowsArgs a, bool bf16_weights,
                                                                      Mixed mixed, int wshift, int zero_count) {
  constexpr int E = kVec<T>;
  bool zero;
  const unsigned wg = mixed.number(&zero);
  if (zero) return zero_rows<T, kTiny>(a, zero_count, wg, mixed.zeros);
  __shared__ float sums[kThreads / 64][N];
  const int lane = threadIdx.x & (kLanes - 1), per = (kThreads / kLanes) >> wshift;
  int group = threadIdx.x / kLanes;
  if (kLanes == 64) group = __builtin_amdgcn_readfirstlane(group);
  const int part = group & ((1 << wshift) - 1);  // of a row's waves
  const auto put = [&](int64_t p, float v) {
    if (bf16_weights)
      static_cast<bf16_t*>(a.dweights)[p] = narrow<bf16_t>(v);
    else
      static_cast<float*>(a.dweights)[p] = v;
  };
  for (int64_t t0 = int64_t(wg) * per; t0 < a.tokens; t0 += int64_t(mixed.tokens) * per) {
    const int64_t t = t0 + (group >> wshift);
    const bool mine = t < a.tokens;
    for (int j0 = 0; j0 < a.choices; j0 += N) {
      const Choices<N> ch(a, mine ? t : 0, mine ? j0 : a.choices, bf16_weights);
      float dot[N] = {};
      if (ch.any)
        for (int64_t c = int64_t(part * kLanes + lane) * E; c < a.dim; c += int64_t(kLanes * E) << wshift) {
          const Columns<T, kTiny> col(c, a.dim);
          const Raw<T, E> d = col.template load<false>(static_cast<const T*>(a.dy) + t * a.dy_stride);
          Raw<T, E> r[N];
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (ch.row[j] >= 0) r[j] = col.template load<(kLanes == 64)>(static_cast<const T*>(a.x) + ch.row[j] * a.x_stride);
          loads_first();
#pragma unroll
          for (int j = 0; j < N; ++j) {
            if (ch.row[j] < 0) continue;
            float f[E];
#pragma unroll
            for (int k = 0; k < E; ++k) {
              if (kTiny || k >= col.shared) dot[j] = fmaf(d.get(k), r[j].get(k), dot[j]);
              f[k] = ch.w[j] * d.get(k);
            }
            T* to = static_cast<T*>(a.out) + ch.row[j] * a.out_stride;
            if (kOwn && col.shared > 0)
              col.store_own(to, f);
            else
              col.template store<(kLanes == 64)>(to, f);
          }
          if constexpr (kLanes < 64) break;  // lanes for all of a row
        }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float sum = lanes_sum<kLanes>(dot[j]);
        if (wshift > 0) {
          if (lane == 0) sums[group][j] = sum;
        } else if (lane == 0 && mine && j0 + j < a.choices) {
          put(t * a.choices + j0 + j, sum);
        }
      }
      if (wshift > 0) {
        __syncthreads();
        if (part == 0 && lane < N && mine && j0 + lane < a.choices) {
          float sum = 0.0f;
          for (int p = 0; p < 1 << wshift; ++p) sum += sums[group + p][lane];
          put(t * a.choices + j0 + lane, sum);
        }
        __syncthreads();
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------------------------

template <typename I>
int sort(const ExpertSortArgs& a, hipStream_t s) {
  const int parts = expert_parts(a.pairs, a.experts);
  SortShape g{ceil_div(ceil_div(a.pairs, parts), 64) * 64, 0, 0};
  int waves = sort_waves(a.experts);
  while (waves > 1 && g.part <= 64 * waves) waves /= 2;  // 128 pairs a wave, if there are: what its lanes hold
  while ((1 << g.bits) < a.experts) ++g.bits;
  g.share = int32_t(ceil_div(ceil_div(g.part, waves), 64) * 64);
  if (parts > 1)
    if (const int e = launch(expert_count_kernel<I>, unsigned(parts), 1024, size_t(a.experts) * 4, s, a, g)) return e;
  const size_t lds = (size_t(waves + 3) * a.experts + 1 + waves) * 4;
  const auto place = g.share <= 64 * kHeldIds ? expert_place_kernel<I, kHeldIds, true>
                     : waves < kWaves         ? expert_place_kernel<I, kLongIds, false>
                                              : expert_place_kernel<I, kIds, false>;
  return launch(place, unsigned(parts), waves * 64, lds, s, a, g);
}

template <typename F>
int with_bool(bool b, F&& f) {
  return b ? f(std::true_type()) : f(std::false_type());
}

// Zeros are written through the caches, which take them up beside what goes past them: with at least an eighth of the
// pairs as many rows of no pair, pairs' rows past the caches make the best of both (8192 tokens of 2048 bf16 to eight
// experts each, a quarter of that of no pair: 62 us instead of 71); without, all go through them (57 us instead of 63).
// Rows of less than 64 vectors share their ends' cache lines with others (30000 x 100 bf16 to six experts 13 us, past
// the caches 20).
template <typename T>
int dispatch(const ExpertRowsArgs& a, hipStream_t s) {
  const int64_t vecs = ceil_div(a.dim, kVec<T>), pairs = a.tokens * a.choices;
  const auto call = [&](auto tiny, auto once) {
    const int lshift = lanes_shift(vecs);
    const Mixed mixed(a.tokens > 0 ? grid_of(a.tokens, kThreads >> lshift) : 0, zeroing_of(a, vecs));
    return launch(expert_dispatch_kernel<T, decltype(tiny)::value, decltype(once)::value>, mixed.tokens + mixed.zeros,
                  kThreads, 0, s, a, mixed, lshift, zero_rows_of(vecs));
  };
  if (a.dim < kVec<T>) return call(std::true_type(), std::false_type());
  return with_bool(vecs >= 64 && a.dim % kVec<T> == 0 && a.rows - pairs >= pairs / 8,
                   [&](auto once) { return call(std::false_type(), once); });
}

// f(choices in flight) as a constant.
template <typename F>
int with_choices(int choices, F&& f) {
  if (choices > 4) return f(std::integral_constant<int, 8>());
  if (choices > 2) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 2>());
}

// A sorted buffer of more bytes is read past the caches on its way back, and what it gives written past them: 8192
// tokens of 2048 bf16 by eight experts (256 MiB) 52 us instead of 59, 40000 251 instead of 283; 4099 x 3 rows of 1001 fp32
// (49 MB) 11.3 us, past the caches 12.2.
constexpr int64_t kReadOnce = int64_t(128) << 20;
template <typename T>
int64_t bytes_of(const ExpertRowsArgs& a) {
  return a.rows * a.dim * int64_t(sizeof(T));
}

template <typename T>
int combine(const ExpertRowsArgs& a, bool bf16_weights, hipStream_t s) {
  const auto call = [&](auto tiny, auto nt) {
    return with_choices(a.choices, [&](auto n) {
      const int lshift = lanes_shift(ceil_div(a.dim, kVec<T>));
      return launch(expert_combine_kernel<T, decltype(n)::value, decltype(tiny)::value, decltype(nt)::value>,
                    grid_of(a.tokens, kThreads >> lshift), kThreads, 0, s, a, bf16_weights, lshift);
    });
  };
  if (a.dim < kVec<T>) return call(std::true_type(), std::false_type());
  return with_bool(bytes_of<T>(a) > kReadOnce, [&](auto nt) { return call(std::false_type(), nt); });
}

template <typename T>
int combine_bwd(const ExpertRowsArgs& a, bool bf16_weights, hipStream_t s) {
  const int64_t vecs = ceil_div(a.dim, kVec<T>);
  const auto call = [&](auto tiny, auto lanes, auto own) {
    return with_choices(a.choices, [&](auto n) {
      const int wshift = vecs <= 64 ? 0 : vecs <= 128 ? 1 : 2;
      const Mixed mixed(a.tokens > 0 ? grid_of(a.tokens, (kThreads / decltype(lanes)::value) >> wshift) : 0,
                        zeroing_of(a, vecs));
      return launch(expert_combine_bwd_kernel<T, decltype(n)::value, decltype(tiny)::value, decltype(lanes)::value,
                                              decltype(own)::value>,
                    mixed.tokens + mixed.zeros, kThreads, 0, s, a, bf16_weights, mixed, wshift, zero_rows_of(vecs));
    });
  };
  if (a.dim < kVec<T>) return call(std::true_type(), std::integral_constant<int, 1>(), std::false_type());
  return with_bool(a.out == a.x && a.dim % kVec<T> != 0, [&](auto own) {
    if (vecs <= 4) return call(std::false_type(), std::integral_constant<int, 4>(), own);
    if (vecs <= 16) return call(std::false_type(), std::integral_constant<int, 16>(), own);
    return call(std::false_type(), std::integral_constant<int, 64>(), own);
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
  const bool bf16_weights = weight_dtype == TIDE_BF16;
  return dtype == TIDE_BF16 ? combine<bf16_t>(a, bf16_weights, s) : combine<float>(a, bf16_weights, s);
}
int launch_expert_combine_bwd(const ExpertRowsArgs& a, int dtype, int weight_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf16_weights = weight_dtype == TIDE_BF16;
  return dtype == TIDE_BF16 ? combine_bwd<bf16_t>(a, bf16_weights, s) : combine_bwd<float>(a, bf16_weights, s);
}

}  // namespace tide_step
