// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = table[ids[t]] * scale                      (zeros for ids outside the table)
//   dtable[v] = scale * sum of dy[t] over ids[t] = v    (in ascending t)
//
// HBM bounds the lookup: rows are read and written once in 16-byte vectors.
//
// The gradient has to write every row of the table, and most rows have no token.  Its first kernel
// brings tokens of equal id together.  Workgroup b of 2^k owns the rows v with v mod 2^k = b, so that
// low, frequent ids are shared evenly.  It reads all ids (which stay in the L2), counts those of each of
// its rows and those of lower workgroups -- the place where its tokens begin -- and then places its
// tokens in ascending order: a stable counting sort with no traffic between workgroups.  The rows are
// filled with zeros beside that or before it.  The second kernel sums the sorted tokens in pieces of
// equal length, so a frequent id is shared by many waves, and a third adds the partial sums of ids that
// cross pieces, in a fixed order.
//
// Measured: lookup of 65536 rows of 4096 bf16 128 us; gradient of 8192 such rows in a table of 131072
// 200 us (zeros 160, sort 8, sums 23, join 6), of 50021 rows of 1001 fp32 in 20011 75 us (sort beside the
// zeros 20, sums 48 -- 5.1 TB/s, rows at 4-byte boundaries --, join 7).
#include "step_device.h"
#include "step_internal.h"

namespace tide_step {
namespace {

constexpr int kThreads = 256;

// Workgroups for n items, `per` each: a launch holds less than 2^32 threads, so kernels go on to the
// items a grid further.
constexpr int64_t kMaxGrid = int64_t(1) << 21;
__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline unsigned grid_of(int64_t n, int64_t per) {
  const int64_t g = ceil_div(n, per);
  return unsigned(g < kMaxGrid ? g : kMaxGrid);
}

// ---------------------------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------------------------

template <typename T, int E, bool kWhole>
__device__ __forceinline__ void store_scaled(T* out, int n, const Raw<T, E>& r, bool inside, float scale) {
  float f[E];
#pragma unroll
  for (int k = 0; k < E; ++k) f[k] = inside ? r.get(k) * scale : 0.0f;
  store_vec<T, E, true, kWhole>(out, n, f);
}
template <int E>
__device__ __forceinline__ int tail(int64_t n) {
  return int(n < E ? n : E);
}

// Rows of 64 vectors and more: a row goes to 1 << wshift waves of a workgroup of four, a lane holding
// NV vectors at a time.
template <typename T, typename I, int NV, bool kWhole>
__global__ __launch_bounds__(kThreads) void embedding_rows_kernel(int64_t tokens, const I* __restrict__ ids,
                                                                  int64_t vocab, int64_t dim,
                                                                  const T* __restrict__ table, float scale,
                                                                  T* __restrict__ out, int wshift) {
  constexpr int E = kVec<T>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t step = int64_t(64 * NV * E) << wshift;
  for (int64_t t = (int64_t(blockIdx.x) << (2 - wshift)) + (wave >> wshift); t < tokens;
       t += int64_t(gridDim.x) << (2 - wshift)) {
    const int64_t id = ids[t];
    const bool inside = id >= 0 && id < vocab;
    const T* row = table + (inside ? id * dim : 0);
    T* o = out + t * dim;
    for (int64_t c0 = int64_t(wave & ((1 << wshift) - 1)) * (64 * NV * E); c0 < dim; c0 += step) {
      Raw<T, E> r[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t c = c0 + (v * 64 + lane) * E;
        r[v] = load_vec<T, E, false, kWhole>(row + c, inside ? tail<E>(dim - c) : 0, true);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t c = c0 + (v * 64 + lane) * E;
        if (c < dim) store_scaled<T, E, kWhole>(o + c, tail<E>(dim - c), r[v], inside, scale);
      }
    }
  }
}

// Narrow rows: a group of 1 << lshift lanes for each of NT tokens in turn.
template <typename T, typename I, int NT, bool kWhole>
__global__ __launch_bounds__(kThreads) void embedding_narrow_kernel(int64_t tokens, const I* __restrict__ ids,
                                                                    int64_t vocab, int dim,
                                                                    const T* __restrict__ table, float scale,
                                                                    T* __restrict__ out, int lshift) {
  constexpr int E = kVec<T>;
  const int groups = kThreads >> lshift, c = (threadIdx.x & ((1 << lshift) - 1)) * E;
  for (int64_t t0 = int64_t(blockIdx.x) * groups * NT + (threadIdx.x >> lshift); t0 < tokens;
       t0 += int64_t(gridDim.x) * groups * NT) {
    int64_t id[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) id[i] = t0 + i * groups < tokens ? int64_t(ids[t0 + i * groups]) : -1;
    Raw<T, E> r[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const bool inside = id[i] >= 0 && id[i] < vocab;
      r[i] = load_vec<T, E, false, kWhole>(table + (inside ? id[i] * dim : 0) + c, inside ? dim - c : 0, dim >= E);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int64_t t = t0 + i * groups;
      if (t < tokens && c < dim)
        store_scaled<T, E, kWhole>(out + t * dim + c, dim - c, r[i], id[i] >= 0 && id[i] < vocab, scale);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Gradient: sorting tokens by id, and the rows without tokens
// ---------------------------------------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kRowBits = 9;   // of a row's number within its range
constexpr int kListed = 448;  // tokens of a wave's list (with the counts less than 64 KiB of LDS)
static_assert((1 << kRowBits) == kSortMaxRows, "a list's entry is a token of the wave's part and a row");

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

// Lanes of m below this one.
__device__ __forceinline__ int lanes_before(uint64_t m) {
  return int(__builtin_amdgcn_mbcnt_hi(unsigned(m >> 32), __builtin_amdgcn_mbcnt_lo(unsigned(m), 0)));
}

// The lanes whose `row` equals this lane's, of those in `active`.  A range seldom has more than two
// different rows among 64 tokens: the first few are taken one by one, what is left by the rows' bits.
__device__ __forceinline__ uint64_t same_row(int row, uint64_t active, int bits, int lane) {
  uint64_t same = 0, todo = active;
  for (int k = 0; k < 3 && todo != 0; ++k) {
    const int r = __builtin_amdgcn_readlane(row, __ffsll((unsigned long long)todo) - 1);
    const uint64_t of_r = __ballot(row == r) & todo;
    if (row == r) same = of_r;
    todo &= ~of_r;
  }
  if (todo != 0) {
    uint64_t rest = todo;
    for (int k = 0; k < bits; ++k) {
      const uint64_t set = __ballot((row >> k) & 1);
      rest &= (row >> k) & 1 ? set : ~set;
    }
    if ((todo >> lane) & 1) same = rest;
  }
  return same;
}

// Workgroups below `sorting` sort, the ranges from `first_range` on; the others, if any, write zeros to the
// table, one 16-byte store a thread: short-lived workgroups in order of address write fastest (131072 x 4096
// bf16 with 256 threads 157 us, 1024 threads 169, a wave for each row 194).  Rows that have tokens are written
// again by the sums, which costs less than asking for each row whether it has any (237 us with the sums, 30
// more).
//
// 50021 tokens of a text over 20011 rows: 20 us; with the ids read once more for the places 24, without
// a queue or list, a few tokens at a time, 28, and with a row's lanes found by all of its bits 44.
template <typename T, typename I>
__global__ __launch_bounds__(kSortThreads) void embedding_sort_kernel(EmbeddingBwdArgs a, unsigned first_range,
                                                                      unsigned sorting, unsigned ranges, int shift,
                                                                      int most_rows, int bits) {
  if (blockIdx.x >= sorting) {
    constexpr int N = kVec<T>;
    const float none[N] = {};
    const int64_t end = a.vocab * a.dim;
    for (int64_t e = (int64_t(blockIdx.x - sorting) * kSortThreads + threadIdx.x) * N; e < end;
         e += int64_t(gridDim.x - sorting) * kSortThreads * N)
      store_vec<T, N, false, false>(static_cast<T*>(a.dtable) + e, tail<N>(end - e), none);
    return;
  }
  extern __shared__ int count[];  // [kSortWaves][most_rows]: tokens of a wave's part, then their places
  __shared__ int lds[kSortWaves];
  __shared__ alignas(16) unsigned lists[kSortWaves][kListed];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const unsigned vocab = unsigned(a.vocab), range = first_range + blockIdx.x, mask = (1u << shift) - 1;
  const int rows = int((vocab - range + mask) >> shift);  // range, range + 2^shift, ...: at least one
  for (int i = threadIdx.x; i < kSortWaves * most_rows; i += kSortThreads) count[i] = 0;

  // each wave reads a part of the tokens of its own, in order
  constexpr int kAhead = 16;  // loads in flight (32 take more than 64 registers: fewer workgroups write zeros)
  const int64_t part = ceil_div(ceil_div(a.tokens, kSortWaves), 64) * 64;
  const int64_t first_token = __builtin_amdgcn_readfirstlane(wave) * part;
  const int end = int(first_token + part < a.tokens ? part : a.tokens > first_token ? a.tokens - first_token : 0);
  const I* __restrict__ from = static_cast<const I*>(a.ids) + first_token;
  const auto for_ids = [&](auto&& f) {  // f(token of the part, id), all lanes together; id -1 beyond the end
    for (int t0 = 0; t0 < end; t0 += 64 * kAhead) {
      I v[kAhead];
      if (end - t0 >= 64 * kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = from[t0 + (lane + j * 64)];
      } else {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = lane + j * 64 < end - t0 ? from[t0 + (lane + j * 64)] : I(-1);
      }
      loads_first();
#pragma unroll
      for (int j = 0; j < kAhead; ++j) f(t0 + j * 64 + lane, v[j]);
    }
  };
  const auto range_of = [&](I id) {  // ~0: outside the table
    const bool inside = sizeof(I) == 4 || unsigned(uint64_t(id) >> 32) == 0;
    return inside && unsigned(id) < vocab ? unsigned(id) & mask : ~0u;
  };
  // A wave lists its tokens of the range, so that most ranges read the ids once; those of a range that
  // holds more than the list are found again.  Only this wave uses its list and its row of `count`, and
  // its LDS accesses stay in order.
  unsigned* list = lists[wave];
  int* mine = count + wave * most_rows;
  int below = 0, listed = 0;
  for_ids([&](int t, I id) {
    const unsigned r = range_of(id);
    below += r < range;
    const uint64_t here = __ballot(r == range);
    if (here == 0) return;
    const int at = listed + lanes_before(here);
    if (r == range && at < kListed) list[at] = unsigned(t) << kRowBits | unsigned(id) >> shift;
    listed += __popcll(here);
  });
  const bool all_listed = listed <= kListed && part <= (int64_t(1) << (32 - kRowBits));
  __syncthreads();  // `count` is zero
  if (all_listed) {
    for (int i = lane; i < listed; i += 64) atomicAdd(mine + (list[i] & ((1 << kRowBits) - 1)), 1);
  } else {
    for_ids([&](int, I id) {
      if (range_of(id) == range) atomicAdd(mine + (unsigned(id) >> shift), 1);
    });
  }
  int base;
  block_exclusive(below, lds, &base);  // its barriers also end the counting

  // places: the range's rows in order, a row's tokens by wave
  int of_row = 0;
  if (int(threadIdx.x) < rows)
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) of_row += count[w * most_rows + threadIdx.x];
  int found;
  int place = base + block_exclusive(of_row, lds, &found);
  if (int(threadIdx.x) < rows) {
    // of a run that crosses a border of pieces: the piece it ends in
    const int first_piece = place / kPiece, last_piece = (place + of_row - 1) / kPiece;
    if (of_row > 0 && first_piece != last_piece) a.last_piece[first_piece] = last_piece;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = count[w * most_rows + threadIdx.x];
      count[w * most_rows + threadIdx.x] = place;
      place += n;
    }
  }
  if (threadIdx.x == 0) {
    if (range == ranges - 1) a.num_sorted[0] = base + found;
    if (range == 0) a.num_sorted[1] = a.num_sorted[2] = 0;
  }
  if (found == 0) return;
  __syncthreads();

  // up to 64 tokens in order, one a lane
  const auto place_tokens = [&](int n, int token, int row) {
    const uint64_t active = n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1;
    const uint64_t same = same_row(row, active, bits, lane);
    if (lane < n) {
      const int first = __hip_atomic_load(mine + row, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      const int at = first + lanes_before(same);
      a.sorted_token[at] = token;
      a.sorted_row[at] = int(unsigned(row) << shift | range);
      if (lane == 63 - __clzll((long long)same))  // the last of its row: the next place
        __hip_atomic_store(mine + row, at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
  };
  if (all_listed) {
    for (int i = 0; i < listed; i += 64) {
      const unsigned e = i + lane < listed ? list[i + lane] : 0;
      place_tokens(listed - i, int(first_token) + int(e >> kRowBits), int(e & ((1 << kRowBits) - 1)));
    }
    return;
  }
  // the list's memory as a queue of tokens that wait until there are 64
  int2* queue = reinterpret_cast<int2*>(list);
  static_assert(sizeof(lists[0]) >= 128 * sizeof(int2), "a queue of 128 tokens");
  int waiting = 0;
  const auto take = [&](int n) {
    const int2 q = lane < n ? queue[lane] : int2{0, 0};
    place_tokens(n, q.x, q.y);
  };
  for_ids([&](int t, I id) {
    const unsigned r = range_of(id);
    const uint64_t here = __ballot(r == range);
    if (here == 0) return;
    if (r == range) queue[waiting + lanes_before(here)] = int2{int(first_token) + t, int(unsigned(id) >> shift)};
    waiting += __popcll(here);
    if (waiting < 64) return;
    __builtin_amdgcn_wave_barrier();
    take(64);
    waiting -= 64;
    if (lane < waiting) queue[lane] = queue[64 + lane];
    __builtin_amdgcn_wave_barrier();
  });
  __builtin_amdgcn_wave_barrier();
  take(waiting);
}

// ---------------------------------------------------------------------------------------------
// Gradient: sums
// ---------------------------------------------------------------------------------------------

template <typename T, int E, bool kWhole>
__device__ __forceinline__ void write_row(const EmbeddingBwdArgs& a, int row, int64_t c, int n, const float (&acc)[E]) {
  T* out = static_cast<T*>(a.dtable) + int64_t(row) * a.dim + c;
  float f[E];
#pragma unroll
  for (int k = 0; k < E; ++k) f[k] = acc[k] * a.scale;
  if (a.accumulate) {
    const Raw<T, E> old = load_vec<T, E, false, kWhole>(out, n, a.dim >= E);
#pragma unroll
    for (int k = 0; k < E; ++k) f[k] += old.get(k);
  }
  store_vec<T, E, false, kWhole>(out, n, f);
}

// A wave's item: 64 vectors of columns of a piece of kPiece sorted tokens.  Sixteen
// rows of dy are in flight at a time; they are added in order.
template <typename T, bool kWhole>
__device__ __forceinline__ void sum_piece(const EmbeddingBwdArgs& a, int64_t piece, int64_t c, int total) {
  constexpr int E = kVec<T>, kAhead = 16;
  const int lane = threadIdx.x & 63;
  const int64_t begin = piece * kPiece;
  const int cnt = int(total - begin < kPiece ? total - begin : kPiece);
  // lane i holds token i of the piece; lanes kPiece and kPiece + 1 the rows after and before it
  static_assert(kPiece + 2 <= 64, "a piece and its neighbours are held by one wave");
  const int64_t at = lane < cnt ? begin + lane : lane == kPiece + 1 ? begin - 1 : lane == kPiece ? begin + cnt : -1;
  const int rows = at >= 0 && at < total ? a.sorted_row[at] : -1;
  const int tokens = lane < cnt ? a.sorted_token[at] : 0;
  const int after = __builtin_amdgcn_readlane(rows, kPiece);
  const int n = tail<E>(a.dim - c);
  float acc[E] = {};
  int row = __builtin_amdgcn_readlane(rows, 0);
  bool open = row == __builtin_amdgcn_readlane(rows, kPiece + 1);  // the run began in an earlier piece
  for (int i0 = 0; i0 < cnt; i0 += kAhead) {
    const T* from[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {  // beyond the end the last token again
      const int64_t t = __builtin_amdgcn_readlane(tokens, i0 + j < cnt ? i0 + j : cnt - 1);
      from[j] = static_cast<const T*>(a.dy) + t * a.dim;
    }
    Raw<T, E> r[kAhead];
    load_vecs<T, E, kAhead, true, kWhole>(r, from, c, n, a.dim >= E);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j;
      if (i >= cnt) break;
#pragma unroll
      for (int k = 0; k < E; ++k) acc[k] += r[j].get(k);
      const int next = i + 1 < cnt ? __builtin_amdgcn_readlane(rows, i + 1) : after;
      if (next == row && i + 1 < cnt) continue;
      if (n > 0) {
        if (!open && next == row && c == 0) {  // short runs from the front of the list, long ones from its end
          const int last = a.last_piece[piece], pieces = int(ceil_div(a.tokens, kPiece));
          const int at = last - piece < kShortRun ? atomicAdd(a.num_sorted + 1, 1)
                                                  : pieces - 1 - atomicAdd(a.num_sorted + 2, 1);
          a.runs[at] = EmbeddingRun{int(piece), last, row};
        }
        if (open || next == row)
          store_vec<float, E, false, kWhole>(a.partial + (2 * piece + (open ? 0 : 1)) * a.dim + c, n, acc);
        else
          write_row<T, E, kWhole>(a, row, c, n, acc);
      }
#pragma unroll
      for (int k = 0; k < E; ++k) acc[k] = 0.0f;
      row = next;
      open = false;
    }
  }
}

template <typename T, bool kWhole>
__global__ __launch_bounds__(kThreads) void embedding_sum_kernel(EmbeddingBwdArgs a) {
  constexpr int E = kVec<T>;
  const int total = a.num_sorted[0];
  const int64_t chunks = ceil_div(a.dim, 64 * E), items = ceil_div(total, kPiece) * chunks;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  for (int64_t item = int64_t(blockIdx.x) * 4 + wave; item < items; item += int64_t(gridDim.x) * 4) {
    const int64_t piece = item / chunks;
    sum_piece<T, kWhole>(a, piece, ((item - piece * chunks) * 64 + lane) * E, total);
  }
}

// Sum of the partial sums of pieces q0 to q1 - 1 of a run that begins in `piece`, in order.
template <int E, bool kWhole>
__device__ __forceinline__ void sum_partials(const EmbeddingBwdArgs& a, int64_t piece, int64_t q0, int64_t q1,
                                             int64_t c, int n, float (&acc)[E]) {
  constexpr int kAhead = 64 / E;
  for (int64_t q = q0; q < q1; q += kAhead) {
    const float* from[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t p = q + j < q1 ? q + j : q1 - 1;
      from[j] = a.partial + (2 * p + (p == piece ? 1 : 0)) * a.dim;
    }
    Raw<float, E> r[kAhead];
    load_vecs<float, E, kAhead, false, kWhole>(r, from, c, n, a.dim >= E);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (q + j < q1) {
#pragma unroll
        for (int k = 0; k < E; ++k) acc[k] += r[j].get(k);
      }
  }
}

// Adds the partial sums of the runs that begin in a piece and end in a later one, 64 vectors of columns
// at a time.  Most runs are of a few pieces: a wave's task.  The others are shared by a workgroup's waves,
// an equal part of the run's pieces each, in order; the parts meet in LDS.  The time is a chain of waits
// (the count and a run, then its partial sums in turns), so all tasks have to run at once.
constexpr int kJoinWaves = 8;
constexpr int kJoinLongWgs = 32;
constexpr int kJoinShortWgs = 96;
template <typename T, bool kWhole>
__global__ __launch_bounds__(kJoinWaves * 64) void embedding_join_kernel(EmbeddingBwdArgs a) {
  constexpr int E = kVec<T>;
  __shared__ float part[kJoinWaves - 1][64 * E];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int pieces = int(ceil_div(a.tokens, kPiece));
  const int64_t step = int64_t(gridDim.y) * 64 * E;
  if (blockIdx.x >= kJoinLongWgs) {
    const int first = int(blockIdx.x - kJoinLongWgs) * kJoinWaves + wave;
    const int runs = a.num_sorted[1];
    for (int k = first; k < runs; k += kJoinShortWgs * kJoinWaves) {
      const EmbeddingRun run = a.runs[k];
      for (int64_t c0 = int64_t(blockIdx.y) * 64 * E; c0 < a.dim; c0 += step) {
        const int64_t c = c0 + lane * E;
        const int n = tail<E>(a.dim - c);
        float acc[E] = {};
        sum_partials<E, kWhole>(a, run.first, run.first, int64_t(run.last) + 1, c, n, acc);
        if (n > 0) write_row<T, E, kWhole>(a, run.row, c, n, acc);
      }
    }
    return;
  }
  const int runs = a.num_sorted[2];
  for (int k = blockIdx.x; k < runs; k += kJoinLongWgs) {
    const EmbeddingRun run = a.runs[pieces - 1 - k];
    const int64_t end = int64_t(run.last) + 1, share = ceil_div(end - run.first, kJoinWaves);
    const int64_t q0 = run.first + wave * share, q1 = q0 + share < end ? q0 + share : end;
    for (int64_t c0 = int64_t(blockIdx.y) * 64 * E; c0 < a.dim; c0 += step) {
      const int64_t c = c0 + lane * E;
      const int n = tail<E>(a.dim - c);
      float acc[E] = {};
      sum_partials<E, kWhole>(a, run.first, q0, q1, c, n, acc);
      __syncthreads();  // the last columns' parts are read
      if (wave > 0) {
#pragma unroll
        for (int j = 0; j < E; ++j) part[wave - 1][j * 64 + lane] = acc[j];
      }
      __syncthreads();
      if (wave == 0 && n > 0) {
#pragma unroll
        for (int w = 0; w < kJoinWaves - 1; ++w)
#pragma unroll
          for (int j = 0; j < E; ++j) acc[j] += part[w][j * 64 + lane];
        write_row<T, E, kWhole>(a, run.row, c, n, acc);
      }
    }
  }
}

// Few tokens (up to kMost): a workgroup for each, which looks at all ids, goes on if its own is the first of its row,
// and sums the row's tokens, in ascending order or in ascending quarters.
template <typename T, typename I, bool kWhole, int kMost>
__global__ __launch_bounds__(kThreads) void embedding_direct_kernel(EmbeddingBwdArgs a) {
  constexpr int E = kVec<T>, kAhead = 16, kMasks = kMost / 64;
  __shared__ uint64_t masks[kMasks];
  __shared__ int list[kMost];
  const I* __restrict__ ids = static_cast<const I*>(a.ids);
  const int tokens = int(a.tokens), lane = threadIdx.x & 63;
  const int64_t row = ids[blockIdx.x];
  if (uint64_t(row) >= uint64_t(a.vocab)) return;
  I id[kMost / kThreads];
#pragma unroll
  for (int j = 0; j < kMost / kThreads; ++j) {
    const int t = j * kThreads + threadIdx.x;
    id[j] = t < tokens ? ids[t] : I(-1);
  }
#pragma unroll
  for (int j = 0; j < kMost / kThreads; ++j) {
    const uint64_t same = __ballot(int64_t(id[j]) == row);
    if (lane == 0) masks[(j * kThreads + threadIdx.x) / 64] = same;
  }
  __syncthreads();
  int before[kMasks + 1] = {};
#pragma unroll
  for (int k = 0; k < kMasks; ++k) before[k + 1] = before[k] + __popcll(masks[k]);
  // this workgroup's token is the row's first one?
  const int first = blockIdx.x / 64;
#pragma unroll
  for (int k = 0; k < kMasks; ++k) {
    const uint64_t earlier = k < first ? ~uint64_t(0) : k == first ? (uint64_t(1) << (blockIdx.x & 63)) - 1 : 0;
    if ((masks[k] & earlier) != 0) return;
  }
#pragma unroll
  for (int j = 0; j < kMost / kThreads; ++j) {
    const int t = j * kThreads + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kMasks; ++k)
      if (t / 64 == k && ((masks[k] >> lane) & 1)) list[before[k] + __popcll(masks[k] & ((uint64_t(1) << lane) - 1))] = t;
  }
  __syncthreads();
  const int n = before[kMasks];
  // A wave takes 64 vectors of columns; all of its lanes go along, those beyond the last column too.  Rows
  // of no more than that are shared: each wave adds a quarter of the tokens.
  constexpr int kWaves = kThreads / 64;
  __shared__ float part[kWaves - 1][64 * E];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool shared = a.dim <= 64 * E;
  const int share = shared ? (n + kWaves - 1) / kWaves : n;
  const int t0 = shared ? wave * share : 0, t1 = t0 + share < n ? t0 + share : n;
  for (int64_t c0 = shared ? 0 : int64_t(wave) * 64 * E; c0 < a.dim; c0 += kThreads * E) {
    const int64_t c = c0 + lane * E;
    const int m = tail<E>(a.dim - c);
    float acc[E] = {};
    for (int i0 = t0; i0 < t1; i0 += kAhead) {
      const int token = list[i0 + lane < t1 ? i0 + lane : t1 - 1];
      const T* from[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        from[j] = static_cast<const T*>(a.dy) + int64_t(__builtin_amdgcn_readlane(token, j)) * a.dim;
      Raw<T, E> r[kAhead];
      load_vecs<T, E, kAhead, true, kWhole>(r, from, c, m, a.dim >= E);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j < t1) {
#pragma unroll
          for (int k = 0; k < E; ++k) acc[k] += r[j].get(k);
        }
    }
    if (shared) {  // one turn of the loop
      if (wave > 0) {
#pragma unroll
        for (int k = 0; k < E; ++k) part[wave - 1][k * 64 + lane] = acc[k];
      }
      __syncthreads();
      if (wave > 0) return;
#pragma unroll
      for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
        for (int k = 0; k < E; ++k) acc[k] += part[w][k * 64 + lane];
    }
    if (m > 0) write_row<T, E, kWhole>(a, int(row), c, m, acc);
  }
}
template <typename T>
__global__ __launch_bounds__(kThreads) void embedding_zero_kernel(T* table, int64_t n) {
  constexpr int E = kVec<T>;
  const float none[E] = {};
  for (int64_t e = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * E; e < n; e += int64_t(gridDim.x) * kThreads * E)
    store_vec<T, E, false, false>(table + e, tail<E>(n - e), none);
}

// Up to so many bytes the zeros are written beside the sort: 76 MB with 50021 tokens 84 us instead of 90 in
// a launch of its own, 156 MB with 8192 tokens 56 instead of 58.  Beyond, the shorter-lived workgroups of
// a launch of its own gain more: 500 MB 122 us instead of 127, 1 GB 202 instead of 214.
constexpr int64_t kZeroBesideSort = int64_t(256) << 20;

// Up to 1024 tokens are not sorted, 512 where rows are wide: 500 tokens of a text, 512 columns of bf16, 7 us
// instead of 20, 4096 columns 45 instead of 55; 1000 tokens 10 instead of 22, 4096 columns 57 and 57.  One
// workgroup sums all tokens of a row, so a long run of a wide row takes longer (500 of 4096 columns 85 us
// instead of 18).  How long runs are is known on the device only: tables so small that some row has more than
// 32 tokens are left to the sort, one frequent id in a larger table is not noticed.
inline bool sum_directly(int64_t tokens, int64_t vocab, int64_t vecs) {
  if (vecs <= 64) return tokens <= 1024;
  return tokens <= (vecs <= 256 ? 1024 : 512) && tokens <= 32 * vocab;
}

template <typename T, typename I, bool kWhole>
int gradient(const EmbeddingBwdArgs& a, hipStream_t s) {
  const int64_t elems = a.accumulate ? 0 : a.vocab * a.dim;
  const bool direct = sum_directly(a.tokens, a.vocab, ceil_div(a.dim, kVec<T>));
  const bool zero_first = direct || elems * int64_t(sizeof(T)) > kZeroBesideSort;
  int e = 0;
  if (zero_first && elems > 0)
    e = launch(embedding_zero_kernel<T>, grid_of(elems, kThreads * kVec<T>), kThreads, 0, s, static_cast<T*>(a.dtable),
               elems);
  if (e != 0) return e;
  if (direct) {
    if (a.tokens > 512)
      return launch(embedding_direct_kernel<T, I, kWhole, 1024>, unsigned(a.tokens), kThreads, 0, s, a);
    if (a.tokens > 0) return launch(embedding_direct_kernel<T, I, kWhole, 512>, unsigned(a.tokens), kThreads, 0, s, a);
    return e;
  }
  const int shift = sort_shift(a.vocab);
  const int64_t owners = int64_t(1) << shift, rows = ceil_div(a.vocab, owners);
  int bits = 0;
  while ((1 << bits) < rows) ++bits;
  const unsigned ranges = unsigned(a.vocab < owners ? a.vocab : owners);
  unsigned zeroing = zero_first || elems == 0 ? 0 : grid_of(elems, kSortThreads * kVec<T>);
  // workgroups do not go on to another range: tables of more than 2^30 rows take a second launch
  for (unsigned first = 0; first < ranges && e == 0; first += unsigned(kMaxGrid), zeroing = 0) {
    const unsigned sorting = ranges - first < kMaxGrid ? ranges - first : unsigned(kMaxGrid);
    e = launch(embedding_sort_kernel<T, I>, sorting + zeroing, kSortThreads, kSortWaves * rows * sizeof(int), s, a, first,
               sorting, ranges, shift, int(rows), bits);
  }
  if (e != 0) return e;
  const int64_t pieces = ceil_div(a.tokens, kPiece), chunks = ceil_div(ceil_div(a.dim, kVec<T>), 64);
  e = launch(embedding_sum_kernel<T, kWhole>, grid_of(pieces * chunks, 4), kThreads, 0, s, a);
  if (e != 0) return e;
  // how many runs there are is known on the device only
  return launch(embedding_join_kernel<T, kWhole>,
                dim3(kJoinLongWgs + kJoinShortWgs, unsigned(chunks < 64 ? chunks : 64)), kJoinWaves * 64, 0, s, a);
}
template <typename T, typename I>
int gradient(const EmbeddingBwdArgs& a, hipStream_t s) {
  return with_whole<kVec<T>>(a.dim, [&](auto w) { return gradient<T, I, decltype(w)::value>(a, s); });
}

// Two vectors a lane and up to four waves a row: 65536 rows of 4096 bf16 (20132 distinct of 131072) in
// 129 us, 5.4 TB/s of the bytes that have to move; four vectors 131, eight 134, one wave a row 140.  The
// output is written past the caches, which keep the table's frequent rows: with plain stores 142 us, and
// 18 us against 19 at 8192 rows, where it would fit.
template <typename T, typename I>
int lookup(int64_t tokens, const void* ids, int64_t vocab, int64_t dim, const void* table, float scale, void* out,
            hipStream_t s) {
  constexpr int NV = 2, NT = 4;
  const int64_t vecs = ceil_div(dim, kVec<T>);
  const auto* i = static_cast<const I*>(ids);
  const auto* w = static_cast<const T*>(table);
  auto* o = static_cast<T*>(out);
  return with_whole<kVec<T>>(dim, [&](auto wh) {
    constexpr bool whole = decltype(wh)::value;
    if (vecs < 64) {
      int lshift = 0;
      while ((1 << lshift) < vecs) ++lshift;
      const int64_t per = int64_t(kThreads >> lshift) * NT;
      return launch(embedding_narrow_kernel<T, I, NT, whole>, grid_of(tokens, per), kThreads, 0, s, tokens, i, vocab,
                    int(dim), w, scale, o, lshift);
    }
    const int wshift = vecs <= 64 * NV ? 0 : vecs <= 128 * NV ? 1 : 2;
    return launch(embedding_rows_kernel<T, I, NV, whole>, grid_of(tokens, 4 >> wshift), kThreads, 0, s, tokens, i, vocab,
                  dim, w, scale, o, wshift);
  });
}

}  // namespace

int launch_embedding(int64_t tokens, const void* ids, int ids_dtype, int64_t vocab, int64_t dim, const void* table,
                     int dtype, float scale, void* out, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const auto call = [&](auto f) { return f(tokens, ids, vocab, dim, table, scale, out, s); };
  if (dtype == TIDE_BF16) return call(ids_dtype == TIDE_INT32 ? lookup<bf16_t, int32_t> : lookup<bf16_t, int64_t>);
  return call(ids_dtype == TIDE_INT32 ? lookup<float, int32_t> : lookup<float, int64_t>);
}

int launch_embedding_bwd(const EmbeddingBwdArgs& a, int dtype, int ids_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == TIDE_BF16)
    return ids_dtype == TIDE_INT32 ? gradient<bf16_t, int32_t>(a, s) : gradient<bf16_t, int64_t>(a, s);
  return ids_dtype == TIDE_INT32 ? gradient<float, int32_t>(a, s) : gradient<float, int64_t>(a, s);
}

}  // namespace tide_step
