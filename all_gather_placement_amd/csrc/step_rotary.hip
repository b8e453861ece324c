// Rotary positions of several axes: pair i of a head is turned by a = positions[axis of i][t] * freqs[i],
//
//   (u, v) -> (u cos a - v sin a, v cos a + u sin a)
//
// HBM bounds it: every element is read and written once in 16-byte vectors.  A token's angles are the same
// for all of its heads, so a workgroup makes those of its tokens once, in LDS, and no table is read.
//
// A workgroup has one turn: all of a thread's loads, then the angles while they are in flight, then its stores.
// Loads and stores are counted together and in order, so a thread that went on to further vectors would wait
// for its stores with every load: 32760 x 40 x 128 bf16 took 343 us that way, and 108 now (6.2 TB/s).  Heads of
// few tokens or one head of many are bound by the angles, some 60 instructions each.
#include "step_device.h"
#include "step_grid.h"
#include "step_internal.h"

namespace tide_step {
namespace {

// Items of a thread: all of its loads are in flight before the angles are made, and none waits for a store.
template <bool kHalves>
constexpr int kItems = kHalves ? 2 : 4;
// A thread has fewer items where it would make more than four angles for them, which all wait for each other (100000
// tokens of one head of 64 bf16 13.0 us instead of 15.3), and where there would be few workgroups (512 tokens of 32
// heads of 128 3.7 us instead of 4.1).
template <typename T, bool kHalves>
constexpr int kAnglesOf = kHalves ? kVec<T> : kVec<T> / 2;  // of an item
constexpr int64_t kFewThreads = 512 * 256;
constexpr int kMaxThreads = 512;
static_assert(TIDE_ROTARY_MAX_DIM / 4 + 2 <= kMaxThreads, "a workgroup takes at least one head, whose parts may end in vectors");
constexpr int kAngleBytes = 32768;  // of LDS

// Quotients by a number that is known before the launch, of numbers below 2^31, by a product with its reciprocal rounded
// up (Granlund and Montgomery, "Division by invariant integers using multiplication", 1994).
struct Divisor {
  uint32_t d, factor, shift;
  explicit Divisor(uint32_t by) : d(by), factor(0), shift(0) {
    while ((uint64_t(1) << shift) < by) ++shift;
    factor = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - by)) / by + 1);
  }
  __device__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, factor) + n) >> shift; }
};

struct RotaryShape {
  int64_t first_token; // of the launch
  int32_t tokens;      // of a workgroup
  int32_t heads;       // of a workgroup
  int32_t padded;      // pairs of a token in LDS, whole vectors
  int32_t units;       // vectors (halves: pairs of vectors) of a head that are turned
  Divisor per_head;    // items of a head: turned and copied
  Divisor per_token;   // items of a token's heads
  Divisor pairs;
};

// cos and sin of an angle of up to 2^64, as their values rounded to fp32.  Whole turns are taken off the product with
// 1 / (2 pi) before it is rounded, and that factor has two parts: far positions keep their place within a turn to 2^-43.
// What is left of the angle beside whole quarters is at most pi / 4, where the series of sine and cosine up to the 11th
// and 12th power are within 2^-36.
__device__ __forceinline__ void turn(double angle, float* cos, float* sin) {
  constexpr double kTurn = 0.15915494309189533577, kTurnRest = -9.839338337591243e-18;  // 1 / (2 pi)
  double turns = fma(angle, kTurnRest, fma(angle, kTurn, -rint(angle * kTurn)));
  turns -= rint(turns);
  const double quarters = rint(4.0 * turns);
  const double x = fma(-0.25, quarters, turns) * 6.28318530717958647692, y = x * x;
  double s = fma(y, -1.0 / 39916800.0, 1.0 / 362880.0);
  s = fma(y, s, -1.0 / 5040.0);
  s = fma(y, s, 1.0 / 120.0);
  s = fma(y, s, -1.0 / 6.0);
  s = fma(x * y, s, x);
  double c = fma(y, 1.0 / 479001600.0, -1.0 / 3628800.0);
  c = fma(y, c, 1.0 / 40320.0);
  c = fma(y, c, -1.0 / 720.0);
  c = fma(y, c, 1.0 / 24.0);
  c = fma(y, c, -0.5);
  c = fma(y, c, 1.0);
  const int q = int(quarters);  // from -2 to 2
  const float fs = float(s), fc = float(c);
  const float u = q & 1 ? fs : fc, v = q & 1 ? fc : fs;
  *cos = (q + 1) & 2 ? -u : u;
  *sin = q & 2 ? -v : v;
}

// A pair turned.  Which products are rounded is written out: lanes whose vectors overlap turn the same pair as different
// elements of theirs, and have to write the same values.
__device__ __forceinline__ void turn_pair(float u, float v, float cos, float sin, float* first, float* second) {
  *first = fmaf(u, cos, -(v * sin));
  *second = fmaf(u, sin, v * cos);
}

// A vector, or the two vectors that are turned against each other.
template <typename T>
struct Item {
  uint32_t t, u;
  T* to;
  Raw<T, kVec<T>> first, second;
};

// Where a part of a head -- the turned elements, of halves each half; the others -- is no whole number of vectors, its
// last vector is the one that ends with it, and shares elements with the one before: both lanes turn them and write the
// same values.  In place, a lane must not read what another has turned: a workgroup has all of a head, and its loads
// are complete before its barrier, its stores behind it.
template <int E, bool kWhole>
__device__ __forceinline__ int vector_at(int c, int length) {
  return kWhole || c + E <= length ? c : length - E;
}
// The same for a part of less than a vector, its elements.
template <typename T, bool kTiny, bool kOnce>
__device__ __forceinline__ Raw<T, kVec<T>> load_part(const T* p, int length) {
  if (!kTiny || length >= kVec<T>) return load_whole<T, kVec<T>, kOnce>(p);
  return load_vec<T, kVec<T>, kOnce, false>(p, length, false);
}
template <typename T, bool kTiny, bool kOnce>
__device__ __forceinline__ void store_part(T* p, int length, const float (&f)[kVec<T>]) {
  store_vec<T, kVec<T>, kOnce, !kTiny>(p, kTiny ? length : kVec<T>, f);
}

// How the parts of a head end: with whole vectors, inside one, or before the first.
enum Ends { kWholeVectors, kInsideVectors, kTinyParts };

// kOnce: vectors are read past the caches.
template <typename T, typename P, bool kHalves, Ends kEnds, bool kOnce>
__global__ __launch_bounds__(kMaxThreads) void rotary_kernel(RotaryArgs a, RotaryShape g) {
  constexpr int E = kVec<T>, N = kItems<kHalves>;
  constexpr bool kWhole = kEnds == kWholeVectors, kTiny = kEnds == kTinyParts;
  extern __shared__ f32x4 lds[];
  float* cosines = reinterpret_cast<float*>(lds);  // [tokens][padded]
  float* sines = cosines + g.tokens * g.padded;
  const int64_t h0 = int64_t(blockIdx.y) * g.heads;
  const uint32_t heads = uint32_t(a.heads - h0 < g.heads ? a.heads - h0 : g.heads);
  const int turned = 2 * a.pairs, plain = a.dim - turned;
  const int64_t t0 = g.first_token + int64_t(blockIdx.x) * g.tokens;
  const uint32_t tokens = uint32_t(a.tokens - t0 < g.tokens ? a.tokens - t0 : g.tokens);
  Item<T> item[N];
  bool there[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t i = threadIdx.x + j * blockDim.x;
    const uint32_t t = g.per_token(i), rest = i - t * g.per_token.d, h = g.per_head(rest), u = rest - h * g.per_head.d;
    there[j] = t < tokens && h < heads;
    item[j].t = t;
    item[j].u = u;
    const T* from = static_cast<const T*>(a.x) + (t0 + t) * a.x_token + (h0 + h) * a.x_head;
    item[j].to = static_cast<T*>(a.out) + (t0 + t) * a.out_token + (h0 + h) * a.out_head;
    if (!there[j]) continue;
    if (int(u) >= g.units) {
      const int c = vector_at<E, kWhole || kTiny>((int(u) - g.units) * E, plain);
      item[j].first = load_part<T, kTiny, kOnce>(from + turned + c, kTiny ? plain - c : plain);
    } else if constexpr (kHalves) {
      const int c = vector_at<E, kWhole || kTiny>(int(u) * E, a.pairs);
      item[j].first = load_part<T, kTiny, kOnce>(from + c, kTiny ? a.pairs - c : a.pairs);
      item[j].second = load_part<T, kTiny, kOnce>(from + a.pairs + c, kTiny ? a.pairs - c : a.pairs);
    } else {
      const int c = vector_at<E, kWhole || kTiny>(int(u) * E, turned);
      item[j].first = load_part<T, kTiny, kOnce>(from + c, kTiny ? turned - c : turned);
    }
  }
  loads_first();
  for (uint32_t i = threadIdx.x; i < tokens * g.pairs.d; i += blockDim.x) {
    const uint32_t t = g.pairs(i), p = i - t * g.pairs.d;
    int axis = 0;
    while (int(p) >= a.ends[axis]) ++axis;
    const double at = double(static_cast<const P*>(a.positions)[axis * a.tokens + t0 + t]);
    float c, s;
    turn(at * a.freqs[p], &c, &s);
    cosines[t * g.padded + p] = c;
    sines[t * g.padded + p] = s * a.sign;
  }
  if constexpr (kEnds == kInsideVectors) {  // the loads are complete
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (there[j]) {
        item[j].first.forget();
        if constexpr (kHalves) item[j].second.forget();
      }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (!there[j]) continue;
    const int u = int(item[j].u);
    if (u >= g.units) {
      const int c = vector_at<E, kWhole || kTiny>((u - g.units) * E, plain);
      float f[E];
#pragma unroll
      for (int k = 0; k < E; ++k) f[k] = item[j].first.get(k);
      store_part<T, kTiny, kWhole>(item[j].to + turned + c, plain - c, f);
      continue;
    }
    constexpr int A = kAnglesOf<T, kHalves>;
    typedef float Angles __attribute__((ext_vector_type(A), aligned(kWhole ? 4 * A : 4)));
    const int p = vector_at<A, kWhole || kTiny>(u * A, a.pairs);
    const Angles c = *reinterpret_cast<const Angles*>(cosines + item[j].t * g.padded + p);
    const Angles s = *reinterpret_cast<const Angles*>(sines + item[j].t * g.padded + p);
    if constexpr (kHalves) {
      float f[E], f2[E];
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float x = item[j].first.get(k), y = item[j].second.get(k);
        turn_pair(x, y, c[k], s[k], &f[k], &f2[k]);
      }
      store_part<T, kTiny, kWhole>(item[j].to + p, a.pairs - p, f);
      store_part<T, kTiny, kWhole>(item[j].to + a.pairs + p, a.pairs - p, f2);
    } else {
      float f[E];
#pragma unroll
      for (int k = 0; k < A; ++k) {
        const float x = item[j].first.get(2 * k), y = item[j].first.get(2 * k + 1);
        turn_pair(x, y, c[k], s[k], &f[2 * k], &f[2 * k + 1]);
      }
      store_part<T, kTiny, kWhole>(item[j].to + 2 * p, turned - 2 * p, f);
    }
  }
}

template <typename T, typename P, bool kHalves, Ends kEnds, bool kOnce>
int rotary(const RotaryArgs& a, hipStream_t s) {
  constexpr int E = kVec<T>, N = kItems<kHalves>;
  const int units = int(kHalves ? ceil_div(a.pairs, E) : ceil_div(2 * a.pairs, E));
  const int copied = a.x == a.out ? 0 : int(ceil_div(a.dim - 2 * a.pairs, E));
  const int padded = int(ceil_div(a.pairs, E) * E);
  // heads of a workgroup, then its tokens: as many as give each of its threads its items
  const int64_t most = int64_t(kMaxThreads) * N, per_head = units + copied;
  int64_t heads = most / per_head < a.heads ? most / per_head : a.heads;
  heads = ceil_div(a.heads, ceil_div(a.heads, heads));
  int64_t per_thread = N;
  while (per_thread > 1 && (per_thread * kAnglesOf<T, kHalves> > 4 * heads ||
                            a.tokens * a.heads * per_head < kFewThreads * per_thread))
    per_thread /= 2;
  int64_t tokens = 256 * per_thread / (heads * per_head);
  const int64_t fit = kAngleBytes / (padded * 8);
  if (tokens > fit) tokens = fit;
  if (tokens > a.tokens) tokens = a.tokens;
  if (tokens < 1) tokens = 1;
  RotaryShape g{0, int32_t(tokens), int32_t(heads), padded, units, Divisor(uint32_t(per_head)),
                      Divisor(uint32_t(heads * per_head)), Divisor(uint32_t(a.pairs))};
  int64_t threads = ceil_div(ceil_div(tokens * heads * per_head, per_thread), 64) * 64;
  if (threads > kMaxThreads) threads = kMaxThreads;
  // workgroups have one turn: more tokens than a launch holds take another
  int e = 0;
  for (; g.first_token < a.tokens && e == 0; g.first_token += kMaxGrid * tokens)
    e = launch(rotary_kernel<T, P, kHalves, kEnds, kOnce>,
               dim3(grid_of(a.tokens - g.first_token, tokens), unsigned(ceil_div(a.heads, heads))), int(threads),
               size_t(tokens) * padded * 8, s, a, g);
  return e;
}
// More than the last-level cache holds, read and written, is read past it: 32760 x 40 x 128 bf16 108 us instead of
// 112, a seventh of that 17.5 instead of 16.2.  Loads of vectors that end inside others' cache lines need the caches
// (50000 x 8 x 100 with 64 turned 34 us, past them 43).
constexpr int64_t kPastCaches = int64_t(256) << 20;

template <typename T, typename P, bool kHalves>
int rotary(const RotaryArgs& a, hipStream_t s) {
  constexpr int E = kVec<T>;
  const int part = kHalves ? a.pairs : 2 * a.pairs, plain = a.x == a.out ? 0 : a.dim - 2 * a.pairs;
  if (part < E || (plain > 0 && plain < E)) return rotary<T, P, kHalves, kTinyParts, false>(a, s);
  if (part % E != 0 || plain % E != 0) return rotary<T, P, kHalves, kInsideVectors, false>(a, s);
  const bool once = 2 * a.tokens * a.heads * a.dim * int64_t(sizeof(T)) > kPastCaches;
  return once ? rotary<T, P, kHalves, kWholeVectors, true>(a, s) : rotary<T, P, kHalves, kWholeVectors, false>(a, s);
}
template <typename T, typename P>
int rotary(const RotaryArgs& a, int pairing, hipStream_t s) {
  return pairing == TIDE_ROTARY_HALVES ? rotary<T, P, true>(a, s) : rotary<T, P, false>(a, s);
}
template <typename T>
int rotary(const RotaryArgs& a, int positions_dtype, int pairing, hipStream_t s) {
  if (positions_dtype == TIDE_INT32) return rotary<T, int32_t>(a, pairing, s);
  if (positions_dtype == TIDE_INT64) return rotary<T, int64_t>(a, pairing, s);
  return rotary<T, float>(a, pairing, s);
}

}  // namespace

int launch_rotary(const RotaryArgs& a, int dtype, int positions_dtype, int pairing, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == TIDE_BF16 ? rotary<bf16_t>(a, positions_dtype, pairing, s)
                            : rotary<float>(a, positions_dtype, pairing, s);
}

}  // namespace tide_step
