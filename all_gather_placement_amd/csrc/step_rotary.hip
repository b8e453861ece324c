// Rotary positions of several axes: pair i of a head is turned by a = positions[axis of i][t] * freqs[i],
//
//   (u, v) -> (u cos a - v sin a, v cos a + u sin a)
//
// HBM bounds it: every element is read and written once in 16-byte vectors.  A token's angles are the same
// for all of its heads, so a workgroup makes those of its tokens once, in LDS, and no table is read.
#include "step_device.h"
#include "step_grid.h"
#include "step_internal.h"

namespace tide_step {
namespace {

constexpr int kThreads = 256;
constexpr int kAngleBytes = 32768;  // of LDS

// Quotients by a number that is known before the launch, of numbers below 2^31.
struct Divisor {
  uint32_t d, factor, shift;
  explicit Divisor(uint32_t by) : d(by), factor(0), shift(0) {
    while ((uint64_t(1) << shift) < by) ++shift;
    factor = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - by)) / by + 1);
  }
  __device__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, factor) + n) >> shift; }
};

struct RotaryShape {
  int32_t tokens;      // of a workgroup at a time
  int32_t heads;       // of a workgroup
  int32_t padded;      // pairs of a token in LDS, whole vectors
  int32_t units;       // vectors (halves: pairs of vectors) of a head that are turned
  Divisor per_head;    // items of a head: turned and copied
  Divisor per_token;   // items of a token's heads
  Divisor pairs;
};

// cos and sin of an angle, as their values rounded to fp32.  In 64 bits, far positions keep their place within a
// turn; what is left of the angle beside whole quarters is at most pi / 4, where the series of sine and cosine up
// to the 11th and 12th power are within 2^-36.
__device__ __forceinline__ void turn(double angle, float* cos, float* sin) {
  double turns = angle * 0.15915494309189533577;  // 1 / (2 pi)
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

template <typename T, typename P, bool kHalves>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, RotaryShape g) {
  constexpr int E = kVec<T>;
  extern __shared__ float angles[];  // cos [tokens][padded], then sin
  float* sines = angles + g.tokens * g.padded;
  const T* x = static_cast<const T*>(a.x);
  T* out = static_cast<T*>(a.out);
  const int64_t h0 = int64_t(blockIdx.y) * g.heads;
  const int heads = int(a.heads - h0 < g.heads ? a.heads - h0 : g.heads);
  for (int64_t t0 = int64_t(blockIdx.x) * g.tokens; t0 < a.tokens; t0 += int64_t(gridDim.x) * g.tokens) {
    const int tokens = int(a.tokens - t0 < g.tokens ? a.tokens - t0 : g.tokens);
    for (uint32_t i = threadIdx.x; i < uint32_t(tokens) * g.pairs.d; i += kThreads) {
      const uint32_t t = g.pairs(i), p = i - t * g.pairs.d;
      int axis = 0;
      while (int(p) >= a.ends[axis]) ++axis;
      const double at = double(static_cast<const P*>(a.positions)[axis * a.tokens + t0 + t]);
      float c, s;
      turn(at * a.freqs[p], &c, &s);
      angles[t * g.padded + p] = c;
      sines[t * g.padded + p] = s * a.sign;
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < uint32_t(tokens) * g.per_token.d; i += kThreads) {
      const uint32_t t = g.per_token(i), rest = i - t * g.per_token.d, h = g.per_head(rest), u = rest - h * g.per_head.d;
      if (int(h) >= heads) continue;
      const T* from = x + (t0 + t) * a.x_token + (h0 + h) * a.x_head;
      T* to = out + (t0 + t) * a.out_token + (h0 + h) * a.out_head;
      if (int(u) >= g.units) {  // columns that are not turned
        const int c = 2 * a.pairs + (int(u) - g.units) * E, n = tail<E>(a.dim - c);
        const Raw<T, E> v = load_vec<T, E, true, false>(from + c, n, a.dim - 2 * a.pairs >= E);
        float f[E];
  #pragma unroll
        for (int k = 0; k < E; ++k) f[k] = v.get(k);
        store_vec<T, E, true, false>(to + c, n, f);
        continue;
      }
      if constexpr (kHalves) {
        const int p = u * E, n = tail<E>(a.pairs - p);
        const float* c = angles + t * g.padded + p;
        const float* s = sines + t * g.padded + p;
        const Raw<T, E> first = load_vec<T, E, true, false>(from + p, n, a.pairs >= E);
        const Raw<T, E> second = load_vec<T, E, true, false>(from + a.pairs + p, n, a.pairs >= E);
        float f[E], f2[E];
  #pragma unroll
        for (int k = 0; k < E; ++k) {
          f[k] = first.get(k) * c[k] - second.get(k) * s[k];
          f2[k] = second.get(k) * c[k] + first.get(k) * s[k];
        }
        store_vec<T, E, true, false>(to + p, n, f);
        store_vec<T, E, true, false>(to + a.pairs + p, n, f2);
      } else {
        const int p = u * (E / 2), n = tail<E>(2 * (a.pairs - p));
        const float* c = angles + t * g.padded + p;
        const float* s = sines + t * g.padded + p;
        const Raw<T, E> v = load_vec<T, E, true, false>(from + 2 * p, n, 2 * a.pairs >= E);
        float f[E];
  #pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          f[2 * k] = v.get(2 * k) * c[k] - v.get(2 * k + 1) * s[k];
          f[2 * k + 1] = v.get(2 * k + 1) * c[k] + v.get(2 * k) * s[k];
        }
        store_vec<T, E, true, false>(to + 2 * p, n, f);
      }
    }
    __syncthreads();  // the angles are used until here
  }
}

template <typename T, typename P>
int rotary(const RotaryArgs& a, int pairing, hipStream_t s) {
  constexpr int E = kVec<T>;
  const bool halves = pairing == TIDE_ROTARY_HALVES, in_place = a.x == a.out;
  const int units = int(halves ? ceil_div(a.pairs, E) : ceil_div(2 * a.pairs, E));
  const int copied = in_place ? 0 : int(ceil_div(a.dim - 2 * a.pairs, E));
  const int padded = int(ceil_div(a.pairs, E) * E);
  constexpr int64_t kMaxHeadParts = 65535;
  const int64_t heads = ceil_div(a.heads, kMaxHeadParts), items = heads * (units + copied);
  // items of about four a thread; the angles of so many tokens fit LDS
  int64_t tokens = ceil_div(4 * kThreads, items);
  const int64_t fit = kAngleBytes / (padded * 8);
  if (tokens > fit) tokens = fit;
  if (tokens > a.tokens) tokens = a.tokens;
  const RotaryShape g{int32_t(tokens), int32_t(heads), padded, units, Divisor(uint32_t(units + copied)), Divisor(uint32_t(items)),
                      Divisor(uint32_t(a.pairs))};
  const dim3 grid(grid_of(a.tokens, tokens), unsigned(ceil_div(a.heads, heads)));
  const size_t lds = size_t(tokens) * padded * 8;
  return halves ? launch(rotary_kernel<T, P, true>, grid, kThreads, lds, s, a, g)
                : launch(rotary_kernel<T, P, false>, grid, kThreads, lds, s, a, g);
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
