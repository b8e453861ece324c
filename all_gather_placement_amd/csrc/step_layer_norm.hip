// Layer norm and its gradient.
//
//   mean = sum(x)/D, var = sum((x-mean)^2)/D, rstd = 1/sqrt(var+eps), y = (x-mean)*rstd*w + b
//   xhat = (x-mean)*rstd, g = dy*w, dx = rstd*(g - sum(g)/D - xhat*sum(g*xhat)/D)
//   dw = sum over rows dy*xhat, db = sum over rows dy
//
// HBM bounds both directions: a row is read once into registers, where the mean and then the
// centred squares are summed in fp32 (two passes over registers, so a large mean costs no digits),
// and written once.  A lane holds 16-byte vectors; a row belongs to a part of a wave, to a wave or to
// the waves of a workgroup.  Rows too wide for the registers are streamed instead, and read again from
// the caches.
//
// The parameter gradients are sums down the columns: each workgroup keeps the sums of its rows in
// registers, in row order, and leaves them in the workspace; a second kernel adds the workgroups'
// sums in a fixed order.
//
// Measured: 32760 x 5120 bf16 forward 114 us (5.9 TB/s; a copy of the same bytes takes 109), 8192 x 8192
// bf16 backward 72 us and 6 of the second kernel (437 MB move in the first, 6.1 TB/s).
#include "step_device.h"
#include "step_internal.h"

namespace tide_step {
namespace {

constexpr int kMaxWaves = 16;

template <int E>
__device__ __forceinline__ int tail(int64_t n) {
  return int(n < E ? n : E);
}
__host__ __device__ constexpr int64_t padded(int64_t cols) { return layer_norm_bwd_padded(cols); }

// K sums over the workgroup, each the same in every thread, with one barrier.  `lds` has to be another
// one at the next call.  A lane holds one wave's part of one sum, so a wave joins four sums at a time.
template <int K>
__device__ __forceinline__ void block_sums(float (&v)[K], float (&lds)[K * kMaxWaves]) {
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lanes_sum<64>(v[k]);
  if (waves == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) lds[k * kMaxWaves + wave] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; k += 4) {
    const int at = k * kMaxWaves + lane;
    float t = at < K * kMaxWaves && (lane & 15) < waves ? lds[at] : 0.0f;
    t = lanes_sum<16>(t);
#pragma unroll
    for (int j = 0; j < 4 && k + j < K; ++j)
      v[k + j] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(t), 16 * j));
  }
}
__device__ __forceinline__ float block_sum(float v, float (&lds)[kMaxWaves]) {
  float s[1] = {v};
  block_sums<1>(s, lds);
  return s[0];
}

// ---------------------------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------------------------

template <typename T, typename PT, bool kWhole>
struct Affine {
  static constexpr int E = kVec<T>;
  Raw<PT, E> w, b;
  __device__ __forceinline__ void load(const LayerNormArgs& a, int c, int n) {
    const bool wide = a.cols >= E;
    if (a.weight != nullptr) w = load_vec<PT, E, false, kWhole>(static_cast<const PT*>(a.weight) + c, n, wide);
    if (a.bias != nullptr) b = load_vec<PT, E, false, kWhole>(static_cast<const PT*>(a.bias) + c, n, wide);
  }
  template <bool kOnce>
  __device__ __forceinline__ void store(const LayerNormArgs& a, T* y, int n, const Raw<T, E>& r, float mean,
                                        float rstd) const {
    float o[E];
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float xhat = (r.get(k) - mean) * rstd;
      o[k] = (a.weight != nullptr ? xhat * w.get(k) : xhat) + (a.bias != nullptr ? b.get(k) : 0.0f);
    }
    store_vec<T, E, kOnce, kWhole>(y, n, o);
  }
};

// Narrow rows: a group of L lanes for each, one vector a lane.
constexpr int kNarrowThreads = 256;

template <typename T, typename PT, int L, bool kOnce, bool kWhole>
__global__ __launch_bounds__(kNarrowThreads) void layer_norm_narrow_kernel(LayerNormArgs a) {
  constexpr int E = kVec<T>, kGroups = kNarrowThreads / L;
  const int D = int(a.cols), c = (threadIdx.x % L) * E, n = D - c;
  const float inv = 1.0f / float(D);
  Affine<T, PT, kWhole> affine;
  affine.load(a, c, n);
  for (int64_t row = int64_t(blockIdx.x) * kGroups + threadIdx.x / L; row < a.rows;
       row += int64_t(gridDim.x) * kGroups) {
    const Raw<T, E> r = load_vec<T, E, kOnce, kWhole>(static_cast<const T*>(a.x) + row * a.x_stride + c, n, D >= E);
    float sum = 0;
#pragma unroll
    for (int k = 0; k < E; ++k) sum += r.get(k);
    const float mean = lanes_sum<L>(sum) * inv;
    float sq = 0;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float d = r.get(k) - mean;
      sq += k < n ? d * d : 0.0f;
    }
    const float rstd = 1.0f / sqrtf(lanes_sum<L>(sq) * inv + a.eps);
    if (c == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    affine.template store<kOnce>(a, static_cast<T*>(a.y) + row * a.y_stride + c, n, r, mean, rstd);
  }
}

// Rows of up to kMaxWaves * 64 * NV vectors: a workgroup holds RB rows at a time in registers, NV
// vectors of each in a lane, and joins the waves' sums of all of them at one barrier.
template <typename T, typename PT, int NV, int RB, bool kOnce, bool kWhole>
__global__ __launch_bounds__(kMaxWaves * 64) void layer_norm_rows_kernel(LayerNormArgs a) {
  constexpr int E = kVec<T>;
  __shared__ float lds[2][RB * kMaxWaves];
  const int D = int(a.cols);
  const float inv = 1.0f / float(D);
  for (int64_t row0 = int64_t(blockIdx.x) * RB; row0 < a.rows; row0 += int64_t(gridDim.x) * RB) {
    Raw<T, E> r[RB][NV];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const T* x = static_cast<const T*>(a.x) + (row0 + i) * a.x_stride;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * int(blockDim.x) + int(threadIdx.x)) * E;
        r[i][v] = load_vec<T, E, kOnce, kWhole>(x + c, row0 + i < a.rows ? D - c : 0, true);
      }
    }
    Affine<T, PT, kWhole> affine[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * int(blockDim.x) + int(threadIdx.x)) * E;
      affine[v].load(a, c, D - c);
    }
    float mean[RB], rstd[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      mean[i] = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int k = 0; k < E; ++k) mean[i] += r[i][v].get(k);
        r[i][v].forget();
      }
    }
    block_sums<RB>(mean, lds[0]);
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      mean[i] *= inv;
      rstd[i] = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int n = D - (v * int(blockDim.x) + int(threadIdx.x)) * E;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float d = r[i][v].get(k) - mean[i];
          rstd[i] += k < n ? d * d : 0.0f;
        }
        r[i][v].forget();
      }
    }
    block_sums<RB>(rstd, lds[1]);
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      if (row0 + i >= a.rows) break;
      rstd[i] = 1.0f / sqrtf(rstd[i] * inv + a.eps);
      if (threadIdx.x == 0) {
        if (a.mean != nullptr) a.mean[row0 + i] = mean[i];
        if (a.rstd != nullptr) a.rstd[row0 + i] = rstd[i];
      }
      T* y = static_cast<T*>(a.y) + (row0 + i) * a.y_stride;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * int(blockDim.x) + int(threadIdx.x)) * E;
        if (c < D) affine[v].template store<kOnce>(a, y + c, D - c, r[i][v], mean[i], rstd[i]);
      }
    }
  }
}

// Rows wider than the registers: three passes over the row, the later ones from the caches (4096 x 40960
// bf16 196 us, 3.4 TB/s of the bytes that have to move; rows in registers reach 5.9).
constexpr int kWideThreads = 1024;

template <typename T, typename PT>
__global__ __launch_bounds__(kWideThreads) void layer_norm_wide_kernel(LayerNormArgs a) {
  __shared__ float lds[2][16];
  constexpr int E = kVec<T>;
  const int64_t D = a.cols;
  const float inv = 1.0f / float(D);
  const PT* w = static_cast<const PT*>(a.weight);
  const PT* b = static_cast<const PT*>(a.bias);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    T* y = static_cast<T*>(a.y) + row * a.y_stride;
    float sum = 0;
    for (int64_t c = int64_t(threadIdx.x) * E; c < D; c += kWideThreads * E) {
      const Raw<T, E> r = load_vec<T, E, false, false>(x + c, tail<E>(D - c), true);
#pragma unroll
      for (int k = 0; k < E; ++k) sum += r.get(k);
    }
    const float mean = block_sum(sum, lds[0]) * inv;
    float sq = 0;
    for (int64_t c = int64_t(threadIdx.x) * E; c < D; c += kWideThreads * E) {
      const int n = tail<E>(D - c);
      const Raw<T, E> r = load_vec<T, E, false, false>(x + c, n, true);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float d = r.get(k) - mean;
        sq += k < n ? d * d : 0.0f;
      }
    }
    const float var = block_sum(sq, lds[1]) * inv;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    for (int64_t c = int64_t(threadIdx.x) * E; c < D; c += kWideThreads * E) {
      const int n = tail<E>(D - c);
      const Raw<T, E> r = load_vec<T, E, false, false>(x + c, n, true);
      Raw<PT, E> rw, rb;
      if (w != nullptr) rw = load_vec<PT, E, false, false>(w + c, n, true);
      if (b != nullptr) rb = load_vec<PT, E, false, false>(b + c, n, true);
      float o[E];
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float xhat = (r.get(k) - mean) * rstd;
        o[k] = (w != nullptr ? xhat * rw.get(k) : xhat) + (b != nullptr ? rb.get(k) : 0.0f);
      }
      store_vec<T, E, false, false>(y + c, n, o);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------------------------

// Narrow rows: as the forward kernel; the groups' sums over their rows meet in LDS, in order.
template <typename T, typename PT, int L, bool kOnce, bool kWhole>
__global__ __launch_bounds__(kNarrowThreads) void layer_norm_bwd_narrow_kernel(LayerNormBwdArgs a) {
  constexpr int E = kVec<T>, kGroups = kNarrowThreads / L;
  __shared__ float join[kNarrowThreads * E];
  const int D = int(a.cols), c = (threadIdx.x % L) * E, n = D - c;
  const float inv = 1.0f / float(D);
  Raw<PT, E> rw;
  if (a.weight != nullptr) rw = load_vec<PT, E, false, kWhole>(static_cast<const PT*>(a.weight) + c, n, D >= E);
  float dw[E] = {}, db[E] = {};
  for (int64_t row = int64_t(blockIdx.x) * kGroups + threadIdx.x / L; row < a.rows;
       row += int64_t(gridDim.x) * kGroups) {
    const Raw<T, E> rx = load_vec<T, E, kOnce, kWhole>(static_cast<const T*>(a.x) + row * a.x_stride + c, n, D >= E);
    const Raw<T, E> rd = load_vec<T, E, kOnce, kWhole>(static_cast<const T*>(a.dy) + row * a.dy_stride + c, n, D >= E);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0, s2 = 0;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float xhat = k < n ? (rx.get(k) - mean) * rstd : 0.0f;
      const float d = rd.get(k);
      const float g = a.weight != nullptr ? d * rw.get(k) : d;
      s1 += g;
      s2 += g * xhat;
      dw[k] += d * xhat;
      db[k] += d;
    }
    if (a.dx == nullptr) continue;
    s1 = lanes_sum<L>(s1) * inv;
    s2 = lanes_sum<L>(s2) * inv;
    if (n <= 0) continue;
    float o[E];
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float xhat = (rx.get(k) - mean) * rstd;
      const float g = a.weight != nullptr ? rd.get(k) * rw.get(k) : rd.get(k);
      o[k] = rstd * (g - s1 - xhat * s2);
    }
    store_vec<T, E, kOnce, kWhole>(static_cast<T*>(a.dx) + row * a.dx_stride + c, n, o);
  }
  if (a.partial == nullptr) return;
  float* part = a.partial + int64_t(blockIdx.x) * 2 * padded(D);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < E; ++k) join[threadIdx.x * E + k] = s == 0 ? dw[k] : db[k];
    __syncthreads();
    for (int i = threadIdx.x; i < L * E && i < D; i += kNarrowThreads) {
      float t = 0;
      for (int g = 0; g < kGroups; ++g) t += join[g * L * E + i];
      part[s * padded(D) + i] = t;
    }
  }
}

// Rows of up to kMaxWaves * 64 * NV vectors: RB rows at a time, as the forward kernel; the sums down
// the columns stay in registers from the workgroup's first row to its last.
template <typename T, typename PT, int NV, int RB, bool kOnce, bool kWhole>
__global__ __launch_bounds__(kMaxWaves * 64) void layer_norm_bwd_rows_kernel(LayerNormBwdArgs a) {
  constexpr int E = kVec<T>;
  __shared__ float lds[2][2 * RB * kMaxWaves];
  const int D = int(a.cols);
  const float inv = 1.0f / float(D);
  Raw<PT, E> rw[NV];
  float dw[NV][E], db[NV][E];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * int(blockDim.x) + int(threadIdx.x)) * E;
    if (a.weight != nullptr) rw[v] = load_vec<PT, E, false, kWhole>(static_cast<const PT*>(a.weight) + c, D - c, true);
#pragma unroll
    for (int k = 0; k < E; ++k) dw[v][k] = db[v][k] = 0.0f;
  }
  int parity = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RB; row0 < a.rows; row0 += int64_t(gridDim.x) * RB, parity ^= 1) {
    Raw<T, E> rx[RB][NV], rd[RB][NV];
    float mean[RB], rstd[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int64_t row = row0 + i;
      const bool in = row < a.rows;
      const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
      const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
      mean[i] = in ? a.mean[row] : 0.0f;
      rstd[i] = in ? a.rstd[row] : 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * int(blockDim.x) + int(threadIdx.x)) * E;
        rx[i][v] = load_vec<T, E, kOnce, kWhole>(x + c, in ? D - c : 0, true);
        rd[i][v] = load_vec<T, E, kOnce, kWhole>(dy + c, in ? D - c : 0, true);
      }
    }
    float s[2 * RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      s[2 * i] = s[2 * i + 1] = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int n = D - (v * int(blockDim.x) + int(threadIdx.x)) * E;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float xhat = k < n ? (rx[i][v].get(k) - mean[i]) * rstd[i] : 0.0f;
          const float d = rd[i][v].get(k);
          const float g = a.weight != nullptr ? d * rw[v].get(k) : d;
          s[2 * i] += g;
          s[2 * i + 1] += g * xhat;
          dw[v][k] += d * xhat;
          db[v][k] += d;
        }
        rx[i][v].forget();
        rd[i][v].forget();
      }
    }
    if (a.dx == nullptr) continue;
    block_sums<2 * RB>(s, lds[parity]);
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      if (row0 + i >= a.rows) break;
      const float m1 = s[2 * i] * inv, m2 = s[2 * i + 1] * inv;
      T* dx = static_cast<T*>(a.dx) + (row0 + i) * a.dx_stride;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * int(blockDim.x) + int(threadIdx.x)) * E, n = D - c;
        if (n <= 0) continue;
        float o[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float xhat = (rx[i][v].get(k) - mean[i]) * rstd[i];
          const float d = rd[i][v].get(k);
          const float g = a.weight != nullptr ? d * rw[v].get(k) : d;
          o[k] = rstd[i] * (g - m1 - xhat * m2);
        }
        store_vec<T, E, kOnce, kWhole>(dx + c, n, o);
      }
    }
  }
  if (a.partial == nullptr) return;
  float* part = a.partial + int64_t(blockIdx.x) * 2 * padded(D);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * int(blockDim.x) + int(threadIdx.x)) * E, n = D - c;
    if (n <= 0) continue;
    store_vec<float, E, false, kWhole>(part + c, n, dw[v]);
    store_vec<float, E, false, kWhole>(part + padded(D) + c, n, db[v]);
  }
}

// Few rows: one launch without partial sums.  Workgroups below `row_wgs` make a row of dx each; the
// others read all rows of 64 vectors of columns again, four waves every fourth row, and write the
// parameters' gradients.
constexpr int kColWaves = 4;
template <typename T, typename PT, int NV, bool kWhole>
__global__ __launch_bounds__(kMaxWaves * 64) void layer_norm_bwd_few_kernel(LayerNormBwdArgs a, unsigned row_wgs) {
  constexpr int E = kVec<T>;
  const int D = int(a.cols), wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (blockIdx.x < row_wgs) {
    __shared__ float lds[2 * kMaxWaves];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const float mean = a.mean[row], rstd = a.rstd[row], inv = 1.0f / float(D);
    Raw<T, E> rx[NV], rd[NV];
    Raw<PT, E> rw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * int(blockDim.x) + int(threadIdx.x)) * E;
      rx[v] = load_vec<T, E, false, kWhole>(x + c, D - c, D >= E);
      rd[v] = load_vec<T, E, false, kWhole>(dy + c, D - c, D >= E);
      if (a.weight != nullptr) rw[v] = load_vec<PT, E, false, kWhole>(static_cast<const PT*>(a.weight) + c, D - c, D >= E);
    }
    float s[2] = {0, 0};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int n = D - (v * int(blockDim.x) + int(threadIdx.x)) * E;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float xhat = k < n ? (rx[v].get(k) - mean) * rstd : 0.0f;
        const float g = a.weight != nullptr ? rd[v].get(k) * rw[v].get(k) : rd[v].get(k);
        s[0] += g;
        s[1] += g * xhat;
      }
    }
    block_sums<2>(s, lds);
    const float m1 = s[0] * inv, m2 = s[1] * inv;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * int(blockDim.x) + int(threadIdx.x)) * E, n = D - c;
      if (n <= 0) continue;
      float o[E];
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float xhat = (rx[v].get(k) - mean) * rstd;
        const float g = a.weight != nullptr ? rd[v].get(k) * rw[v].get(k) : rd[v].get(k);
        o[k] = rstd * (g - m1 - xhat * m2);
      }
      store_vec<T, E, false, kWhole>(static_cast<T*>(a.dx) + row * a.dx_stride + c, n, o);
    }
    return;
  }
  constexpr int kAhead = 8;
  __shared__ float part[kColWaves - 1][2 * 64 * E];
  const int waves = int(blockDim.x >> 6) < kColWaves ? int(blockDim.x >> 6) : kColWaves;
  const int c = (int(blockIdx.x - row_wgs) * 64 + lane) * E, n = D - c, rows = int(a.rows);
  float dw[E] = {}, db[E] = {};
  if (wave < waves) {
    for (int r0 = wave; r0 < rows; r0 += waves * kAhead) {
      Raw<T, E> rx[kAhead], rd[kAhead];
      float mean[kAhead], rstd[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t row = r0 + j * waves < rows ? r0 + j * waves : rows - 1;
        rx[j] = load_vec<T, E, false, kWhole>(static_cast<const T*>(a.x) + row * a.x_stride + c, n, D >= E);
        rd[j] = load_vec<T, E, false, kWhole>(static_cast<const T*>(a.dy) + row * a.dy_stride + c, n, D >= E);
        mean[j] = a.mean[row];
        rstd[j] = a.rstd[row];
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (r0 + j * waves >= rows) break;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          dw[k] += rd[j].get(k) * ((rx[j].get(k) - mean[j]) * rstd[j]);
          db[k] += rd[j].get(k);
        }
      }
    }
    if (wave > 0) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        part[wave - 1][k * 64 + lane] = dw[k];
        part[wave - 1][(E + k) * 64 + lane] = db[k];
      }
    }
  }
  __syncthreads();
  if (wave > 0) return;
  for (int w = 1; w < waves; ++w) {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      dw[k] += part[w - 1][k * 64 + lane];
      db[k] += part[w - 1][(E + k) * 64 + lane];
    }
  }
#pragma unroll
  for (int k = 0; k < E; ++k) {
    if (k < n && a.dweight != nullptr) static_cast<PT*>(a.dweight)[c + k] = narrow<PT>(dw[k]);
    if (k < n && a.dbias != nullptr) static_cast<PT*>(a.dbias)[c + k] = narrow<PT>(db[k]);
  }
}

// Rows wider than the registers: the input's gradient, two passes over a row (4096 x 40960 bf16 370 us with
// the sums below, a third pass; 2.7 TB/s of the bytes that have to move).
template <typename T, typename PT>
__global__ __launch_bounds__(kWideThreads) void layer_norm_bwd_wide_kernel(LayerNormBwdArgs a) {
  __shared__ float lds[2][2][16];
  constexpr int E = kVec<T>;
  const int64_t D = a.cols;
  const float inv = 1.0f / float(D);
  const PT* w = static_cast<const PT*>(a.weight);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0, s2 = 0;
    for (int64_t c = int64_t(threadIdx.x) * E; c < D; c += kWideThreads * E) {
      const int n = tail<E>(D - c);
      const Raw<T, E> rx = load_vec<T, E, false, false>(x + c, n, true), rd = load_vec<T, E, false, false>(dy + c, n, true);
      Raw<PT, E> rw;
      if (w != nullptr) rw = load_vec<PT, E, false, false>(w + c, n, true);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float xhat = k < n ? (rx.get(k) - mean) * rstd : 0.0f;
        const float g = w != nullptr ? rd.get(k) * rw.get(k) : rd.get(k);
        s1 += g;
        s2 += g * xhat;
      }
    }
    s1 = block_sum(s1, lds[parity][0]) * inv;
    s2 = block_sum(s2, lds[parity][1]) * inv;
    for (int64_t c = int64_t(threadIdx.x) * E; c < D; c += kWideThreads * E) {
      const int n = tail<E>(D - c);
      const Raw<T, E> rx = load_vec<T, E, false, false>(x + c, n, true), rd = load_vec<T, E, false, false>(dy + c, n, true);
      Raw<PT, E> rw;
      if (w != nullptr) rw = load_vec<PT, E, false, false>(w + c, n, true);
      float o[E];
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float xhat = (rx.get(k) - mean) * rstd;
        const float g = w != nullptr ? rd.get(k) * rw.get(k) : rd.get(k);
        o[k] = rstd * (g - s1 - xhat * s2);
      }
      store_vec<T, E, false, false>(dx + c, n, o);
    }
  }
}

// ... and the parameter gradients' sums, a wave for 64 vectors of columns and a group of rows.
template <typename T>
__global__ __launch_bounds__(64) void layer_norm_bwd_cols_kernel(LayerNormBwdArgs a) {
  constexpr int E = kVec<T>;
  const int64_t D = a.cols, c = (int64_t(blockIdx.x) * 64 + threadIdx.x) * E;
  if (c >= D) return;
  const int n = tail<E>(D - c);
  float dw[E] = {}, db[E] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const Raw<T, E> rx = load_vec<T, E, false, false>(static_cast<const T*>(a.x) + row * a.x_stride + c, n, true);
    const Raw<T, E> rd = load_vec<T, E, false, false>(static_cast<const T*>(a.dy) + row * a.dy_stride + c, n, true);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int k = 0; k < E; ++k) {
      dw[k] += rd.get(k) * ((rx.get(k) - mean) * rstd);
      db[k] += rd.get(k);
    }
  }
  float* part = a.partial + int64_t(blockIdx.y) * 2 * padded(D);
  store_vec<float, E, false, false>(part + c, n, dw);
  store_vec<float, E, false, false>(part + padded(D) + c, n, db);
}

// Adds the workgroups' partial sums: a workgroup takes 64 columns (and those a grid further), a thread four
// of them and every sixteenth partial; the sixteen sums of a column meet in LDS, in order.
template <typename PT>
__global__ __launch_bounds__(256) void layer_norm_join_kernel(const float* __restrict__ partial, int groups, int64_t D,
                                                              PT* dweight, PT* dbias) {
  __shared__ float lds[16][64];
  const int64_t P = padded(D);
  const int slice = threadIdx.x >> 4, q = (threadIdx.x & 15) * 4;
  for (int64_t b = blockIdx.x; b * 64 < 2 * P; b += gridDim.x) {
    if (b != int64_t(blockIdx.x)) __syncthreads();  // the last columns' sums are read
    const int64_t c = b * 64 + q;                   // of the 2 * P columns
    f32x4 s = {0, 0, 0, 0};
    if (c < 2 * P) {
#pragma unroll 8
      for (int g = slice; g < groups; g += 16) s += __builtin_bit_cast(f32x4, load16(partial + int64_t(g) * 2 * P + c));
    }
    *reinterpret_cast<f32x4*>(&lds[slice][q]) = s;
    __syncthreads();
    if (threadIdx.x < 64) {
      const int64_t o = b * 64 + threadIdx.x, col = o < P ? o : o - P;
      PT* out = o < P ? dweight : dbias;
      if (o < 2 * P && col < D && out != nullptr) {
        float t = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) t += lds[k][threadIdx.x];
        out[col] = narrow<PT>(t);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------------------------

constexpr int64_t kMaxGrid = 1 << 20;
inline int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int V>
struct Int {
  static constexpr int value = V;
};
// f(L) for the smallest group that holds a row of up to 64 vectors.
template <typename F>
void with_lanes(int64_t vecs, F&& f) {
  if (vecs <= 8) f(Int<8>());
  else if (vecs <= 16) f(Int<16>());
  else if (vecs <= 32) f(Int<32>());
  else f(Int<64>());
}
// f(NV, RB, waves) for rows of more than 64 vectors; false for rows that the registers do not hold.
//
// Forward: three vectors a lane and two rows a workgroup keep about 16 waves with 60 KiB of loads in
// flight on a compute unit and halve the reads of weight and bias (32760 x 5120 bf16: 113 us; two
// vectors 122, four 119, one row 122, ten vectors in one wave, without a barrier, 146; a copy of the same
// bytes takes 109).  Two vectors where they leave fewer lanes of the first waves empty (600 MB of bf16: 96
// vectors 112 us, with three 122; 224 vectors 107 and 117; but 160 vectors 119 and 107).  Of 1024 vectors two
// (109 us, with three 119) and of 2048 four (116 and 155) would be faster; they are not told apart.
// Few rows go to as many waves as they fill: the time is one row's (1024 rows of 1024 vectors 10.8 us, with
// three vectors and two rows 11.3; at 2048 rows both 17.2).
template <typename F>
bool with_rows(int64_t vecs, int64_t rows, F&& f) {
  const auto waves = [&](int nv) { return int(ceil_div(vecs, 64 * nv)); };
  if (vecs > 64 * kMaxWaves * 4) return false;
  if (vecs > 64 * kMaxWaves * 3) f(Int<4>(), Int<1>(), waves(4));
  else if (rows >= 2048 && (vecs <= 128 || (vecs > 192 && vecs <= 256))) f(Int<2>(), Int<2>(), waves(2));
  else if (rows >= 2048) f(Int<3>(), Int<2>(), waves(3));
  else if (vecs <= 64 * kMaxWaves) f(Int<1>(), Int<1>(), waves(1));
  else f(Int<3>(), Int<1>(), waves(3));
  return true;
}
// Backward: the sums down the columns take 16 registers for a vector of bf16 (of fp32 eight, held to the same
// limit), so a lane holds at most two; beyond, rows are streamed.  Two vectors of two rows do not fit (38400 x
// 4096 bf16 598 us instead of 159).  Sixteen waves are resident on a compute unit (8192 x 8192 bf16, two
// vectors, 512 workgroups of 8 waves: 72 us, with the partial sums 6.1 TB/s; 16 waves of one vector 79).
// From two waves' width on, up to eight, one vector of two rows is faster (with the join, bf16: 4096 rows of 192
// vectors 18 us, two vectors of one row 24; 38400 of 512 159 and 178); beyond, and in rows of one wave, where
// many rows count, two vectors of one row (19200 of 1024 162 us and 169; 153600 of 128 168 and 180, but 4096 of
// 128 22 and 17).
template <typename F>
bool with_bwd_rows(int64_t vecs, F&& f) {
  const auto waves = [&](int nv) { return int(ceil_div(vecs, 64 * nv)); };
  if (vecs > 64 * kMaxWaves * 2) return false;
  if (vecs > 128 && vecs <= 512) f(Int<1>(), Int<2>(), waves(1));
  else f(Int<2>(), Int<1>(), waves(2));
  return true;
}

// Rows whose inputs and outputs exceed the last-level cache are accessed as read and written once:
// 8192 x 8192 bf16 backward 72 us instead of 81, 32760 x 5120 forward 119 instead of 124; tensors that
// fit lose up to 10% that way (8192 x 4096 forward: 26 instead of 24).
constexpr int64_t kCacheBytes = int64_t(256) << 20;
template <int E, typename F>
int with_form(int64_t bytes, int64_t cols, F&& f) {
  return with_whole<E>(cols, [&](auto whole) {
    return bytes > kCacheBytes ? f(std::true_type(), whole) : f(std::false_type(), whole);
  });
}

// The backward pass of up to so many rows is one launch: 16 rows of 4096 bf16 3.6 us, with partial sums
// and their join 7.2; 16 rows of 1001 6.9 and 7.4; 64 rows of 1001 would take 21 instead of 8.
constexpr int kFewRows = 16;

template <typename T, typename PT>
int forward(const LayerNormArgs& a, hipStream_t s) {
  const int64_t vecs = ceil_div(a.cols, kVec<T>);
  return with_form<kVec<T>>(2 * a.rows * a.cols * int64_t(sizeof(T)), a.cols, [&](auto o, auto w) {
    constexpr bool once = decltype(o)::value, whole = decltype(w)::value;
    int e = 0;
    if (vecs <= 64) {
      with_lanes(vecs, [&](auto l) {
        constexpr int L = decltype(l)::value;
        const int64_t grid = min64(ceil_div(a.rows, kNarrowThreads / L), kMaxGrid);
        e = launch(layer_norm_narrow_kernel<T, PT, L, once, whole>, unsigned(grid), kNarrowThreads, 0, s, a);
      });
      return e;
    }
    const bool fits = with_rows(vecs, a.rows, [&](auto nv, auto rb, int waves) {
      constexpr int NV = decltype(nv)::value, RB = decltype(rb)::value;
      const int64_t grid = min64(ceil_div(a.rows, RB), kMaxGrid);
      e = launch(layer_norm_rows_kernel<T, PT, NV, RB, once, whole>, unsigned(grid), waves * 64, 0, s, a);
    });
    if (fits) return e;
    return launch(layer_norm_wide_kernel<T, PT>, unsigned(min64(a.rows, kMaxGrid)), kWideThreads, 0, s, a);
  });
}

template <typename T, typename PT>
int backward(LayerNormBwdArgs a, int groups, hipStream_t s) {
  const bool params = a.dweight != nullptr || a.dbias != nullptr;
  const int64_t vecs = ceil_div(a.cols, kVec<T>);
  if (params && a.rows > 0 && a.rows <= kFewRows && vecs <= 64 * kMaxWaves * 2)
    return with_whole<kVec<T>>(a.cols, [&](auto w) {
      constexpr bool whole = decltype(w)::value;
      const unsigned rows = a.dx != nullptr ? unsigned(a.rows) : 0, cols = unsigned(ceil_div(vecs, 64));
      const auto few = [&](unsigned row_wgs, unsigned col_wgs) {
        if (vecs <= 64 * kMaxWaves)
          return launch(layer_norm_bwd_few_kernel<T, PT, 1, whole>, row_wgs + col_wgs, int(cols) * 64, 0, s, a, row_wgs);
        return launch(layer_norm_bwd_few_kernel<T, PT, 2, whole>, row_wgs + col_wgs, int(ceil_div(vecs, 128)) * 64, 0,
                      s, a, row_wgs);
      };
      if (a.dx != a.dy) return few(rows, cols);
      const int e = few(0, cols);  // the sums first: they read dy too
      return e != 0 ? e : few(rows, 0);
    });
  if (!params) a.partial = nullptr;
  int e = 0;
  if (a.rows > 0)
    e = with_form<kVec<T>>(3 * a.rows * a.cols * int64_t(sizeof(T)), a.cols, [&](auto o, auto w) {
      constexpr bool once = decltype(o)::value, whole = decltype(w)::value;
      int e = 0;
      if (vecs <= 64) {
        with_lanes(vecs, [&](auto l) {
          e = launch(layer_norm_bwd_narrow_kernel<T, PT, decltype(l)::value, once, whole>, unsigned(groups),
                     kNarrowThreads, 0, s, a);
        });
        return e;
      }
      const bool fits = with_bwd_rows(vecs, [&](auto nv, auto rb, int waves) {
        e = launch(layer_norm_bwd_rows_kernel<T, PT, decltype(nv)::value, decltype(rb)::value, once, whole>,
                   unsigned(groups), waves * 64, 0, s, a);
      });
      if (fits) return e;
      // the sums first: dx may lie where dy does
      if (params)
        e = launch(layer_norm_bwd_cols_kernel<T>, dim3(unsigned(ceil_div(vecs, 64)), unsigned(groups)), 64, 0, s, a);
      if (e != 0 || a.dx == nullptr) return e;
      return launch(layer_norm_bwd_wide_kernel<T, PT>, unsigned(min64(a.rows, kMaxGrid)), kWideThreads, 0, s, a);
    });
  if (e != 0 || !params) return e;
  return launch(layer_norm_join_kernel<PT>, unsigned(min64(ceil_div(2 * padded(a.cols), 64), kMaxGrid)), 256, 0, s,
                a.partial, groups, a.cols, static_cast<PT*>(a.dweight), static_cast<PT*>(a.dbias));
}

// Workgroups: as many as are resident at 16 waves a compute unit, each with at least two turns.
int64_t bwd_groups(int64_t rows, int64_t vecs) {
  int64_t groups = 0;
  if (vecs <= 64) {
    with_lanes(vecs, [&](auto l) { groups = min64(ceil_div(rows, 2 * kNarrowThreads / decltype(l)::value), 1024); });
    return groups;
  }
  const bool fits = with_bwd_rows(vecs, [&](auto, auto rb, int waves) {
    groups = min64(ceil_div(rows, 2 * decltype(rb)::value), 256 * (waves > 8 ? 1 : min64(16 / waves, 8)));
  });
  return fits ? groups : min64(rows, 64);
}

}  // namespace

int layer_norm_bwd_groups(int64_t rows, int64_t cols, int dtype) {
  return int(bwd_groups(rows, ceil_div(cols, dtype == TIDE_BF16 ? kVec<bf16_t> : kVec<float>)));
}

int launch_layer_norm(const LayerNormArgs& a, int dtype, int param_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == TIDE_BF16) return param_dtype == TIDE_BF16 ? forward<bf16_t, bf16_t>(a, s) : forward<bf16_t, float>(a, s);
  return param_dtype == TIDE_BF16 ? forward<float, bf16_t>(a, s) : forward<float, float>(a, s);
}

int launch_layer_norm_bwd(const LayerNormBwdArgs& a, int dtype, int param_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int groups = layer_norm_bwd_groups(a.rows, a.cols, dtype);
  if (dtype == TIDE_BF16)
    return param_dtype == TIDE_BF16 ? backward<bf16_t, bf16_t>(a, groups, s) : backward<bf16_t, float>(a, groups, s);
  return param_dtype == TIDE_BF16 ? backward<float, bf16_t>(a, groups, s) : backward<float, float>(a, groups, s);
}

}  // namespace tide_step
