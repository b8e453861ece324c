// Layer norm and its gradient.
//
//   mean = sum(x)/D, var = sum((x-mean)^2)/D, rstd = 1/sqrt(var+eps), y = (x-mean)*rstd*w + b
//   xhat = (x-mean)*rstd, g = dy*w, dx = rstd*(g - sum(g)/D - xhat*sum(g*xhat)/D)
//   dw = sum over rows dy*xhat, db = sum over rows dy
//
// HBM bounds both directions: a row is read once into registers, where the mean and then the
// centred squares are summed in fp32 (two passes over registers, so a large mean costs no digits),
// and written once.  A row belongs to a group of L lanes that hold NV vectors of eight elements
// each; a group is part of a wave for narrow rows and a workgroup for wide ones.  Rows too wide for
// the registers are streamed instead, and read again from the caches.
//
// The parameter gradients are sums down the columns: each workgroup keeps the sums of its rows in
// registers, in row order, and leaves them in the workspace; a second kernel adds the workgroups'
// sums in order.
#include "step_device.h"
#include "step_internal.h"

namespace tide_step {
namespace {

template <int L>
constexpr int kThreadsOf = L <= 64 ? 256 : L;

// Sum of v over the group of L lanes, in every lane.  `lds` (wide groups only) holds one float per
// wave and must be another one at the next call, so that one barrier suffices.
template <int L>
__device__ __forceinline__ float group_sum(float v, float* lds) {
  if constexpr (L <= 64) {
    return lanes_sum<L>(v);
  } else {
    v = lanes_sum<64>(v);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0;
#pragma unroll
    for (int w = 0; w < L / 64; ++w) s += lds[w];
    return s;
  }
}

template <typename T, typename PT, int L, int NV>
__global__ __launch_bounds__(kThreadsOf<L>) void layer_norm_kernel(LayerNormArgs a) {
  constexpr int kGroups = kThreadsOf<L> / L;
  __shared__ float lds[2][16];
  const int D = int(a.cols);
  const int lane = threadIdx.x % L;
  const float inv = 1.0f / float(D);
  const PT* w = static_cast<const PT*>(a.weight);
  const PT* b = static_cast<const PT*>(a.bias);
  for (int64_t row = int64_t(blockIdx.x) * kGroups + threadIdx.x / L; row < a.rows;
       row += int64_t(gridDim.x) * kGroups) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    T* y = static_cast<T*>(a.y) + row * a.y_stride;
    Raw8<T> r[NV];
    float sum = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8;
      r[v] = load8(x + c, D - c);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += r[v].get(k);
    const float mean = group_sum<L>(sum, lds[0]) * inv;
    float sq = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int n = D - (v * L + lane) * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = r[v].get(k) - mean;
        sq += k < n ? d * d : 0.0f;
      }
    }
    const float var = group_sum<L>(sq, lds[1]) * inv;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (lane == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8, n = D - c;
      if (n <= 0) continue;
      Raw8<PT> rw, rb;
      if (w != nullptr) rw = load8(w + c, n);
      if (b != nullptr) rb = load8(b + c, n);
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xhat = (r[v].get(k) - mean) * rstd;
        o[k] = (w != nullptr ? xhat * rw.get(k) : xhat) + (b != nullptr ? rb.get(k) : 0.0f);
      }
      store8(y + c, n, o);
    }
  }
}

// Rows wider than the registers: three passes over the row, the later ones from the caches.
constexpr int kWideThreads = 1024;

template <typename T, typename PT>
__global__ __launch_bounds__(kWideThreads) void layer_norm_wide_kernel(LayerNormArgs a) {
  __shared__ float lds[2][16];
  const int64_t D = a.cols;
  const float inv = 1.0f / float(D);
  const PT* w = static_cast<const PT*>(a.weight);
  const PT* b = static_cast<const PT*>(a.bias);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    T* y = static_cast<T*>(a.y) + row * a.y_stride;
    float sum = 0;
    for (int64_t c = int64_t(threadIdx.x) * 8; c < D; c += kWideThreads * 8) {
      const Raw8<T> r = load8(x + c, int(D - c < 8 ? D - c : 8));
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += r.get(k);
    }
    const float mean = group_sum<kWideThreads>(sum, lds[0]) * inv;
    float sq = 0;
    for (int64_t c = int64_t(threadIdx.x) * 8; c < D; c += kWideThreads * 8) {
      const int n = int(D - c < 8 ? D - c : 8);
      const Raw8<T> r = load8(x + c, n);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = r.get(k) - mean;
        sq += k < n ? d * d : 0.0f;
      }
    }
    const float var = group_sum<kWideThreads>(sq, lds[1]) * inv;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    for (int64_t c = int64_t(threadIdx.x) * 8; c < D; c += kWideThreads * 8) {
      const int n = int(D - c < 8 ? D - c : 8);
      const Raw8<T> r = load8(x + c, n);
      Raw8<PT> rw, rb;
      if (w != nullptr) rw = load8(w + c, n);
      if (b != nullptr) rb = load8(b + c, n);
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xhat = (r.get(k) - mean) * rstd;
        o[k] = (w != nullptr ? xhat * rw.get(k) : xhat) + (b != nullptr ? rb.get(k) : 0.0f);
      }
      store8(y + c, n, o);
    }
  }
}

template <typename T, typename PT, int L, int NV>
__global__ __launch_bounds__(kThreadsOf<L>) void layer_norm_bwd_kernel(LayerNormBwdArgs a) {
  constexpr int kThreads = kThreadsOf<L>;
  constexpr int kGroups = kThreads / L;
  __shared__ float lds[2][2][16];
  __shared__ float join[kGroups > 1 ? kThreads * 8 : 1];
  const int D = int(a.cols);
  const int lane = threadIdx.x % L;
  const float inv = 1.0f / float(D);
  const PT* w = static_cast<const PT*>(a.weight);
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[v][k] = db[v][k] = 0.0f;
  int parity = 0;
  for (int64_t row = int64_t(blockIdx.x) * kGroups + threadIdx.x / L; row < a.rows;
       row += int64_t(gridDim.x) * kGroups, parity ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    Raw8<T> rx[NV], rd[NV];
    Raw8<PT> rw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8;
      rx[v] = load8(x + c, D - c);
      rd[v] = load8(dy + c, D - c);
      if (w != nullptr) rw[v] = load8(w + c, D - c);
    }
    float s1 = 0, s2 = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int n = D - (v * L + lane) * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xhat = k < n ? (rx[v].get(k) - mean) * rstd : 0.0f;
        const float d = rd[v].get(k);
        const float g = w != nullptr ? d * rw[v].get(k) : d;
        s1 += g;
        s2 += g * xhat;
        dw[v][k] += d * xhat;
        db[v][k] += d;
      }
    }
    if (a.dx == nullptr) continue;
    s1 = group_sum<L>(s1, lds[parity][0]) * inv;
    s2 = group_sum<L>(s2, lds[parity][1]) * inv;
    T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8, n = D - c;
      if (n <= 0) continue;
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xhat = (rx[v].get(k) - mean) * rstd;
        const float d = rd[v].get(k);
        const float g = w != nullptr ? d * rw[v].get(k) : d;
        o[k] = rstd * (g - s1 - xhat * s2);
      }
      store8(dx + c, n, o);
    }
  }
  if (a.partial == nullptr) return;
  float* part = a.partial + int64_t(blockIdx.x) * 2 * D;
  if constexpr (kGroups > 1) {
    // one vector of every group through LDS at a time, added in group order
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) join[threadIdx.x * 8 + k] = s == 0 ? dw[v][k] : db[v][k];
        __syncthreads();
        for (int i = threadIdx.x; i < L * 8; i += kThreads) {
          float t = 0;
          for (int g = 0; g < kGroups; ++g) t += join[g * L * 8 + i];
          const int c = v * L * 8 + i;
          if (c < D) part[s * D + c] = t;
        }
      }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8, n = D - c;
      if (n <= 0) continue;
      store8(part + c, n, dw[v]);
      store8(part + D + c, n, db[v]);
    }
  }
}

// Rows wider than the registers: the input's gradient, two passes over a row.
template <typename T, typename PT>
__global__ __launch_bounds__(kWideThreads) void layer_norm_bwd_wide_kernel(LayerNormBwdArgs a) {
  __shared__ float lds[2][2][16];
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
    for (int64_t c = int64_t(threadIdx.x) * 8; c < D; c += kWideThreads * 8) {
      const int n = int(D - c < 8 ? D - c : 8);
      const Raw8<T> rx = load8(x + c, n), rd = load8(dy + c, n);
      Raw8<PT> rw;
      if (w != nullptr) rw = load8(w + c, n);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xhat = k < n ? (rx.get(k) - mean) * rstd : 0.0f;
        const float g = w != nullptr ? rd.get(k) * rw.get(k) : rd.get(k);
        s1 += g;
        s2 += g * xhat;
      }
    }
    s1 = group_sum<kWideThreads>(s1, lds[parity][0]) * inv;
    s2 = group_sum<kWideThreads>(s2, lds[parity][1]) * inv;
    for (int64_t c = int64_t(threadIdx.x) * 8; c < D; c += kWideThreads * 8) {
      const int n = int(D - c < 8 ? D - c : 8);
      const Raw8<T> rx = load8(x + c, n), rd = load8(dy + c, n);
      Raw8<PT> rw;
      if (w != nullptr) rw = load8(w + c, n);
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xhat = (rx.get(k) - mean) * rstd;
        const float g = w != nullptr ? rd.get(k) * rw.get(k) : rd.get(k);
        o[k] = rstd * (g - s1 - xhat * s2);
      }
      store8(dx + c, n, o);
    }
  }
}

// ... and the parameter gradients' sums, a wave for each 512 columns and group of rows.
template <typename T>
__global__ __launch_bounds__(64) void layer_norm_bwd_cols_kernel(LayerNormBwdArgs a) {
  const int64_t D = a.cols, c = (int64_t(blockIdx.x) * 64 + threadIdx.x) * 8;
  if (c >= D) return;
  const int n = int(D - c < 8 ? D - c : 8);
  float dw[8] = {}, db[8] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const Raw8<T> rx = load8(static_cast<const T*>(a.x) + row * a.x_stride + c, n);
    const Raw8<T> rd = load8(static_cast<const T*>(a.dy) + row * a.dy_stride + c, n);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      dw[k] += rd.get(k) * ((rx.get(k) - mean) * rstd);
      db[k] += rd.get(k);
    }
  }
  float* part = a.partial + int64_t(blockIdx.y) * 2 * D;
  store8(part + c, n, dw);
  store8(part + D + c, n, db);
}

// Adds the workgroups' partial sums: a lane for each column, four waves taking every fourth partial.
template <typename PT>
__global__ __launch_bounds__(256) void layer_norm_join_kernel(const float* __restrict__ partial, int groups, int64_t D,
                                                              PT* dweight, PT* dbias) {
  __shared__ float lds[4][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t c = int64_t(blockIdx.x) * 64 + lane;  // column of the [2 * D] sums
  float s = 0;
  if (c < 2 * D)
    for (int g = wave; g < groups; g += 4) s += partial[int64_t(g) * 2 * D + c];
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < 2 * D) {
    const float t = ((lds[0][lane] + lds[1][lane]) + lds[2][lane]) + lds[3][lane];
    PT* out = c < D ? dweight : dbias;
    if (out != nullptr) out[c < D ? c : c - D] = narrow<PT>(t);
  }
}

// The narrowest shape that holds a row: f(L, NV) with L * NV * 8 >= cols, or false beyond the widest.
template <int L_, int NV_>
struct Shape {
  static constexpr int L = L_, NV = NV_;
};
template <typename F>
bool with_shape(int64_t cols, bool bwd, F&& f) {
  if (cols <= 64) f(Shape<8, 1>());
  else if (cols <= 256) f(Shape<32, 1>());
  else if (cols <= 512) f(Shape<64, 1>());
  else if (cols <= 1024) f(Shape<64, 2>());
  else if (cols <= 2048) f(Shape<256, 1>());
  else if (cols <= 4096) f(Shape<256, 2>());
  else if (cols <= 6144) f(Shape<256, 3>());
  else if (cols <= 8192) f(Shape<256, 4>());
  else if (cols <= 16384) f(Shape<1024, 2>());
  else if (cols <= 32768 && !bwd) f(Shape<1024, 4>());
  else return false;
  return true;
}

constexpr int64_t kMaxGrid = 1 << 20;
inline int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

template <typename T, typename PT>
void forward(const LayerNormArgs& a, hipStream_t s) {
  const bool fits = with_shape(a.cols, false, [&](auto sh) {
    using S = decltype(sh);
    constexpr int threads = kThreadsOf<S::L>, groups = threads / S::L;
    const int64_t grid = min64((a.rows + groups - 1) / groups, kMaxGrid);
    hipLaunchKernelGGL((layer_norm_kernel<T, PT, S::L, S::NV>), dim3(unsigned(grid)), dim3(threads), 0, s, a);
  });
  if (!fits)
    hipLaunchKernelGGL((layer_norm_wide_kernel<T, PT>), dim3(unsigned(min64(a.rows, kMaxGrid))), dim3(kWideThreads), 0,
                       s, a);
}

template <typename T, typename PT>
void backward(LayerNormBwdArgs a, int groups, hipStream_t s) {
  const bool params = a.dweight != nullptr || a.dbias != nullptr;
  if (!params) a.partial = nullptr;
  if (a.rows > 0) {
    const bool fits = with_shape(a.cols, true, [&](auto sh) {
      using S = decltype(sh);
      hipLaunchKernelGGL((layer_norm_bwd_kernel<T, PT, S::L, S::NV>), dim3(unsigned(groups)), dim3(kThreadsOf<S::L>), 0,
                         s, a);
    });
    if (!fits) {
      // the sums first: dx may lie where dy does
      if (params)
        hipLaunchKernelGGL((layer_norm_bwd_cols_kernel<T>), dim3(unsigned((a.cols + 511) / 512), unsigned(groups)),
                           dim3(64), 0, s, a);
      if (a.dx != nullptr)
        hipLaunchKernelGGL((layer_norm_bwd_wide_kernel<T, PT>), dim3(unsigned(min64(a.rows, kMaxGrid))),
                           dim3(kWideThreads), 0, s, a);
    }
  }
  if (params)
    hipLaunchKernelGGL((layer_norm_join_kernel<PT>), dim3(unsigned((2 * a.cols + 63) / 64)), dim3(256), 0, s, a.partial,
                       groups, a.cols, static_cast<PT*>(a.dweight), static_cast<PT*>(a.dbias));
}

}  // namespace

int layer_norm_bwd_groups(int64_t rows, int64_t cols, int) {
  if (rows == 0) return 0;
  int64_t need = 0;
  const bool fits = with_shape(cols, true, [&](auto sh) {
    using S = decltype(sh);
    constexpr int groups = kThreadsOf<S::L> / S::L;
    need = min64((rows + groups - 1) / groups, kThreadsOf<S::L> == 1024 ? 256 : 1024);
  });
  return int(fits ? need : min64(rows, 64));
}

int launch_layer_norm(const LayerNormArgs& a, int dtype, int param_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == TIDE_BF16) {
    if (param_dtype == TIDE_BF16) forward<bf16_t, bf16_t>(a, s);
    else forward<bf16_t, float>(a, s);
  } else {
    if (param_dtype == TIDE_BF16) forward<float, bf16_t>(a, s);
    else forward<float, float>(a, s);
  }
  return hipGetLastError();
}

int launch_layer_norm_bwd(const LayerNormBwdArgs& a, int dtype, int param_dtype, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int groups = layer_norm_bwd_groups(a.rows, a.cols, dtype);
  if (dtype == TIDE_BF16) {
    if (param_dtype == TIDE_BF16) backward<bf16_t, bf16_t>(a, groups, s);
    else backward<bf16_t, float>(a, groups, s);
  } else {
    if (param_dtype == TIDE_BF16) backward<float, bf16_t>(a, groups, s);
    else backward<float, float>(a, groups, s);
  }
  return hipGetLastError();
}

}  // namespace tide_step
