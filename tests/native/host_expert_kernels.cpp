// The experts' kernels of libtide_step.so on the host, where lanes and waves run in any order that is asked for.
// Exit status 0 = all checks passed.
//
//   host_expert_kernels in_place   gradients written over the rows that they are made of
#include <cstdio>
#include <random>
#include <string>
#include <vector>

#include "../../all_gather_placement_amd/csrc/step_device.h"
#include "../../all_gather_placement_amd/csrc/step_internal.h"

namespace tide_step {
template <typename... P>
int launch_on_host(void (*kernel)(P...), dim3 grid, int threads, size_t, hipStream_t, const typename Same<P>::type&... args) {
  lanes::run(grid, unsigned(threads), [&] { kernel(args...); });
  return hipSuccess;
}
}  // namespace tide_step
#define launch launch_on_host
#include "../../all_gather_placement_amd/csrc/step_experts.hip"
#undef launch

namespace tide_step {
namespace {
thread_local int count[1 << 14], lds[1 << 14];  // the sort's
}  // namespace
}  // namespace tide_step
using namespace tide_step;

// The host compiler's rounding of float to bf16, which its runtime may lack: to nearest, ties to even.
extern "C" __bf16 __truncsfbf2(float f) {
  const uint32_t u = __float_as_uint(f);
  return lanes::bits_of<__bf16>(uint16_t((u + 0x7fff + (u >> 16 & 1)) >> 16));
}

static int failures = 0;
#define CHECK(cond, ...)                                                      \
  do {                                                                        \
    if (!(cond)) {                                                            \
      std::fprintf(stderr, "CHECK failed at line %d: %s: ", __LINE__, #cond); \
      std::fprintf(stderr, __VA_ARGS__);                                      \
      std::fprintf(stderr, "\n");                                             \
      ++failures;                                                             \
    }                                                                         \
  } while (0)

// Whole numbers, of which every product and sum is exact.
template <typename T>
std::vector<T> numbers(size_t n, unsigned seed) {
  std::mt19937 rng(seed);
  std::vector<T> v(n);
  for (T& x : v) x = narrow<T>(float(int(rng() % 7) - 3));
  return v;
}

template <typename T>
void in_place(int dtype, int64_t dim, int choices) {
  const int64_t tokens = 5, pairs = tokens * choices, rows = pairs + 2, stride = dim + 1;
  std::vector<int32_t> place(size_t(pairs), -1), source(size_t(rows), -1);
  for (int64_t p = 1; p < pairs; ++p) {  // the first pair has no row
    place[size_t(p)] = int32_t(rows - 1 - p);
    source[size_t(rows - 1 - p)] = int32_t(p);
  }
  const std::vector<T> x = numbers<T>(size_t(rows * stride), 1), dy = numbers<T>(size_t(tokens * dim), 2);
  const std::vector<float> w = numbers<float>(size_t(pairs), 3);
  std::vector<T> buf = x;
  std::vector<float> dw(size_t(pairs), 77.0f);
  ExpertRowsArgs a{};
  a.tokens = tokens, a.dim = dim, a.rows = rows, a.choices = choices, a.place = place.data(), a.source = source.data();
  a.x = buf.data(), a.x_stride = stride, a.dy = dy.data(), a.dy_stride = dim, a.weights = w.data();
  a.out = buf.data(), a.out_stride = stride, a.dweights = dw.data();
  launch_expert_combine_bwd(a, dtype, TIDE_FP32, nullptr);
  int wrong_dots = 0, wrong_rows = 0;
  for (int64_t p = 0; p < pairs; ++p) {
    float dot = 0.0f;
    for (int64_t c = 0; c < dim && place[size_t(p)] >= 0; ++c)
      dot += widen(dy[size_t(p / choices * dim + c)]) * widen(x[size_t(place[size_t(p)] * stride + c)]);
    wrong_dots += dw[size_t(p)] != dot;
  }
  for (int64_t r = 0; r < rows; ++r) {
    const int64_t s = source[size_t(r)];
    for (int64_t c = 0; c < dim; ++c)
      wrong_rows += widen(buf[size_t(r * stride + c)]) != (s < 0 ? 0.0f : w[size_t(s)] * widen(dy[size_t(s / choices * dim + c)]));
    wrong_rows += widen(buf[size_t(r * stride + dim)]) != widen(x[size_t(r * stride + dim)]);  // between the rows
  }
  CHECK(wrong_dots == 0 && wrong_rows == 0, "%d bytes, %lld columns, %d choices, %s: %d of %lld products, %d elements", int(sizeof(T)),
        (long long)dim, choices, lanes::backwards ? "last lanes first" : "first lanes first", wrong_dots, (long long)pairs, wrong_rows);
}

int main(int argc, char** argv) {
  const std::string what = argc > 1 ? argv[1] : "";
  if (what == "in_place") {
    // rows that end inside a vector, whose last two vectors belong to a lane's neighbour, to two waves, or to a
    // wave's first and next turn
    for (bool backwards : {false, true}) {
      lanes::backwards = backwards;
      for (int choices : {1, 2, 5, 9}) {
        for (int64_t dim : {1, 3, 4, 6, 21, 66, 253, 256, 257, 259, 511, 513, 515, 769, 1001, 1024, 1025, 1027, 2049, 2303})
          in_place<float>(TIDE_FP32, dim, choices);
        for (int64_t dim : {7, 8, 13, 129, 511, 513, 519, 520, 1025, 1031, 1537, 2049, 2055, 4097})
          in_place<bf16_t>(TIDE_BF16, dim, choices);
      }
    }
  } else {
    ++failures;
  }
  std::printf("%d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
