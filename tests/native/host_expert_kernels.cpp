// The experts' kernels of libtide_step.so on the host, where lanes and waves run in any order that is asked for.
// Exit status 0 = all checks passed.
//
//   host_expert_kernels in_place   gradients written over the rows that they are made of
//   host_expert_kernels sort       places, rows and offsets of small calls
//   host_expert_kernels far        a sort whose rows end at the largest number
#include <sys/mman.h>
#include <unistd.h>

#include <algorithm>
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

template <typename I>
void sorted(int dtype, int64_t tokens, int choices, int experts, int align, int more) {
  const int64_t pairs = tokens * choices, rows = pairs + std::min<int64_t>(experts, pairs) * (align - 1) + more;
  std::mt19937 rng(unsigned(pairs + experts));
  std::vector<I> ids(static_cast<size_t>(pairs));
  for (I& id : ids) id = I(int(rng() % unsigned(experts + 2)) - 1);
  std::vector<int32_t> place(size_t(pairs), 77), source(size_t(rows + 1), 77), offsets(size_t(experts) + 1, 77);
  std::vector<int32_t> counts(size_t(expert_parts(pairs, experts)) * size_t(experts));
  launch_expert_sort({pairs, ids.data(), experts, align, place.data(), source.data(), rows, offsets.data(), counts.data()}, dtype, nullptr);
  std::vector<int32_t> p(size_t(pairs), -1), s(size_t(rows + 1), -1), o(size_t(experts) + 1, 0);
  s.back() = 77;
  for (int e = 0; e < experts; ++e) {
    int32_t at = o[size_t(e)];
    for (int64_t i = 0; i < pairs; ++i)
      if (ids[size_t(i)] == e) p[size_t(i)] = at, s[size_t(at++)] = int32_t(i);
    o[size_t(e) + 1] = (at + align - 1) / align * align;
  }
  CHECK(place == p && source == s && offsets == o, "%lld tokens, %d choices of %d, multiples of %d", (long long)tokens, choices, experts, align);
}

// One pair of two experts, whose rows are rounded up to the largest number: the first expert's rows end there, and
// the second's begin.  All of the rows' memory is one piece, mapped over and over; none of what lies before and behind
// it may be touched.
void far() {
  const int64_t rows = (int64_t(1) << 31) - 1, bytes = int64_t(1) << 33, piece = int64_t(1) << 23;
  char* space = static_cast<char*>(mmap(nullptr, size_t(4 * bytes), PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
  const int file = memfd_create("rows", 0);
  CHECK(space != MAP_FAILED && file >= 0 && ftruncate(file, piece) == 0, "no memory");
  if (failures > 0) return;
  char* from = space + 2 * bytes;
  for (int64_t at = 0; at < bytes; at += piece)
    CHECK(mmap(from + at, size_t(piece), PROT_READ | PROT_WRITE, MAP_SHARED | MAP_FIXED, file, 0) != MAP_FAILED, "no memory");
  const int64_t id = 0;
  int32_t place = 77, offsets[3] = {77, 77, 77};
  launch_expert_sort({1, &id, 2, int32_t(rows), &place, reinterpret_cast<int32_t*>(from), rows, offsets, nullptr}, TIDE_INT64, nullptr);
  CHECK(place == 0 && offsets[0] == 0 && offsets[1] == rows && offsets[2] == rows, "%d %d %d", place, offsets[1], offsets[2]);
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
  } else if (what == "sort") {
    for (int more : {0, 5})
      for (int align : {1, 7, 16, 128})
        for (int experts : {1, 2, 9, 63, 200}) {
          for (int64_t tokens : {0, 1, 5, 70, 333}) sorted<int64_t>(TIDE_INT64, tokens, 3, experts, align, more);
          sorted<int32_t>(TIDE_INT32, 2100, 2, experts, align, more);
        }
    sorted<int32_t>(TIDE_INT32, 5000, 1, 2048, 3, 1);
  } else if (what == "far") {
    far();
  } else {
    ++failures;
  }
  std::printf("%d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
