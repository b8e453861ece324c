// Host code of the block operators of libtide_step.so (argument checks, workspace sizes, quotients) under
// AddressSanitizer and UBSan, at the ends of the ranges of every argument.  Built with g++; the kernel
// launchers are stubs that check what reaches them.  Exit status 0 = all checks passed.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>
#include <random>
#include <vector>

#include "../../all_gather_placement_amd/csrc/step_checks.h"
#include "../../all_gather_placement_amd/csrc/step_internal.h"

static int failures = 0, launched = 0;
#define CHECK(cond)                                                           \
  do {                                                                        \
    if (!(cond)) {                                                            \
      std::fprintf(stderr, "CHECK failed at line %d: %s\n", __LINE__, #cond); \
      ++failures;                                                             \
    }                                                                         \
  } while (0)

namespace tide_step {
tide_status status_of(int e) { return e == 0 ? TIDE_OK : TIDE_ERR_HIP; }

static bool far(int64_t rows, int64_t stride) { return rows > 1 && stride > (int64_t(1) << 44) / rows; }

int launch_expert_sort(const ExpertSortArgs& a, int, void*) {
  ++launched;
  CHECK(a.pairs >= 0 && a.pairs < (int64_t(1) << 31) && a.experts >= 1 && a.experts <= TIDE_MAX_EXPERTS && a.align >= 1);
  CHECK(a.rows >= a.pairs && a.rows < (int64_t(1) << 31));
  CHECK(expert_parts(a.pairs, a.experts) >= 1 && expert_parts(a.pairs, a.experts) <= kExpertMaxParts);
  CHECK(expert_parts(a.pairs, a.experts) == 1 || a.counts != nullptr);
  return 0;
}
int launch_expert_dispatch(const ExpertRowsArgs& a, int, void*) {
  ++launched;
  CHECK(a.rows > 0 && a.out != nullptr && !far(a.rows, a.out_stride) && !far(a.tokens, a.x_stride));
  return 0;
}
int launch_expert_combine(const ExpertRowsArgs& a, int, int, void*) {
  ++launched;
  CHECK(a.tokens > 0 && a.out != nullptr && !far(a.tokens, a.out_stride) && !far(a.rows, a.x_stride));
  return 0;
}
int launch_expert_combine_bwd(const ExpertRowsArgs& a, int, int, void*) {
  ++launched;
  CHECK(a.tokens + a.rows > 0 && !far(a.rows, a.out_stride) && !far(a.tokens, a.dy_stride));
  return 0;
}
int launch_rotary(const RotaryArgs& a, int, int, int, void*) {
  ++launched;
  CHECK(a.tokens > 0 && a.heads > 0 && a.pairs >= 1 && 2 * a.pairs <= a.dim && a.ends[a.axes - 1] == a.pairs);
  CHECK(!far(a.tokens, a.x_token) && !far(a.heads, a.x_head) && !far(a.tokens, a.out_token) && !far(a.heads, a.out_head));
  return 0;
}
int launch_dropout(const DropoutArgs& a, int, void*) {
  ++launched;
  CHECK(a.threshold <= 65536 && std::isfinite(a.scale) && (a.threshold == 65536 ? a.scale == 0 : a.scale >= 1));
  CHECK(a.offset + a.rows * a.cols <= (int64_t(1) << 62));
  return 0;
}
}  // namespace tide_step

static void* at(int k) { return reinterpret_cast<void*>(uintptr_t(k) << 50); }

int main() {
  const int64_t lim = std::numeric_limits<int64_t>::max();
  const int64_t sizes[] = {-lim - 1, -1, 0, 1, 7, 4096, 1 << 20, (int64_t(1) << 31) - 1, int64_t(1) << 31, int64_t(1) << 44, lim};
  const int32_t counts[] = {-2147483647 - 1, -1, 0, 1, 2, 64, 65, 2048, 2049, 2147483647};
  int accepted = 0, refused = 0;
  const auto take = [&](tide_status s, int before) {
    CHECK(s == TIDE_OK || s == TIDE_ERR_INVALID);
    CHECK(s == TIDE_OK || launched == before);  // what is refused enqueues nothing
    ++(s == TIDE_OK ? accepted : refused);
  };
  for (int64_t tokens : sizes)
    for (int32_t choices : counts)
      for (int32_t experts : counts)
        for (int32_t align : counts) {
          const int64_t rows = tide_expert_rows(tokens, choices, experts, align);
          const int64_t ws = tide_expert_sort_workspace(tokens, choices, experts);
          CHECK(rows == -1 || (rows >= tokens * choices && ws >= 0));
          for (int64_t r : {rows, rows + 1, int64_t(0), lim}) {
            const int before = launched;
            const tide_status s = tide_expert_sort(tokens, choices, at(1), TIDE_INT64, experts, align, static_cast<int32_t*>(at(2)),
                                                   static_cast<int32_t*>(at(3)), r, static_cast<int32_t*>(at(4)), at(5), ws, nullptr);
            take(s, before);
            CHECK(s != TIDE_OK || (rows >= 0 && r >= rows));
          }
        }
  auto* p = static_cast<const int32_t*>(at(1));
  auto* q = static_cast<const int32_t*>(at(2));
  for (int64_t tokens : sizes)
    for (int32_t choices : {0, 1, 64, 65})
      for (int64_t dim : sizes)
        for (int64_t rows : sizes)
          for (int64_t stride : sizes) {
            int before = launched;
            take(tide_expert_dispatch(tokens, choices, dim, at(3), stride, 0, p, q, rows, at(4), stride, nullptr), before);
            before = launched;
            take(tide_expert_combine(tokens, choices, dim, at(3), stride, rows, 1, at(5), 0, p, at(4), dim, nullptr), before);
            before = launched;
            take(tide_expert_combine_bwd(tokens, choices, dim, at(3), dim, at(4), dim, rows, 1, at(5), 0, p, q, at(6), stride,
                                         at(7), nullptr),
                 before);
          }
  for (int64_t tokens : sizes)
    for (int64_t heads : sizes)
      for (int64_t dim : {int64_t(0), int64_t(2), int64_t(128), int64_t(1024), int64_t(1025), lim})
        for (int64_t token : sizes)
          for (int64_t head : sizes)
            for (int64_t own : {int64_t(0), dim}) {
              const int32_t sections[] = {1, 2147483647, 1};
              const int before = launched;
              take(tide_rotary(tokens, heads, dim, at(1), token, head, 0, at(2), TIDE_FP32, 1, sections,
                               static_cast<double*>(at(3)), 1, 0, at(4), own == 0 ? token : dim, own == 0 ? head : 0, nullptr),
                   before);
              CHECK(tide_rotary(tokens, heads, dim, at(1), token, head, 0, at(2), TIDE_FP32, 3, sections,
                                static_cast<double*>(at(3)), 1, 0, at(4), token, head, nullptr) == TIDE_ERR_INVALID);
            }
  for (int64_t rows : sizes)
    for (int64_t cols : sizes)
      for (int64_t stride : sizes)
        for (int64_t offset : {int64_t(-1), int64_t(0), int64_t(3), int64_t(1) << 61, int64_t(1) << 62, lim})
          for (double prob : {0.0, 1e-9, 0.1, 0.5, 0.99999, 0.999999, 1.0, -0.0, 1.5, std::nan("")}) {
            const int before = launched;
            take(tide_dropout(rows, cols, at(1), stride, 0, prob, ~uint64_t(0), nullptr, offset, at(2), stride, at(3), stride,
                              nullptr),
                 before);
          }
  // views that share memory: random strided vectors over each other, against a list of their elements
  std::mt19937_64 rng(3);
  for (int round = 0; round < 20000; ++round) {
    const int64_t tokens = 1 + int64_t(rng() % 4), heads = 1 + int64_t(rng() % 4), dim = 2 + 2 * int64_t(rng() % 2);
    int64_t st[4];
    for (auto& s : st) s = int64_t(rng() % 24);
    if (round % 3 == 0) st[2] = st[0], st[3] = st[1];
    const int64_t shift = round % 5 == 0 ? 0 : int64_t(rng() % 48);
    std::vector<int> in(400, 0), out(400, 0);
    bool apart = true, meet = false;
    for (int64_t t = 0; t < tokens; ++t)
      for (int64_t h = 0; h < heads; ++h)
        for (int64_t k = 0; k < dim; ++k) {
          in[size_t(t * st[0] + h * st[1] + k)] = 1;
          int& o = out[size_t(shift + t * st[2] + h * st[3] + k)];
          apart &= o == 0;
          o = 1;
        }
    for (size_t i = 0; i < in.size(); ++i) meet |= in[i] && out[i];
    const bool same = shift == 0 && (tokens == 1 || st[0] == st[2]) && (heads == 1 || st[1] == st[3]);
    const int32_t sections[] = {1};
    char* base = static_cast<char*>(at(1));
    const tide_status s = tide_rotary(tokens, heads, dim, base, st[0], st[1], TIDE_FP32, at(2), TIDE_INT32, 1, sections,
                                      static_cast<double*>(at(3)), 0, 0, base + 4 * shift, st[2], st[3], nullptr);
    if (s == TIDE_OK) CHECK(apart && (same || !meet));  // what is accepted is safe
    // outputs behind the inputs, heads within a token's stride or tokens within a head's
    const bool behind = shift >= (tokens - 1) * st[0] + (heads - 1) * st[1] + dim;
    const bool nested = (heads == 1 || st[3] >= dim) && (tokens == 1 || st[2] >= dim) &&
                        (tokens == 1 || heads == 1 || st[2] >= (heads - 1) * st[3] + dim || st[3] >= (tokens - 1) * st[2] + dim);
    if (behind && nested) CHECK(s == TIDE_OK);
  }
  CHECK(accepted > 1000 && refused > 1000);
  std::printf("%d failures (%d accepted, %d refused)\n", failures, accepted, refused);
  return failures == 0 ? 0 : 1;
}
