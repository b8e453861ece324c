// Host code of libtide_step.so (argument checks, tables of tensors, workspace layout) under
// AddressSanitizer and UBSan.  Built with g++; the kernel launchers are stubs that walk their
// arguments as the kernels would and check them.  Exit status 0 = all checks passed.
#include <cstdint>
#include <cstdio>
#include <map>
#include <random>
#include <vector>

#include "../../all_gather_placement_amd/csrc/step_internal.h"

static int failures = 0;
#define CHECK(cond)                                                           \
  do {                                                                        \
    if (!(cond)) {                                                            \
      std::fprintf(stderr, "CHECK failed at line %d: %s\n", __LINE__, #cond); \
      ++failures;                                                             \
    }                                                                         \
  } while (0)

// elements of each (address, output) pair that the launches of a call cover
static std::map<std::pair<uintptr_t, uintptr_t>, int64_t> covered;
static int64_t partials = 0, finished = -1;

namespace tide_step {
namespace {
template <typename Table, typename Out>
void walk(const Table& t, int dtype, int grid, int batch, Out&& out) {
  CHECK(t.count <= batch && grid >= 1 && grid <= kNormMaxWgs);
  const int64_t c = norm_chunk_elems(dtype);
  for (int i = 0; i < t.count; ++i) {
    const uint32_t next = i + 1 < t.count ? t.e[i + 1].first : t.chunks;
    CHECK(next > t.e[i].first && t.e[i].last >= 1 && int64_t(t.e[i].last) <= c);
    covered[{reinterpret_cast<uintptr_t>(t.e[i].p), out(t.e[i])}] += int64_t(next - t.e[i].first - 1) * c + t.e[i].last;
  }
}
}  // namespace

int launch_norm_partial(const NormTable& t, int dtype, double*, int grid, void*) {
  walk(t, dtype, grid, kNormBatch, [](const NormEntry&) { return uintptr_t(0); });
  partials += grid;
  return 0;
}
int launch_norm_finish(const double*, int n, double*, float*, void*) {
  finished = n;
  return 0;
}
int launch_clip(const ClipTable& t, int dtype, const double*, double, float*, int grid, void*) {
  if (t.count > 0)
    walk(t, dtype, grid, kClipBatch, [](const ClipEntry& e) { return reinterpret_cast<uintptr_t>(e.out); });
  return 0;
}
int launch_layer_norm(const LayerNormArgs&, int, int, void*) { return 0; }
int layer_norm_bwd_groups(int64_t rows, int64_t, int) { return rows < 256 ? int(rows) : 256; }
int launch_layer_norm_bwd(const LayerNormBwdArgs&, int, int, void*) { return 0; }
int launch_embedding(int64_t, const void*, int, int64_t, int64_t, const void*, int, float, void*, void*) { return 0; }
int launch_embedding_bwd(const EmbeddingBwdArgs& a, int, int, void*) {
  // the workspace's parts follow each other
  CHECK(reinterpret_cast<char*>(a.sorted_token) >= reinterpret_cast<char*>(a.num_sorted) + 4);
  CHECK(a.sorted_row >= a.sorted_token + a.tokens);
  CHECK(reinterpret_cast<char*>(a.partial) >= reinterpret_cast<char*>(a.sorted_row + a.tokens));
  const int64_t used = reinterpret_cast<char*>(a.partial) - reinterpret_cast<char*>(a.num_sorted) +
                       (a.tokens + kPiece - 1) / kPiece * 2 * a.dim * 4;
  CHECK(used <= tide_embedding_bwd_workspace(a.tokens, a.vocab, a.dim));
  return 0;
}
}  // namespace tide_step

int main() {
  std::mt19937_64 rng(7);
  for (int round = 0; round < 200; ++round) {
    const int n = int(rng() % 700), dtype = int(rng() % 2), size = dtype == TIDE_BF16 ? 2 : 4;
    std::vector<const void*> grads;
    std::vector<void*> outs;
    std::vector<int64_t> numels;
    uintptr_t at = 1 << 20;
    for (int i = 0; i < n; ++i) {
      const int64_t m = rng() % 8 == 0 ? 0 : int64_t(rng() % (round % 10 == 0 ? 50000000 : 20000));
      numels.push_back(m);
      grads.push_back(reinterpret_cast<const void*>(at));
      at += uintptr_t((m + 1) * size);
      outs.push_back(round % 2 ? reinterpret_cast<void*>(at) : const_cast<void*>(grads.back()));
      at += uintptr_t((m + 1) * size);
    }
    at = (at + 4095) / 4096 * 4096;
    void* ws = reinterpret_cast<void*>(at);
    const int64_t need = tide_grad_norm_workspace(n, numels.data(), dtype);
    float* norm = reinterpret_cast<float*>(at + uintptr_t(need));
    covered.clear();
    partials = 0;
    CHECK(tide_grad_norm(n, grads.data(), numels.data(), dtype, nullptr, norm, ws, need, nullptr) == TIDE_OK);
    CHECK(finished == partials && 16 + partials * 8 <= need);
    CHECK(tide_grad_norm(n, grads.data(), numels.data(), dtype, nullptr, norm, ws, need - 16, nullptr) ==
          TIDE_ERR_INVALID);
    for (int i = 0; i < n; ++i)
      if (numels[i] > 0) CHECK((covered[{reinterpret_cast<uintptr_t>(grads[i]), 0}]) == numels[i]);
    covered.clear();
    CHECK(tide_clip_grad_norm(n, grads.data(), outs.data(), numels.data(), dtype, 1.0, nullptr, norm, ws, need,
                              nullptr) == TIDE_OK);
    for (int i = 0; i < n; ++i)
      if (numels[i] > 0)
        CHECK((covered[{reinterpret_cast<uintptr_t>(grads[i]), reinterpret_cast<uintptr_t>(outs[i])}]) == numels[i]);
    if (n > 1 && numels[0] > 0 && numels[1] > 0) {
      outs[1] = outs[0];
      CHECK(tide_clip_grad_norm(n, grads.data(), outs.data(), numels.data(), dtype, 1.0, nullptr, norm, ws, need,
                                nullptr) == TIDE_ERR_INVALID);
    }
  }
  for (int round = 0; round < 200; ++round) {
    const int64_t tokens = int64_t(rng() % 100000), vocab = 1 + int64_t(rng() % 100000), dim = 1 + int64_t(rng() % 5000);
    const int64_t need = tide_embedding_bwd_workspace(tokens, vocab, dim);
    char* base = reinterpret_cast<char*>(uintptr_t(1) << 44);
    CHECK(tide_embedding_bwd(tokens, base, TIDE_INT64, vocab, dim, base + (int64_t(1) << 36), TIDE_FP32, 1.0f, 0,
                             base + (int64_t(1) << 38), base + (int64_t(1) << 40), need, nullptr) == TIDE_OK);
  }
  std::printf("%d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
