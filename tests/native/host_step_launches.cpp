// Launches of libtide_step.so without a GPU: this program stands in for the runtime's launch functions,
// refuses what the runtime refuses, and looks at what each call launches.  Exit status 0 = all checks passed.
//
//   host_step_launches sort     table gradients up to the largest vocabulary that is accepted
//   host_step_launches columns  layer norm and its gradient up to the widest row that is accepted
//   host_step_launches far      lookups and norms up to the largest sizes that are accepted
//   host_step_launches scalars  norm, sum of squares and workspace over a gradient, an output or each other
//   host_step_launches blocks   blocks of columns of one buffer, as inputs and outputs
//   host_step_launches parts    the parts of the table gradient's workspace
//   host_step_launches failed   no kernel follows one that was not launched
//   host_step_launches stale    an error of another library's earlier call is neither reported nor cleared
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <functional>
#include <map>
#include <string>
#include <vector>

#include "../../all_gather_placement_amd/csrc/step_internal.h"

static int failures = 0;
#define CHECK(cond, ...)                                                                \
  do {                                                                                  \
    if (!(cond)) {                                                                      \
      std::fprintf(stderr, "CHECK failed at line %d: %s: ", __LINE__, #cond);           \
      std::fprintf(stderr, __VA_ARGS__);                                                \
      std::fprintf(stderr, "\n");                                                       \
      ++failures;                                                                       \
    }                                                                                   \
  } while (0)

// ---------------------------------------------------------------------------------------------
// The runtime's functions that the library calls
// ---------------------------------------------------------------------------------------------

struct Launch {
  std::string name;
  dim3 grid, block;
  hipError_t status;
  bool is(const char* kernel) const { return name.find(kernel) != std::string::npos; }
};
static std::vector<Launch> launches;
static void (*on_launch)(const Launch&, void** args) = nullptr;
static hipError_t last_error = hipSuccess;
static size_t fail_at = SIZE_MAX;  // the launch of a call that is refused

static std::map<const void*, std::string>& names() {  // the library registers before this file's statics exist
  static std::map<const void*, std::string> m;
  return m;
}
struct Config {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
};
static Config config;

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* module = nullptr;
  return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*, void*, void*, void*,
                           int*) {
  names()[host] = device;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  config = {grid, block, lds, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = config.grid;
  *block = config.block;
  *lds = config.lds;
  *stream = config.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t lds, hipStream_t) {
  // less than 2^32 threads along an axis, up to 1024 in a workgroup, 64 KiB of its memory
  const auto axis = [](unsigned g, unsigned b) { return g > 0 && b > 0 && uint64_t(g) * b < (uint64_t(1) << 32); };
  const bool ok = axis(grid.x, block.x) && axis(grid.y, block.y) && axis(grid.z, block.z) &&
                  block.x * block.y * block.z <= 1024 && grid.y <= 65535 && grid.z <= 65535 && lds <= 65536 && launches.size() != fail_at;
  Launch l{names().at(f), grid, block, ok ? hipSuccess : hipErrorInvalidConfiguration};
  if (ok && on_launch != nullptr) on_launch(l, args);
  launches.push_back(l);
  if (!ok) last_error = l.status;
  return l.status;
}
hipError_t hipGetLastError(void) {
  const hipError_t e = last_error;
  last_error = hipSuccess;
  return e;
}
}

// Made-up addresses, far apart, that are never touched.
static void* at(int k) { return reinterpret_cast<void*>(uintptr_t(k) << 50); }

static std::string describe() {
  std::string s;
  for (const Launch& l : launches)
    s += l.name.substr(0, 60) + " <" + std::to_string(l.grid.x) + "x" + std::to_string(l.grid.y) + ", " +
         std::to_string(l.block.x) + "> " + std::to_string(int(l.status)) + "; ";
  return s;
}

// ---------------------------------------------------------------------------------------------
// Checks
// ---------------------------------------------------------------------------------------------

constexpr int64_t kWorkspace = int64_t(1) << 49;

static tide_status table_gradient(int64_t tokens, int64_t vocab, int64_t dim, int dtype, int ids, int accumulate) {
  launches.clear();
  return tide_embedding_bwd(tokens, at(1), ids, vocab, dim, at(2), dtype, 1.0f, accumulate, at(3), at(4), kWorkspace,
                            nullptr);
}

// Every range of table rows is sorted by one workgroup, in as many launches as that takes.
static uint64_t sorted_ranges;
static void count_ranges(const Launch& l, void** args) {
  if (!l.is("embedding_sort")) return;
  const unsigned first = *static_cast<unsigned*>(args[1]), sorting = *static_cast<unsigned*>(args[2]);
  CHECK(first == sorted_ranges, "from range %u after %llu", first, (unsigned long long)sorted_ranges);
  CHECK(sorting <= l.grid.x, "%u of %u", sorting, l.grid.x);
  sorted_ranges += sorting;
}

static void sort() {
  const int64_t vocabs[] = {1, 255, 256, 257, 131072, 131073, 1 << 24, int64_t(1) << 27, (int64_t(1) << 27) + 1,
                            int64_t(1) << 29, int64_t(1) << 30, (int64_t(1) << 30) + 1, (int64_t(1) << 31) - 1};
  for (int64_t vocab : vocabs)
    for (int64_t tokens : {int64_t(1025), int64_t(100000), (int64_t(1) << 31) - 1})
      for (int64_t dim : {1, 2, 9, 4096})
        for (int dtype : {TIDE_BF16, TIDE_FP32})
          for (int accumulate : {0, 1}) {
            sorted_ranges = 0;
            on_launch = count_ranges;
            const tide_status s = table_gradient(tokens, vocab, dim, dtype, TIDE_INT64, accumulate);
            on_launch = nullptr;
            CHECK(s == TIDE_OK, "%lld rows, %lld tokens: %s", (long long)vocab, (long long)tokens, describe().c_str());
            const uint64_t owners = uint64_t(1) << tide_step::sort_shift(vocab);
            CHECK(sorted_ranges == std::min(owners, uint64_t(vocab)), "%lld rows: %llu ranges", (long long)vocab,
                  (unsigned long long)sorted_ranges);
          }
}

static tide_status layer_norm(int64_t rows, int64_t cols, int dtype = TIDE_BF16) {
  return tide_layer_norm(rows, cols, at(1), cols, dtype, at(2), at(3), TIDE_BF16, 1e-5f, at(4), cols,
                         static_cast<float*>(at(5)), static_cast<float*>(at(6)), nullptr);
}
static tide_status layer_norm_bwd(int64_t rows, int64_t cols, bool in_place = false, int dtype = TIDE_BF16) {
  return tide_layer_norm_bwd(rows, cols, at(1), cols, at(2), cols, dtype, at(3), TIDE_FP32, static_cast<float*>(at(4)),
                             static_cast<float*>(at(5)), in_place ? at(1) : at(6), cols, at(7), at(8), at(9), kWorkspace,
                             nullptr);
}

static void columns() {
  for (int64_t cols : {int64_t(1), int64_t(40), int64_t(40000), int64_t(1) << 25, int64_t(1) << 28,
                       (int64_t(1) << 29) - 4, int64_t(1) << 29, int64_t(1) << 30, (int64_t(1) << 31) - 1})
    for (int64_t rows : {0, 1, 16, 17, 1000})
      for (int dtype : {TIDE_BF16, TIDE_FP32}) {
        launches.clear();
        CHECK(layer_norm(rows, cols, dtype) == TIDE_OK, "%lld x %lld: %s", (long long)rows, (long long)cols,
              describe().c_str());
        launches.clear();
        CHECK(layer_norm_bwd(rows, cols, false, dtype) == TIDE_OK, "%lld x %lld: %s", (long long)rows, (long long)cols,
              describe().c_str());
      }
}

static void far() {
  const int64_t most = (int64_t(1) << 31) - 1;
  for (int64_t tokens : {int64_t(1), most})
    for (int64_t dim : {int64_t(1), int64_t(9), int64_t(512), int64_t(8191), most})
      for (int ids : {TIDE_INT32, TIDE_INT64}) {
        if (tokens > (int64_t(1) << 44) / dim) continue;
        launches.clear();
        CHECK(tide_embedding(tokens, at(1), ids, 100, dim, at(2), TIDE_BF16, 1.0f, at(3), nullptr) == TIDE_OK, "%lld x %lld: %s",
              (long long)tokens, (long long)dim, describe().c_str());
        launches.clear();
        CHECK(tide_embedding_bwd(tokens, at(1), ids, 100, dim, at(2), TIDE_BF16, 1.0f, 0, at(3), at(4), kWorkspace,
                                 nullptr) == TIDE_OK, "%lld x %lld: %s", (long long)tokens, (long long)dim, describe().c_str());
      }
  const int64_t numel = int64_t(1) << 42;
  const void* grad = at(1);
  void* out = at(1);
  for (int dtype : {TIDE_BF16, TIDE_FP32}) {
    launches.clear();
    CHECK(tide_clip_grad_norm(1, &grad, &out, &numel, dtype, 1.0, static_cast<double*>(at(2)), static_cast<float*>(at(3)),
                              at(4), kWorkspace, nullptr) == TIDE_OK, "%s", describe().c_str());
  }
}

// Refused before anything is launched, or not at all.
static void expect(bool refused, tide_status s, const char* what, int64_t where) {
  CHECK((s == TIDE_ERR_INVALID) == refused && (refused ? launches.empty() : s == TIDE_OK), "%s %lld: status %d, %zu launches",
        what, (long long)where, int(s), launches.size());
  launches.clear();
}

static void scalars() {
  // two gradients of 1000 floats, outputs elsewhere, one long list
  char* base = static_cast<char*>(at(1));
  char* far = static_cast<char*>(at(2));
  const int64_t numels[] = {1000, 1000};
  const void* grads[] = {base, base + 8192};
  void* outs[] = {base + 65536, base + 65536 + 8192};
  void* same[] = {base, base + 8192};
  const int64_t need = tide_grad_norm_workspace(2, numels, TIDE_FP32);
  const auto f64 = [](char* p) { return reinterpret_cast<double*>(p); };
  const auto f32 = [](char* p) { return reinterpret_cast<float*>(p); };
  const auto norm = [&](char* sumsq, char* value, char* ws) {
    launches.clear();
    return tide_grad_norm(2, grads, numels, TIDE_FP32, f64(sumsq), f32(value), ws, need, nullptr);
  };
  const auto clip = [&](void* const* to, char* sumsq, char* value) {
    launches.clear();
    return tide_grad_clip(2, grads, to, numels, TIDE_FP32, f64(sumsq), 1.0, f32(value), nullptr);
  };
  const auto both = [&](void* const* to, char* sumsq, char* value, char* ws) {
    launches.clear();
    return tide_clip_grad_norm(2, grads, to, numels, TIDE_FP32, 1.0, f64(sumsq), f32(value), ws, need, nullptr);
  };
  // where 4, 8 and `need` bytes lie over one of the gradients, of 4000 bytes each
  for (int64_t o : {0, 16, 3984, 8192, 8192 + 3984, 8192 + 2000 - 2000 % 16}) {
    char* p = base + o;
    expect(true, norm(nullptr, p, far), "norm over a gradient", o);
    expect(true, norm(p, nullptr, far), "sum over a gradient", o);
    expect(true, norm(nullptr, nullptr, p), "workspace over a gradient", o);
    expect(true, clip(outs, far, p), "clip: norm over a gradient", o);
    expect(false, clip(outs, p, far), "clip: the given sum may be part of a gradient that is not written", o);
    expect(true, clip(same, p, far), "clip: the given sum over an output", o);
    for (void* const* to : {outs, same}) {
      expect(true, both(to, nullptr, p, far), "norm and clip: norm over a gradient", o);
      expect(true, both(to, p, nullptr, far), "norm and clip: sum over a gradient", o);
      expect(true, both(to, nullptr, nullptr, p), "norm and clip: workspace over a gradient", o);
    }
  }
  for (int64_t o : {-64, 4000, 8192 + 4000}) {  // beside them
    char* p = base + o;
    expect(false, norm(nullptr, p, far), "norm beside a gradient", o);
    expect(false, norm(p, nullptr, far), "sum beside a gradient", o);
    expect(false, clip(outs, far, p), "clip: norm beside a gradient", o);
    expect(false, both(outs, nullptr, p, far), "norm and clip: norm beside a gradient", o);
    expect(false, both(same, p, nullptr, far), "norm and clip: sum beside a gradient", o);
  }
  expect(true, norm(base - 32, nullptr, base - need + 8), "workspace's end over a gradient", 0);
  // each other: a norm in either half of the sum of squares, either of them in the workspace
  for (int64_t o : {0, 4}) {
    expect(true, norm(far, far + o, far + 4096), "norm in the sum", o);
    expect(true, clip(outs, far, far + o), "clip: norm in the given sum", o);
    expect(true, clip(same, far, far + o), "clip in place: norm in the given sum", o);
    expect(true, both(outs, far, far + o, far + 4096), "norm and clip: norm in the sum", o);
  }
  for (int64_t o : {int64_t(0), int64_t(8), need - 8}) {
    expect(true, norm(far + o, nullptr, far), "sum in the workspace", o);
    expect(true, norm(nullptr, far + o, far), "norm in the workspace", o);
    expect(true, both(same, far + o, nullptr, far), "norm and clip: sum in the workspace", o);
    expect(true, both(outs, nullptr, far + o, far), "norm and clip: norm in the workspace", o);
  }
  expect(false, norm(far, far + 8, far + 16), "next to each other", 0);
  expect(false, clip(outs, far, far + 8), "next to each other", 1);
  expect(false, both(same, far, far + 8, far + 16), "next to each other", 2);
  const int64_t none[] = {0, 0};
  expect(false, tide_grad_norm(2, grads, none, TIDE_FP32, f64(base), f32(base + 8192), far, need, nullptr),
         "gradients without elements lie over nothing", 0);
}

static void blocks() {
  constexpr int64_t R = 5, S = 256;
  char* base = static_cast<char*>(at(1));
  // bf16 rows of `cols` elements from column `c` of a buffer with rows of S elements
  const auto ln = [&](int64_t cols, int64_t xc, int64_t yc, int64_t ys, char* weight, char* mean) {
    launches.clear();
    return tide_layer_norm(R, cols, base + 2 * xc, S, TIDE_BF16, weight, nullptr, TIDE_BF16, 1e-5f, base + 2 * yc, ys,
                           reinterpret_cast<float*>(mean), nullptr, nullptr);
  };
  const auto bwd = [&](int64_t cols, int64_t dyc, int64_t xc, int64_t dxc) {
    launches.clear();
    return tide_layer_norm_bwd(R, cols, base + 2 * dyc, S, base + 2 * xc, S, TIDE_BF16, nullptr, TIDE_BF16,
                               static_cast<float*>(at(2)), static_cast<float*>(at(3)), base + 2 * dxc, S, at(4), at(5), at(6),
                               kWorkspace, nullptr);
  };
  for (int64_t cols : {1, 7, 64, 128})
    for (int64_t xc : {0, 3, 100})
      for (int64_t yc = 0; yc < 2 * S; ++yc) {
        // from element to element: the buffer's elements that either writes or reads
        std::vector<int> used(size_t(R + 4) * S, 0);
        for (int64_t r = 0; r < R; ++r)
          for (int64_t c = 0; c < cols; ++c) used[size_t(xc + r * S + c)] = 1;
        bool meet = false;
        for (int64_t r = -1; r <= R; ++r)  // rows before and after count: a block is a block of all rows
          for (int64_t c = 0; c < cols; ++c) {
            const int64_t e = yc % S + r * S + c;
            if (e >= 0) meet |= used[size_t(e)] != 0;
          }
        expect(meet, ln(cols, xc, yc, S, nullptr, nullptr), "blocks", yc);
        expect(meet, bwd(cols, 2 * S * R, xc, yc), "blocks of x and dx", yc);
        if (yc != xc && yc < S) expect(meet, bwd(cols, yc, 2 * S * R, xc), "blocks of dy and dx", yc);
      }
  expect(false, bwd(64, 0, 64, 128), "three blocks", 0);
  expect(false, bwd(64, 0, 64, 0), "three blocks, in place", 0);
  expect(true, ln(64, 0, 100, S + 8, nullptr, nullptr), "other strides", 0);
  // vectors within a row's gap, over its end, over the next row's start, longer than the gap
  expect(false, ln(64, 0, 64, S, base + 2 * 128, nullptr), "weight in the gap", 0);
  expect(false, ln(64, 0, 64, S, base + 2 * (S - 64), nullptr), "weight at the gap's end", 0);
  expect(true, ln(64, 0, 64, S, base + 2 * 127, nullptr), "weight over y", 0);
  expect(false, ln(64, 0, 64, S, base + 2 * (S - 63), nullptr), "weight over x: both are read", 0);
  expect(true, ln(64, 64, 0, S, base + 2 * (S - 63), nullptr), "weight over the next row of y", 0);
  expect(false, ln(64, 0, 64, S, nullptr, base + 2 * 128), "mean in the gap", 0);
  expect(true, ln(64, 0, 64, S, nullptr, base + 2 * (S - 8)), "mean over x", 0);
}

// The workspace's parts lie one behind the other within the bytes that are asked for.
static int64_t workspace_bytes;
static int looked_at;
static void check_parts(const Launch& l, void** args) {
  if (!l.is("embedding_sort") && !l.is("embedding_sum") && !l.is("embedding_join")) return;
  ++looked_at;
  const auto& a = *static_cast<const tide_step::EmbeddingBwdArgs*>(args[0]);
  const int64_t pieces = (a.tokens + tide_step::kPiece - 1) / tide_step::kPiece;
  struct Part {
    const void* p;
    int64_t bytes, align;
  };
  const Part parts[] = {{a.num_sorted, 3 * 4, 4},
                        {a.sorted_token, a.tokens * 4, 4},
                        {a.sorted_row, a.tokens * 4, 4},
                        {a.last_piece, pieces * 4, 4},
                        {a.runs, pieces * int64_t(sizeof(tide_step::EmbeddingRun)), 4},
                        {a.partial, pieces * 2 * a.dim * 4, 16}};
  uintptr_t end = reinterpret_cast<uintptr_t>(at(4));
  for (const Part& p : parts) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p.p);
    CHECK(lo >= end && lo % uintptr_t(p.align) == 0, "part %d of %lld tokens of %lld", int(&p - parts), (long long)a.tokens,
          (long long)a.dim);
    end = lo + uintptr_t(p.bytes);
  }
  CHECK(end <= reinterpret_cast<uintptr_t>(at(4)) + uintptr_t(workspace_bytes), "%lld tokens of %lld", (long long)a.tokens,
        (long long)a.dim);
}

static void parts() {
  for (int64_t tokens : {513, 1025, 1056, 1057, 99999, 1 << 24})
    for (int64_t dim : {1, 3, 8, 1001, 4096})
      for (int64_t vocab : {int64_t(1), int64_t(20011), int64_t(1) << 30}) {
        workspace_bytes = tide_embedding_bwd_workspace(tokens, vocab, dim);
        on_launch = check_parts;
        launches.clear();
        CHECK(tide_embedding_bwd(tokens, at(1), TIDE_INT64, vocab, dim, at(2), TIDE_FP32, 1.0f, 0, at(3), at(4),
                                 workspace_bytes, nullptr) == TIDE_OK, "%s", describe().c_str());
        on_launch = nullptr;
      }
  CHECK(looked_at > 100, "%d", looked_at);
}

// Every operator in every sequence of launches.
struct Call {
  const char* name;
  std::function<tide_status()> run;
};
static std::vector<Call> calls() {
  std::vector<Call> c;
  static std::vector<const void*> grads;
  static std::vector<void*> outs;
  static std::vector<int64_t> few(300, 1), some(100, 100000), many(300, 1000000);
  if (grads.empty())
    for (int i = 0; i < 300; ++i) {
      grads.push_back(reinterpret_cast<void*>((uintptr_t(1) << 40) + (uintptr_t(i) << 30)));
      outs.push_back(const_cast<void*>(grads.back()));
    }
  double* sumsq = static_cast<double*>(at(2));
  float* norm = static_cast<float*>(at(3));
  for (const std::vector<int64_t>* n : {&few, &some, &many}) {
    const int32_t count = int32_t(n->size());
    c.push_back({"grad_norm", [=] {
                   return tide_grad_norm(count, grads.data(), n->data(), TIDE_BF16, sumsq, norm, at(4), kWorkspace, nullptr);
                 }});
    c.push_back({"grad_clip", [=] {
                   return tide_grad_clip(count, grads.data(), outs.data(), n->data(), TIDE_FP32, sumsq, 1.0, norm, nullptr);
                 }});
    c.push_back({"clip_grad_norm", [=] {
                   return tide_clip_grad_norm(count, grads.data(), outs.data(), n->data(), TIDE_FP32, 1.0, sumsq, norm,
                                              at(4), kWorkspace, nullptr);
                 }});
  }
  for (int64_t cols : {40, 4096, 16384, 40000})
    for (int64_t rows : {3, 5000}) {
      c.push_back({"layer_norm", [=] { return layer_norm(rows, cols); }});
      for (bool in_place : {false, true})
        c.push_back({"layer_norm_bwd", [=] { return layer_norm_bwd(rows, cols, in_place); }});
    }
  for (int64_t tokens : {40, 600, 5000})
    for (int64_t vocab : {int64_t(100), int64_t(200000), (int64_t(1) << 31) - 1}) {
      c.push_back({"embedding", [=] {
                     return tide_embedding(tokens, at(1), TIDE_INT32, vocab, 700, at(2), TIDE_FP32, 1.0f, at(3), nullptr);
                   }});
      for (int accumulate : {0, 1})
        c.push_back({"embedding_bwd", [=] { return table_gradient(tokens, vocab, 700, TIDE_FP32, TIDE_INT32, accumulate); }});
    }
  return c;
}

static void failed() {
  size_t most = 0;
  for (const Call& c : calls()) {
    launches.clear();
    CHECK(c.run() == TIDE_OK, "%s: %s", c.name, describe().c_str());
    const size_t n = launches.size();
    most = std::max(most, n);
    for (size_t k = 0; k < n; ++k) {
      launches.clear();
      fail_at = k;
      CHECK(c.run() == TIDE_ERR_HIP, "%s", c.name);
      fail_at = SIZE_MAX;
      CHECK(launches.size() == k + 1, "%s goes on after launch %zu of %zu: %s", c.name, k + 1, n, describe().c_str());
      CHECK(tide_step_last_hip_error() == hipErrorInvalidConfiguration, "%s", c.name);
      CHECK(last_error == hipSuccess, "%s leaves its own error", c.name);
      last_error = hipSuccess;
    }
  }
  CHECK(most >= 5, "%zu", most);  // zeros, two sorts, sums, join
}

static void stale() {
  for (const Call& c : calls()) {
    launches.clear();
    last_error = hipErrorNotReady;
    CHECK(c.run() == TIDE_OK, "%s reports another call's error", c.name);
    CHECK(last_error == hipErrorNotReady, "%s clears another call's error", c.name);
    last_error = hipSuccess;
  }
}

int main(int argc, char** argv) {
  const std::string what = argc > 1 ? argv[1] : "";
  if (what == "sort") sort();
  else if (what == "columns") columns();
  else if (what == "far") far();
  else if (what == "scalars") scalars();
  else if (what == "blocks") blocks();
  else if (what == "parts") parts();
  else if (what == "failed") failed();
  else if (what == "stale") stale();
  else ++failures;
  std::printf("%d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
