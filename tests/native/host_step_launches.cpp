// Launches of libtide_step.so without a GPU: this program stands in for the runtime's launch functions,
// refuses what the runtime refuses, and looks at what each call launches.  Exit status 0 = all checks passed.
//
//   host_step_launches sort     table gradients up to the largest vocabulary that is accepted
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstring>
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
                  block.x * block.y * block.z <= 1024 && grid.y <= 65535 && grid.z <= 65535 && lds <= 65536;
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

int main(int argc, char** argv) {
  const std::string what = argc > 1 ? argv[1] : "";
  if (what == "sort") sort();
  else ++failures;
  std::printf("%d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
