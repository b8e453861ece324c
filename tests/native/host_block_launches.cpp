// Launches of the block operators of libtide_step.so without a GPU: this program stands in for the runtime's launch
// functions, refuses what the runtime refuses, and looks at what each call launches.  Exit status 0 = all checks passed.
//
//   host_block_launches far      sizes up to the largest that are accepted
//   host_block_launches turns    rotary launches: every token in one of them, once
//   host_block_launches failed   no kernel follows one that was not launched
#include <hip/hip_runtime_api.h>

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

static int32_t* ints(int k) { return static_cast<int32_t*>(at(k)); }
constexpr int64_t kMost = (int64_t(1) << 31) - 1;
static const char* shown() {
  static std::string s;
  s = describe();
  return s.c_str();
}

static tide_status sort(int64_t tokens, int choices, int experts, int align, int64_t more = 0) {
  launches.clear();
  const int64_t rows = tide_expert_rows(tokens, choices, experts, align);
  return tide_expert_sort(tokens, choices, at(1), TIDE_INT64, experts, align, ints(2), ints(3), rows + more, ints(4), at(5),
                          int64_t(1) << 49, nullptr);
}
static tide_status rotary(int64_t tokens, int64_t heads, int dim, int pairs, int pairing, int dtype, bool in_place = false) {
  launches.clear();
  const int32_t sections[] = {pairs};
  return tide_rotary(tokens, heads, dim, at(1), heads * dim, dim, dtype, at(2), TIDE_INT32, 1, sections,
                     static_cast<double*>(at(3)), pairing, 0, in_place ? at(1) : at(4), heads * dim, dim, nullptr);
}

static void far() {
  for (int experts : {1, 2, 100, 128, 512, 513, 1023, 1025, 2047, 2048})
    for (int64_t tokens : {int64_t(0), int64_t(1), int64_t(500), int64_t(4097), int64_t(1) << 20, (int64_t(1) << 25) - 1})
      for (int choices : {1, 64})
        for (int align : {1, 128}) {
          if (tide_expert_rows(tokens, choices, experts, align) < 0) continue;
          CHECK(sort(tokens, choices, experts, align) == TIDE_OK, "%lld x %d of %d: %s", (long long)tokens, choices, experts, shown());
          CHECK(!launches.empty() && launches.size() <= 2, "%s", shown());
        }
  CHECK(sort(kMost, 1, 2048, 1) == TIDE_OK && sort(1, 1, 1, 1, kMost - 1) == TIDE_OK, "%s", shown());
  for (int64_t tokens : {int64_t(0), int64_t(1), int64_t(1) << 20, kMost / 64})
    for (int choices : {1, 2, 3, 5, 64})
      for (int64_t dim : {int64_t(1), int64_t(3), int64_t(4), int64_t(100), int64_t(129), int64_t(2048), int64_t(8192), kMost})
        for (int64_t rows : {int64_t(0), int64_t(1), tokens * choices, kMost})
          for (int dtype : {TIDE_BF16, TIDE_FP32}) {
            if (tokens > (int64_t(1) << 44) / dim || rows > (int64_t(1) << 44) / dim) continue;
            launches.clear();
            CHECK(tide_expert_dispatch(tokens, choices, dim, at(1), dim, dtype, ints(2), ints(3), rows, at(8), dim, nullptr) == TIDE_OK, "%s", shown());
            CHECK((rows > 0) == (launches.size() == 1), "%s", shown());
            launches.clear();
            CHECK(tide_expert_combine(tokens, choices, dim, at(8), dim, rows, dtype, at(4), dtype, ints(2), at(1), dim, nullptr) == TIDE_OK, "%s", shown());
            CHECK((tokens > 0) == (launches.size() == 1), "%s", shown());
            launches.clear();
            CHECK(tide_expert_combine_bwd(tokens, choices, dim, at(1), dim, at(8), dim, rows, dtype, at(4), TIDE_FP32, ints(2),
                                          ints(3), at(12), dim, at(5), nullptr) == TIDE_OK, "%s", shown());
            CHECK((tokens + rows > 0) == (launches.size() == 1), "%s", shown());
          }
  for (int64_t cols : {int64_t(1), int64_t(7), int64_t(4096), kMost, int64_t(1) << 44})
    for (int64_t rows : {int64_t(0), int64_t(1), int64_t(1) << 20, kMost})
      for (int gap : {0, 1})
        for (int64_t offset : {int64_t(0), int64_t(5), (int64_t(1) << 62) - (int64_t(1) << 44)}) {
          if (rows > (int64_t(1) << 44) / (cols + gap)) continue;
          launches.clear();
          CHECK(tide_dropout(rows, cols, at(1), cols + gap, TIDE_BF16, 0.5, 1, nullptr, offset, at(2), cols, at(3), cols, nullptr) == TIDE_OK, "%s", shown());
          CHECK((rows > 0) == (launches.size() == 1), "%s", shown());
        }
}

// Every token of a call is in one launch, and a workgroup has room for its items.
static int64_t next_token, call_tokens, call_items;
static int items_of_thread;
static void count_tokens(const Launch& l, void** args) {
  if (!l.is("rotary")) return;
  struct {
    int64_t first;
    int32_t tokens, heads;
  } g;
  std::memcpy(&g, args[1], sizeof(g));
  CHECK(g.first == next_token, "token %lld after %lld", (long long)g.first, (long long)next_token);
  CHECK(g.tokens >= 1 && g.heads >= 1, "%d tokens of %d heads", g.tokens, g.heads);
  next_token += int64_t(l.grid.x) * g.tokens;
  CHECK(next_token - call_tokens < g.tokens || l.grid.x == (1u << 21), "%s", shown());
  CHECK(int64_t(g.tokens) * g.heads * call_items <= int64_t(l.block.x) * items_of_thread, "%d tokens of %d heads of %lld items, %u threads",
        g.tokens, g.heads, (long long)call_items, l.block.x);
}
static void turns() {
  for (int64_t tokens : {int64_t(1), int64_t(2), int64_t(63), int64_t(5000), int64_t(1) << 22, kMost})
    for (int64_t heads : {int64_t(1), int64_t(2), int64_t(5), int64_t(40), int64_t(1000), int64_t(65535)})
      for (int dim : {2, 3, 8, 40, 64, 100, 128, 576, 1023, 1024})
        for (int pairs : {1, dim / 2, dim / 4})
          for (int pairing : {TIDE_ROTARY_HALVES, TIDE_ROTARY_NEIGHBOURS})
            for (int dtype : {TIDE_BF16, TIDE_FP32})
              for (bool in_place : {false, true}) {
                if (pairs < 1 || 2 * pairs > dim || heads > (int64_t(1) << 44) / dim / tokens) continue;
                const int e = dtype == TIDE_BF16 ? 8 : 4, turned = pairing == TIDE_ROTARY_HALVES ? pairs : 2 * pairs;
                call_tokens = tokens;
                call_items = (turned + e - 1) / e + (in_place ? 0 : (dim - 2 * pairs + e - 1) / e);
                items_of_thread = pairing == TIDE_ROTARY_HALVES ? 2 : 4;
                next_token = 0;
                on_launch = count_tokens;
                const tide_status s = rotary(tokens, heads, dim, pairs, pairing, dtype, in_place);
                on_launch = nullptr;
                CHECK(s == TIDE_OK && next_token >= tokens, "%lld x %lld x %d: %s", (long long)tokens, (long long)heads, dim, shown());
              }
}

static void failed() {
  CHECK(sort(100000, 8, 128, 16) == TIDE_OK && launches.size() == 2, "%s", shown());
  for (size_t at_launch : {0, 1}) {
    fail_at = at_launch;
    CHECK(sort(100000, 8, 128, 16) == TIDE_ERR_HIP, "%s", shown());
    CHECK(launches.size() == at_launch + 1 && tide_step_last_hip_error() == hipErrorInvalidConfiguration, "%s", shown());
    fail_at = SIZE_MAX;
  }
  CHECK(rotary(kMost, 128, 32, 16, 0, TIDE_FP32) == TIDE_OK && launches.size() > 2, "%s", shown());
  fail_at = 1;
  CHECK(rotary(kMost, 128, 32, 16, 0, TIDE_FP32) == TIDE_ERR_HIP && launches.size() == 2, "%s", shown());
  fail_at = 0;
  launches.clear();
  CHECK(tide_dropout(1, 100, at(1), 100, TIDE_BF16, 0.5, 1, nullptr, 0, nullptr, 0, at(3), 100, nullptr) == TIDE_ERR_HIP, "%s", shown());
  launches.clear();
  CHECK(tide_expert_dispatch(4, 1, 8, at(1), 8, TIDE_BF16, ints(2), ints(3), 4, at(8), 8, nullptr) == TIDE_ERR_HIP, "%s", shown());
  fail_at = SIZE_MAX;
  CHECK(sort(100, 8, 128, 16) == TIDE_OK && launches.size() == 1, "%s", shown());
}

int main(int argc, char** argv) {
  const std::string what = argc > 1 ? argv[1] : "";
  if (what == "far") far();
  else if (what == "turns") turns();
  else if (what == "failed") failed();
  else ++failures;
  std::printf("%d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
