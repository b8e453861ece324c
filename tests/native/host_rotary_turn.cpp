// Sines and cosines of libtide_step.so's rotary positions on the host, against the host library's in 80 bits.  Exit
// status 0 = all checks passed.
#include <cstdio>
#include <random>

#include "../../all_gather_placement_amd/csrc/step_device.h"
#define launch(...) hipSuccess  // only sines and cosines are looked at
#include "../../all_gather_placement_amd/csrc/step_rotary.hip"

namespace tide_step {
namespace {
[[maybe_unused]] thread_local f32x4 lds[1];
}
}  // namespace tide_step

static int failures = 0;
static double worst = 0.0;
// An fp32 value between -1 and 1 is rounded by at most 2^-25; what is rounded is off by less than 2^-35.
constexpr double kOff = 1.0 / (1 << 25) + 1.0 / (int64_t(1) << 35);

static void look(double angle) {
  float c = 0, s = 0;
  tide_step::turn(angle, &c, &s);
  const double off = std::max(std::fabs(double(c - cosl(angle))), std::fabs(double(s - sinl(angle))));
  worst = std::max(worst, off);
  if (off <= kOff) return;
  if (failures++ < 20) std::fprintf(stderr, "angle %.17g: %.9g %.9g, off by %.3g\n", angle, c, s, off);
}

int main() {
  std::mt19937_64 rng(1);
  std::uniform_real_distribution<double> unit(1.0, 2.0);
  for (int sign : {-1, 1})
    for (int e = -60; e < 64; ++e) {
      look(sign * std::ldexp(1.0, e));
      for (int i = 0; i < 3000; ++i) look(sign * std::ldexp(unit(rng), e));
    }
  look(std::ldexp(1.0, 64));
  look(-std::ldexp(1.0, 64));
  look(0.0);
  // beside multiples of an eighth of a turn, where a sine or cosine is 0 or the series change
  for (int64_t k : {1, 2, 3, 4, 5, 6, 7, 8, 1001, 1 << 20, 1 << 30, (1 << 30) + 1})
    for (int i = -3; i <= 3; ++i) look(double(k) * 0.78539816339744830962 * (1.0 + i * 0x1p-52));
  for (double far : {1e30, 3.4e38, 1e300}) {  // no place within a turn is left, but a sine and cosine are
    float c = 9, s = 9;
    tide_step::turn(far, &c, &s);
    if (!(std::fabs(c) <= 1 && std::fabs(s) <= 1)) ++failures;
  }
  for (double none : {HUGE_VAL, -HUGE_VAL, std::nan("")}) {
    float c = 9, s = 9;
    tide_step::turn(none, &c, &s);
    if (!std::isnan(c) || !std::isnan(s)) ++failures;
  }
  std::printf("%d failures, off by %.3g at most\n", failures, worst);
  return failures == 0 ? 0 : 1;
}
