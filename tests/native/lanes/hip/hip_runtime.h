// Stands in for the HIP runtime so that kernels compile for the host and run there, a fiber for each lane.
//
// A lane runs until it meets another: at a barrier, or where lanes of a wave exchange values.  Between two such
// places lanes run one after another, in an order that the program chooses, so what passes must hold for any order
// that the GPU may take between them, and for more: there, lanes of a wave take each instruction together.
#pragma once

#include <stddef.h>
#include <stdint.h>
#include <string.h>
#include <ucontext.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <memory>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __shared__ thread_local
#define __launch_bounds__(...)

struct dim3 {
  unsigned x, y, z;
  dim3(unsigned a = 1, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {}
};
typedef int hipError_t;
typedef void* hipStream_t;
enum { hipSuccess = 0 };
inline hipError_t hipGetLastError() { return hipSuccess; }
inline hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) { std::abort(); }

inline dim3 threadIdx, blockIdx, blockDim, gridDim;

namespace lanes {

struct Lane {
  ucontext_t context;
  std::unique_ptr<char[]> stack;
  bool done = false;
  unsigned meetings = 0, barriers = 0;  // reached so far
  uint32_t given[2] = {0, 0};           // to the meetings of even and odd numbers
};
inline std::vector<Lane> group;
inline ucontext_t scheduler;
inline unsigned current = 0, moves = 0;
inline bool backwards = false;  // the lanes' order
inline std::function<void()> kernel;

inline void rest() { swapcontext(&group[current].context, &scheduler); }
template <typename Reached>
void wait_for(unsigned from, unsigned to, Reached&& reached) {
  ++moves;
  for (bool all = false; !all;) {
    rest();  // also the last one, so that lanes go on in their order
    all = true;
    for (unsigned i = from; i < to && i < group.size(); ++i) all &= group[i].done || reached(group[i]);
  }
  ++moves;
}
inline unsigned lane() { return current & 63; }
// Gives v to the lanes of the wave; what they gave is then read by its place.
struct Meeting {
  unsigned first, which, number;
  explicit Meeting(uint32_t v) : first(current & ~63u) {
    Lane& me = group[current];
    const unsigned n = number = ++me.meetings;
    which = n & 1;
    me.given[which] = v;
    wait_for(first, first + 64, [n](const Lane& l) { return l.meetings >= n; });
  }
  uint32_t operator[](unsigned i) const { return group[first + i].given[which]; }
  bool here(unsigned i) const { return first + i < group.size() && group[first + i].meetings >= number; }
};
inline uint64_t ballot(bool v) {
  const Meeting m(v);
  uint64_t r = 0;
  for (unsigned i = 0; i < 64; ++i)
    if (m.here(i) && m[i]) r |= uint64_t(1) << i;
  return r;
}
// The lane that a data-parallel move reads, -1 for none.
inline int moved_from(int control, int i) {
  const int row = i & ~15;
  if (control < 0x100) return (i & ~3) | (control >> (2 * (i & 3)) & 3);
  if (control > 0x110 && control < 0x120) return (i & 15) >= control - 0x110 ? i - (control - 0x110) : -1;
  if (control == 0x140) return row | (15 - (i & 15));
  if (control == 0x141) return (i & ~7) | (7 - (i & 7));
  if (control == 0x142) return row > 0 ? row - 1 : -1;
  if (control == 0x143) return i >= 32 ? 31 : -1;
  std::abort();
}
inline int move(int old, int v, int control, int rows, int, bool) {
  const Meeting m(static_cast<uint32_t>(v));
  const int i = int(lane()), from = moved_from(control, i);
  return from >= 0 && (rows >> (i >> 4) & 1) ? int(m[unsigned(from)]) : old;
}
struct Pair {
  uint32_t v[2];
  uint32_t operator[](int i) const { return v[i]; }
};
inline Pair swapped(uint32_t v, unsigned distance) {
  const Meeting m(v);
  return {{m[lane() & ~distance], m[lane() | distance]}};
}
inline double shuffle_xor(double v, int mask) {
  uint64_t bits;
  memcpy(&bits, &v, 8);
  const Meeting low(static_cast<uint32_t>(bits));
  const uint64_t from_low = low[lane() ^ unsigned(mask)];
  const Meeting high(static_cast<uint32_t>(bits >> 32));
  bits = uint64_t(high[lane() ^ unsigned(mask)]) << 32 | from_low;
  memcpy(&v, &bits, 8);
  return v;
}
inline void barrier() {
  const unsigned n = ++group[current].barriers;
  wait_for(0, unsigned(group.size()), [n](const Lane& l) { return l.barriers >= n; });
}

inline void enter() {
  kernel();
  group[current].done = true;
  ++moves;
  rest();
}
inline void run(dim3 grid, unsigned threads, std::function<void()> call) {
  constexpr size_t kStack = 1 << 16;
  kernel = std::move(call);
  gridDim = grid;
  blockDim = dim3(threads);
  for (unsigned y = 0; y < grid.y; ++y)
    for (unsigned x = 0; x < grid.x; ++x) {
      blockIdx = dim3(x, y);
      group = std::vector<Lane>(threads);
      for (Lane& l : group) {
        l.stack.reset(new char[kStack]);
        getcontext(&l.context);
        l.context.uc_stack.ss_sp = l.stack.get();
        l.context.uc_stack.ss_size = kStack;
        l.context.uc_link = nullptr;
        makecontext(&l.context, enter, 0);
      }
      for (bool left = true; left;) {
        const unsigned before = moves;
        left = false;
        for (unsigned k = 0; k < threads; ++k) {
          current = backwards ? threads - 1 - k : k;
          if (group[current].done) continue;
          threadIdx = dim3(current);
          swapcontext(&scheduler, &group[current].context);
          left |= !group[current].done;
        }
        if (left && moves == before) {
          std::fprintf(stderr, "lanes wait for each other\n");
          std::abort();
        }
      }
    }
}

template <typename To, typename From>
To bits_of(From v) {
  static_assert(sizeof(To) == sizeof(From), "");
  To r;
  memcpy(&r, &v, sizeof(r));
  return r;
}

}  // namespace lanes

#define __syncthreads() lanes::barrier()
#define __ballot(v) lanes::ballot((v) != 0)
#define __shfl_xor(v, mask, width) lanes::shuffle_xor(v, mask)
#define __umulhi(a, b) uint32_t(uint64_t(uint32_t(a)) * uint32_t(b) >> 32)
#define __ffsll(v) __builtin_ffsll(v)
#define __clzll(v) __builtin_clzll(v)
#define __uint_as_float(v) lanes::bits_of<float>(uint32_t(v))
#define __int_as_float(v) lanes::bits_of<float>(int32_t(v))
#define __float_as_uint(v) lanes::bits_of<uint32_t>(float(v))
#define __float_as_int(v) lanes::bits_of<int32_t>(float(v))
#define __HIP_MEMORY_SCOPE_WORKGROUP 0
#define __hip_atomic_load(p, order, scope) (*(p))
#define __hip_atomic_store(p, v, order, scope) (void)(*(p) = (v))
#define __builtin_amdgcn_readfirstlane(v) int(v)  // of a value that is the wave's
#define __builtin_amdgcn_sched_barrier(v) (void)(v)
#define __builtin_amdgcn_update_dpp lanes::move
#define __builtin_amdgcn_permlane16_swap(a, b, c, d) lanes::swapped(a, 16)
#define __builtin_amdgcn_permlane32_swap(a, b, c, d) lanes::swapped(a, 32)
#define __builtin_amdgcn_sbfe(v, at, bits) (int(unsigned(v) << (32 - (at) - (bits))) >> (32 - (bits)))
#define __builtin_amdgcn_mbcnt_lo(m, v) ((v) + __builtin_popcount(unsigned(m) & unsigned((uint64_t(1) << (lanes::lane() < 32 ? lanes::lane() : 32)) - 1)))
#define __builtin_amdgcn_mbcnt_hi(m, v) ((v) + __builtin_popcount(unsigned(m) & (lanes::lane() < 32 ? 0u : unsigned((uint64_t(1) << (lanes::lane() - 32)) - 1))))
template <typename T>
T atomicAdd(T* p, T v) {
  const T old = *p;
  *p = old + v;
  return old;
}
