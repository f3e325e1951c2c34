// Shared pieces of the e4m3 and the microscaled 4-bit products: direct-to-LDS
// loads and their waits, the dealing of tiles, the host's division of K.
#pragma once

#include "pipe_device.hpp"
#include "pipe_linear.hpp"

namespace pipe {

template <int T>
struct Step {
  static constexpr int value = T;
};

__device__ __forceinline__ void dma_block_at(const uint8_t* base, uint32_t offset,
                                             uint32_t lds_base) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(offset), "s"(base), "{m0}"(lds_base)
               : "memory");
}

// Waits for the loads of stage ks of `count` in a ring of S slots, LOADS a stage
// and wave: those of younger stages may stay under way.
template <int S, int LOADS>
__device__ __forceinline__ void wait_stage(int ks, int count) {
  if (ks + S - 1 <= count)
    wait_vmcnt<(S - 2) * LOADS>();
  else
    wait_vmcnt_mul<LOADS>(count - 1 - ks);
}

template <int OUT>
struct Out16;
template <>
struct Out16<0> {
  using type = __bf16;
};
template <>
struct Out16<1> {
  using type = _Float16;
};
// Output tile and K range of a work item. Workgroups go to the 8 XCDs in turn:
// the items are dealt so that each XCD walks one contiguous run of the order,
// and the order runs down bands of 4 tile rows, column by column, so that the
// tiles an XCD holds at once share few A and B rows.
template <class P>
__device__ __forceinline__ void tile_item(const P& p, int item, int items, int& tm, int& tn,
                                          int& split) {
  constexpr int kBand = 4;
  const int per = items >> 3, odd = items & 7, xcd = item & 7;
  int q = xcd * per + min(xcd, odd) + (item >> 3);
  split = q % p.splits;
  q /= p.splits;
  const int band = kBand * p.tiles_n;
  const int first = q / band * kBand;
  const int rows = min(p.tiles_m - first, kBand);
  const int local = q % band;
  tm = first + local % rows;
  tn = local / rows;
}

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Equal shares of `steps` stages for at most `most` workgroups a tile, `least`
// stages each; no share is empty.
inline int shares(int steps, int64_t most, int least) {
  int64_t n = most < steps / least ? most : steps / least;
  if (n <= 1) return 1;
  return ceil_div(steps, ceil_div(steps, n));
}

}  // namespace pipe
