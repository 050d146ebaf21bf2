// block128.cuh -- what the FP8 block-128 kernels share: the launch descriptions
// and the group table of padded 128-row blocks, built by one warp.
//
// The format ("Scaling and Optimizing Frontier Model Training": DeepSeek-V3-class
// experts, whose weights are stored this way): E4M3 codes with one fp32 scale for
// each 128 values along the contraction (activations, gradients) or for each
// 128 x 128 block (weights).
#pragma once

#include "fme_device.cuh"
#include "fme_launch.h"

namespace fme {

// Programmatic serialization: a kernel launched with it may start once the one before it in the stream
// lets it (or ends), and waits here for all of that one's writes; before this it touches no
// global memory.  Ordinary loads see those writes then, non-coherent ones (__ldg) need not: their data must not change
// while the kernel runs, so such a kernel reads what the one before it may write with ordinary loads.  The
// row-wise quantizer and the products let their successors start at once: a product sets up its barriers and
// tensor memory while the last CTAs of the kernel before it end (about 1 us of 11 and of 20 for the gradients of
// 1999 rows).
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void start_next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Groups of up to 32 at a time: lane l of the calling warp holds group g0 + l.
// Calls fn(g, first row, rows, first unit) for the lane's group, where a group of
// n rows takes ceil(n / unit) units; returns the total units, or -1 if the offsets
// do not rise from 0 to rows (offsets NULL = one group of `rows`).  The whole warp
// calls it; the table of 32 groups costs two loads and five shuffles, and the loads of 128 groups are in flight
// together (256 experts: 0.7 us sooner than 32 by 32).  Up to 32 groups go without that loop: every CTA of the quantizers
// reads the table, and its instructions cost them 1.3% there (65536 x 7168 both ways, 32 groups 291 us, without 288).
// (Ordinary loads, see above.)
template <typename Fn>
__device__ __forceinline__ int32_t scan_groups(const int32_t *offsets, int32_t num_groups, int64_t rows, int32_t unit,
                                               Fn fn) {
  const int lane = threadIdx.x & 31;
  int32_t base = 0;
  bool ok = true;
  auto load = [&](int g, int32_t &lo, int32_t &hi) {
    lo = hi = 0;
    if (g < num_groups) {
      lo = offsets ? offsets[g] : 0;
      hi = offsets ? offsets[g + 1] : static_cast<int32_t>(rows);
    }
  };
  auto groups32 = [&](int g, int32_t lo, int32_t hi) {
    if (g < num_groups && (lo > hi || lo < 0 || hi > rows || (g == 0 && lo != 0) || (g == num_groups - 1 && hi != rows)))
      ok = false;
    const int32_t units = hi > lo ? (hi - lo - 1) / unit + 1 : 0;
    int32_t incl = units;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int32_t up = __shfl_up_sync(0xFFFFFFFFu, incl, s);
      if (lane >= s) incl += up;
    }
    if (g < num_groups) fn(g, lo, hi - lo, base + incl - units);
    base += __shfl_sync(0xFFFFFFFFu, incl, 31);
  };
  if (num_groups <= 32) {
    int32_t lo, hi;
    load(lane, lo, hi);
    groups32(lane, lo, hi);
  } else {
    for (int g0 = 0; g0 < num_groups; g0 += 128) {
      int32_t lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) load(g0 + 32 * j + lane, lo[j], hi[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (g0 + 32 * j >= num_groups) break;
        groups32(g0 + 32 * j + lane, lo[j], hi[j]);
      }
    }
  }
  return __all_sync(0xFFFFFFFFu, ok) ? base : -1;
}

}  // namespace fme
