// Launches of the tiled products.
#pragma once

#include "mm_wide.hpp"

namespace m3 {

template <typename T, int EPI, int ACT, int BM, int BN>
void mm_join_launch(const MmArgs& a, const MmPlan& pl, hipStream_t s) {
  const int cut = pl.ntm * pl.ntn - pl.full;
  if (cut == 0) return;
  constexpr int pieces = BM / 64 * (EPI == MM_GATED ? BN / 128 : BN / 64);
  hipLaunchKernelGGL((mm_join_kernel<T, EPI, ACT, BM, BN>), dim3((unsigned)(cut * pieces)), dim3(256), 0, s, a, pl);
}

template <typename T, int LAYOUT, int EPI, int ACT>
hipError_t mm_tile_run(const MmArgs& a, const MmPlan& pl, hipStream_t s) {
  const int room = mm_room(pl.tile);
  const dim3 grid((unsigned)(pl.items < room ? pl.items : room)), blk(256);
  const bool alone = pl.items <= 256;
  constexpr int B64 = EPI == MM_GATED ? 128 : 64, N64 = EPI == MM_GATED ? 3 : 4;
  if (pl.tile == 256) {
    hipLaunchKernelGGL((mm_wide_kernel<T, LAYOUT, EPI, ACT>), grid, blk, 0, s, a, pl);
    mm_join_launch<T, EPI, ACT, 256, 256>(a, pl, s);
  } else if (pl.tile == 128) {
    if (alone) hipLaunchKernelGGL((mm_tile_kernel<T, LAYOUT, EPI, ACT, 128, 128, 4, 1>), grid, blk, 0, s, a, pl);
    else hipLaunchKernelGGL((mm_tile_kernel<T, LAYOUT, EPI, ACT, 128, 128, 2, 2>), grid, blk, 0, s, a, pl);
    mm_join_launch<T, EPI, ACT, 128, 128>(a, pl, s);
  } else if (pl.tile == 64) {
    if (alone) hipLaunchKernelGGL((mm_tile_kernel<T, LAYOUT, EPI, ACT, 64, B64, 2 * N64, 1>), grid, blk, 0, s, a, pl);
    else hipLaunchKernelGGL((mm_tile_kernel<T, LAYOUT, EPI, ACT, 64, B64, N64, 2>), grid, blk, 0, s, a, pl);
    mm_join_launch<T, EPI, ACT, 64, B64>(a, pl, s);
  } else {
    return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <typename T>
hipError_t mm_pair_run(const MmArgs& a, const MmPlan& pa, const MmArgs& b, const MmPlan& pb, hipStream_t s) {
  // each product's blocks start on the first XCD
  const int na = (pa.items + 7) / 8 * 8;
  hipLaunchKernelGGL((mm_pair_kernel<T>), dim3((unsigned)(na + pb.items)), dim3(256), 0, s, a, pa, b, pb, na);
  return hipGetLastError();
}

}  // namespace m3
