// Launches of the tiled products.
#pragma once

#include "mm_wide.hpp"

namespace m3 {

template <typename T, int EPI, int ACT, int TILE>
void mm_join_launch(const MmArgs& a, const MmPlan& pl, hipStream_t s) {
  const int cut = pl.ntm * pl.ntn - pl.full;
  if (cut == 0) return;
  constexpr int pieces = TILE / 64 * (EPI == MM_GATED ? TILE / 128 : TILE / 64);
  hipLaunchKernelGGL((mm_join_kernel<T, EPI, ACT, TILE, TILE>), dim3((unsigned)(cut * pieces)), dim3(256), 0, s, a, pl);
}

template <typename T, int LAYOUT, int EPI, int ACT>
hipError_t mm_tile_run(const MmArgs& a, const MmPlan& pl, hipStream_t s) {
  const int room = mm_room(pl.tile);
  const dim3 grid((unsigned)(pl.items < room ? pl.items : room)), blk(256);
  if (pl.tile == 256) {
    hipLaunchKernelGGL((mm_wide_kernel<T, LAYOUT, EPI, ACT>), grid, blk, 0, s, a, pl);
    mm_join_launch<T, EPI, ACT, 256>(a, pl, s);
  } else if (pl.tile == 128) {
    hipLaunchKernelGGL((mm_tile_kernel<T, LAYOUT, EPI, ACT, 128, 128>), grid, blk, 0, s, a, pl);
    mm_join_launch<T, EPI, ACT, 128>(a, pl, s);
  } else {
    return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace m3
