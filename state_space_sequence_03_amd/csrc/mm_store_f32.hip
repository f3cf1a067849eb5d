// Products of the backward (no epilogue), f32 io.
#include "mm_parts.hpp"
#include "mm_run.hpp"

namespace m3 {

hipError_t mm_store_f32(MmLayout layout, const MmArgs& a, const MmPlan& plan, hipStream_t s) {
  if (layout == MM_P_K) return mm_tile_run<float, MM_P_K, MM_STORE, ACT_NONE>(a, plan, s);
  if (layout == MM_NONE_K) return mm_tile_run<float, MM_NONE_K, MM_STORE, ACT_NONE>(a, plan, s);
  return hipErrorInvalidValue;
}

hipError_t mm_pair_f32(const MmArgs& a, const MmPlan& pa, const MmArgs& b, const MmPlan& pb, hipStream_t s) {
  return mm_pair_run<float>(a, pa, b, pb, s);
}

}  // namespace m3
