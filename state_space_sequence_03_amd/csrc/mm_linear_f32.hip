// Products with the linear epilogue, f32 io.
#include "mm_few.hpp"
#include "mm_parts.hpp"
#include "mm_run.hpp"

namespace m3 {

hipError_t mm_linear_f32(const MmArgs& a, const MmPlan& plan, hipStream_t s) {
  return with_act(a.act, [&](auto act) {
    return plan.tile == 0 ? mm_few_run<float, MM_LINEAR, act.value>(a, s)
                          : mm_tile_run<float, MM_PQ_K, MM_LINEAR, act.value>(a, plan, s);
  });
}

}  // namespace m3
