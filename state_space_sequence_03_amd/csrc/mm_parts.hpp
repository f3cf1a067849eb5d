// The products' instances, one translation unit each.
#pragma once

#include "m3_launch.hpp"

namespace m3 {

hipError_t mm_store_bf16(MmLayout layout, const MmArgs& a, const MmPlan& plan, hipStream_t s);
hipError_t mm_store_f32(MmLayout layout, const MmArgs& a, const MmPlan& plan, hipStream_t s);
hipError_t mm_linear_bf16(const MmArgs& a, const MmPlan& plan, hipStream_t s);
hipError_t mm_linear_f32(const MmArgs& a, const MmPlan& plan, hipStream_t s);
hipError_t mm_gated_bf16(const MmArgs& a, const MmPlan& plan, hipStream_t s);
hipError_t mm_gated_f32(const MmArgs& a, const MmPlan& plan, hipStream_t s);
hipError_t mm_pair_bf16(const MmArgs& a, const MmPlan& pa, const MmArgs& b, const MmPlan& pb, hipStream_t s);
hipError_t mm_pair_f32(const MmArgs& a, const MmPlan& pa, const MmArgs& b, const MmPlan& pb, hipStream_t s);

}  // namespace m3
