// Windowed attention, backward, fp32.
#include "attn_bwd.hpp"

namespace m3 {
template hipError_t launch_attn_bwd<float>(const AttnArgs&, hipStream_t);
}  // namespace m3
