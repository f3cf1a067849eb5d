// Windowed attention, forward, fp32.
#include "attn_fwd.hpp"

namespace m3 {
template hipError_t launch_attn_fwd<float>(const AttnArgs&, hipStream_t);
}  // namespace m3
