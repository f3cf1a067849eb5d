// Windowed attention, forward, bf16.
#include "attn_fwd.hpp"

namespace m3 {
template hipError_t launch_attn_fwd<bf16_t>(const AttnArgs&, hipStream_t);
}  // namespace m3
