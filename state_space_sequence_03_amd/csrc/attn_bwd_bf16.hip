// Windowed attention, backward, bf16.
#include "attn_bwd.hpp"

namespace m3 {
template hipError_t launch_attn_bwd<bf16_t>(const AttnArgs&, hipStream_t);
}  // namespace m3
