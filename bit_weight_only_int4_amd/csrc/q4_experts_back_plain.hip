// Tiles of q4_experts_back.h.
#include "q4_experts_back.h"

namespace q4 {
template hipError_t launch_back_tile<float, 64, false>(const BackParams&, hipStream_t);
template hipError_t launch_back_tile<float, 128, false>(const BackParams&, hipStream_t);
}  // namespace q4
