// Tiles of q4_experts_back.h.
#include "q4_experts_back.h"

namespace q4 {
template hipError_t launch_back_tile<_Float16, 64, true>(const BackParams&, hipStream_t);
template hipError_t launch_back_tile<_Float16, 128, true>(const BackParams&, hipStream_t);
}  // namespace q4
