// Tiles of q4_experts_back.h whose row operand is complete in memory.
#include "q4_experts_back.h"

namespace q4 {
template hipError_t launch_back_direct<64>(const BackParams&, hipStream_t);
template hipError_t launch_back_direct<128>(const BackParams&, hipStream_t);
}  // namespace q4
