// Kernels of q4_experts_few.h.
#include "q4_experts_few.h"

namespace q4 {
template hipError_t few_scales<1, float, false>(const FewParams&, int32_t, hipStream_t);
}  // namespace q4
