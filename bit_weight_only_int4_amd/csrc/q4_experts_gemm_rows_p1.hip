// The tiles of q4_experts_gemm.h with activations of 1 binary16 part(s), for the experts.
#include "q4_experts_gemm.h"

namespace q4 {
template hipError_t launch_gemm_tile<1, 64, kGatedRows>(const GemmParams&, hipStream_t);
template hipError_t launch_gemm_tile<1, 128, kGatedRows>(const GemmParams&, hipStream_t);
}  // namespace q4
