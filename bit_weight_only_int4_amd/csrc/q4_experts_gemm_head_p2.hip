// The tiles of q4_experts_gemm.h with activations of 2 binary16 part(s), for the head.
#include "q4_experts_gemm.h"

namespace q4 {
template hipError_t launch_gemm_tile<2, 64, kHeadStats>(const GemmParams&, hipStream_t);
template hipError_t launch_gemm_tile<2, 128, kHeadStats>(const GemmParams&, hipStream_t);
template hipError_t launch_gemm_tile<2, 64, kHeadGrad>(const GemmParams&, hipStream_t);
template hipError_t launch_gemm_tile<2, 128, kHeadGrad>(const GemmParams&, hipStream_t);
}  // namespace q4
