// q4_experts_few.hip -- the choice of a kernel for few rows (q4_experts_few.h).
#include "q4_experts_few.h"

namespace q4 {

#define Q4_FEW(P, T, GATED) \
  extern template hipError_t few_scales<P, T, GATED>(const FewParams&, int32_t, hipStream_t);
Q4_FEW(2, float, true)
Q4_FEW(1, _Float16, true)
Q4_FEW(1, bf16, true)
Q4_FEW(2, float, false)
#undef Q4_FEW

hipError_t launch_few(const FewParams& p, int32_t tile_rows, bool gated, hipStream_t s) {
  if (gated) {
    switch (p.dtype) {
      case Q4_DTYPE_F32: return few_scales<2, float, true>(p, tile_rows, s);
      case Q4_DTYPE_F16: return few_scales<1, _Float16, true>(p, tile_rows, s);
      default: return few_scales<1, bf16, true>(p, tile_rows, s);
    }
  }
  // the gated rows are fp32
  return few_scales<2, float, false>(p, tile_rows, s);
}

}  // namespace q4
