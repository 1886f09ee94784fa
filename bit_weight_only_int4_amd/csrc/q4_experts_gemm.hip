// q4_experts_gemm.hip -- the choice of a tile for products of many rows
// (q4_experts_gemm.h).
#include "q4_experts_gemm.h"

namespace q4 {

#define Q4_TILES(EPI)                                                              \
  extern template hipError_t launch_gemm_tile<1, 64, EPI>(const GemmParams&, hipStream_t);  \
  extern template hipError_t launch_gemm_tile<2, 64, EPI>(const GemmParams&, hipStream_t);  \
  extern template hipError_t launch_gemm_tile<1, 128, EPI>(const GemmParams&, hipStream_t); \
  extern template hipError_t launch_gemm_tile<2, 128, EPI>(const GemmParams&, hipStream_t);
Q4_TILES(kGatedRows)
Q4_TILES(kPlainRows)
Q4_TILES(kHeadStats)
Q4_TILES(kHeadGrad)
#undef Q4_TILES

namespace {
template <Epilogue EPI>
hipError_t by_tile(const GemmParams& p, int32_t tile_rows, hipStream_t s) {
  if (tile_rows == 128)
    return p.a.parts == 2 ? launch_gemm_tile<2, 128, EPI>(p, s) : launch_gemm_tile<1, 128, EPI>(p, s);
  return p.a.parts == 2 ? launch_gemm_tile<2, 64, EPI>(p, s) : launch_gemm_tile<1, 64, EPI>(p, s);
}
}  // namespace

hipError_t launch_gemm(const GemmParams& in, int32_t tile_rows, Epilogue epi, hipStream_t s) {
  GemmParams p = in;
  p.b_wide = reinterpret_cast<uintptr_t>(p.w.qw) % 16 == 0 && p.w.K % 32 == 0;
  switch (epi) {
    case kGatedRows: return by_tile<kGatedRows>(p, tile_rows, s);
    case kPlainRows: return by_tile<kPlainRows>(p, tile_rows, s);
    case kHeadStats: return by_tile<kHeadStats>(p, tile_rows, s);
    default: return by_tile<kHeadGrad>(p, tile_rows, s);
  }
}

}  // namespace q4
