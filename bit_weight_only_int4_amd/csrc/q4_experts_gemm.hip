// q4_experts_gemm.hip -- the choice of a tile for products of many rows
// (q4_experts_gemm.h).
#include "q4_experts_gemm.h"

namespace q4 {

#define Q4_TILES(P, EPI)                                                           \
  extern template hipError_t launch_gemm_tile<P, 64, EPI>(const GemmParams&, hipStream_t);  \
  extern template hipError_t launch_gemm_tile<P, 128, EPI>(const GemmParams&, hipStream_t);
Q4_TILES(1, kGatedRows)
Q4_TILES(2, kGatedRows)
Q4_TILES(2, kPlainRows)  // fp32 values
Q4_TILES(1, kHeadStats)
Q4_TILES(2, kHeadStats)
Q4_TILES(1, kHeadGrad)
Q4_TILES(2, kHeadGrad)
#undef Q4_TILES

namespace {
template <int P, Epilogue EPI>
hipError_t by_rows(const GemmParams& p, int32_t tile_rows, hipStream_t s) {
  return tile_rows == 128 ? launch_gemm_tile<P, 128, EPI>(p, s) : launch_gemm_tile<P, 64, EPI>(p, s);
}
template <Epilogue EPI>
hipError_t by_tile(const GemmParams& p, int32_t tile_rows, hipStream_t s) {
  return p.a.parts == 2 ? by_rows<2, EPI>(p, tile_rows, s) : by_rows<1, EPI>(p, tile_rows, s);
}
}  // namespace

hipError_t launch_gemm(const GemmParams& in, int32_t tile_rows, Epilogue epi, hipStream_t s) {
  GemmParams p = in;
  p.b_wide = reinterpret_cast<uintptr_t>(p.w.qw) % 16 == 0 && p.w.K % 32 == 0;
  switch (epi) {
    case kGatedRows: return by_tile<kGatedRows>(p, tile_rows, s);
    case kPlainRows: return by_rows<2, kPlainRows>(p, tile_rows, s);
    case kHeadStats: return by_tile<kHeadStats>(p, tile_rows, s);
    default: return by_tile<kHeadGrad>(p, tile_rows, s);
  }
}

}  // namespace q4
