// q4_experts_back.hip -- the choice of a tile for input gradients of many rows
// (q4_experts_back.h).
#include "q4_experts_back.h"

namespace q4 {

#define Q4_TILES(T, GATE)                                                            \
  extern template hipError_t launch_back_tile<T, 64, GATE>(const BackParams&, hipStream_t); \
  extern template hipError_t launch_back_tile<T, 128, GATE>(const BackParams&, hipStream_t);
Q4_TILES(_Float16, true)
Q4_TILES(bf16, true)
Q4_TILES(float, true)
Q4_TILES(float, false)
#undef Q4_TILES
extern template hipError_t launch_back_direct<64>(const BackParams&, hipStream_t);
extern template hipError_t launch_back_direct<128>(const BackParams&, hipStream_t);

namespace {
template <typename T, bool GATE>
hipError_t by_tile(const BackParams& p, int32_t tile_rows, hipStream_t s) {
  return tile_rows == 128 ? launch_back_tile<T, 128, GATE>(p, s) : launch_back_tile<T, 64, GATE>(p, s);
}
}  // namespace

hipError_t launch_back(const BackParams& in, int32_t tile_rows, bool gate, hipStream_t s) {
  BackParams p = in;
  if (p.d_parts) return tile_rows == 128 ? launch_back_direct<128>(p, s) : launch_back_direct<64>(p, s);
  const int64_t e = p.d_dtype == Q4_DTYPE_F32 ? 4 : 2;
  p.d_vec = reinterpret_cast<uintptr_t>(p.d) % 16 == 0 && p.ldd * e % 16 == 0;
  if (!gate) return by_tile<float, false>(p, tile_rows, s);
  switch (p.d_dtype) {
    case Q4_DTYPE_F32: return by_tile<float, true>(p, tile_rows, s);
    case Q4_DTYPE_F16: return by_tile<_Float16, true>(p, tile_rows, s);
    default: return by_tile<bf16, true>(p, tile_rows, s);
  }
}

}  // namespace q4
