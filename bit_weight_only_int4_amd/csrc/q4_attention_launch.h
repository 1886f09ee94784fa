// q4_attention_launch.h -- the attention kernel for one number of digits;
// included by q4_attention_d3.hip and q4_attention_d4.hip.
#pragma once

#include "q4_attention_wide.h"

namespace q4 {

template <int DT, int ND, int W, bool UNIFORM>
static hipError_t launch_attention_waves(const AttnParams& p, hipStream_t s) {
  using namespace attn;
  const size_t lds = (size_t)W * kRows * (16 * DT + 6) * sizeof(float);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void*)attention_kernel<DT, ND, W, UNIFORM>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)((int64_t)p.batch * p.c.heads * p.row_blocks * p.splits));
  hipLaunchKernelGGL((attention_kernel<DT, ND, W, UNIFORM>), grid, dim3(64 * W), lds, s, p);
  return hipGetLastError();
}

template <int DT, int ND, bool UNIFORM>
static hipError_t launch_attention_pages(const AttnParams& p, hipStream_t s) {
  using namespace attn;
  if (p.block_rows > kRows) {
    const size_t bytes = (size_t)4 * (4 * ((DT + 3) / 4) + DT) * 1024;
    const dim3 grid((unsigned)((int64_t)p.batch * p.c.heads * p.row_blocks * p.splits));
    auto run = attention_wide_kernel<DT, ND, 1, UNIFORM>;
    if constexpr (ND == 3 || DT > 12)
      if (p.block_rows == 2 * kWaves * kRows) run = attention_wide_kernel<DT, ND, 2, UNIFORM>;
    if (bytes > 65536) {
      const hipError_t e = hipFuncSetAttribute(
          (const void*)run, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(run, grid, dim3(kThreads), bytes, s, p);
    return hipGetLastError();
  }
  // where CUs have a workgroup or two at most, eight waves shorten each
  if constexpr (DT <= 8)
    if (p.few) return launch_attention_waves<DT, ND, 8, UNIFORM>(p, s);
  return launch_attention_waves<DT, ND, 4, UNIFORM>(p, s);
}

template <int DT, int ND>
static hipError_t launch_attention_dim(const AttnParams& p, hipStream_t s) {
  return p.c.page >= attn::kTile ? launch_attention_pages<DT, ND, true>(p, s)
                                 : launch_attention_pages<DT, ND, false>(p, s);
}

// The kernel holds a head in 16-wide tiles; head sizes between the instances
// run the next one up (past-the-end tiles are computed and not stored).
template <int ND>
hipError_t launch_attention_digits(const AttnParams& p, hipStream_t s) {
  const int d16 = p.c.dim / 16;
  if (d16 <= 4) return launch_attention_dim<4, ND>(p, s);
  if (d16 <= 6) return launch_attention_dim<6, ND>(p, s);
  if (d16 <= 8) return launch_attention_dim<8, ND>(p, s);
  if (d16 <= 12) return launch_attention_dim<12, ND>(p, s);
  return launch_attention_dim<16, ND>(p, s);
}

}  // namespace q4
