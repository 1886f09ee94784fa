// q4_attention.hip -- plan and launch of attention over the paged cache.
#include "q4_attention_kernels.h"

namespace q4 {

namespace attn {

// Joins the splits of one query row: the weights of its parts first, a lane
// each, then their outputs, a wave every fourth part.
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnParams p, int32_t max_rows) {
  __shared__ float acc_s[kWaves][256];
  __shared__ float den_s[kWaves];
  // rows of a sequence and kv head are consecutive
  const int64_t rr = blockIdx.x % max_rows;
  const uint32_t bh = blockIdx.x / max_rows;
  const Block k = block_of(p, bh * p.row_blocks + (uint32_t)(rr / kRows));
  if (rr >= k.rows) return;
  const int n = (k.tiles + p.split_tiles - 1) / p.split_tiles;
  if (n <= 1) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, dim = p.c.dim;
  const int64_t tk = rr / p.group;
  const int64_t tq = k.sp.t0 + tk, hq = k.h * p.group + (rr - tk * p.group);
  const int64_t stride = p.T * p.heads, at = tq * p.heads + hq;
  float m = -__builtin_inff();
  for (int s = lane; s < n; s += 64) m = fmaxf(m, p.part_ml[2 * (at + s * stride)]);
#pragma unroll
  for (int i = 32; i >= 1; i >>= 1) m = fmaxf(m, __shfl_xor(m, i, 64));
  const float ref = m > -__builtin_inff() ? m : 0.0f;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, den = 0.0f;
  for (int s = wave; s < n; s += kWaves) {
    const int64_t a = at + s * stride;
    const float f = exp2_fast(p.part_ml[2 * a] - ref), d = p.part_ml[2 * a + 1];
    den += d != d ? d : f * d;  // a part without a maximum: 0, or NaN
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < dim) acc[i] += f * p.part_o[a * dim + lane + 64 * i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) acc_s[wave][lane + 64 * i] = acc[i];
  if (lane == 0) den_s[wave] = den;
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= dim) return;
  float o = 0.0f, total = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    o += acc_s[w][d];
    total += den_s[w];
  }
  store_elem(p.out, tq * p.o_ts + hq * p.o_hs + d, total == 0.0f ? 0.0f : o / total, p.dtype);
}

}  // namespace attn

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// The keys of a row block go to several workgroups, for two reasons: row
// blocks alone may leave CUs without work, and sequences differ in length,
// so that the longest would run alone at the end.  A split of kMinTiles tiles
// already costs little beside them (its part of the output is 1 / 32 of the
// keys it reads at 4 rows of 128).  max_len and the window bound the tiles:
// neither the grid nor the workspace depends on device-side lengths.
AttnPlan plan_attention(int32_t dtype, int64_t T, int64_t batch, int64_t heads, int64_t kv_heads,
                        int64_t dim, int64_t page, int64_t max_new, int64_t max_len,
                        int64_t window) {
  (void)dtype;
  (void)page;
  constexpr int64_t kTargetBlocks = 4096, kMinTiles = 16;
  AttnPlan pl;
  const int64_t group = heads / kv_heads;
  pl.max_rows = (int32_t)(max_new * group);
  pl.row_blocks = (int32_t)ceil_div(max_new * group, attn::kRows);
  // a block's queries span at most kRows positions
  int64_t span = max_len;
  if (window > 0 && window + attn::kRows < span) span = window + attn::kRows;
  const int64_t tiles = ceil_div(span, attn::kTile) + (window > 0 ? 1 : 0);
  const int64_t blocks = batch * kv_heads * pl.row_blocks;
  int64_t splits = ceil_div(kTargetBlocks, blocks > 0 ? blocks : 1);
  if (splits > tiles / kMinTiles) splits = tiles / kMinTiles;
  if (splits < 1) splits = 1;
  pl.split_tiles = (int32_t)ceil_div(tiles > 0 ? tiles : 1, splits);
  pl.splits = (int32_t)ceil_div(tiles > 0 ? tiles : 1, pl.split_tiles);
  pl.workspace = pl.splits > 1
                     ? (size_t)pl.splits * (size_t)(T * heads) * (size_t)(dim + 2) * sizeof(float)
                     : 0;
  return pl;
}

hipError_t launch_attention(const AttnParams& p, hipStream_t s) {
  const hipError_t e = p.dtype == Q4_DTYPE_F32 ? launch_attention_digits<3>(p, s)
                                               : launch_attention_digits<2>(p, s);
  if (e != hipSuccess || p.splits <= 1) return e;
  const dim3 grid((unsigned)((int64_t)p.batch * p.c.heads * p.max_rows));
  hipLaunchKernelGGL(attn::attention_join_kernel, grid, dim3(attn::kThreads), 0, s, p, p.max_rows);
  return hipGetLastError();
}

}  // namespace q4
