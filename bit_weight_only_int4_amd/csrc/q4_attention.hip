// q4_attention.hip -- plan and launch of attention over the paged cache.
#include "q4_attention_kernels.h"

namespace q4 {

namespace attn {

// Joins the splits of the row blocks that have more than one.
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnParams p) {
  const Block k = block_of(p, blockIdx.x);
  if (k.row0 >= k.rows) return;
  const int n_splits = (k.tiles + p.split_tiles - 1) / p.split_tiles;
  if (n_splits <= 1) return;
  const int dim = p.c.dim;
  const int64_t stride = p.T * p.heads;
  for (int i = threadIdx.x; i < kRows * dim; i += kThreads) {
    const int row = i / dim, d = i - row * dim;
    const int64_t rr = k.row0 + row;
    if (rr >= k.rows) break;
    const int64_t tk = rr / p.group;
    const int64_t tq = k.sp.t0 + tk, hq = k.h * p.group + (rr - tk * p.group);
    const int64_t at = tq * p.heads + hq;
    float m = -__builtin_inff(), acc = 0.0f, den = 0.0f;
    for (int s = 0; s < n_splits; ++s) m = fmaxf(m, p.part_ml[2 * (at + s * stride)]);
    const float ref = m > -__builtin_inff() ? m : 0.0f;
    for (int s = 0; s < n_splits; ++s) {
      const int64_t a = at + s * stride;
      const float f = exp2_fast(p.part_ml[2 * a] - ref);
      const float sw = p.part_ml[2 * a + 1];
      den += sw != sw ? sw : f * sw;
      acc += f * p.part_o[a * dim + d];
    }
    store_elem(p.out, tq * p.o_ts + hq * p.o_hs + d, den == 0.0f ? 0.0f : acc / den, p.dtype);
  }
}

}  // namespace attn

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// The keys of a row block go to several workgroups where the row blocks alone
// leave CUs without work: as many as give the chip kTargetBlocks workgroups,
// each at least one tile per wave.  max_len and the window bound the tiles,
// so that neither the grid nor the workspace depends on device-side lengths.
AttnPlan plan_attention(int32_t dtype, int64_t T, int64_t batch, int64_t heads, int64_t kv_heads,
                        int64_t dim, int64_t page, int64_t max_new, int64_t max_len,
                        int64_t window) {
  (void)dtype;
  (void)page;
  constexpr int64_t kTargetBlocks = 1024;
  AttnPlan pl;
  const int64_t group = heads / kv_heads;
  pl.row_blocks = (int32_t)ceil_div(max_new * group, attn::kRows);
  // a block's queries span at most kRows positions
  int64_t span = max_len;
  if (window > 0 && window + attn::kRows < span) span = window + attn::kRows;
  const int64_t tiles = ceil_div(span, attn::kTile) + 1;
  const int64_t blocks = batch * kv_heads * pl.row_blocks;
  int64_t splits = ceil_div(kTargetBlocks, blocks > 0 ? blocks : 1);
  if (splits > ceil_div(tiles, attn::kWaves)) splits = ceil_div(tiles, attn::kWaves);
  if (splits < 1) splits = 1;
  pl.split_tiles = (int32_t)ceil_div(tiles, splits);
  pl.splits = (int32_t)ceil_div(tiles, pl.split_tiles);
  pl.workspace = pl.splits > 1
                     ? (size_t)pl.splits * (size_t)(T * heads) * (size_t)(dim + 2) * sizeof(float)
                     : 0;
  return pl;
}

hipError_t launch_attention(const AttnParams& p, hipStream_t s) {
  const hipError_t e = p.dtype == Q4_DTYPE_F32 ? launch_attention_digits<3>(p, s)
                                               : launch_attention_digits<2>(p, s);
  if (e != hipSuccess || p.splits <= 1) return e;
  const dim3 grid((unsigned)((int64_t)p.batch * p.c.heads * p.row_blocks));
  hipLaunchKernelGGL(attn::attention_join_kernel, grid, dim3(attn::kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace q4
