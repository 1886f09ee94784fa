// q4_attention.hip -- plan and launch of attention over the paged cache.
#include "q4_attention_wide.h"

namespace q4 {

namespace attn {

// Joins the splits of a query row, a workgroup each, where there may be many.
// The parts' weights come first, a thread each, so that their outputs then
// load without waiting for one another: 4 elements a thread, dim / 4 threads a
// part, four parts a step.
__global__ __launch_bounds__(kThreads) void attention_join_many_kernel(AttnParams p) {
  extern __shared__ float lds[];  // weights [splits], then [parts at once][dim]
  __shared__ float red[2 * kWaves];
  const uint32_t rr = blockIdx.x % (uint32_t)p.max_rows;
  const uint32_t bh = blockIdx.x / (uint32_t)p.max_rows;
  const Block k = block_of(p, bh / p.c.heads, bh % p.c.heads, (int)((uint32_t)rr / (uint32_t)p.block_rows));
  if (rr >= k.rows) return;
  const int n = (k.tiles + p.split_tiles - 1) / p.split_tiles;
  if (n <= 1) return;
  const int64_t tk = row_token(p, rr);
  const int64_t tq = k.sp.t0 + tk, hq = k.h * p.group + (rr - tk * p.group);
  const int64_t at = tq * p.heads + hq, stride = p.T * p.heads;
  const int64_t out = tq * p.o_ts + hq * p.o_hs;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, dim = p.c.dim;
  float* weight = lds;
  float m = -__builtin_inff();
  for (int s = tid; s < n; s += kThreads) m = fmaxf(m, p.part_ml[2 * (at + s * stride)]);
#pragma unroll
  for (int i = 32; i >= 1; i >>= 1) m = fmaxf(m, __shfl_xor(m, i, 64));
  if (lane == 0) red[wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = fmaxf(m, red[w]);
  const float ref = m > -__builtin_inff() ? m : 0.0f;
  float den = 0.0f;
  for (int s = tid; s < n; s += kThreads) {
    const int64_t a = at + s * stride;
    const float f = exp2_fast(p.part_ml[2 * a] - ref), d = p.part_ml[2 * a + 1];
    weight[s] = f;
    den += d != d ? d : f * d;  // a part without a maximum: 0, or NaN
  }
#pragma unroll
  for (int i = 32; i >= 1; i >>= 1) den += __shfl_xor(den, i, 64);
  if (lane == 0) red[kWaves + wave] = den;
  __syncthreads();
  const int quads = dim >> 2, at_once = kThreads / quads;
  const int part = tid / quads, d = 4 * (tid - part * quads);
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  if (part < at_once) {
    const float* src = p.part_o + at * dim + d;
    int s = part;
    for (; s + 3 * at_once < n; s += 4 * at_once) {
      f32x4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *(const f32x4*)(src + (s + i * at_once) * stride * dim);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc += weight[s + i * at_once] * v[i];
    }
    for (; s < n; s += at_once) acc += weight[s] * *(const f32x4*)(src + s * stride * dim);
    float* o = lds + p.splits + part * dim + d;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = acc[e];
  }
  __syncthreads();
  if (tid >= dim) return;
  float o = 0.0f, total = 0.0f;
  for (int i = 0; i < at_once; ++i) o += lds[p.splits + i * dim + tid];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) total += red[kWaves + w];
  store_elem(p.out, out + tid, total == 0.0f ? 0.0f : o / total, p.dtype);
}

// Joins few splits: dim / 4 threads a query row, so that many rows share a
// workgroup; maxima, sums and outputs of kJoinAtOnce parts load together.
constexpr int kJoinAtOnce = 8;
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnParams p) {
  const int quads = p.c.dim >> 2, at_once = kThreads / quads;
  const int mine = threadIdx.x / quads, d = 4 * (threadIdx.x - mine * quads);
  const int per_bh = (p.max_rows + at_once - 1) / at_once;
  const int64_t rr = (int64_t)(blockIdx.x % per_bh) * at_once + mine;
  const uint32_t bh = blockIdx.x / per_bh;
  if (mine >= at_once || rr >= p.max_rows) return;
  const Block k = block_of(p, bh / p.c.heads, bh % p.c.heads, (int)((uint32_t)rr / (uint32_t)p.block_rows));
  if (rr >= k.rows) return;
  const int n = (k.tiles + p.split_tiles - 1) / p.split_tiles;
  if (n <= 1) return;
  const int64_t tk = row_token(p, rr);
  const int64_t tq = k.sp.t0 + tk, hq = k.h * p.group + (rr - tk * p.group);
  const int64_t at = tq * p.heads + hq, stride = p.T * p.heads;
  float m = -__builtin_inff(), den = 0.0f;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < n; s += kJoinAtOnce) {
    float top[kJoinAtOnce], sum[kJoinAtOnce];
    f32x4 o[kJoinAtOnce];
#pragma unroll
    for (int i = 0; i < kJoinAtOnce; ++i) {
      const int64_t a = at + (s + i < n ? s + i : n - 1) * stride;
      top[i] = p.part_ml[2 * a];
      sum[i] = p.part_ml[2 * a + 1];
      o[i] = *(const f32x4*)&p.part_o[a * p.c.dim + d];
    }
    const float before = m;
#pragma unroll
    for (int i = 0; i < kJoinAtOnce; ++i) m = fmaxf(m, top[i]);
    const float ref = m > -__builtin_inff() ? m : 0.0f, keep = exp2_fast(before - ref);
    den *= keep;
    acc *= keep;
#pragma unroll
    for (int i = 0; i < kJoinAtOnce; ++i) {
      if (s + i >= n) break;
      const float f = exp2_fast(top[i] - ref);
      den += sum[i] != sum[i] ? sum[i] : f * sum[i];  // a part without a maximum: 0, or NaN
      acc += f * o[i];
    }
  }
  const float inv = den == 0.0f ? 0.0f : 1.0f / den;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    store_elem(p.out, tq * p.o_ts + hq * p.o_hs + d + e, acc[e] * inv, p.dtype);
}

}  // namespace attn

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// Which kernel, and how much of it.
//
// Where sequences may bring more rows to a kv head than two blocks of 16, and
// there is work enough, the wide kernel, whose workgroups share keys and values
// between 128 rows, or 64 where those would leave CUs without a workgroup.
// Enough is kWideAll rows in all, or kWideWork rows times tiles, with the keys
// split into pieces of at least kWideTiles tiles.  Below, its barriers and its
// longer way to the first key cost more than the sharing gives.  Bf16, 32 query
// and 8 kv heads of 128, 16-row workgroups against wide ones, us:
//   new tokens x sequences over positions   rows   rows x tiles   16-row   wide
//   128 x 1 over 1000                       4096          2^16      12.5   29.8
//   64 x 1 over 4000                        2048          2^17      24.5   31.3
//   64 x 4 over 1000                        8192          2^17      19.0   30.6
//   128 x 1 over 4000                       4096          2^18      34.5   39.0
//   64 x 1 over 16000                       2048          2^19      56.7   49.1
//   32 x 4 over 16000                       4096          2^20       105   82.4
//   256 x 4 over 256                       32768          2^17      32.3   21.9
//   64 x 64 over 64                       131072          2^17       109   51.9
//   16 x 64 over 2000                      32768          2^20       160    127
//   12 x 16 over 4000                       6144          2^19      57.2   48.3
//   8 x 256 over 100 (32 rows a head)      65536          2^17      61.7   83.6
// (the fourth is 63 tiles, just below the limit).  Fp32, the same: 128 x 1 over
// 4000 36.4 and 43.7, 64 x 1 over 16000 60.6 and 55.3, 256 x 4 over 256 31.6 and
// 24.4, 64 x 64 over 64 99.5 and 65.0, 12 x 16 over 4000 58.8 and 54.6.
//
// 128 rows a workgroup of the wide kernel, except for fp32 queries up to heads
// of 192: two row blocks of four digits a wave leave no registers there.  64
// against 128 rows, us, 3 x 300 to 2048 tokens over up to 8192, heads of 32
// 227 and 249, 64 229 and 251, 80 313 and 325, 96 371 and 354, 128 338 and 394,
// 192 736 and 789, 256 (a wave a SIMD either way) 1120 and 984.
//
// Else 16 rows a workgroup.  The keys of a row block go to several workgroups,
// each at least kMinTiles tiles, where row blocks alone do not give every CU
// one (kTargetBlocks); and, where they do, to at most kRagged, each at least
// kRaggedTiles tiles, as sequences differ in length and the longest would run
// alone at the end (64 sequences of 500 to 8000 tokens, 8 kv heads of 128, fp32:
// 103 us with one, 79 with four; of 9000 tokens each, where nothing is gained,
// 201 and 212).  Equal pieces for all workgroups, cut from the tiles of all
// sequences in a row, were measured and not kept: the longer way to the first
// key and the second launch cost what the balance gave (84 and 231 us).
// max_len and the window bound the tiles: neither the grid nor the workspace
// depends on device-side lengths.
AttnPlan plan_attention(int32_t dtype, int64_t T, int64_t batch, int64_t heads, int64_t kv_heads,
                        int64_t dim, int64_t page, int64_t max_new, int64_t max_len,
                        int64_t window) {
  (void)page;
  constexpr int64_t kTargetBlocks = 256, kWideTarget = 512, kMinTiles = 4, kWideTiles = 12;
  constexpr int64_t kRagged = 4, kRaggedTiles = 24, kWideMin = 33, kWideAll = 16384, kWideWork = 1 << 18;
  AttnPlan pl{};
  const int64_t group = heads / kv_heads;
  constexpr int kBlock = attn::kWaves * attn::kRows;
  // positions that a block's queries span
  auto span_of = [&](int64_t rows) {
    return window > 0 && window + rows < max_len ? window + rows : max_len;
  };
  const int64_t rows = batch * kv_heads * max_new * group;
  const bool wide = max_new * group >= kWideMin &&
                    (rows >= kWideAll || rows * ceil_div(span_of(kBlock), attn::kTile) >= kWideWork);
  pl.max_rows = (int32_t)(max_new * group);
  const bool large = (dtype != Q4_DTYPE_F32 || dim > 192) &&
                     batch * kv_heads * ceil_div(max_new * group, 2 * kBlock) >= 512;
  pl.block_rows = !wide ? attn::kRows : large ? 2 * kBlock : kBlock;
  pl.row_blocks = (int32_t)ceil_div(max_new * group, pl.block_rows);
  int64_t tiles = ceil_div(span_of(pl.block_rows), attn::kTile) + (window > 0 ? 1 : 0);
  if (tiles < 1) tiles = 1;
  const int64_t blocks = batch * kv_heads * pl.row_blocks;
  const int64_t target = wide ? kWideTarget : kTargetBlocks, least = wide ? kWideTiles : kMinTiles;
  int64_t splits = ceil_div(target, blocks > 0 ? blocks : 1);
  if (splits > tiles / least) splits = tiles / least;
  if (!wide && blocks >= kTargetBlocks) splits = tiles / kRaggedTiles < kRagged ? tiles / kRaggedTiles : kRagged;
  if (splits < 1) splits = 1;
  pl.split_tiles = (int32_t)ceil_div(tiles, splits);
  pl.splits = (int32_t)ceil_div(tiles, pl.split_tiles);
  pl.few = !wide && blocks * pl.splits <= 256;
  pl.parts = pl.splits > 1 ? (size_t)pl.splits * (size_t)(T * heads) : 0;
  pl.workspace = pl.parts * (size_t)(dim + 2) * sizeof(float);
  return pl;
}

hipError_t launch_attention(const AttnParams& p, hipStream_t s) {
  const hipError_t e = p.dtype == Q4_DTYPE_F32 ? launch_attention_digits<4>(p, s)
                                               : launch_attention_digits<3>(p, s);
  if (e != hipSuccess || p.splits <= 1) return e;
  const int64_t bh = (int64_t)p.batch * p.c.heads, at_once = attn::kThreads / (p.c.dim / 4);
  if (p.splits > attn::kJoinAtOnce) {
    const size_t lds = (p.splits + (size_t)at_once * p.c.dim) * sizeof(float);
    hipLaunchKernelGGL(attn::attention_join_many_kernel, dim3((unsigned)(bh * p.max_rows)),
                       dim3(attn::kThreads), lds, s, p);
  } else {
    hipLaunchKernelGGL(attn::attention_join_kernel,
                       dim3((unsigned)(bh * ((p.max_rows + at_once - 1) / at_once))),
                       dim3(attn::kThreads), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace q4
