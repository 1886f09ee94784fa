// q4_attention_wide.h -- attention of many query rows of one sequence (chunks
// of a prompt) over the paged 8-bit cache.
//
// The mathematics and the operand layouts are those of
// q4_attention_kernels.h.  Here a workgroup holds 128 rows of a kv head, 32 in
// each of its four waves, and all of them read a tile's keys and values from
// LDS, where global loads have put them directly, 1 KB to an operand of 16
// rows and 64 columns in the order of the lanes that read it (so that neither
// side has a bank conflict).  Two buffers: the next tile loads while one is
// worked on, with one barrier a tile.
//
// Bound by the vector unit: a score takes 11 issue slots (4 of them the
// exponential) and an output element 3 a tile, together 1200 cycles for 16
// rows and 64 tokens of a head of 128, where the matrix unit needs 512 (two
// digits).  What keeps them few:
//   * with two digits scores stay integers until the maximum is known;
//   * the running maximum is only a reference that keeps the exponentials in
//     range: outputs are rescaled when a row's maximum passes it by 2^8, not
//     at every new maximum;
//   * tiles that all rows of a wave see whole skip the masks.
#pragma once

#include "q4_attention_kernels.h"

namespace q4 {
namespace attn {

constexpr int kColumns = 2;                              // 16-row blocks of a wave
constexpr int kWideRows = kWaves * kColumns * kRows;     // 128
constexpr float kSlack = 8.0f;                           // log2 that a maximum may pass the reference by

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef const __attribute__((address_space(1))) void* global_ptr;

// Scores of a tile before the maximum is taken: integers where two digits
// make them (below 2^31: 256 products of 2^14 times 257), else fp32.
template <int ND>
struct Raw {
  typedef float type;
};
template <>
struct Raw<2> {
  typedef int32_t type;
};

template <int ND>
__device__ __forceinline__ typename Raw<ND>::type raw_join(const int32_t (&a)[ND]) {
  if constexpr (ND == 2) return a[1] * 256 + a[0];
  else return join_digits<ND>(a);
}

__device__ __forceinline__ int32_t column_max(int32_t x) {
  auto r = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
  x = (int32_t)r[0] > (int32_t)r[1] ? (int32_t)r[0] : (int32_t)r[1];
  r = __builtin_amdgcn_permlane32_swap((uint32_t)x, (uint32_t)x, false, false);
  return (int32_t)r[0] > (int32_t)r[1] ? (int32_t)r[0] : (int32_t)r[1];
}

// Probabilities of a tile that the row sees whole and one page covers, as
// tile_softmax.  mx is a reference, at most kSlack below the maximum.
template <int ND>
__device__ __forceinline__ void whole_tile_softmax(const typename Raw<ND>::type (&raw)[4][4],
                                                   float unit, float vs, float& mx, float& sum,
                                                   i32x4 (&pd)[ND], float& alpha, float& w) {
  typename Raw<ND>::type best = raw[0][0];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) best = raw[a][i] > best ? raw[a][i] : best;
  const float top = (float)column_max(best) * unit;
  float part = 0.0f;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    uint32_t bits[4], out[ND];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // at most 1 but for the product's rounding, and NaN only where unit is
      const float e = __builtin_amdgcn_fmed3f(
          exp2_fast(__builtin_fmaf((float)raw[a][i], unit, -top)), 0.0f, 1.0f);
      part += e;
      bits[i] = f32_bits(__builtin_fmaf(e, digit_max<ND>(), 8388608.0f + (float)digit_bias<ND>()));
    }
    pack_digits<ND>(bits[0], bits[1], bits[2], bits[3], out);
#pragma unroll
    for (int i = 0; i < ND; ++i) pd[i][a] = (int32_t)out[i];
  }
  alpha = 1.0f;
  if (__any(top > mx + kSlack)) {
    const float to = top > mx + kSlack ? top : mx;
    alpha = to > mx ? exp2_fast(mx - to) : 1.0f;
    mx = to;
  }
  const float beta = exp2_fast(top - mx);
  sum = sum * alpha + (beta * part + (unit - unit));  // NaN shows
  w = beta * vs * (1.0f / digit_max<ND>());
}

template <int DT, int ND, bool UNIFORM>
__global__ __launch_bounds__(kThreads, DT <= 8 ? 2 : 1) void attention_wide_kernel(AttnParams p) {
  constexpr int NS = (DT + 3) / 4;
  constexpr int KF = 4 * NS, FR = KF + DT;  // operands (1 KB each) of a tile: keys, all
  extern __shared__ char tiles[];           // [2][FR][1024]
  // Heads vary fastest, so that an XCD keeps to few of them, then row blocks,
  // the last first as they have the most keys: those that run together share
  // their keys in L2.
  uint32_t id = blockIdx.x;
  const int h = id % p.c.heads;
  id /= p.c.heads;
  const int rb = p.row_blocks - 1 - (int)(id % p.row_blocks);
  id /= p.row_blocks;
  const int b = id % p.batch, split = id / p.batch;
  const Block k = block_of(p, b, h, rb);
  if (k.row0 >= k.rows) return;
  const int n_splits = (k.tiles + p.split_tiles - 1) / p.split_tiles;
  if (split > 0 && split >= n_splits) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int col = lane & 15, g = lane >> 4;
  const KvCache& c = p.c;
  const int dim = c.dim, d16 = dim >> 4;
  const int32_t* table = c.table + (int64_t)k.b * c.table_ld;
  const int page_mask = c.page - 1;
  const float nan = bits_f32(0x7fc00000u);
  const int t_end = (split + 1) * p.split_tiles < k.tiles ? (split + 1) * p.split_tiles : k.tiles;

  // pages of the tile's keys that this lane loads, and of its 16 tokens
  auto pages_of = [&](int tile, int32_t& key, int32_t& own) {
    const int64_t token0 = (int64_t)(k.tile0 + tile) * kTile;
    if (UNIFORM) {
      own = key = __builtin_amdgcn_readfirstlane(
          page_at(table, c.max_pages, c.pages, token0 >> c.page_log2));
    } else {
      own = segment_page(p, table, k.keys, token0 + 16 * g);
      key = segment_page(p, table, k.keys, token0 + 16 * (col >> 2));
    }
  };
  float ks_next = 0.0f, vs_next = 0.0f;
  // every fourth operand of the tile, straight to LDS, and the lane's scales
  auto fetch = [&](int tile, int buf, int32_t key, int32_t own) {
    const int64_t token0 = (int64_t)(k.tile0 + tile) * kTile;
    const int k_slot = (int)((token0 + (UNIFORM ? 0 : 16 * (col >> 2))) & page_mask);
    const int v_slot = (int)((token0 + (UNIFORM ? 0 : 16 * g)) & page_mask);
    const int64_t ph = (int64_t)(own > 0 ? own : 0) * c.heads + k.h;
    const int8_t* kb =
        c.k + ((((int64_t)(key > 0 ? key : 0) * c.heads + k.h) << c.page_log2) + k_slot) * dim;
    const int8_t* vb = c.v + ph * ((int64_t)dim << c.page_log2) + v_slot;
    const uint32_t k_off = (uint32_t)(((UNIFORM ? 16 * (col >> 2) : 0) + (col & 3)) * dim);
    const uint32_t v_off = (uint32_t)((col << c.page_log2) + (UNIFORM ? 16 * g : 0));
    char* to = tiles + buf * FR * 1024;
#pragma unroll
    for (int i = 0; i < (FR + kWaves - 1) / kWaves; ++i) {
      const int f = kWaves * i + wave;
      if (FR % kWaves != 0 && f >= FR) break;
      const int8_t* src;
      if (f < KF) {
        const int a = f / NS, s = f % NS, d = 64 * s + 16 * g;
        src = kb + 4 * a * dim + (k_off + (d < dim ? d : 0));
      } else {
        const int dt = f - KF;
        src = vb + ((dt < d16 ? 16 * dt : 0) << c.page_log2) + v_off;
      }
      __builtin_amdgcn_global_load_lds((global_ptr)src, (lds_ptr)(to + f * 1024), 16, 0, 0);
    }
    ks_next = own >= 0 ? c.ks[ph] : nan;
    vs_next = own >= 0 ? c.vs[ph] : nan;
  };
  int32_t key = 0, own = 0, buf = 0;
  int t = split * p.split_tiles;
  if (t < t_end) {
    pages_of(t, key, own);
    fetch(t, 0, key, own);
    if (t + 1 < t_end) pages_of(t + 1, key, own);
  }

  // the lane's query rows and what they see
  Column<DT> st[kColumns];
  i32x4 qd[kColumns][NS][ND];
  float q_unit[kColumns];
  int64_t see_lo[kColumns], see_hi[kColumns];
  const int64_t wave_row = k.row0 + wave * kColumns * kRows;
#pragma unroll
  for (int n = 0; n < kColumns; ++n) {
    const int64_t r = wave_row + n * kRows + col;
    const bool valid = r < k.rows;
    const int64_t tok = valid ? r / p.group : 0;
    const int head = k.h * p.group + (int)(valid ? r - tok * p.group : 0);
    const int64_t pos = valid ? k.sp.pos0 + tok : -1;
    see_lo[n] = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
    see_hi[n] = pos < k.keys.hi ? pos : k.keys.hi - 1;
    column_init(st[n]);
    q_unit[n] = row_digits<NS, ND>(p, (k.sp.t0 + tok) * p.q_ts + (int64_t)head * p.q_hs, valid, g,
                                   qd[n]);
  }
  // positions that some and all of the wave's rows see
  const int64_t rows_end = wave_row + kColumns * kRows < k.rows ? wave_row + kColumns * kRows : k.rows;
  const int64_t pos_first = k.sp.pos0 + wave_row / p.group;
  const int64_t pos_last = k.sp.pos0 + (rows_end - 1) / p.group;
  const bool idle = wave_row >= k.rows;
  const KeyRange some = key_range(pos_first, pos_last, p.window, k.keys.hi);
  const int64_t all_hi = pos_first < k.keys.hi ? pos_first : k.keys.hi - 1;
  const int64_t all_lo = p.window > 0 ? pos_last - p.window + 1 : 0;

  for (; t < t_end; ++t, buf ^= 1) {
    // this wave's part of the tile has landed; past the barrier all of it has,
    // and every wave is done with the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const float ks = ks_next, vs = vs_next;
    if (t + 1 < t_end) {
      fetch(t + 1, buf ^ 1, key, own);
      if (t + 2 < t_end) pages_of(t + 2, key, own);
    }
    const int64_t token0 = (int64_t)(k.tile0 + t) * kTile;
    if (idle || token0 >= some.hi || token0 + kTile <= some.lo) continue;
    const bool whole = token0 >= all_lo && token0 + kTile - 1 <= all_hi;
    const char* from = tiles + buf * FR * 1024 + 16 * lane;
    typename Raw<ND>::type raw[kColumns][4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      i32x4 kd[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) kd[s] = *(const i32x4*)(from + (a * NS + s) * 1024);
#pragma unroll
      for (int n = 0; n < kColumns; ++n) {
        i32x4 acc[ND];
#pragma unroll
        for (int i = 0; i < ND; ++i) {
          acc[i] = i32x4{0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < NS; ++s)
            acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(kd[s], qd[n][s][i], acc[i], 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int32_t part[ND];
#pragma unroll
          for (int i = 0; i < ND; ++i) part[i] = acc[i][e];
          raw[n][a][e] = raw_join<ND>(part);
        }
      }
    }
    i32x4 pd[kColumns][ND];
    float w[kColumns];
#pragma unroll
    for (int n = 0; n < kColumns; ++n) {
      float alpha;
      const float unit = q_unit[n] * ks;
      if (UNIFORM && whole) {
        whole_tile_softmax<ND>(raw[n], unit, vs, st[n].mx, st[n].sum, pd[n], alpha, w[n]);
      } else {
        float sc[4][4];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[a][e] = (float)raw[n][a][e];
        const int64_t base = token0 + 16 * g;
        const int64_t lo = see_lo[n] - base, hi = see_hi[n] - base;
        tile_softmax<ND, true, UNIFORM>(sc, unit, vs, (int)(lo > 16 ? 16 : lo < 0 ? 0 : lo),
                                        (int)(hi < -1 ? -1 : hi > 15 ? 15 : hi), st[n].mx,
                                        st[n].sum, pd[n], alpha, w[n]);
      }
      if (__any(alpha != 1.0f)) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int e = 0; e < 4; ++e) st[n].o[dt][e] *= alpha;
      }
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const i32x4 vd = *(const i32x4*)(from + (KF + dt) * 1024);
#pragma unroll
      for (int n = 0; n < kColumns; ++n) {
        i32x4 acc[ND];
#pragma unroll
        for (int i = 0; i < ND; ++i)
          acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vd, pd[n][i], i32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int32_t part[ND];
#pragma unroll
          for (int i = 0; i < ND; ++i) part[i] = acc[i][e];
          st[n].o[dt][e] = __builtin_fmaf((float)raw_join<ND>(part), w[n], st[n].o[dt][e]);
        }
      }
    }
  }

#pragma unroll
  for (int n = 0; n < kColumns; ++n) {
    const int64_t r = wave_row + n * kRows + col;
    const float sum = column_sum(st[n].sum);
    if (r >= k.rows) continue;
    const int64_t tok = r / p.group;
    const int64_t tq = k.sp.t0 + tok, hq = k.h * p.group + (r - tok * p.group);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // no key seen: 0
    const int64_t at = (int64_t)split * p.T * p.heads + tq * p.heads + hq;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      if (16 * dt >= dim) break;
      if (n_splits <= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          store_elem(p.out, tq * p.o_ts + hq * p.o_hs + 16 * dt + 4 * g + e, st[n].o[dt][e] * inv,
                     p.dtype);
      } else {
        *(f32x4*)&p.part_o[at * dim + 16 * dt + 4 * g] =
            f32x4{st[n].o[dt][0], st[n].o[dt][1], st[n].o[dt][2], st[n].o[dt][3]};
      }
    }
    if (n_splits > 1 && g == 0) {
      p.part_ml[2 * at] = st[n].mx;
      p.part_ml[2 * at + 1] = sum;
    }
  }
}

}  // namespace attn
}  // namespace q4
