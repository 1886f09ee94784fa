// q4_attention_wide.h -- attention of many query rows of one sequence (chunks
// of a prompt) over the paged 8-bit cache.
//
// The mathematics and the operand layouts are those of
// q4_attention_kernels.h.  Here a workgroup holds 128 (or 64) rows of a kv
// head, 32 (16) in each of its four waves, and all of them read the keys and
// values of two tiles at a time from LDS, where global loads have put them
// directly, 1 KB to an operand of 16 rows and 64 columns in the order of the
// lanes that read it (so that neither side has a bank conflict).  Two buffers:
// the next pair of tiles loads while one is worked on, with one barrier a pair.
//
// Bound by the vector unit: with three digits a score takes 14 issue slots (4
// of them the exponential) and an output element 5 a pair of tiles.  What keeps
// them few:
//   * two tiles share a maximum and their outputs' way from integers to fp32
//     (one tile at a time took 1398 us where this took 1277, both with two
//     digits: 4 x 2048 tokens over 8192 each, 32 query and 8 kv heads of 128,
//     bf16; now 1532);
//   * the running maximum is only a reference that keeps the exponentials in
//     range: outputs are rescaled when a row's maximum passes it by 2^8, not
//     at every new maximum;
//   * tiles that all rows of a wave see whole skip the masks;
//   * nothing after a pair's loads waits for them before the next barrier: a
//     page number is checked a pair after its load (1277 to 1208 us with two
//     digits).
#pragma once

#include "q4_attention_kernels.h"

namespace q4 {
namespace attn {

constexpr float kSlack = 8.0f;                           // log2 that a maximum may pass the reference by

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef const __attribute__((address_space(1))) void* global_ptr;

// The digits' range of pair_softmax: its exponentials may pass 1 by the
// rounding of a product below kFarScore, 2^-8.
template <int ND>
__device__ __forceinline__ constexpr float pair_digit_max() {
  return ND == 4 ? 2113929216.0f : 8257536.0f;  // 126 * 256^(ND - 1)
}
constexpr float kFarScore = 65536.0f;

// Probabilities of two tiles that the row sees whole.  unit, vs: of the lane's
// tokens of each tile.  mx is a reference, at most kSlack below the
// maximum.  False, with nothing changed, where scores or scales are far out or
// not finite (tile_softmax takes those).
template <int ND>
__device__ __forceinline__ bool pair_softmax(const float (&raw)[2][4][4],
                                             const float (&unit)[2], const float (&vs)[2],
                                             float& mx, float& sum, i32x4 (&pd)[2][ND],
                                             float& alpha, float& w) {
  float tops[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float best = raw[t][0][0];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) best = fmaxf(best, raw[t][a][i]);
    tops[t] = best * unit[t];
  }
  const float top = column_max(fmaxf(tops[0], tops[1]));
  const bool fine = __builtin_fabsf(tops[0]) < kFarScore && __builtin_fabsf(tops[1]) < kFarScore &&
                    vs[0] < 1e30f && vs[1] < 1e30f;
  if (__any(!fine)) return false;
  // the largest p * scale is the digits' unit
  const float big = fmaxf(column_max(fmaxf(exp2_fast(tops[0] - top) * vs[0],
                                           exp2_fast(tops[1] - top) * vs[1])), 1e-30f);
  float part = 0.0f;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float to_digits = pair_digit_max<ND>() * (vs[t] / big);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      uint32_t bits[4], out[ND];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = exp2_fast(__builtin_fmaf(raw[t][a][i], unit[t], -top));
        part += e;
        bits[i] = digit_bits<ND>(e, to_digits);
      }
      pack_digits<ND>(bits[0], bits[1], bits[2], bits[3], out);
#pragma unroll
      for (int i = 0; i < ND; ++i) pd[t][i][a] = (int32_t)out[i];
    }
  }
  alpha = 1.0f;
  if (__any(top > mx + kSlack)) {
    const float to = top > mx + kSlack ? top : mx;
    alpha = to > mx ? exp2_fast(mx - to) : 1.0f;
    mx = to;
  }
  const float beta = exp2_fast(top - mx);
  sum = sum * alpha + beta * part;
  w = beta * big * (1.0f / pair_digit_max<ND>());
  return true;
}

// NC: 16-row blocks of a wave.
template <int DT, int ND, int NC, bool UNIFORM>
__global__ __launch_bounds__(kThreads, DT <= 8 ? 2 : 1) void attention_wide_kernel(AttnParams p) {
  constexpr int NS = (DT + 3) / 4;
  constexpr int KF = 4 * NS, FR = KF + DT;  // operands (1 KB each) of a tile: keys, all
  extern __shared__ char tiles[];           // [2 buffers][2 tiles][FR][1024]
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

  auto first_token = [&](int tile) { return (int64_t)(k.tile0 + tile) * kTile; };
  float ks_next[2] = {0.0f, 0.0f}, vs_next[2] = {0.0f, 0.0f};
  bool in_next[2] = {false, false};
  // every fourth operand of a tile, straight to LDS, and the lane's scales
  auto fetch = [&](int tile, int buf, int at, const Pages& pg) {
    const int32_t key = pg.key, own = pg.own;
    const int64_t token0 = first_token(tile);
    const int k_slot = (int)((token0 + (UNIFORM ? 0 : 16 * (col >> 2))) & page_mask);
    const int v_slot = (int)((token0 + (UNIFORM ? 0 : 16 * g)) & page_mask);
    const int64_t ph = (int64_t)(own > 0 ? own : 0) * c.heads + k.h;
    const int8_t* kb =
        c.k + ((((int64_t)(key > 0 ? key : 0) * c.heads + k.h) << c.page_log2) + k_slot) * dim;
    const int8_t* vb = c.v + ph * ((int64_t)dim << c.page_log2) + v_slot;
    const uint32_t k_off = (uint32_t)(((UNIFORM ? 16 * (col >> 2) : 0) + (col & 3)) * dim);
    const uint32_t v_off = (uint32_t)((col << c.page_log2) + (UNIFORM ? 16 * g : 0));
    char* to = tiles + (2 * buf + at) * FR * 1024;
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
    ks_next[at] = c.ks[ph];
    vs_next[at] = c.vs[ph];
    in_next[at] = own >= 0;
  };
  int32_t buf = 0;
  // table entries of the next pair of tiles, checked when it is fetched
  Pages raw[2];
  auto load_pair = [&](int tile) {
#pragma unroll
    for (int i = 0; i < 2; ++i) raw[i] = load_pages<UNIFORM>(p, table, first_token(tile + i));
  };
  auto fetch_pair = [&](int tile, int to) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (tile + i < t_end)
        fetch(tile + i, to, i, check_pages<UNIFORM>(p, raw[i], k.keys, first_token(tile + i)));
  };
  int t = split * p.split_tiles;
  load_pair(t);
  fetch_pair(t, 0);
  load_pair(t + 2);

  // the lane's query rows and what they see
  Column<DT> st[NC];
  i32x4 qd[NC][NS][ND];
  float q_unit[NC];
  int64_t see_lo[NC], see_hi[NC];
  const int64_t wave_row = k.row0 + wave * NC * kRows;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int64_t r = wave_row + n * kRows + col;
    const bool valid = r < k.rows;
    const int64_t tok = valid ? row_token(p, r) : 0;
    const int head = k.h * p.group + (int)(valid ? r - tok * p.group : 0);
    const int64_t pos = valid ? k.sp.pos0 + tok : -1;
    see_lo[n] = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
    see_hi[n] = pos < k.keys.hi ? pos : k.keys.hi - 1;
    column_init(st[n]);
    q_unit[n] = row_digits<NS, ND>(p, (k.sp.t0 + tok) * p.q_ts + (int64_t)head * p.q_hs, valid, g,
                                   qd[n]);
  }
  // positions that some and all of the wave's rows see
  const int64_t rows_end = wave_row + NC * kRows < k.rows ? wave_row + NC * kRows : k.rows;
  const int64_t pos_first = k.sp.pos0 + row_token(p, wave_row);
  const int64_t pos_last = k.sp.pos0 + row_token(p, rows_end - 1);
  const bool idle = wave_row >= k.rows;
  const KeyRange some = key_range(pos_first, pos_last, p.window, k.keys.hi);
  const int64_t all_hi = pos_first < k.keys.hi ? pos_first : k.keys.hi - 1;
  const int64_t all_lo = p.window > 0 ? pos_last - p.window + 1 : 0;

  for (; t < t_end; t += 2, buf ^= 1) {
    // this wave's part of the tiles has landed; past the barrier all of them
    // have, and every wave is done with the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    float ks[2], vs[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ks[i] = in_next[i] ? key_scale(ks_next[i]) : nan;
      vs[i] = in_next[i] ? scale_or_nan(vs_next[i]) : nan;
    }
    fetch_pair(t + 2, buf ^ 1);
    load_pair(t + 4);
    // A wave in its matrix instructions goes before one in its exponentials, so
    // that the two units are busy at once (2890 tokens over up to 5441, bf16: 269
    // us, 278 without it)
    __builtin_amdgcn_s_setprio(0);
    const int64_t token0 = (int64_t)(k.tile0 + t) * kTile;
    if (idle || token0 >= some.hi || token0 + 2 * kTile <= some.lo) continue;
    const bool whole =
        t + 1 < t_end && token0 >= all_lo && token0 + 2 * kTile - 1 <= all_hi;
    const char* from = tiles + 2 * buf * FR * 1024 + 16 * lane;
    i32x4 pd[NC][2][ND];
    float w[NC];
    bool pairs = false;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      bool done = false;
      if (whole) {
        float raw[2][4][4];
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            i32x4 acc[ND];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              const i32x4 kd = *(const i32x4*)(from + (i * FR + a * NS + s) * 1024);
#pragma unroll
              for (int m = 0; m < ND; ++m)
                acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                    kd, qd[n][s][m], s == 0 ? i32x4{0, 0, 0, 0} : acc[m], 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              int32_t part[ND];
#pragma unroll
              for (int m = 0; m < ND; ++m) part[m] = acc[m][e];
              raw[i][a][e] = join_digits<ND>(part);
            }
          }
        __builtin_amdgcn_s_setprio(0);
        const float unit[2] = {q_unit[n] * ks[0], q_unit[n] * ks[1]};
        float alpha = 1.0f;
        done = pair_softmax<ND>(raw, unit, vs, st[n].mx, st[n].sum, pd[n], alpha, w[n]);
        if (done && __any(alpha != 1.0f)) {
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int e = 0; e < 4; ++e) st[n].o[dt][e] *= alpha;
        }
      }
      if (!done) {
        // a tile at a time, with masks; the pair adds nothing below
        w[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int m = 0; m < ND; ++m) pd[n][i][m] = i32x4{0, 0, 0, 0};
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int64_t first = token0 + i * kTile;
          if (t + i >= t_end || first >= some.hi || first + kTile <= some.lo) continue;
          i32x4 kd[4][NS], vd[DT], digits[ND];
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int s = 0; s < NS; ++s)
              kd[a][s] = *(const i32x4*)(from + (i * FR + a * NS + s) * 1024);
          float sc[4][4], alpha, worth;
          tile_scores<NS, ND>(kd, qd[n], sc);
          const int64_t lo = see_lo[n] - (first + 16 * g), hi = see_hi[n] - (first + 16 * g);
          tile_softmax<ND, true, UNIFORM>(
              sc, q_unit[n] * (i ? ks[1] : ks[0]), i ? vs[1] : vs[0],
              (int)(lo > 16 ? 16 : lo < 0 ? 0 : lo), (int)(hi < -1 ? -1 : hi > 15 ? 15 : hi),
              st[n].mx, st[n].sum, digits, alpha, worth);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
            vd[dt] = *(const i32x4*)(from + (i * FR + KF + dt) * 1024);
          tile_values<DT, ND>(vd, digits, alpha, worth, st[n].o);
        }
      }
      pairs |= done;
    }
    if (!pairs) continue;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const i32x4 v0 = *(const i32x4*)(from + (KF + dt) * 1024);
      const i32x4 v1 = *(const i32x4*)(from + (FR + KF + dt) * 1024);
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        i32x4 acc[ND];
#pragma unroll
        for (int m = 0; m < ND; ++m) {
          acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v0, pd[n][0][m], i32x4{0, 0, 0, 0}, 0, 0, 0);
          acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v1, pd[n][1][m], acc[m], 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int32_t part[ND];
#pragma unroll
          for (int m = 0; m < ND; ++m) part[m] = acc[m][e];
          st[n].o[dt][e] = __builtin_fmaf(join_digits<ND>(part), w[n], st[n].o[dt][e]);
        }
      }
    }
  }

#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int64_t r = wave_row + n * kRows + col;
    const float sum = column_sum(st[n].sum);
    if (r >= k.rows) continue;
    const int64_t tok = row_token(p, r);
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
