// q4_experts_gemm.h -- activations times packed 4-bit matrices for many rows,
// on MFMA; instantiated by q4_experts_gemm_*.hip.
//
//   z[r, n] = sum_g s[g, n] * sum_{k in g} a[r, k] c[n, k]
//
// with the rows of an expert (or of the head) in tiles of BM and 128 columns,
// four waves (WaveGrid) as 32x32x16 products.  A step is 64 k: rows of a and
// packed words come by direct loads into LDS (chunks of 16 bytes of a turned by
// row so that the reads meet no bank twice) in a ring of S stages, a barrier
// each.  A wave unpacks the words it needs itself.  A group's products are summed
// by MFMA and added to the result in fp32 times the column's scale; with a scale
// per row of the matrix there is one group and one multiplication.
//
// Bound: MFMA against the vector unit's unpacking (9 operations a word) and group
// sums (64 a group and wave).  Head of 128257 x 2048, a scale per row: 2048 rows
// of bf16 1.07 ms, 1000 TFLOP/s; 512 of fp32 0.49 ms, twice 550 (a library
// product of binary16, 8192^3, reaches 1324).  4099 tokens by 8 over 64 experts
// of 2048 x 1024 in groups of 128, bf16: gate and up 402 us, 685 TFLOP/s, down (two
// parts) 335, twice 410, where a ninth of the tiles' rows are empty.
#pragma once

#include "q4_experts.h"
#include "q4_experts_device.h"

namespace q4 {

typedef const __attribute__((address_space(1))) void* global_cptr;
typedef __attribute__((address_space(3))) void* lds_vptr;

enum GroupMode : int { kOneGroup = 0, kGroups64 = 1, kGroups32 = 2 };

constexpr int kBN = 128;
constexpr int kBK = 64;

template <int P, int BM, int GM>
struct GemmTile {
  static constexpr int kGroupsPerStep = GM == kGroups32 ? 2 : 1;
  static constexpr int kA = P * BM * kBK * 2;
  static constexpr int kB = kBN * kBK / 2;
  static constexpr int kScale = GM == kOneGroup ? 0 : kGroupsPerStep * kBN * 4;
  static constexpr int kStage = kA + kB + kScale;
  // one group: two stages (three workgroups a CU, or two of 128 rows in two
  // parts); else two workgroups, of three stages where LDS allows it
  static constexpr int kStages = GM != kOneGroup && 3 * kStage <= 76 * 1024 ? 3 : 2;
  // vector memory operations a wave issues per step
  static constexpr int kIssue = P * BM / 32 + 1 + (GM == kOneGroup ? 0 : 1);
};

// The four waves of a tile.  Of 64 rows in one part, each has all rows of 32
// columns: a word is unpacked once, at the price of reading the rows from LDS by
// four waves and not two.  With two parts LDS would bound it (32003 x 2048, 96
// rows of fp32: 52 us so, 44 with waves of 32 rows by 64 columns).
template <int P, int BM>
struct WaveGrid {
  static constexpr int WC = BM == 64 && P == 1 ? 4 : 2;  // waves side by side
  static constexpr int CB = 4 / WC;                      // column blocks of 32 of a wave
  static constexpr int RB = BM * WC / 128;               // and of rows
};

template <int N>
__device__ __forceinline__ void wait_loads() {
  // vmcnt(N), other counters left free; no load moves past it
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Loads before it are issued before those after it: a wait that counts the newest
// loads relies on their order, which the compiler is otherwise free to change.
__device__ __forceinline__ void keep_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Maximum or sum over the 32 lanes of a half for 16 values: each step halves
// the values a lane holds, so 16 exchanges do where 80 would.  Lane l ends with
// value (l & 15) for lanes 0..15 of its half (and again for 16..31).
template <typename F>
__device__ __forceinline__ float reduce16(const float (&v)[16], int lane, F f) {
  float a[8], b[4], c[2], d;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool up = lane & 8;
    const float keep = up ? v[i + 8] : v[i], give = up ? v[i] : v[i + 8];
    a[i] = f(keep, __shfl_xor(give, 8, 64));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 4;
    const float keep = up ? a[i + 4] : a[i], give = up ? a[i] : a[i + 4];
    b[i] = f(keep, __shfl_xor(give, 4, 64));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 2;
    const float keep = up ? b[i + 2] : b[i], give = up ? b[i] : b[i + 2];
    c[i] = f(keep, __shfl_xor(give, 2, 64));
  }
  {
    const bool up = lane & 1;
    const float keep = up ? c[1] : c[0], give = up ? c[0] : c[1];
    d = f(keep, __shfl_xor(give, 1, 64));
  }
  return f(d, __shfl_xor(d, 16, 64));
}

template <bool B>
struct Flag {
  static constexpr bool value = B;
};
typedef Flag<true> Yes;
typedef Flag<false> No;

template <int P, int BM, int GM, Epilogue EPI>
__global__ void __launch_bounds__(256, GM == kOneGroup && P == 1 ? 3 : 2) gemm_kernel(const GemmParams p) {
  typedef GemmTile<P, BM, GM> L;
  typedef WaveGrid<P, BM> G;
  constexpr int WC = G::WC, CB = G::CB, RB = G::RB;
  constexpr int S = L::kStages;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int32_t sh_slot[BM], sh_exp[BM];
  constexpr bool kHead = EPI == kHeadStats || EPI == kHeadGrad;
  __shared__ int32_t sh_target[kHead ? BM : 1];
  __shared__ float sh_lse[EPI == kHeadGrad ? BM : 1], sh_g[EPI == kHeadGrad ? BM : 1];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = w / WC, wc = w % WC, c = lane & 31, q = lane >> 5;

  // which tile
  const int32_t row_tiles = p.tiles ? *p.n_tiles : p.row_tiles;
  const uint32_t total = (uint32_t)row_tiles * (uint32_t)p.col_tiles;
  if (blockIdx.x >= total) return;
  const uint32_t at = xcd_swizzle(blockIdx.x, total);
  int mt, ct, expert = 0, first, rows;
  if (p.tiles) {
    // an XCD takes the column tiles of one expert's rows one after the other
    mt = (int)(at / (uint32_t)p.col_tiles);
    ct = (int)(at % (uint32_t)p.col_tiles);
    const Tile t = p.tiles[mt];
    expert = t.expert;
    first = t.first;
    rows = t.rows;
  } else {
    // the head: all rows of a column tile together, so that the matrix is read once
    mt = (int)(at % (uint32_t)row_tiles);
    ct = (int)(at / (uint32_t)row_tiles);
    first = mt * BM;
    rows = (int)(p.M - first < BM ? p.M - first : BM);
  }

  // the tile's rows; those past its end repeat the last
  auto row_of = [&](int r) { return r < rows ? r : rows - 1; };
  if (tid < BM) {
    const int r = row_of(tid);
    const int32_t slot = p.slots ? p.slots[first + r] : first + r;
    const int64_t ar = p.slots ? slot / p.slots_per_row : slot;
    sh_slot[tid] = tid < rows ? slot : -1;
    sh_exp[tid] = p.a.e[ar];
    if constexpr (kHead) {
      const int64_t t = p.targets[ar] - p.n0 - (int64_t)ct * kBN;
      sh_target[tid] = p.targets[ar] >= 0 && t >= 0 && t < kBN ? (int32_t)t : -1;
    }
    if constexpr (EPI == kHeadGrad) {
      sh_lse[tid] = p.lse[ar];
      sh_g[tid] = p.targets[ar] >= 0 ? p.g[ar] : 0.0f;
    }
  }

  // sources of this lane's direct loads
  const _Float16* asrc[BM / 32];
#pragma unroll
  for (int i = 0; i < BM / 32; ++i) {
    const int r = w * (BM / 4) + i * 8 + (lane >> 3);
    const int rr = row_of(r);
    const int32_t slot = p.slots ? p.slots[first + rr] : first + rr;
    const int64_t ar = p.slots ? slot / p.slots_per_row : slot;
    asrc[i] = p.a.a + ar * p.a.Kp + ((lane & 7) ^ ((r >> 1) & 7)) * 8;
  }
  const int64_t piece = p.a.rows * p.a.Kp;
  // packed row of a local column
  auto packed_row = [&](int n) -> int64_t {
    if constexpr (EPI == kGatedRows) {
      constexpr int side = CB * 16;  // columns of a wave's gate, up's beside them
      const int64_t h = (int64_t)ct * 64 + n / (2 * side) * side + n % side;
      const int64_t hc = h < p.width ? h : p.width - 1;
      return (n & side) ? p.width + hc : hc;
    } else {
      const int64_t col = (int64_t)ct * kBN + n;
      return p.n0 + (col < p.n_cols ? col : p.n_cols - 1);
    }
  };
  // packed words: 16 bytes a lane (half a row's step), or 4 where rows are not
  // so aligned
  const int64_t ldq = p.w.K >> 1;
  const bool wide = p.b_wide != 0;
  const uint8_t* bbase = p.w.qw + expert * p.w.expert_bytes;
  const uint8_t* bsrc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    bsrc[i] = bbase + packed_row(wide ? tid >> 1 : w * 32 + i * 8 + (lane >> 3)) * ldq;
  // (within a step of a row; its halves change places by the row's eighth, so that
  // the reads of 16 lanes meet no bank twice)
  const int b_byte = wide ? ((tid ^ (tid >> 4)) & 1) * 16 : (lane & 7) * 4;
  // scales of a step's groups, 4 bytes a lane
  const float* ssrc = nullptr;
  int sslot = 0, sgroup = 0;
  if constexpr (GM != kOneGroup) {
    sgroup = GM == kGroups32 ? w >> 1 : 0;
    ssrc = p.w.scales + expert * p.w.expert_scales + packed_row((w & 1) * 64 + lane);
    sslot = sgroup * kBN + (w & 1) * 64;
  }

  const int steps = (int)(p.a.Kp / kBK);
  const int per_group = GM == kGroups64 ? p.w.group / kBK : 1;  // steps of a group

  auto issue = [&](int step) {
    // past the last step it loads that one again, so that every step waits for as many loads
    const int st = step < steps ? step : steps - 1;
    uint8_t* base = smem + (step % S) * L::kStage;
#pragma unroll
    for (int pc = 0; pc < P; ++pc)
#pragma unroll
      for (int i = 0; i < BM / 32; ++i)
        __builtin_amdgcn_global_load_lds(
            (global_cptr)(asrc[i] + pc * piece + (int64_t)st * kBK),
            (lds_vptr)(base + pc * BM * 128 + (w * (BM / 4) + i * 8) * 128), 16, 0, 0);
    if constexpr (GM != kOneGroup) {
      const int g0 = GM == kGroups32 ? 2 * st : st / per_group;
      // (the second half of the last step may be past the last group: a sum of
      // zeros, times any scale)
      const int sg = g0 + sgroup < p.w.G ? g0 + sgroup : p.w.G - 1;
      __builtin_amdgcn_global_load_lds((global_cptr)(ssrc + (int64_t)sg * p.w.N),
                                       (lds_vptr)(base + L::kA + L::kB + sslot * 4), 4, 0, 0);
    }
    // words past K are other rows' (here the row's first): activations are 0 there
    auto from = [&](int at) {
      const int64_t byte = (int64_t)st * (kBK / 2) + at;
      return byte < ldq ? byte : 0;
    };
    if (wide) {
      __builtin_amdgcn_global_load_lds((global_cptr)(bsrc[0] + from(b_byte)),
                                       (lds_vptr)(base + L::kA + w * 1024), 16, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_global_load_lds((global_cptr)(bsrc[i] + from(b_byte ^ (i & 1) * 16)),
                                         (lds_vptr)(base + L::kA + w * 1024 + i * 256), 4, 0, 0);
    }
  };

  f32x16 out[RB][CB], acc[RB][CB];
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int b = 0; b < CB; ++b) {
      out[r][b] = f32x16{};
      acc[r][b] = f32x16{};
    }

  // where this lane reads
  int a_at[RB], a_turn[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int row = (wr * RB + r) * 32 + c;
    a_at[r] = row * 128;
    a_turn[r] = (row >> 1) & 7;
  }
  const int b_at = (wc * CB * 32 + c) * 32 + (c >> 3 & 1) * 16 + q * 8;

  const Magic magic = Magic::make();
  auto fold = [&](const uint8_t* base, int g) {
    const float* s = (const float*)(base + L::kA + L::kB) + g * kBN + wc * CB * 32 + c;
#pragma unroll
    for (int b = 0; b < CB; ++b) {
      const float sc = s[b * 32];
#pragma unroll
      for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i) out[r][b][i] = __builtin_fmaf(acc[r][b][i], sc, out[r][b][i]);
    }
  };
  // a step's products; FIRST: its (or its groups') sums start anew
  auto products = [&](const uint8_t* base, auto first_step) {
    constexpr bool FIRST = decltype(first_step)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t words[CB][2];
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const u32x2 x = *(const u32x2*)(base + L::kA + (b_at ^ h * 16) + b * 32 * 32);
        words[b][0] = x[0];
        words[b][1] = x[1];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        h8 bo[CB];
#pragma unroll
        for (int b = 0; b < CB; ++b) bo[b] = codes_of(words[b][j], magic);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
#pragma unroll
          for (int pc = 0; pc < P; ++pc) {
            const int chunk = (h * 4 + q * 2 + j) ^ a_turn[r];
            const h8 a = *(const h8*)(base + pc * BM * 128 + a_at[r] + chunk * 16);
            const bool start = GM == kGroups32 ? j == 0 && pc == 0
                                               : GM == kGroups64 && FIRST && h == 0 && j == 0 && pc == 0;
#pragma unroll
            for (int b = 0; b < CB; ++b)
              acc[r][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, bo[b], start ? f32x16{} : acc[r][b], 0, 0, 0);
          }
        }
      }
      if constexpr (GM == kGroups32) fold(base, h);
    }
  };
  // a wave without rows (of a tile that is not full) loads for the others
  const bool idle = wr * RB * 32 >= rows;
  issue(0);
  if constexpr (S == 3) {
    keep_order();
    issue(1);
  }
  auto begin = [&](int step) -> const uint8_t* {
    wait_loads<(S - 2) * L::kIssue>();
    lds_barrier();
    issue(step + S - 1);
    return smem + (step % S) * L::kStage;
  };
  if constexpr (GM == kGroups64) {
    for (int st = 0; st < steps;) {
      const uint8_t* base = begin(st++);
      if (!idle) products(base, Yes{});
      const int end = st + per_group - 1 < steps ? st + per_group - 1 : steps;
      for (; st < end;) {
        base = begin(st++);
        if (!idle) products(base, No{});
      }
      settle(acc);
      fold(base, 0);
    }
  } else {
    for (int st = 0; st < steps; ++st) {
      const uint8_t* base = begin(st);
      if (!idle) products(base, No{});
    }
    settle(acc);
  }

  // ---- results -------------------------------------------------------------
  wait_loads<0>();  // loads past the last step write LDS
  float scale0[2] = {1.0f, 1.0f};
  if constexpr (GM == kOneGroup) {
#pragma unroll
    for (int b = 0; b < CB; ++b)
      scale0[b] = p.w.scales[expert * p.w.expert_scales + packed_row((wc * CB + b) * 32 + c)];
  }
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int r0 = (wr * RB + r) * 32 + 4 * q;
    float z[CB][16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = r0 + 8 * (i >> 2) + (i & 3);
      const int e = sh_exp[row];
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        if constexpr (GM == kOneGroup)
          z[b][i] = __builtin_ldexpf(acc[r][b][i] * scale0[b], -e);
        else
          z[b][i] = __builtin_ldexpf(out[r][b][i], -e);
      }
    }
    if constexpr (EPI == kGatedRows) {
      auto put = [&](int i, float g, float u, int64_t h) {
        const int slot = sh_slot[r0 + 8 * (i >> 2) + (i & 3)];
        if (slot < 0 || h >= p.width) return;
        p.out[(int64_t)slot * p.out_ld + h] = g * sigmoid(g) * u;
        if (p.pre) {
          float* pre = p.pre + (int64_t)slot * 2 * p.width + h;
          pre[0] = g;
          pre[p.width] = u;
        }
      };
      if constexpr (CB == 2) {
#pragma unroll
        for (int i = 0; i < 16; ++i) put(i, z[0][i], z[1][i], (int64_t)ct * 64 + wc * 32 + c);
      } else {
        // lanes of the gate and of up change halves of their rows
        const bool up = c & 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float other = __shfl_xor(up ? z[0][i] : z[0][i + 8], 16, 64);
          const float mine = up ? z[0][i + 8] : z[0][i];
          put(up ? i + 8 : i, up ? other : mine, up ? mine : other, (int64_t)ct * 64 + wc * 16 + (c & 15));
        }
      }
    } else if constexpr (EPI == kPlainRows) {
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const int64_t col = (int64_t)ct * kBN + (wc * CB + b) * 32 + c;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int slot = sh_slot[r0 + 8 * (i >> 2) + (i & 3)];
          if (slot >= 0 && col < p.n_cols) p.out[(int64_t)slot * p.out_ld + col] = z[b][i];
        }
      }
    } else if constexpr (EPI == kHeadStats) {
      float m[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = r0 + 8 * (i >> 2) + (i & 3), slot = sh_slot[row], t = sh_target[row];
        m[i] = -__builtin_inff();
#pragma unroll
        for (int b = 0; b < CB; ++b) {
          const int col = (wc * CB + b) * 32 + c;
          if (slot >= 0 && t == col) p.chosen[slot] = z[b][i];
          if ((int64_t)ct * kBN + col >= p.n_cols) z[b][i] = -__builtin_inff();
          m[i] = b == 0 || z[b][i] > m[i] ? z[b][i] : m[i];
        }
      }
      // lane l of a half ends with row value l & 15's maximum, and hands it back
      const float mine = reduce16(m, lane, [](float x, float y) { return x > y ? x : y; });
      float s[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float top = __shfl(mine, (lane & 48) | i, 64);
        const float base = top > -__builtin_inff() ? top : 0.0f;
        s[i] = 0.0f;
#pragma unroll
        for (int b = 0; b < CB; ++b) s[i] += exp2_fast((z[b][i] - base) * kLog2e);
      }
      const float sum = reduce16(s, lane, [](float x, float y) { return x + y; });
      if ((lane & 16) == 0) {
        const int i = lane & 15, row = r0 + 8 * (i >> 2) + (i & 3), slot = sh_slot[row];
        if (slot >= 0) {
          float* st = p.stats + (((int64_t)slot * p.col_tiles + ct) * WC + wc) * 2;
          st[0] = mine;
          st[1] = sum;
        }
      }
    } else if constexpr (GM != kOneGroup) {
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const int col = (wc * CB + b) * 32 + c;
        if ((int64_t)ct * kBN + col >= p.n_cols) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = r0 + 8 * (i >> 2) + (i & 3), slot = sh_slot[row];
          if (slot < 0) continue;
          const float g = sh_g[row];
          const float pr = exp_full(z[b][i] - sh_lse[row]) - (sh_target[row] == col ? 1.0f : 0.0f);
          p.d[(int64_t)slot * p.out_ld + (int64_t)ct * kBN + col] = g != 0.0f ? g * pr : 0.0f;
        }
      }
    } else {
      // a scale per column: the gradient's operand is complete here, zeros up
      // to the tile's end
      const int s_exp = top_exponent(*p.s_bits);
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const int col = (wc * CB + b) * 32 + c;
        const float s = (int64_t)ct * kBN + col < p.n_cols ? __builtin_ldexpf(scale0[b], 15 - s_exp) : 0.0f;
        _Float16* to = p.d_parts + (int64_t)ct * kBN + (col & ~7) + operand_place(col & 7);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = r0 + 8 * (i >> 2) + (i & 3), slot = sh_slot[row];
          if (slot < 0) continue;
          const float g = sh_g[row];
          const float pr = exp_full(z[b][i] - sh_lse[row]) - (sh_target[row] == col ? 1.0f : 0.0f);
          const float x = s != 0.0f && g != 0.0f ? settled(__builtin_ldexpf(g, -top_exponent(finite_bits(g))) * pr * s) : 0.0f;
          _Float16* dst = to + (int64_t)slot * p.out_ld;
          const _Float16 hi = part_hi(x);
          *dst = hi;
          dst[p.a.rows * p.out_ld] = part_lo(x, hi);
        }
      }
    }
  }
}

template <int P, int BM, Epilogue EPI>
hipError_t launch_gemm_tile(const GemmParams& p, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.row_tiles * p.col_tiles));
#define Q4_GEMM(GM)                                                                        \
  do {                                                                                     \
    typedef GemmTile<P, BM, GM> L;                                                         \
    constexpr int lds = L::kStages * L::kStage;                                            \
    if (lds > 64 * 1024) {                                                                 \
      const hipError_t e = hipFuncSetAttribute((const void*)gemm_kernel<P, BM, GM, EPI>,    \
                                               hipFuncAttributeMaxDynamicSharedMemorySize, \
                                               lds);                                       \
      if (e != hipSuccess) return e;                                                       \
    }                                                                                      \
    hipLaunchKernelGGL((gemm_kernel<P, BM, GM, EPI>), grid, dim3(256), lds, s, p);         \
  } while (0)
  if (p.w.group == 0)
    Q4_GEMM(kOneGroup);
  else if (p.w.group == 32)
    Q4_GEMM(kGroups32);
  else
    Q4_GEMM(kGroups64);
#undef Q4_GEMM
  return hipGetLastError();
}

}  // namespace q4
