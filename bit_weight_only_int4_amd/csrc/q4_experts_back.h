// q4_experts_back.h -- the input gradient through packed 4-bit matrices for
// many rows, on MFMA; instantiated by q4_experts_back_*.hip.
//
//   z[r, k] = sum_n (d[r, n] s[g(k), n]) c[n, k]
//
// contracted over the rows n of the packed matrix.  The scale of a column's
// group belongs to the row operand here: d times the scales of the tile's
// group is formed in fp32 on the way into LDS and split into binary16 parts
// there (d against its row's largest magnitude, the scales against their
// group's), so codes stay exact integers.  128 columns of one group need one
// such operand; with groups of 32 or 64 each 32 columns have their own (NG = 4).
//
// Codes lie along k, the contraction runs along n: a thread takes a word (8 k)
// of four rows n, turns its 4 x 8 nibbles around in registers (12 operations)
// and writes 16 bits for each k, so LDS holds the tile packed along n and a
// wave unpacks it as the forward product does.  Within each 32 columns the order
// is (k in word, word % 4), and pieces of 8 bytes are turned, so that writes and
// reads spread over the banks.
//
// Tiles of BM rows by 128 columns, four waves of 64 rows by BM/2 columns; the
// next two steps' loads are in registers while a step's products run (the next
// step's where LDS holds one stage: 128 rows, NG = 4).
//
// Bound: the vector unit, which forms the row operand anew for every tile of
// columns (6 operations an element) beside the codes'.  2048 tokens by 4 over 32
// experts of 2048 x 1408 in groups of 128, bf16: through down 230 us, through gate
// and up 275, 205 and 345 TFLOP/s (twice that in its two parts).
#pragma once

#include "q4_experts.h"
#include "q4_experts_device.h"
#include "q4_experts_gemm.h"

namespace q4 {

// The row operand is a value computed on the way: two binary16 parts (22 bits)
// whatever the activations' type.
constexpr int kParts = 2;

template <int BM, int NG>
struct BackTile {
  static constexpr int kN = NG == 1 ? 64 : 32;  // n of a step
  static constexpr int kPart = BM * kN * 2;     // bytes of one part of one operand
  static constexpr int kA = NG * kParts * kPart;
  static constexpr int kB = 128 * kN / 2;
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = 2 * kStage <= 76 * 1024 ? 2 : 1;
};

// Words of rows n .. n + 3 at the same 8 k, as 8 half words: element i holds
// nibble i of the four rows, the first row lowest.  Pairs (0, 4), (1, 5), (2,
// 6), (3, 7) share a register: low half first.
__device__ __forceinline__ void turn_words(const uint32_t (&w)[4], uint32_t (&t)[4]) {
  constexpr uint32_t m = 0x0F0F0F0Fu;
  const uint32_t e01 = (w[0] & m) | ((w[1] << 4) & ~m), e23 = (w[2] & m) | ((w[3] << 4) & ~m);
  const uint32_t o01 = ((w[0] >> 4) & m) | (w[1] & ~m), o23 = ((w[2] >> 4) & m) | (w[3] & ~m);
  // bytes j of the e's are nibble 2 j of two rows each, of the o's nibble 2 j + 1
  t[0] = __builtin_amdgcn_perm(e23, e01, 0x06020400u);  // nibbles 0 and 4
  t[1] = __builtin_amdgcn_perm(o23, o01, 0x06020400u);  // 1, 5
  t[2] = __builtin_amdgcn_perm(e23, e01, 0x07030501u);  // 2, 6
  t[3] = __builtin_amdgcn_perm(o23, o01, 0x07030501u);  // 3, 7
}

// Where 8 bytes of a column's codes lie (of NS / 16 such pieces): turned by the
// column's eighth of 32 and by its 32, so that reads of 16 lanes and writes of 64
// meet no bank twice.
template <int NS>
__device__ __forceinline__ int turned(int piece, int eighth, int block) {
  return piece ^ ((eighth ^ block) & (NS / 16 - 1));
}
// A word (8 k) of rows n .. n + 3 into LDS: word kw of 16, rows' place u of NS /
// 4.  Element i is column (kw / 4) * 32 + kw % 4 + 4 i, in the eighth i / 2 (the
// words' low element second if flip).
template <int NS>
__device__ __forceinline__ void store_turned(uint8_t* b, const uint32_t (&w)[4], int kw, int u, bool flip) {
  uint32_t t[4];
  turn_words(w, t);
  const uint32_t e[4] = {flip ? t[1] : t[0], flip ? t[0] : t[1], flip ? t[3] : t[2], flip ? t[2] : t[3]};
  const int at = ((kw >> 2) * 32 + (kw & 3)) * (NS / 2) + turned<NS>(u >> 2, 0, kw >> 2) * 8 + (u & 3) * 2;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint8_t *lo = b + (at ^ turned<NS>(0, j, 0) * 8), *hi = b + (at ^ turned<NS>(0, j + 2, 0) * 8);
#pragma unroll
    for (int i = 2 * j; i < 2 * j + 2; ++i) {
      *(uint16_t*)(lo + i * 4 * (NS / 2)) = (uint16_t)e[i];
      *(uint16_t*)(hi + (i + 4) * 4 * (NS / 2)) = (uint16_t)(e[i] >> 16);
    }
  }
}

template <typename T, int BM, int NG, bool GATE>
__global__ void __launch_bounds__(256, 2) back_kernel(const BackParams p) {
  typedef BackTile<BM, NG> L;
  constexpr int CB = BM / 64, WC = 4 / CB, NS = L::kN, S = L::kStages;
  constexpr int kChunks = NS / 8;            // 16-byte pieces of a row
  constexpr int kPasses = BM * kChunks / 256;  // rows of a thread
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int32_t sh_slot[BM], sh_exp[BM];
  __shared__ float sh_weight[GATE ? BM : 1];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = w / WC, wc = w % WC, c = lane & 31, q = lane >> 5;

  const int32_t row_tiles = p.tiles ? *p.n_tiles : p.row_tiles;
  const uint32_t total = (uint32_t)row_tiles * (uint32_t)p.col_tiles * (uint32_t)p.splits;
  if (blockIdx.x >= total) return;
  uint32_t at = xcd_swizzle(blockIdx.x, total);
  int mt, ct, split = 0, expert = 0, first, rows;
  if (p.tiles) {
    mt = (int)(at / (uint32_t)p.col_tiles);
    ct = (int)(at % (uint32_t)p.col_tiles);
    const Tile t = p.tiles[mt];
    expert = t.expert;
    first = t.first;
    rows = t.rows;
  } else {
    // rows of d, the larger operand, stay with one XCD
    const uint32_t plane = (uint32_t)row_tiles * (uint32_t)p.col_tiles;
    split = (int)(at / plane);
    at %= plane;
    mt = (int)(at / (uint32_t)p.col_tiles);
    ct = (int)(at % (uint32_t)p.col_tiles);
    first = mt * BM;
    rows = (int)(p.M - first < BM ? p.M - first : BM);
  }
  const int64_t K = p.w.K, N = p.w.N, ldq = K >> 1;
  const int64_t k0 = (int64_t)ct * 128;
  // this split's rows of the matrix
  const int64_t per = ((p.n_rows + p.splits - 1) / p.splits + NS - 1) / NS * NS;
  const int64_t nb = per * split < p.n_rows ? per * split : p.n_rows;
  const int64_t ne = nb + per < p.n_rows ? nb + per : p.n_rows;
  const int steps = (int)((ne - nb + NS - 1) / NS);

  auto row_of = [&](int r) { return r < rows ? r : rows - 1; };
  if (tid < BM) {
    const int r = row_of(tid);
    const int32_t slot = p.slots ? p.slots[first + r] : first + r;
    const int64_t dr = p.slots ? slot / p.slots_per_row : slot;
    sh_slot[tid] = tid < rows ? slot : -1;
    sh_exp[tid] = top_exponent(p.d_bits[dr]);
    if constexpr (GATE) sh_weight[tid] = p.weights[slot];
  }

  // this thread's part of the row operand: 8 n of kPasses rows
  const int chunk = tid % kChunks, arow = tid / kChunks;
  const T* dsrc[kPasses];
  int de[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row_of(arow + i * (256 / kChunks));
    const int32_t slot = p.slots ? p.slots[first + r] : first + r;
    const int64_t dr = p.slots ? slot / p.slots_per_row : slot;
    dsrc[i] = (const T*)p.d + dr * p.ldd;
    de[i] = -top_exponent(p.d_bits[dr]);
  }
  const float* scales = p.w.scales + expert * p.w.expert_scales + p.n0;
  // (a group's scales against its largest: a group far below the others keeps its bits)
  const uint32_t* s_bits = p.s_bits + (int64_t)expert * p.w.G;
  auto group_of = [&](int64_t k) {
    const int64_t g = p.w.group ? k / p.w.group : 0;
    return g < p.w.G ? g : p.w.G - 1;
  };
  int64_t group_at[NG];
  int s_exp[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    group_at[g] = group_of(k0 + g * 32) * N;
    s_exp[g] = top_exponent(s_bits[group_of(k0 + g * 32)]);
  }
  // and of the codes: a word of four rows
  const int kw = tid & 15, u = tid >> 4;
  const bool codes_mine = u < NS / 4;
  // (addresses are a step's base, the same for all lanes, and a lane's 32-bit offset)
  const uint32_t code_at = (uint32_t)(k0 + kw * 8 < K ? k0 / 8 + kw : 0) * 4u + (uint32_t)(4 * u) * (uint32_t)ldq;
  const uint8_t* codes = p.w.qw + expert * p.w.expert_bytes + (p.n0 + nb) * ldq;
  const uint32_t scale_at = (uint32_t)chunk * 8u;

  const bool d_vec = p.d_vec != 0;
  struct Fetch {
    float d[kPasses][8], s[NG][8];
    uint32_t w[4];
  };
  // (past the last step it loads that one again: the waits count on as many
  // loads whatever the way through the loop)
  auto fetch = [&](Fetch& f, int at_step) {
    const int step = at_step < steps ? at_step : steps - 1;
    const int64_t n0 = nb + (int64_t)step * NS, n = n0 + chunk * 8;
    const uint8_t* code = codes + (int64_t)step * NS * ldq;
    if (n0 + NS <= ne) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        if (d_vec) {
          constexpr int v = 16 / sizeof(T);
          typedef T tv __attribute__((ext_vector_type(v)));
#pragma unroll
          for (int j = 0; j < 8 / v; ++j) {
            const tv x = *(const tv*)(dsrc[i] + n + j * v);
#pragma unroll
            for (int e = 0; e < v; ++e) f.d[i][j * v + e] = to_f32(x[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) f.d[i][e] = to_f32(dsrc[i][n + e]);
        }
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float* s = scales + (group_at[g] + n0);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f32x4_a4 x = *(const f32x4_a4*)(s + (scale_at + 4 * j));
#pragma unroll
          for (int e = 0; e < 4; ++e) f.s[g][j * 4 + e] = x[e];
        }
      }
      if (codes_mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f.w[i] = *(const uint32_t*)(code + i * ldq + code_at);
      }
    } else {
      // the last step: zeros past the end (and any codes)
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) f.d[i][e] = n + e < ne ? to_f32(dsrc[i][n + e]) : 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) f.s[g][e] = n + e < ne ? scales[group_at[g] + n + e] : 0.0f;
      if (codes_mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t r = n0 + 4 * u + i;
          f.w[i] = *(const uint32_t*)(codes + ((r < ne ? r : ne - 1) - nb) * ldq + (code_at - (uint32_t)(4 * u) * (uint32_t)ldq));
        }
      }
    }
  };
  auto turn_of = [](int row) { return NS == 64 ? (row >> 1) & 7 : (row >> 2) & 3; };
  auto store = [&](const Fetch& f, int step) {
    uint8_t* base = smem + (S == 2 ? (step & 1) * L::kStage : 0);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float s[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = __builtin_ldexpf(f.s[g][operand_nibble(e)], 15 - s_exp[g]);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int row = arow + i * (256 / kChunks);
        h8 hi, lo;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = settled(__builtin_ldexpf(f.d[i][operand_nibble(e)], de[i]) * s[e]);
          hi[e] = part_hi(x);
          lo[e] = part_lo(x, hi[e]);
        }
        uint8_t* dst = base + g * kParts * L::kPart + row * (NS * 2) + ((chunk ^ turn_of(row)) * 16);
        *(h8*)dst = hi;
        *(h8*)(dst + L::kPart) = lo;
      }
    }
    if (codes_mine) store_turned<NS>(base + L::kA, f.w, kw, u, p.nibble_order != Q4_ORDER_LOW_FIRST);
  };

  f32x16 acc[2][CB];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int b = 0; b < CB; ++b) acc[r][b] = f32x16{};
  const Magic magic = Magic::make();
  auto products = [&](int step) {
    const uint8_t* base = smem + (S == 2 ? (step & 1) * L::kStage : 0);
#pragma unroll
    for (int h = 0; h < NS / 32; ++h) {
      uint32_t words[CB][2];
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const u32x2 x = *(const u32x2*)(base + L::kA + ((wc * CB + b) * 32 + c) * (NS / 2) + turned<NS>(h * 2 + q, c >> 3, wc * CB + b) * 8);
        words[b][0] = x[0];
        words[b][1] = x[1];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        h8 bo[CB];
#pragma unroll
        for (int b = 0; b < CB; ++b) bo[b] = codes_of(words[b][j], magic);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = wr * 64 + r * 32 + c;
          const int at_ = row * (NS * 2) + (((h * 4 + q * 2 + j) ^ turn_of(row)) * 16);
#pragma unroll
          for (int pc = 0; pc < kParts; ++pc) {
#pragma unroll
            for (int b = 0; b < CB; ++b) {
              const int g = NG == 1 ? 0 : wc * CB + b;
              const h8 a = *(const h8*)(base + (g * kParts + pc) * L::kPart + at_);
              acc[r][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, bo[b], acc[r][b], 0, 0, 0);
            }
          }
        }
      }
    }
  };

  const bool idle = wr * 64 >= rows;  // a wave without rows
  if constexpr (S == 2) {
    // loads two steps ahead of their use: a step's products are shorter than
    // the way from memory
    Fetch f0, f1;
    if (steps > 0) {
      fetch(f0, 0);
      fetch(f1, 1);
      store(f0, 0);
      fetch(f0, 2);
      lds_barrier();
      for (int st = 0; st < steps; st += 2) {
        if (!idle) products(st);
        store(f1, st + 1);
        fetch(f1, st + 3);
        lds_barrier();
        if (st + 1 < steps && !idle) products(st + 1);
        store(f0, st + 2);
        fetch(f0, st + 4);
        lds_barrier();
      }
    } else {
      lds_barrier();
    }
  } else {
    Fetch f;
    if (steps > 0) fetch(f, 0);
    lds_barrier();
    for (int st = 0; st < steps; ++st) {
      lds_barrier();
      store(f, st);
      lds_barrier();
      fetch(f, st + 1);
      if (!idle) products(st);
    }
  }
  settle(acc);

  // ---- results -------------------------------------------------------------
  int b_exp[CB];  // of the wave's blocks of columns
#pragma unroll
  for (int b = 0; b < CB; ++b)
    b_exp[b] = (NG == 1 ? s_exp[0] : top_exponent(s_bits[group_of(k0 + (wc * CB + b) * 32)])) - 15;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int r0 = wr * 64 + r * 32 + 4 * q;
    if constexpr (GATE) {
      float dot[16], top[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) dot[i] = top[i] = 0.0f;
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const int64_t k = k0 + (wc * CB + b) * 32 + (c & 3) * 8 + (c >> 2);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = r0 + 8 * (i >> 2) + (i & 3), slot = sh_slot[row];
          if (slot < 0 || k >= K) continue;
          const float z = __builtin_ldexpf(acc[r][b][i], sh_exp[row] + b_exp[b]);
          const float* pre = p.pre + (int64_t)slot * 2 * K + k;
          const float g = pre[0], up = pre[K];
          const float sig = sigmoid(g), silu = g * sig;
          dot[i] = __builtin_fmaf(silu * up, z, dot[i]);
          const float dh = sh_weight[row] * z;
          // (the slope first: dh times up may pass fp32's range)
          const float dg = dh * (up * (sig * __builtin_fmaf(g, sigmoid(-g), 1.0f))), du = dh * silu;
          float* dst = p.dpre + (int64_t)slot * 2 * K + k;
          dst[0] = dg;
          dst[K] = du;
          const uint32_t m = umax(finite_bits(dg), finite_bits(du));
          top[i] = bits_f32(umax(f32_bits(top[i]), m));
        }
      }
      const float sum = reduce16(dot, lane, [](float x, float y) { return x + y; });
      const float most = reduce16(top, lane, [](float x, float y) { return x > y ? x : y; });
      if ((lane & 16) == 0) {
        const int i = lane & 15, row = r0 + 8 * (i >> 2) + (i & 3), slot = sh_slot[row];
        if (slot >= 0) {
          p.dw_part[((int64_t)slot * p.col_tiles + ct) * WC + wc] = sum;
          atomicMax(p.dpre_bits + slot, f32_bits(most));
        }
      }
    } else {
      float* out = p.out + (int64_t)split * p.M * p.out_ld;
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const int64_t k = k0 + (wc * CB + b) * 32 + (c & 3) * 8 + (c >> 2);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = r0 + 8 * (i >> 2) + (i & 3), slot = sh_slot[row];
          if (slot < 0 || k >= K) continue;
          const float z = __builtin_ldexpf(acc[r][b][i], sh_exp[row] + b_exp[b]);
          float* dst = out + (int64_t)slot * p.out_ld + k;
          *dst = p.accumulate ? *dst + z : z;
        }
      }
    }
  }
}

// The same with the row operand complete in memory (d_parts): it comes by direct
// loads, as the forward product's, and only the codes are turned around.
template <int BM>
struct DirectTile {
  static constexpr int kA = kParts * BM * kBK * 2;
  static constexpr int kB = 128 * kBK / 2;
  static constexpr int kLds = 2 * (kA + kB);
};

template <int BM>
__global__ void __launch_bounds__(256, 2) back_direct_kernel(const BackParams p) {
  typedef DirectTile<BM> L;
  constexpr int RB = BM / 64;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int32_t sh_exp[BM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = w >> 1, wc = w & 1, c = lane & 31, q = lane >> 5;

  // rows of d stay with one XCD
  const uint32_t total = (uint32_t)p.row_tiles * (uint32_t)p.col_tiles * (uint32_t)p.splits;
  uint32_t at = xcd_swizzle(blockIdx.x, total);
  const uint32_t plane = (uint32_t)p.row_tiles * (uint32_t)p.col_tiles;
  const int split = (int)(at / plane);
  at %= plane;
  const int mt = (int)(at / (uint32_t)p.col_tiles), ct = (int)(at % (uint32_t)p.col_tiles);
  const int first = mt * BM, rows = (int)(p.M - first < BM ? p.M - first : BM);
  const int64_t K = p.w.K, ldq = K >> 1, k0 = (int64_t)ct * 128;
  const int s_exp = top_exponent(*p.s_bits);
  const int64_t per = ((p.n_rows + p.splits - 1) / p.splits + kBK - 1) / kBK * kBK;
  const int64_t nb = per * split < p.n_rows ? per * split : p.n_rows;
  const int64_t ne = nb + per < p.n_rows ? nb + per : p.n_rows;
  const int steps = (int)((ne - nb + kBK - 1) / kBK);
  if (tid < BM) sh_exp[tid] = top_exponent(p.d_bits[first + (tid < rows ? tid : rows - 1)]);

  const _Float16* asrc[BM / 32];
#pragma unroll
  for (int i = 0; i < BM / 32; ++i) {
    const int r = w * (BM / 4) + i * 8 + (lane >> 3);
    asrc[i] = p.d_parts + (int64_t)(first + (r < rows ? r : rows - 1)) * p.ldd + nb +
              ((lane & 7) ^ ((r >> 1) & 7)) * 8;
  }
  const int64_t piece = p.d_rows * p.ldd;
  const int kw = tid & 15, u = tid >> 4;
  const uint32_t word_at = (uint32_t)(k0 + kw * 8 < K ? k0 / 8 + kw : 0) * 4u;
  const uint32_t code_at = word_at + (uint32_t)(4 * u) * (uint32_t)ldq;
  const uint8_t* codes = p.w.qw + (p.n0 + nb) * ldq;

  auto issue = [&](int step) {
    const int st = step < steps ? step : steps - 1;
    uint8_t* base = smem + (step & 1) * L::kA;
#pragma unroll
    for (int pc = 0; pc < kParts; ++pc)
#pragma unroll
      for (int i = 0; i < BM / 32; ++i)
        __builtin_amdgcn_global_load_lds(
            (global_cptr)(asrc[i] + pc * piece + (int64_t)st * kBK),
            (lds_vptr)(base + pc * BM * 128 + (w * (BM / 4) + i * 8) * 128), 16, 0, 0);
  };
  struct Words {
    uint32_t w[4];
  };
  auto fetch = [&](Words& f, int step) {
    const int64_t n0 = (int64_t)step * kBK;
    if (nb + n0 + kBK <= ne) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f.w[i] = *(const uint32_t*)(codes + (n0 + i) * ldq + code_at);
    } else {
      // (rows past the end: any codes, the other operand is 0)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t r = n0 + 4 * u + i;
        f.w[i] = *(const uint32_t*)(codes + (nb + r < ne ? r : ne - 1 - nb) * ldq + word_at);
      }
    }
  };
  auto store = [&](const Words& f, int step) {
    store_turned<kBK>(smem + 2 * L::kA + (step & 1) * L::kB, f.w, kw, u, p.nibble_order != Q4_ORDER_LOW_FIRST);
  };

  f32x16 acc[RB][2];
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int b = 0; b < 2; ++b) acc[r][b] = f32x16{};
  const Magic magic = Magic::make();
  auto products = [&](int step) {
    const uint8_t *a_base = smem + (step & 1) * L::kA, *b_base = smem + 2 * L::kA + (step & 1) * L::kB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t words[2][2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const u32x2 x = *(const u32x2*)(b_base + (wc * 64 + b * 32 + c) * 32 + turned<kBK>(h * 2 + q, c >> 3, wc * 2 + b) * 8);
        words[b][0] = x[0];
        words[b][1] = x[1];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const h8 bo[2] = {codes_of(words[0][j], magic), codes_of(words[1][j], magic)};
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const int row = wr * (BM / 2) + r * 32 + c;
          const int chunk = (h * 4 + q * 2 + j) ^ ((row >> 1) & 7);
#pragma unroll
          for (int pc = 0; pc < kParts; ++pc) {
            const h8 a = *(const h8*)(a_base + pc * BM * 128 + row * 128 + chunk * 16);
#pragma unroll
            for (int b = 0; b < 2; ++b)
              acc[r][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, bo[b], acc[r][b], 0, 0, 0);
          }
        }
      }
    }
  };

  // Step st: its rows were asked for a step ago, its codes two; then the next
  // step's rows, the codes after them (in this order: the wait counts on it), and
  // the next step's codes into LDS.  The compiler waits for all loads before it
  // takes a step's codes, as their addresses depend on a branch.
  const bool idle = wr * (BM / 2) >= rows;
  Words f0, f1;
  if (steps > 0) {
    fetch(f0, 0);
    keep_order();
    issue(0);
    keep_order();
    fetch(f1, 1);
    store(f0, 0);
    auto step = [&](int st, Words& next, Words& after) {
      wait_loads<4>();  // (the four after them are the next step's codes)
      lds_barrier();
      issue(st + 1);
      keep_order();
      fetch(after, st + 2);
      if (!idle) products(st);
      store(next, st + 1);
    };
    for (int st = 0; st < steps; st += 2) {
      step(st, f1, f0);
      if (st + 1 < steps) step(st + 1, f0, f1);
    }
  }
  lds_barrier();
  wait_loads<0>();
  settle(acc);

  float* out = p.out + (int64_t)split * p.M * p.out_ld;
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int r0 = wr * (BM / 2) + r * 32 + 4 * q;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t k = k0 + wc * 64 + b * 32 + (c & 3) * 8 + (c >> 2);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = r0 + 8 * (i >> 2) + (i & 3);
        if (row >= rows || k >= K) continue;
        const float z = __builtin_ldexpf(acc[r][b][i], sh_exp[row] + s_exp - 15);
        float* dst = out + (int64_t)(first + row) * p.out_ld + k;
        *dst = p.accumulate ? *dst + z : z;
      }
    }
  }
}

template <int BM>
hipError_t launch_back_direct(const BackParams& p, hipStream_t s) {
  constexpr int lds = DirectTile<BM>::kLds;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)back_direct_kernel<BM>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((uint32_t)((int64_t)p.row_tiles * p.col_tiles * p.splits));
  hipLaunchKernelGGL((back_direct_kernel<BM>), grid, dim3(256), lds, s, p);
  return hipGetLastError();
}

template <typename T, int BM, bool GATE>
hipError_t launch_back_tile(const BackParams& p, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)p.row_tiles * p.col_tiles * p.splits));
#define Q4_BACK(NG)                                                                          \
  do {                                                                                       \
    typedef BackTile<BM, NG> L;                                                              \
    constexpr int lds = L::kStages * L::kStage;                                              \
    if (lds > 64 * 1024) {                                                                   \
      const hipError_t e = hipFuncSetAttribute((const void*)back_kernel<T, BM, NG, GATE>,  \
                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds); \
      if (e != hipSuccess) return e;                                                         \
    }                                                                                        \
    hipLaunchKernelGGL((back_kernel<T, BM, NG, GATE>), grid, dim3(256), lds, s, p);       \
  } while (0)
  if (p.w.group % 128 == 0)
    Q4_BACK(1);
  else
    Q4_BACK(4);
#undef Q4_BACK
  return hipGetLastError();
}

}  // namespace q4
