// q4_experts_few.h -- packed experts for few rows each (decode), for gfx950;
// instantiated by q4_experts_few_*.hip.
//
//   z[r, n] = sum_g s[g, n] * sum_{k in g} x[r, k] c[n, k]
//
// A workgroup owns an expert's next rows, up to 8 (of fp32, in two binary16
// parts, the second parts are rows 8 .. 15 of the same products; the second half
// reads fp32 whatever the type, so both halves take 8), and CG blocks of 32 of its columns: for the gated half 16
// columns of the gate and the 16 of up beside them.  The depth is divided
// between NW waves (4, 8 or 16), up to four chunks of 128 k for each: a wave
// splits the rows' elements there into binary16 parts, in LDS, scaled by what
// is largest among its own k, and its lanes load 16 bytes of one column's codes
// (32 k) straight into registers, from where 16x16x32 products take them.  The
// waves' sums meet in LDS, scaled back.  Up to there a wave waits for nobody
// but the wave it shares its k with (CS = 2: two sets of waves take turns at
// the columns and at splitting rows), and its first codes are on their way
// while it reads the rows.
//
// Where a group of 32 or 64 has its own scale, a product must not reach past
// it: the words of the four lane groups are exchanged (4 x 4 words by two
// steps of lane swaps) so that a product's 32 k are consecutive.
//
// Bound: HBM over the codes when many experts are in use, else the chain of
// arguments, ids, rows, maximum, products and join.  48 tokens over all of 64
// experts of 2048 x 1024 (8 each, fp32, groups of 128): gate and up 44 us, down
// 30, for 142 and 71 MB of codes and scales (3.2 and 2.4 TB/s; the loads alone
// reach 5.1).  One token by 8 in groups of 32: 10.8 and 6.4 us.
#pragma once

#include "q4_experts.h"
#include "q4_experts_device.h"

namespace q4 {

constexpr int kChunk = 128;   // k of a wave's step
constexpr int kHold = 4;      // chunks of a wave
constexpr int kPitch = kChunk * kHold + 8;  // halves: 16 rows of a read fall on different banks
constexpr int kBatch = 4;     // rows whose loads are under way at once

template <typename T>
struct Raw {
  T v[8];
};

// vec: 4-byte aligned (always so for fp32)
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, bool vec) {
  Raw<T> r;
  if (sizeof(T) == 4 || vec) {
    constexpr int n = 16 / sizeof(T);
    typedef T tv __attribute__((ext_vector_type(n), aligned(4)));
#pragma unroll
    for (int i = 0; i < 8 / n; ++i) {
      const tv x = *(const tv*)(p + n * i);
#pragma unroll
      for (int j = 0; j < n; ++j) r.v[i * n + j] = x[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = p[i];
  }
  return r;
}

// Lane group q (lane >> 4) holds words q * 4 + j in w[j]; afterwards words j * 4 + q.
__device__ __forceinline__ void exchange(u32x4& w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w[0] = c[0];
  w[1] = c[1];
  w[2] = d[0];
  w[3] = d[1];
}

// The value of each lane group, in all lanes.
__device__ __forceinline__ void spread(float x, float (&s)[4]) {
  const uint32_t b = f32_bits(x);
  const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  s[0] = bits_f32(lo[0]);
  s[1] = bits_f32(lo[1]);
  s[2] = bits_f32(hi[0]);
  s[3] = bits_f32(hi[1]);
}

// (as settle() of q4_experts_device.h)
__device__ __forceinline__ void wait_products(f32x4 (&a)[2]) {
  asm volatile("s_nop 7\n\ts_nop 7" : "+v"(a[0]), "+v"(a[1]));
}

// The largest of 64 lanes, in all of them.
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
  x = umax(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xf, 0xf, false));   // lane ^ 1
  x = umax(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xf, 0xf, false));   // lane ^ 2
  x = umax(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, false));  // 7 - lane of 8
  x = umax(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xf, 0xf, false));  // 15 - lane of 16
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = umax(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return umax(b[0], b[1]);
}

enum FewScales : int { kRowScale = 0, kChunkScale = 1, kStepScale = 2 };

// Exact quotients of small numbers (x up to 2^24, divisors up to 2^11, x times
// the divisor below 2^31): div is 2^31 / divisor, rounded up.
inline uint32_t divisor(uint32_t d) { return (uint32_t)((((uint64_t)1 << 31) + d - 1) / d); }
__device__ __forceinline__ int quotient(int x, uint32_t div) { return (int)__umulhi((uint32_t)x * 2, div); }

struct FewShape {
  int32_t col_groups, xcd_groups, tile_rows;
  uint32_t group_div;  // steps of 32 k in a group
  uint32_t slot_div;   // slots of a row
  int32_t vec;
};

// The kernel's arguments lie in host memory: fetched where each is first used
// they cost a microsecond a cache line, one after the other.
__device__ __forceinline__ void fetch_at_once(FewParams& p, FewShape& f) {
  asm volatile(""
               : "+s"(p.w.qw), "+s"(p.w.scales), "+s"(p.w.N), "+s"(p.w.K), "+s"(p.w.G),
                 "+s"(p.w.expert_bytes), "+s"(p.w.expert_scales), "+s"(p.x), "+s"(p.ldx),
                 "+s"(p.nibble_order), "+s"(p.n), "+s"(p.experts), "+s"(p.out));
  asm volatile(""
               : "+s"(p.ids), "+s"(p.slots), "+s"(p.tiles), "+s"(p.n_tiles), "+s"(p.out_ld),
                 "+s"(p.pre), "+s"(p.width), "+s"(f.col_groups), "+s"(f.xcd_groups),
                 "+s"(f.tile_rows),
                 "+s"(f.group_div), "+s"(f.slot_div), "+s"(f.vec));
}

// EVEN: K is a multiple of 32, so a lane's 32 k are a row's or not
template <int P, typename T, bool GATED, int FS, int NW, int CG, int CS, bool EVEN>
__global__ void __launch_bounds__(64 * NW * CS, NW * CS <= 4 ? 2 : 4)
few_kernel(const FewParams pa, const FewShape fa) {
  FewParams p = pa;
  FewShape f = fa;
  fetch_at_once(p, f);
  constexpr bool TR = FS == kStepScale;
  constexpr int kBlock = GATED ? 16 : 32;  // results of a column block
  constexpr int kMine = CG / CS;           // column blocks of a wave
  constexpr int kRedPitch = CG * 32 + 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int32_t sh_slot[16], sh_exp[NW][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane((tid >> 6) % NW);
  const int cs = __builtin_amdgcn_readfirstlane((tid >> 6) / NW);
  const int n16 = lane & 15, q = lane >> 4;
  // neighbouring columns share cache lines of scales: an XCD (workgroups go to
  // the eight in turn) takes an eighth of the column groups of every tile
  const int cg = (int)(blockIdx.x % 8u) * f.xcd_groups + (int)(blockIdx.x / 8u) % f.xcd_groups;
  const int tile = (int)(blockIdx.x / 8u) / f.xcd_groups;
  if (cg >= f.col_groups) return;
  const int cg0 = cg * CG;

  // the tile's expert and slots (lane r has the r-th)
  int expert, rows, slot = 0;
  if (p.tiles) {
    if (tile >= *p.n_tiles) return;
    const Tile t = p.tiles[tile];
    expert = t.expert;
    rows = t.rows;
    if (lane < rows) slot = p.slots[t.first + lane];
  } else {
    // the slot `tile` leads if it is its expert's 0th, tile_rows-th, ... in slot order
    const int32_t id = lane < p.n ? p.ids[lane] : -1;
    expert = __builtin_amdgcn_readlane(id, tile);
    if (!id_ok(expert, p.experts)) return;
    const uint64_t same = __ballot(id == expert), before = same & (((uint64_t)1 << tile) - 1);
    if (__popcll(before) % f.tile_rows != 0) return;
    uint64_t from = same & ~before;
    rows = __popcll(from);
    rows = rows < f.tile_rows ? rows : f.tile_rows;
    for (int r = 0; r < rows; ++r) {
      slot = lane == r ? __ffsll((unsigned long long)from) - 1 : slot;
      from &= from - 1;
    }
  }
  if (tid < rows) sh_slot[tid] = slot;

  // offsets within an expert's matrix are 32-bit
  const int K = (int)p.w.K, N = (int)p.w.N;
  const uint32_t ldq = (uint32_t)K >> 1;

  // this wave's elements of row r, 8 of them a lane; past K the row's first
  const int k_lane = ((lane >> 4) * NW + w) * kChunk + n16 * 8;
  auto load_row = [&](int r) -> Raw<T> {
    const int s = __builtin_amdgcn_readlane(slot, r < rows ? r : rows - 1);
    const T* row = (const T*)p.x + (int64_t)quotient(s, f.slot_div) * p.ldx;
    return load_raw(row + (k_lane < K ? k_lane : 0), f.vec);
  };
  Raw<T> raw[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) raw[i] = load_row(i * CS + cs);

  const uint8_t* codes = p.w.qw + expert * p.w.expert_bytes;
  const float* scales = p.w.scales + expert * p.w.expert_scales;
  const int width = GATED ? (int)p.width : N;
  // packed row of this lane's column in half b of a column block
  auto packed_row = [&](int cg, int b) -> uint32_t {
    if constexpr (GATED) {
      const int h = cg * 16 + n16, hc = h < width ? h : width - 1;
      return (uint32_t)(b ? width + hc : hc);
    } else {
      const int c = cg * 32 + b * 16 + n16;
      return (uint32_t)(c < N ? c : N - 1);
    }
  };
  struct Codes {
    u32x4 c[2][kHold];
    float s[2][FS == kRowScale ? 1 : kHold];  // kStepScale: of the lane group's 32 k
  };
  // a wave's codes and scales of chunk i of a column block; past K
  // the activations are 0 and codes and scales any
  Codes now = {};
  auto load_codes = [&](int cg, int i) {
    if ((i * NW + w) * kChunk >= K) return;
    const uint32_t row[2] = {packed_row(cg, 0), packed_row(cg, 1)};
    const int k0 = (i * NW + w) * kChunk, k = k0 + q * 32;
    if constexpr (EVEN) {
      const uint32_t at = k < K ? (uint32_t)k >> 1 : 0;
#pragma unroll
      for (int b = 0; b < 2; ++b) now.c[b][i] = *(const u32x4_a4*)(codes + (row[b] * ldq + at));
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint32_t at = k + v * 8 < K ? (uint32_t)(k + v * 8) >> 1 : 0;
#pragma unroll
        for (int b = 0; b < 2; ++b) now.c[b][i][v] = *(const uint32_t*)(codes + (row[b] * ldq + at));
      }
    }
    if constexpr (FS != kRowScale) {
      const int g = quotient(k0 / 32 + (FS == kStepScale ? q : 0), f.group_div);
      const uint32_t at = (uint32_t)((g < p.w.G ? g : p.w.G - 1) * N);
#pragma unroll
      for (int b = 0; b < 2; ++b) now.s[b][i] = *(const float*)((const uint8_t*)scales + (at + row[b]) * 4u);
    }
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i) load_codes(cg0 + cs, i);
  float row_scale[kMine][2];
  if constexpr (FS == kRowScale) {
#pragma unroll
    for (int g = 0; g < kMine; ++g)
#pragma unroll
      for (int b = 0; b < 2; ++b) row_scale[g][b] = scales[packed_row(cg0 + g * CS + cs, b)];
  }

  // the rows' elements among this wave's k, split: rows of binary16 operands,
  // first parts, then second parts
  _Float16* mine = (_Float16*)smem + w * f.tile_rows * P * kPitch;
  for (int r0 = 0; r0 * CS + cs < rows; r0 += kBatch) {
    if (r0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) raw[i] = load_row((r0 + i) * CS + cs);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = (r0 + i) * CS + cs;
      if (r >= rows) break;
      uint32_t m = 0;
#pragma unroll
      for (int v = 0; v < 8; ++v) m = umax(m, finite_bits(to_f32(raw[i].v[v])));
      const int e = row_exponent(lanes_max(m));
      if (lane == 0) sh_exp[w][r] = e;
      float x[8];
#pragma unroll
      for (int v = 0; v < 8; ++v)
        x[v] = settled(k_lane < K ? __builtin_ldexpf(to_f32(raw[i].v[v]), e) : 0.0f);
      h8 hi, lo;
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        hi[v] = part_hi(x[operand_nibble(v)]);
        if constexpr (P == 2) lo[v] = part_lo(x[operand_nibble(v)], hi[v]);
      }
      if (p.nibble_order != Q4_ORDER_LOW_FIRST) {
        // nibbles i and i ^ 1 are operands v and v ^ 2
        hi = __builtin_shufflevector(hi, hi, 2, 3, 0, 1, 6, 7, 4, 5);
        if constexpr (P == 2) lo = __builtin_shufflevector(lo, lo, 2, 3, 0, 1, 6, 7, 4, 5);
      }
      _Float16* dst = mine + r * kPitch + lane * 8;
      *(h8*)dst = hi;
      if constexpr (P == 2) *(h8*)(dst + f.tile_rows * kPitch) = lo;
    }
  }
  // (a wave's own LDS operations are in order)
  if constexpr (CS > 1) lds_barrier();
  else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  // this lane's operand row; rows that the tile has not repeat one it has
  const int my = P == 2 ? n16 & 7 : n16;
  const _Float16* arow = mine + ((my < rows ? my : 0) + (P == 2 && n16 >= 8 ? f.tile_rows : 0)) * kPitch;

  const Magic magic = Magic::make();
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 out[kMine][2];
#pragma unroll
  for (int g = 0; g < kMine; ++g) out[g][0] = out[g][1] = zero;
#pragma unroll
  for (int g = 0; g < kMine; ++g) {
    f32x4 acc[2] = {zero, zero};
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if ((i * NW + w) * kChunk >= K) continue;
      // (operands are made chunk by chunk, not all at once)
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      float sc[2][4];
      if constexpr (TR) {
        exchange(now.c[0][i]);
        exchange(now.c[1][i]);
        spread(now.s[0][i], sc[0]);
        spread(now.s[1][i], sc[1]);
      }
      if constexpr (FS == kChunkScale) acc[0] = acc[1] = zero;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const h8 a = *(const h8*)(arow + i * kChunk + (TR ? j * 32 + q * 8 : q * 32 + j * 8));
        f32x4 sum[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const h8 c = codes_of(now.c[b][i][j], magic);
          sum[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, c, TR ? zero : acc[b], 0, 0, 0);
          if constexpr (!TR) acc[b] = sum[b];
        }
        if constexpr (TR) {
          wait_products(sum);
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              out[g][b][v] = __builtin_fmaf(sum[b][v], sc[b][j], out[g][b][v]);
        }
      }
      if constexpr (FS == kChunkScale) {
        wait_products(acc);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            out[g][b][v] = __builtin_fmaf(acc[b][v], now.s[b][i], out[g][b][v]);
      }
      // the chunk's registers take the next block's codes
      if (g + 1 < kMine) load_codes(cg0 + (g + 1) * CS + cs, i);
    }
    if constexpr (FS == kRowScale) {
      wait_products(acc);
#pragma unroll
      for (int b = 0; b < 2; ++b) out[g][b] += acc[b];
    }
  }
  lds_barrier();

  // rows 4 q + v of column n16: into LDS, the second parts' rows onto the first's
  float* red = (float*)smem;
  constexpr int kRows = 16 / P;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int r = P == 1 ? q * 4 + v : (q & 1) * 4 + v;
    const int e = r < rows ? sh_exp[w][r] : 0;
#pragma unroll
    for (int g = 0; g < kMine; ++g)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float x = out[g][b][v];
        if constexpr (P == 2) x += __shfl_xor(x, 32, 64);
        // (before the exponent: a sum of codes times large rows may pass fp32's range)
        if constexpr (FS == kRowScale) x *= row_scale[g][b];
        if (P == 1 || q < 2)
          red[(w * kRows + r) * kRedPitch + (g * CS + cs) * 32 + b * 16 + n16] = __builtin_ldexpf(x, -e);
      }
  }
  lds_barrier();
  for (int t = tid; t < rows * CG * kBlock; t += 64 * NW * CS) {
    const int r = t / (CG * kBlock), c = t % (CG * kBlock);
    const int g = c / kBlock, cc = c % kBlock;
    const int to = sh_slot[r];
    auto value = [&](int col) {
      float x = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) x += red[(i * kRows + r) * kRedPitch + g * 32 + col];
      return x;
    };
    const int col = (cg0 + g) * kBlock + cc;
    if (col >= width) continue;
    if constexpr (GATED) {
      const float gate = value(cc), up = value(16 + cc);
      p.out[(int64_t)to * p.out_ld + col] = gate * sigmoid(gate) * up;
      if (p.pre) {
        float* pre = p.pre + (int64_t)to * 2 * width + col;
        pre[0] = gate;
        pre[width] = up;
      }
    } else {
      p.out[(int64_t)to * p.out_ld + col] = value(cc);
    }
  }
}

template <int P, typename T, bool GATED, int FS>
hipError_t few_blocks(const FewParams& p, int32_t tile_rows, hipStream_t s) {
  const int64_t cols = GATED ? (p.width + 15) / 16 : (p.w.N + 31) / 32;
  const int64_t tiles = p.tiles ? p.row_tiles : p.n;
  const int64_t busy = p.tiles ? tiles : (p.n < p.experts ? p.n : p.experts);
  const int nw = p.w.K <= 4 * kHold * kChunk ? 4 : p.w.K <= 8 * kHold * kChunk ? 8 : 16;
  // Four column blocks share a workgroup's rows, which pays where there are
  // many workgroups, or several rows to split.  One / four blocks, us (fp32; bf16
  // alike): 64 experts of 2048 x 1024, 4 tokens by 8 35.6 / 31.4, 16 81 / 57, 48
  // 128 / 70, 96 215 / 104; 16 of 2048 x 1408, 4 tokens by 2 17.8 / 19.8, 32
  // 46 / 33; 8 of 4096 x 3584, 4 tokens by 2 38 / 52, 16 104 / 71; 4 of 2144 x
  // 384, 12 tokens by 2 21.6 / 26.3.
  const bool even = p.w.K % 32 == 0;
  const int64_t enough = p.n >= 2 * p.experts ? 1024 : 2048;
  const int cg = even && nw < 16 && cols * busy >= enough ? 4 : 1;
  FewShape f;
  f.col_groups = (int32_t)((cols + cg - 1) / cg);
  f.xcd_groups = (f.col_groups + 7) / 8;
  f.tile_rows = tile_rows;
  f.group_div = divisor(p.w.group ? p.w.group / 32 : 1);
  f.slot_div = divisor(p.slots_per_row);
  f.vec = reinterpret_cast<uintptr_t>(p.x) % 4 == 0 && p.ldx * sizeof(T) % 4 == 0;
  const dim3 grid((uint32_t)(8 * f.xcd_groups * tiles));
  const int stage = nw * tile_rows * P * kPitch * 2, join = nw * (16 / P) * (cg * 32 + 1) * 4;
  const int lds = stage > join ? stage : join;
#define Q4_FEW(NW, CG, CS, EVEN)                                                                  \
  do {                                                                                            \
    const void* k = (const void*)few_kernel<P, T, GATED, FS, NW, CG, CS, EVEN>;                   \
    const hipError_t e = lds <= 64 * 1024 ? hipSuccess                                            \
        : hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);                \
    if (e != hipSuccess) return e;                                                                \
    hipLaunchKernelGGL((few_kernel<P, T, GATED, FS, NW, CG, CS, EVEN>), grid, dim3(64 * NW * CS),  \
                       lds, s, p, f);                                                             \
    return hipGetLastError();                                                                     \
  } while (0)
  if (nw == 4) {
    if (cg == 4) Q4_FEW(4, 4, 2, true);
    if (even) Q4_FEW(4, 1, 1, true);
    Q4_FEW(4, 1, 1, false);
  }
  if (nw == 8) {
    if (cg == 4) Q4_FEW(8, 4, 1, true);
    if (even) Q4_FEW(8, 1, 1, true);
    Q4_FEW(8, 1, 1, false);
  }
  if (even) Q4_FEW(16, 1, 1, true);
  Q4_FEW(16, 1, 1, false);
#undef Q4_FEW
}

template <int P, typename T, bool GATED>
hipError_t few_scales(const FewParams& p, int32_t tile_rows, hipStream_t s) {
  if (p.w.group == 0) return few_blocks<P, T, GATED, kRowScale>(p, tile_rows, s);
  if (p.w.group % kChunk == 0) return few_blocks<P, T, GATED, kChunkScale>(p, tile_rows, s);
  return few_blocks<P, T, GATED, kStepScale>(p, tile_rows, s);
}

}  // namespace q4
