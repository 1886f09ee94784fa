// q4_experts_few.hip -- packed experts for few rows each (decode), for gfx950.
//
//   z[r, n] = sum_g s[g, n] * sum_{k in g} x[r, k] c[n, k]
//
// A workgroup owns an expert's next 16 rows of binary16 operands (16 rows of a
// 16-bit type; 8 of fp32, whose second parts are rows 8 .. 15 of the same
// products) and 32 of its columns at a time: for the gated half 16 columns of
// the gate and the 16 of up beside them.  Its waves divide the depth in chunks
// of 128 k, wave w taking chunks w, w + waves, ...; a lane loads 16 bytes of
// one column's codes (32 k) straight into registers, and 16x16x32 products
// take them from there.  A wave keeps its part of the rows, split into binary16
// parts, in registers for all columns of the workgroup.  The waves' sums meet
// in LDS.
//
// Where a group of 32 or 64 has its own scale, a product must not reach past
// it: the words of the four lane groups are exchanged (4 x 4 words by two
// steps of lane swaps) so that a product's 32 k are consecutive.
//
// Bound: HBM over the codes when many experts are in use, else the chain of
// ids, rows, maximum, products and join.
#include <hip/hip_runtime.h>

#include "q4_experts.h"
#include "q4_experts_device.h"

namespace q4 {
namespace {

constexpr int kChunk = 128;  // k of a wave's step
constexpr int kHold = 4;     // chunks of rows a wave keeps

// 8 elements of a row as they lie in memory
template <typename T>
struct Raw {
  T v[8];
};

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, bool vec) {
  Raw<T> r;
  if (vec) {
    constexpr int n = 16 / sizeof(T);
    typedef T tv __attribute__((ext_vector_type(n)));
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

// (as settle() of q4_experts_device.h)
__device__ __forceinline__ void wait_products(f32x4 (&a)[2]) {
  asm volatile("s_nop 7\n\ts_nop 7" : "+v"(a[0]), "+v"(a[1]));
}

enum FewScales : int { kRowScale = 0, kChunkScale = 1, kStepScale = 2 };

template <int P, typename T, bool GATED, int FS, int NW>
__global__ void __launch_bounds__(64 * NW) few_kernel(const FewParams p, int col_groups, int per_wg,
                                                      bool vec) {
  constexpr int R = 16 / P;  // rows of a tile
  constexpr bool TR = FS == kStepScale;
  __shared__ float red[NW][16][33];
  __shared__ int32_t sh_slot[R], sh_rows, sh_exp[R];
  __shared__ uint32_t sh_max[NW][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, q = lane >> 4;
  const int cg0 = (int)(blockIdx.x % (uint32_t)col_groups) * per_wg;
  const int tile = (int)(blockIdx.x / (uint32_t)col_groups);

  // the tile's expert and slots
  int expert;
  if (p.tiles) {
    if (tile >= *p.n_tiles) return;
    const Tile t = p.tiles[tile];
    expert = t.expert;
    if (tid < R) sh_slot[tid] = tid < t.rows ? p.slots[t.first + tid] : -1;
    if (tid == 0) sh_rows = t.rows;
  } else {
    // the slot `tile` leads if it is its expert's 0th, R-th, ... in slot order
    expert = p.ids[tile];
    if (!id_ok(expert, p.experts)) return;
    int rank = 0;
    for (int i = 0; i < tile; i += 64) {
      const bool same = i + lane < tile && p.ids[i + lane] == expert;
      rank += __popcll(__ballot(same));
    }
    if (rank % R != 0) return;
    if (w == 0) {
      int have = 0;
      for (int i = tile & ~63; i < p.n && have < R; i += 64) {
        const bool same = i + lane >= tile && i + lane < p.n && p.ids[i + lane] == expert;
        const uint64_t m = __ballot(same);
        const int at = have + __popcll(m & ((1ull << lane) - 1));
        if (same && at < R) sh_slot[at] = i + lane;
        have += __popcll(m);
      }
      have = have < R ? have : R;
      if (lane >= have && lane < R) sh_slot[lane] = -1;
      if (lane == 0) sh_rows = have;
    }
  }

  const int64_t K = p.w.K, N = p.w.N, ldq = K >> 1;
  const int chunks = (int)((K + kChunk - 1) / kChunk);
  const int rounds = (chunks + kHold * NW - 1) / (kHold * NW);
  const uint8_t* codes = p.w.qw + expert * p.w.expert_bytes;
  const float* scales = p.w.scales + expert * p.w.expert_scales;
  const int64_t width = GATED ? p.width : N;
  // packed row of this lane's column in block b of a column group
  auto packed_row = [&](int cg, int b) -> int64_t {
    if constexpr (GATED) {
      const int64_t h = (int64_t)cg * 16 + n16, hc = h < width ? h : width - 1;
      return b ? width + hc : hc;
    } else {
      const int64_t c = (int64_t)cg * 32 + b * 16 + n16;
      return c < N ? c : N - 1;
    }
  };
  auto load_codes = [&](int64_t row, int chunk) -> u32x4 {
    u32x4 r;
    const int64_t k = (int64_t)chunk * kChunk + q * 32;
    const uint8_t* src = codes + row * ldq + (k >> 1);
    if (k + 32 <= K) {
      r = *(const u32x4_a4*)src;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = k + 8 * i < K ? ((const uint32_t*)src)[i] : 0u;
    }
    return r;
  };

  __syncthreads();
  const int rows = sh_rows;
  const int lm = lane & 15, my = P == 2 ? lm & 7 : lm;
  const bool second = P == 2 && lm >= 8;
  const bool live = my < rows;
  const T* xrow = (const T*)p.x + (live ? sh_slot[my] / p.slots_per_row : 0) * p.ldx;
  auto k_of = [&](int chunk, int j) -> int64_t {
    return (int64_t)chunk * kChunk + (TR ? j * 32 + q * 8 : q * 32 + j * 8);
  };
  auto load_row = [&](int chunk, int j) -> Raw<T> {
    const int64_t k = k_of(chunk, j);
    if (live && k < K) return load_raw(xrow + k, vec);
    return Raw<T>{};
  };

  // the rows' exponents; what was read for them is kept where registers allow
  constexpr bool KEEP = NW == 4 || sizeof(T) == 2;
  Raw<T> raw[KEEP ? kHold : 1][4];
  uint32_t m = 0;
  for (int rd = 0; rd < rounds; ++rd) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int chunk = (rd * kHold + i) * NW + w;
#pragma unroll
      for (int j = 0; j < 4; ++j) raw[KEEP ? i : 0][j] = load_row(chunk, j);
      if constexpr (!KEEP) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < 8; ++v) m = umax(m, finite_bits(to_f32(raw[0][j].v[v])));
      }
    }
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < kHold; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < 8; ++v) m = umax(m, finite_bits(to_f32(raw[i][j].v[v])));
    }
  }
  m = umax(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = umax(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  if (q == 0) sh_max[w][lm] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NW; ++i) m = umax(m, sh_max[i][lm]);
  const int e = row_exponent(m);
  if (w == 0 && q == 0 && lm < R) sh_exp[lm] = e;

  h8 a[kHold][4];
  auto split = [&](int rd, bool again) {
#pragma unroll
    for (int i = 0; i < kHold; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        Raw<T> r;
        if constexpr (KEEP) {
          r = raw[i][j];
          if (again) r = load_row((rd * kHold + i) * NW + w, j);
        } else {
          r = load_row((rd * kHold + i) * NW + w, j);
        }
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const int nib = operand_nibble(v);
          const float x0 = to_f32(r.v[nib]), x1 = to_f32(r.v[nib ^ 1]);
          const float x = settled(__builtin_ldexpf(p.nibble_order == Q4_ORDER_LOW_FIRST ? x0 : x1, e));
          const _Float16 hi = part_hi(x);
          a[i][j][v] = P == 2 && second ? part_lo(x, hi) : hi;
        }
      }
  };
  const Magic magic = Magic::make();
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  const int cg_end_all = (int)(GATED ? (width + 15) / 16 : (N + 31) / 32);
  const int cg1 = cg0 + per_wg < cg_end_all ? cg0 + per_wg : cg_end_all;
  for (int cg = cg0; cg < cg1; ++cg) {
    const int64_t prow[2] = {packed_row(cg, 0), packed_row(cg, 1)};
    f32x4 out[2] = {zero, zero};
    for (int rd = 0; rd < rounds; ++rd) {
      u32x4 cw[2][kHold];
#pragma unroll
      for (int i = 0; i < kHold; ++i) {
        const int chunk = (rd * kHold + i) * NW + w;
#pragma unroll
        for (int b = 0; b < 2; ++b)
          cw[b][i] = chunk < chunks ? load_codes(prow[b], chunk) : u32x4{0, 0, 0, 0};
      }
      constexpr int kScales = FS == kStepScale ? 4 : 1;
      float sc[2][kHold][kScales];
      if constexpr (FS != kRowScale) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          const int chunk = (rd * kHold + i) * NW + w;
#pragma unroll
          for (int j = 0; j < kScales; ++j) {
            // (past the last group: zero activations times any scale)
            const int64_t k = (int64_t)chunk * kChunk + j * 32;
            const int g = k < K ? (int)(k / p.w.group) : p.w.G - 1;
#pragma unroll
            for (int b = 0; b < 2; ++b) sc[b][i][j] = scales[(int64_t)g * N + prow[b]];
          }
        }
      }
      if (rounds > 1 || cg == cg0) split(rd, rounds > 1);
      f32x4 acc[2] = {zero, zero};
#pragma unroll
      for (int i = 0; i < kHold; ++i) {
        const int chunk = (rd * kHold + i) * NW + w;
        if (chunk >= chunks) continue;
        if constexpr (TR) {
          exchange(cw[0][i]);
          exchange(cw[1][i]);
        }
        if constexpr (FS == kChunkScale) acc[0] = acc[1] = zero;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const h8 c = codes_of(cw[b][i][j], magic);
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i][j], c, TR ? zero : acc[b], 0, 0, 0);
          }
          if constexpr (TR) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int v = 0; v < 4; ++v)
                out[b][v] = __builtin_fmaf(acc[b][v], sc[b][i][j], out[b][v]);
          }
        }
        if constexpr (FS == kChunkScale) {
          wait_products(acc);
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              out[b][v] = __builtin_fmaf(acc[b][v], sc[b][i][0], out[b][v]);
        }
      }
      if constexpr (FS == kRowScale) {
        wait_products(acc);
#pragma unroll
        for (int b = 0; b < 2; ++b) out[b] += acc[b];
      }
    }
    // rows 4 q + v of column n16: into LDS, the second parts' rows onto the first's
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float x = out[b][v];
        if constexpr (P == 2) x += __shfl_xor(x, 32, 64);
        if (P == 1 || q < 2) red[w][q * 4 + v][b * 16 + n16] = x;
      }
    __syncthreads();
    constexpr int kCols = GATED ? 16 : 32;
    for (int t = tid; t < R * kCols; t += 64 * NW) {
      const int r = t / kCols, c = t % kCols;
      if (r < rows) {
        const int slot = sh_slot[r], ex = sh_exp[r];
        auto value = [&](int col, int64_t prow_) {
          float x = 0.0f;
#pragma unroll
          for (int i = 0; i < NW; ++i) x += red[i][r][col];
          if constexpr (FS == kRowScale) x *= scales[prow_];
          return __builtin_ldexpf(x, -ex);
        };
        if constexpr (GATED) {
          const int64_t h = (int64_t)cg * 16 + c;
          if (h < width) {
            const float g = value(c, h), u = value(16 + c, width + h);
            p.out[(int64_t)slot * p.out_ld + h] = g * sigmoid(g) * u;
            if (p.pre) {
              float* pre = p.pre + (int64_t)slot * 2 * width + h;
              pre[0] = g;
              pre[width] = u;
            }
          }
        } else {
          const int64_t col = (int64_t)cg * 32 + c;
          if (col < N) p.out[(int64_t)slot * p.out_ld + col] = value(c, col);
        }
      }
    }
    __syncthreads();
  }
}

template <int P, typename T, bool GATED, int NW>
hipError_t few_scales(const FewParams& p, hipStream_t s) {
  const int64_t cols = GATED ? (p.width + 15) / 16 : (p.w.N + 31) / 32;
  const int64_t tiles = p.tiles ? p.row_tiles : p.n;
  // columns of a workgroup: as many as leave two workgroups for every CU; deep
  // rows are split again for every column group, so there it is one
  const int64_t chunks = (p.w.K + kChunk - 1) / kChunk;
  const int64_t busy = p.tiles ? tiles : (p.n < p.experts ? p.n : p.experts);
  int64_t per = chunks > kHold * NW ? 1 : cols * busy / (2 * 256);
  per = per < 1 ? 1 : per > 8 ? 8 : per;
  const int64_t groups = (cols + per - 1) / per;
  const bool vec = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx * sizeof(T) % 16 == 0;
  const dim3 grid((uint32_t)(groups * tiles)), block(64 * NW);
  if (p.w.group == 0)
    hipLaunchKernelGGL((few_kernel<P, T, GATED, kRowScale, NW>), grid, block, 0, s, p, (int)groups, (int)per, vec);
  else if (p.w.group % kChunk == 0)
    hipLaunchKernelGGL((few_kernel<P, T, GATED, kChunkScale, NW>), grid, block, 0, s, p, (int)groups, (int)per, vec);
  else
    hipLaunchKernelGGL((few_kernel<P, T, GATED, kStepScale, NW>), grid, block, 0, s, p, (int)groups, (int)per, vec);
  return hipGetLastError();
}

template <int P, typename T, bool GATED>
hipError_t few_waves(const FewParams& p, hipStream_t s) {
  return p.w.K <= 4 * kHold * kChunk ? few_scales<P, T, GATED, 4>(p, s) : few_scales<P, T, GATED, 8>(p, s);
}

}  // namespace

hipError_t launch_few(const FewParams& p, bool gated, hipStream_t s) {
  if (gated) {
    switch (p.dtype) {
      case Q4_DTYPE_F32: return few_waves<2, float, true>(p, s);
      case Q4_DTYPE_F16: return few_waves<1, _Float16, true>(p, s);
      default: return few_waves<1, bf16, true>(p, s);
    }
  }
  // the gated rows are fp32
  return p.parts == 2 ? few_waves<2, float, false>(p, s) : few_waves<1, float, false>(p, s);
}

}  // namespace q4
