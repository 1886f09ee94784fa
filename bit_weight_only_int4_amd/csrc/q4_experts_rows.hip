// q4_experts_rows.hip -- what goes on around the matrix kernels of packed
// experts: rows listed by expert, activations split into binary16 parts, sums
// over a token's slots, largest magnitudes, and the head's last steps.  All of
// them read their input once or twice and are bound by HBM, or by their launch
// where rows are few: 32792 rows of 1024 fp32 split into two parts 44 us (6.1 TB/s),
// the same summed into 4099 rows of 2048 45 us (6.3).
#include <hip/hip_runtime.h>

#include "q4_experts.h"
#include "q4_experts_device.h"

namespace q4 {
namespace {

__device__ __forceinline__ uint32_t block_umax(uint32_t v, uint32_t* sh) {
  v = wave_umax(v);
  const int w = threadIdx.x >> 6, nw = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) sh[w] = v;
  __syncthreads();
  for (int i = 0; i < nw; ++i) v = umax(v, sh[i]);
  __syncthreads();
  return v;
}

// Eight elements of a row from k, zeros past K.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t k, int64_t K, bool vec, float (&v)[8]) {
  if (vec) {  // K is a multiple of 8
    if constexpr (sizeof(T) == 4) {
      const f32x4 a = *(const f32x4*)(row + k), b = *(const f32x4*)(row + k + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else {
      typedef T t8 __attribute__((ext_vector_type(8)));
      const t8 a = *(const t8*)(row + k);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? to_f32(row[k + i]) : 0.0f;
  }
}

// ---- rows by expert --------------------------------------------------------

// One workgroup: a histogram of the ids, its prefix sums (rows and tiles), and
// the slots scattered behind their expert's start.  The order within an expert
// is that of arrival and changes nothing: a row's result does not depend on its
// place in a tile.
constexpr int kListThreads = 1024;
// The ids of this thread, four loads under way at once.
template <typename F>
__device__ __forceinline__ void each_id(const int32_t* __restrict__ ids, int32_t n, F f) {
  for (int64_t i0 = threadIdx.x; i0 < n; i0 += 4 * kListThreads) {
    int32_t id[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + j * kListThreads;
      id[j] = i < n ? ids[i] : -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) f(id[j], i0 + j * kListThreads);
  }
}
__global__ void __launch_bounds__(kListThreads)
lists_kernel(const int32_t* __restrict__ ids, int32_t n, int32_t experts, int32_t tile_rows,
             const RowLists r) {
  __shared__ int32_t count[kMaxExperts], next[kMaxExperts];
  __shared__ int32_t wave_rows[kListThreads / 64], wave_tiles[kListThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  count[tid] = 0;
  __syncthreads();
  each_id(ids, n, [&](int32_t id, int64_t) {
    if (id_ok(id, experts)) atomicAdd(&count[id], 1);
  });
  __syncthreads();
  // thread e: expert e
  const int32_t c = count[tid], mine = (c + tile_rows - 1) / tile_rows;
  int32_t rows = c, tiles = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t a = __shfl_up(rows, d, 64), b = __shfl_up(tiles, d, 64);
    if (lane >= d) rows += a, tiles += b;
  }
  if (lane == 63) wave_rows[w] = rows, wave_tiles[w] = tiles;
  __syncthreads();
  int32_t rows0 = 0, tiles0 = 0, all = 0;
  for (int i = 0; i < kListThreads / 64; ++i) {
    if (i < w) rows0 += wave_rows[i], tiles0 += wave_tiles[i];
    all += wave_tiles[i];
  }
  rows0 += rows - c;
  tiles0 += tiles - mine;
  next[tid] = rows0;
  for (int32_t i = 0; i < mine; ++i) {
    const int32_t left = c - i * tile_rows;
    r.tiles[tiles0 + i] = Tile{tid, rows0 + i * tile_rows, left < tile_rows ? left : tile_rows, 0};
  }
  if (tid == 0) *r.n_tiles = all;
  __syncthreads();
  each_id(ids, n, [&](int32_t id, int64_t i) {
    if (id_ok(id, experts)) r.slots[atomicAdd(&next[id], 1)] = (int32_t)i;
  });
}

// ---- activations into binary16 parts -----------------------------------------

// A wave a row: its largest magnitude, then every word of 8 elements in the
// order of the codes' operands.  HOLD: rows of up to 512 HOLD elements stay in
// registers in between, longer ones (0) are read again.
typedef float f32x8 __attribute__((ext_vector_type(8)));
template <typename T>
__device__ __forceinline__ f32x8 row_word(const T* __restrict__ src, int64_t k, int64_t K, bool vec) {
  f32x8 r = {0, 0, 0, 0, 0, 0, 0, 0};
  if (k < K) {
    float v[8];
    load8(src, k, K, vec, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = v[j];
  }
  return r;
}
__device__ __forceinline__ void store_parts(const SplitRows& r, int64_t row, int64_t k, int e,
                                            int32_t order, f32x8 y) {
  h8 hi, lo;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int nib = operand_nibble(i);
    const float s = settled(__builtin_ldexpf(order == Q4_ORDER_LOW_FIRST ? y[nib] : y[nib ^ 1], e));
    hi[i] = part_hi(s);
    lo[i] = part_lo(s, hi[i]);
  }
  *(h8*)(r.a + row * r.Kp + k) = hi;
  if (r.parts == 2) *(h8*)(r.a + (r.rows + row) * r.Kp + k) = lo;
}
template <typename T, int HOLD>
__global__ void __launch_bounds__(256)
split_kernel(const T* __restrict__ x, int64_t ldx, int64_t K, int32_t order,
             const int32_t* __restrict__ ids, int32_t experts, const SplitRows r, bool vec) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= r.rows) return;  // whole waves; no barrier follows
  if (ids && !id_ok(ids[row], experts)) return;
  const T* src = x + row * ldx;
  uint32_t m = 0;
  if constexpr (HOLD > 0) {
    f32x8 v[HOLD];
#pragma unroll
    for (int i = 0; i < HOLD; ++i) v[i] = row_word(src, 8 * (lane + 64 * i), K, vec);
#pragma unroll
    for (int i = 0; i < HOLD; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = umax(m, finite_bits(v[i][j]));
    const int e = row_exponent(wave_umax(m));
    if (lane == 0) r.e[row] = e;
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int64_t k = 8 * (lane + 64 * i);
      if (k < r.Kp) store_parts(r, row, k, e, order, v[i]);
    }
  } else {
    for (int64_t k = 8 * lane; k < K; k += 512) {
      const f32x8 v = row_word(src, k, K, vec);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = umax(m, finite_bits(v[j]));
    }
    const int e = row_exponent(wave_umax(m));
    if (lane == 0) r.e[row] = e;
    for (int64_t k = 8 * lane; k < r.Kp; k += 512)
      store_parts(r, row, k, e, order, row_word(src, k, K, vec));
  }
}

// ---- sums over a token's slots -------------------------------------------------

// Eight slots' loads are under way at once; a lane has a slot's id and weight.
template <typename T>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p, bool vec) {
  const int64_t n = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  const int lane = threadIdx.x & 63;
  const bool in = n < p.N;  // N is a multiple of 8
  for (int64_t t = blockIdx.y; t < p.T; t += gridDim.y) {
    int32_t id = -1;
    float w = 0.0f;
    if (lane < p.top_k) {
      id = p.ids[t * p.top_k + lane];
      w = p.weights ? p.weights[t * p.top_k + lane] : 1.0f;
    }
    const bool bad = __any(id >= p.experts);
    const uint64_t used = __ballot(id_ok(id, p.experts));
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < p.top_k; j0 += 8) {
      f32x4 y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (in && (used >> (j0 + j) & 1)) y[j] = *(const f32x4*)(p.y + (t * p.top_k + j0 + j) * p.N + n);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!(used >> (j0 + j) & 1)) continue;
        const float wj = bits_f32((uint32_t)__builtin_amdgcn_readlane((int)f32_bits(w), j0 + j));
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(wj, y[j][i], sum[i]);
      }
    }
    if (!in) continue;
    if (bad) sum = f32x4{} + bits_f32(0x7fc00000u);
    T* dst = (T*)p.out + t * p.ldo + n;
    typedef T t4 __attribute__((ext_vector_type(4)));
    if (vec) {
      t4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = from_f32<T>(sum[i]);
      *(t4*)dst = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = from_f32<T>(sum[i]);
    }
  }
}

// ---- largest magnitudes ----------------------------------------------------------

// (a wave a row; the waves after the last row clear)
template <typename T>
__global__ void __launch_bounds__(256)
row_bits_kernel(const T* __restrict__ x, int64_t ldx, int64_t rows, int64_t K, uint32_t* bits,
                uint32_t* zero, int64_t zeros, bool vec) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) {
    const int64_t i = (row - rows) * 64 + lane;
    if (i < zeros) zero[i] = 0;
    return;
  }
  uint32_t m = 0;
  for (int64_t k = 8 * lane; k < K; k += 512) {
    float v[8];
    load8(x + row * ldx, k, K, vec, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, finite_bits(v[i]));
  }
  m = wave_umax(m);
  if (lane == 0) bits[row] = m;
}

constexpr int kScaleRun = 4096;  // scales of a workgroup, `runs` of them a group
__global__ void __launch_bounds__(256)
scale_bits_kernel(const float* __restrict__ s, int64_t n, uint32_t runs, uint32_t* bits) {
  __shared__ uint32_t sh[4];
  const uint32_t group = blockIdx.x / runs;
  const float* src = s + (int64_t)group * n;
  const int64_t at = (int64_t)(blockIdx.x % runs) * kScaleRun + 4 * threadIdx.x;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kScaleRun / 1024; ++i) {
    const int64_t k = at + 1024 * i;
    if (k + 4 <= n) {
      const f32x4_a4 x = *(const f32x4_a4*)(src + k);
#pragma unroll
      for (int j = 0; j < 4; ++j) m = umax(m, finite_bits(x[j]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k + j < n) m = umax(m, finite_bits(src[k + j]));
    }
  }
  m = block_umax(m, sh);
  if (threadIdx.x == 0) atomicMax(bits + group, m);
}

__global__ void __launch_bounds__(256)
gate_sums_kernel(const float* __restrict__ part, int32_t parts, const int32_t* __restrict__ ids,
                 int64_t n, int32_t experts, float* dweights) {
  const int64_t slot = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (slot >= n) return;
  const int32_t id = ids[slot];
  float s = 0.0f;
  if (id_ok(id, experts))
    for (int i = 0; i < parts; ++i) s += part[slot * parts + i];
  if (id >= experts) s = bits_f32(0x7fc00000u);
  dweights[slot] = s;
}

// ---- the head's last steps -------------------------------------------------------

// A workgroup a row: parts (maximum, sum of e^(z - maximum)) of the vocabulary's
// tiles joined, and the loss.  A part that is NaN or +inf makes the row NaN.
__global__ void __launch_bounds__(256) head_finish_kernel(const HeadFinish p) {
  __shared__ float sh[4];
  __shared__ uint32_t sh_nan[4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t m = blockIdx.x;
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2* st = (const f32x2*)(p.stats + m * p.parts * 2);
  float top = -__builtin_inff();
  bool nan = false;
  for (int i = threadIdx.x; i < p.parts; i += 256) {
    const f32x2 v = st[i];
    nan |= v[0] != v[0] || v[1] != v[1] || v[0] == __builtin_inff();
    top = v[0] > top ? v[0] : top;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const float o = __shfl_xor(top, d, 64);
    top = o > top ? o : top;
  }
  if (lane == 0) sh[w] = top;
  const bool any = __any(nan);
  if (lane == 0) sh_nan[w] = any;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top = sh[i] > top ? sh[i] : top;
    nan |= sh_nan[i] != 0;
  }
  __syncthreads();
  float sum = 0.0f;
  for (int i = threadIdx.x; i < p.parts; i += 256) {
    const f32x2 v = st[i];
    sum += v[0] == top ? v[1] : exp2_fast((v[0] - top) * kLog2e) * v[1];
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
  if (lane == 0) sh[w] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  sum = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  float lse = top + log2_fast(sum) * kLn2;
  if (nan) lse = bits_f32(0x7fc00000u);
  p.lse[m] = lse;
  const int64_t t = p.targets[m];
  p.loss[m] = t < 0 ? 0.0f : t >= p.V ? bits_f32(0x7fc00000u) : lse - p.chosen[m];
}

template <typename T>
__global__ void __launch_bounds__(256)
head_store_kernel(const float* __restrict__ acc, int32_t splits, int64_t M, int64_t K,
                  const int64_t* __restrict__ targets, int64_t V, T* dx, int64_t lddx) {
  const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (k >= K) return;
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
    const int64_t t = targets[m];
    float v = 0.0f;
    for (int i = 0; i < splits; ++i) v += acc[(i * M + m) * K + k];
    v = t < 0 ? 0.0f : t >= V ? bits_f32(0x7fc00000u) : v;
    dx[m * lddx + k] = from_f32<T>(v);
  }
}

bool aligned16(const void* p, int64_t ld, int64_t e) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * e % 16 == 0;
}

constexpr int64_t kGridY = 65535;

}  // namespace

hipError_t launch_lists(const int32_t* ids, int64_t n, int64_t experts, int32_t tile_rows,
                        const RowLists& r, hipStream_t s) {
  static_assert(kMaxExperts == kListThreads, "a thread an expert");
  hipLaunchKernelGGL(lists_kernel, dim3(1), dim3(kListThreads), 0, s, ids, (int32_t)n,
                     (int32_t)experts, tile_rows, r);
  return hipGetLastError();
}

template <typename T>
static void split_of(const void* x, int64_t ldx, int64_t K, int32_t order, const int32_t* ids,
                     int64_t experts, const SplitRows& r, hipStream_t s) {
  const dim3 grid((uint32_t)((r.rows + 3) / 4));
  const bool vec = aligned16(x, ldx, sizeof(T));
#define Q4_SPLIT(HOLD)                                                                             \
  hipLaunchKernelGGL((split_kernel<T, HOLD>), grid, dim3(256), 0, s, (const T*)x, ldx, K, order, ids, \
                     (int32_t)experts, r, vec)
  if (r.Kp <= 1024)
    Q4_SPLIT(2);
  else if (r.Kp <= 2048)
    Q4_SPLIT(4);
  else if (r.Kp <= 4096)
    Q4_SPLIT(8);
  else
    Q4_SPLIT(0);
#undef Q4_SPLIT
}

hipError_t launch_split(const void* x, int64_t ldx, int32_t dtype, int64_t K, int32_t nibble_order,
                        const int32_t* ids, int64_t experts, const SplitRows& r, hipStream_t s) {
  if (dtype == Q4_DTYPE_F32)
    split_of<float>(x, ldx, K, nibble_order, ids, experts, r, s);
  else if (dtype == Q4_DTYPE_F16)
    split_of<_Float16>(x, ldx, K, nibble_order, ids, experts, r, s);
  else
    split_of<bf16>(x, ldx, K, nibble_order, ids, experts, r, s);
  return hipGetLastError();
}

hipError_t launch_combine(const CombineParams& p, int32_t dtype, hipStream_t s) {
  const dim3 grid((uint32_t)((p.N + 1023) / 1024), (uint32_t)(p.T < kGridY ? p.T : kGridY));
  if (dtype == Q4_DTYPE_F32)
    hipLaunchKernelGGL(combine_kernel<float>, grid, dim3(256), 0, s, p, aligned16(p.out, p.ldo, 4));
  else if (dtype == Q4_DTYPE_F16)
    hipLaunchKernelGGL(combine_kernel<_Float16>, grid, dim3(256), 0, s, p, aligned16(p.out, p.ldo, 2));
  else
    hipLaunchKernelGGL(combine_kernel<bf16>, grid, dim3(256), 0, s, p, aligned16(p.out, p.ldo, 2));
  return hipGetLastError();
}

hipError_t launch_row_bits(const void* x, int64_t ldx, int32_t dtype, int64_t rows, int64_t K,
                           uint32_t* bits, uint32_t* zero, int64_t zeros, hipStream_t s) {
  const dim3 grid((uint32_t)((rows + (zeros + 63) / 64 + 3) / 4));
  if (dtype == Q4_DTYPE_F32)
    hipLaunchKernelGGL(row_bits_kernel<float>, grid, dim3(256), 0, s, (const float*)x, ldx, rows, K,
                       bits, zero, zeros, aligned16(x, ldx, 4));
  else if (dtype == Q4_DTYPE_F16)
    hipLaunchKernelGGL(row_bits_kernel<_Float16>, grid, dim3(256), 0, s, (const _Float16*)x, ldx,
                       rows, K, bits, zero, zeros, aligned16(x, ldx, 2));
  else
    hipLaunchKernelGGL(row_bits_kernel<bf16>, grid, dim3(256), 0, s, (const bf16*)x, ldx, rows, K,
                       bits, zero, zeros, aligned16(x, ldx, 2));
  return hipGetLastError();
}

hipError_t launch_scale_bits(const float* sc, int64_t n, int64_t groups, uint32_t* bits,
                             hipStream_t s) {
  const uint32_t runs = (uint32_t)((n + kScaleRun - 1) / kScaleRun);
  hipLaunchKernelGGL(scale_bits_kernel, dim3((uint32_t)groups * runs), dim3(256), 0, s, sc, n, runs, bits);
  return hipGetLastError();
}

hipError_t launch_gate_sums(const float* part, int32_t parts, const int32_t* ids, int64_t n,
                            int64_t experts, float* dweights, hipStream_t s) {
  hipLaunchKernelGGL(gate_sums_kernel, dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, s, part,
                     parts, ids, n, (int32_t)experts, dweights);
  return hipGetLastError();
}

hipError_t launch_head_finish(const HeadFinish& p, hipStream_t s) {
  hipLaunchKernelGGL(head_finish_kernel, dim3((uint32_t)p.M), dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_head_store(const float* acc, int32_t splits, int64_t M, int64_t K, const int64_t* targets,
                             int64_t V, void* dx, int64_t lddx, int32_t dtype, hipStream_t s) {
  const dim3 grid((uint32_t)((K + 255) / 256), (uint32_t)(M < kGridY ? M : kGridY));
  if (dtype == Q4_DTYPE_F32)
    hipLaunchKernelGGL(head_store_kernel<float>, grid, dim3(256), 0, s, acc, splits, M, K, targets, V,
                       (float*)dx, lddx);
  else if (dtype == Q4_DTYPE_F16)
    hipLaunchKernelGGL(head_store_kernel<_Float16>, grid, dim3(256), 0, s, acc, splits, M, K, targets, V,
                       (_Float16*)dx, lddx);
  else
    hipLaunchKernelGGL(head_store_kernel<bf16>, grid, dim3(256), 0, s, acc, splits, M, K, targets, V,
                       (bf16*)dx, lddx);
  return hipGetLastError();
}

}  // namespace q4
