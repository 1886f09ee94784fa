// q4_experts.h -- host-side interface between the C ABI of the expert and
// head-loss operators (q4_experts_abi.hip) and their kernels.  Not part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "q4experts.h"

namespace q4 {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;

struct RouteParams {
  const void* x;
  int64_t ld, T;
  int32_t E, top_k, score, groups, top_groups, renormalize;
  const float* bias;
  float scale;
  int32_t* ids;
  float* weights;
};
hipError_t launch_route(const RouteParams& p, int32_t dtype, hipStream_t s);

struct RouteBwdParams {
  const void* x;
  int64_t ld, T;
  int32_t E, top_k, score, renormalize;
  float scale;
  const int32_t* ids;
  const float* g;
  void* dx;
  int64_t ldd;
};
hipError_t launch_route_backward(const RouteBwdParams& p, int32_t dtype, hipStream_t s);

// One packed matrix per expert (one in all for the head).
struct Packed {
  const uint8_t* qw;
  const float* scales;
  int64_t N, K;         // rows, depth
  int32_t group;        // 0: a scale per row
  int32_t G;            // groups of a row
  int64_t expert_bytes; // N * K / 2
  int64_t expert_scales;
};
inline int64_t groups_of(int64_t K, int64_t group) {
  return group == 0 || group >= K ? 1 : (K + group - 1) / group;
}
inline Packed packed(const uint8_t* qw, const float* scales, int64_t N, int64_t K, int64_t group) {
  const int64_t gs = group >= K ? 0 : group;
  // a group of the whole depth indexes like a scale per row
  const int64_t G = groups_of(K, group);
  return Packed{qw, scales, N, K, (int32_t)gs, (int32_t)G, N * (K / 2), G * N};
}

// Tiles of rows that one expert's weights are multiplied with.  Rows are slots
// (token * top_k + j), listed expert by expert.
struct Tile {
  int32_t expert, first, rows, pad;  // first: index into `slots`
};
struct RowLists {
  int32_t* slots;    // [n] slot ids by expert
  Tile* tiles;       // [tile bound]
  int32_t* n_tiles;  // [1]
};
// At most so many tiles of `rows` rows: every expert in use has one that is not full.
inline int64_t tile_bound(int64_t n, int64_t experts, int64_t rows) {
  return n / rows + (experts < n ? experts : n);
}
hipError_t launch_lists(const int32_t* ids, int64_t n, int64_t experts, int32_t tile_rows,
                        const RowLists& r, hipStream_t s);

// Rows of activations as the matrix kernels read them: row r is scaled by
// 2^e[r] and held as `parts` binary16 numbers per element, [parts][rows][Kp].
struct SplitRows {
  _Float16* a;
  int64_t rows, Kp;   // Kp: K rounded up to a multiple of 64, zeros past K
  int32_t parts;
  int32_t* e;         // [rows]
};
inline int64_t split_pitch(int64_t K) { return (K + 63) / 64 * 64; }
// ids: rows whose id is outside [0, experts) are skipped (NULL: none)
hipError_t launch_split(const void* x, int64_t ldx, int32_t dtype, int64_t K,
                        int32_t nibble_order, const int32_t* ids, int64_t experts,
                        const SplitRows& r, hipStream_t s);

enum Epilogue : int32_t { kGatedRows = 0, kPlainRows = 1, kHeadStats = 2, kHeadGrad = 3 };

struct GemmParams {
  Packed w;
  SplitRows a;
  const int32_t* slots;   // NULL: row r of the tile is row r of a
  const Tile* tiles;      // NULL: tile m is rows m * rows per tile ...
  const int32_t* n_tiles; // NULL: row_tiles
  int32_t row_tiles;      // bound of the tiles
  int32_t slots_per_row;  // a slot's row of a is slot / slots_per_row
  int64_t M;              // rows without tiles
  int32_t col_tiles;
  int64_t n0;             // first row of the packed matrix (the head's pieces)
  int64_t n_cols;         // columns of this launch
  int32_t b_wide;         // packed rows are 16-byte aligned
  // epilogues
  float* out;             // kGatedRows: h [slot][width]; kPlainRows: [slot][N]
  int64_t out_ld;
  float* pre;             // kGatedRows, optional: [slot][2 width]
  int64_t width;
  float* stats;           // kHeadStats: [M][col_tiles][waves side by side][2]
  float* chosen;          // kHeadStats: [M] logit of the target
  const int64_t* targets;
  const float* lse;       // kHeadGrad
  const float* g;         // kHeadGrad
  float* d;               // kHeadGrad: [M][out_ld], or with a scale per row
  _Float16* d_parts;      // [2][rows of a][out_ld]: times it, scaled as BackParams says
  const uint32_t* s_bits;
};
hipError_t launch_gemm(const GemmParams& p, int32_t tile_rows, Epilogue epi, hipStream_t s);

// Few rows per expert: up to 8 a tile, weights straight from memory into the
// matrix operands.
struct FewParams {
  Packed w;
  const void* x;          // rows of dtype
  int64_t ldx;
  int32_t dtype;
  int32_t nibble_order;
  const int32_t* ids;     // direct: tiles are found from the n ids by each workgroup
  int32_t n, experts;
  const int32_t* slots;   // else lists
  const Tile* tiles;
  const int32_t* n_tiles;
  int32_t row_tiles;
  int32_t slots_per_row;
  float* out;             // gated: h [slot][width]; plain: [slot][N]
  int64_t out_ld;
  float* pre;
  int64_t width;
};
constexpr int64_t kFewDepth = 8192;  // of their rows, at most
constexpr int kFewDirect = 48;  // slots up to which workgroups find their rows themselves
hipError_t launch_few(const FewParams& p, int32_t tile_rows, bool gated, hipStream_t s);

// out[t] = sum_j weights[t, j] y[t * top_k + j]; weights NULL: all 1
struct CombineParams {
  const float* y;
  const int32_t* ids;
  const float* weights;
  int64_t T, N;
  int32_t top_k, experts;
  void* out;
  int64_t ldo;
};
hipError_t launch_combine(const CombineParams& p, int32_t dtype, hipStream_t s);

// The input gradient: rows d [rows][N] times the packed matrix [N][K],
// contracted over N.
struct BackParams {
  Packed w;
  int32_t nibble_order;
  const void* d;           // rows of d_dtype
  int64_t ldd;
  // or, with a scale per row of the matrix: d times it, against the row's and
  // the scales' largest (times 2^15), as two binary16 parts [2][d_rows][ldd] in
  // the operands' order, zeros from n_rows to the next multiple of 64
  const _Float16* d_parts;
  int64_t d_rows;
  int32_t d_dtype;
  const uint32_t* d_bits;  // [row of d]: bits of a magnitude that none of the row's passes
  const uint32_t* s_bits;  // [experts][groups]: of the group's largest scale
  const int32_t* slots;
  const Tile* tiles;
  const int32_t* n_tiles;
  int32_t row_tiles, slots_per_row;
  int64_t M;
  int64_t n0, n_rows;      // rows of the packed matrix contracted (the head's pieces)
  int32_t splits;          // of those rows, each into its own [M][out_ld] of out
  int32_t col_tiles;
  int32_t d_vec;           // rows of d are 16-byte aligned
  // plain: out [slot][K]; accumulate adds to what is there
  float* out;
  int64_t out_ld;
  int32_t accumulate;
  // through the gate: dh = weight * (out of this product); dpre [slot][2 width]
  const float* pre;
  const float* weights;
  float* dpre;
  float* dw_part;          // [slot][col_tiles][waves side by side: 4 of 64 rows, 2 of 128]
  uint32_t* dpre_bits;     // [slot]: the largest magnitude, by maximum
};
hipError_t launch_back(const BackParams& p, int32_t tile_rows, bool gate, hipStream_t s);

// Bits of rows' largest finite magnitudes; `zero` words beside them become 0.
hipError_t launch_row_bits(const void* x, int64_t ldx, int32_t dtype, int64_t rows, int64_t K,
                           uint32_t* bits, uint32_t* zero, int64_t zeros, hipStream_t s);
// and of n scales each of so many groups, as maxima over what is there
hipError_t launch_scale_bits(const float* s, int64_t n, int64_t groups, uint32_t* bits,
                             hipStream_t st);
// dweights from its parts
hipError_t launch_gate_sums(const float* part, int32_t parts, const int32_t* ids, int64_t n,
                            int64_t experts, float* dweights, hipStream_t s);

struct HeadFinish {
  const float* stats;
  int32_t parts;
  const float* chosen;
  const int64_t* targets;
  int64_t M, V;
  float *loss, *lse;
};
hipError_t launch_head_finish(const HeadFinish& p, hipStream_t s);
// dx rows, the sum of `splits` fp32 arrays, into dtype
hipError_t launch_head_store(const float* acc, int32_t splits, int64_t M, int64_t K, const int64_t* targets,
                             int64_t V, void* dx, int64_t lddx, int32_t dtype, hipStream_t s);

}  // namespace q4
