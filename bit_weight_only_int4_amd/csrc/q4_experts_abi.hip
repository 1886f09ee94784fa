// q4_experts_abi.hip -- the C ABI of include/q4experts.h: argument checks and
// launches on the caller's stream.  As in q4_abi.hip every check runs before
// anything is queued, errors are return codes and no exception can leave.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_experts.h"
#include "q4_serve.h"

namespace {

using q4::Packed;
using q4::RowLists;
using q4::SplitRows;
using q4::Tile;

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
// Bytes of `rows` rows of n elements, ld apart.
Range span(const void* p, int64_t rows, int64_t ld, int64_t n, int64_t elem) {
  if (!p || rows <= 0 || n <= 0) return Range{0, 0};
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + (uintptr_t)(((rows - 1) * ld + n) * elem)};
}
Range flat(const void* p, int64_t n, int64_t elem) { return span(p, 1, 0, n, elem); }
bool overlap(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// every output apart from every input and from each other
template <int NO, int NI>
bool apart(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return false;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return false;
  }
  return true;
}

constexpr int64_t kMaxRows = (int64_t)1 << 24;   // rows, slots
constexpr int64_t kMaxDepth = (int64_t)1 << 15;  // hidden, width
constexpr int64_t kMaxVocab = (int64_t)1 << 30;
constexpr int64_t kMaxPitch = (int64_t)1 << 37;

bool dtype_ok(int32_t d) { return d == Q4_DTYPE_F32 || d == Q4_DTYPE_F16 || d == Q4_DTYPE_BF16; }
int64_t dtype_size(int32_t d) { return d == Q4_DTYPE_F32 ? 4 : 2; }
int32_t parts_of(int32_t d) { return d == Q4_DTYPE_F32 ? 2 : 1; }
bool depth_ok(int64_t k) { return k >= 8 && k <= kMaxDepth && k % 8 == 0; }
bool pitch_ok(int64_t ld, int64_t rows, int64_t n) {
  return ld >= 0 && ld < kMaxPitch && (rows <= 1 || ld >= n);
}
bool order_ok(int32_t o) { return o == Q4_ORDER_LOW_FIRST || o == Q4_ORDER_HIGH_FIRST; }

q4_status status_of(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_DEVICE; }

// A group size the kernels take for a depth (one group may be of any size).
q4_status group_status(int64_t gs, int64_t K) {
  if (gs < 0) return Q4_ERR_INVALID_ARG;
  return gs == 0 || gs >= K || gs == 32 || gs % 64 == 0 ? Q4_OK : Q4_ERR_UNSUPPORTED;
}

// Pieces of a workspace, each 256-byte aligned within it.
struct Carve {
  uint8_t* base;
  size_t at = 0;
  explicit Carve(void* p) : base((uint8_t*)p) {}
  template <typename T>
  T* take(int64_t n) {
    T* r = (T*)(base + at);
    at += ((size_t)n * sizeof(T) + 255) / 256 * 256;
    return r;
  }
};

SplitRows take_split(Carve& c, int64_t rows, int64_t K, int32_t parts) {
  SplitRows r{};
  r.rows = rows;
  r.Kp = q4::split_pitch(K);
  r.parts = parts;
  r.a = c.take<_Float16>(parts * rows * r.Kp);
  r.e = c.take<int32_t>(rows);
  return r;
}
RowLists take_lists(Carve& c, int64_t n, int64_t experts, int64_t tile_rows) {
  RowLists r{};
  r.slots = c.take<int32_t>(n);
  r.tiles = c.take<Tile>(q4::tile_bound(n, experts, tile_rows));
  r.n_tiles = c.take<int32_t>(1);
  return r;
}

bool experts_sizes_ok(int32_t dtype, int64_t T, int64_t H, int64_t W, int64_t E, int64_t k) {
  return dtype_ok(dtype) && T >= 0 && T < kMaxRows && depth_ok(H) && depth_ok(W) && E >= 1 &&
         E <= q4::kMaxExperts && k >= 1 && k <= q4::kMaxTopK && T * k < kMaxRows;
}

// ---- the experts' forward pass -------------------------------------------------

struct ExpertsPlan {
  bool few, direct;
  int32_t tile_rows;
  int64_t n, bound;
  float *h, *y;
  RowLists lists;
  SplitRows xs, hs;
  size_t bytes;
};

// Tiles of 128 rows unpack a word for twice the rows; tiles of 64 waste less
// where an expert's rows end.  64 / 128, us: 32 experts of 2048 x 1408 in groups
// of 128, fp32, 128 rows each 249 / 287, 192 332 / 341, 256 425 / 418, 512
// 782 / 719; bf16, 128 212 / 226, 256 342 / 325, 512 608 / 558, 1024 1123 /
// 1017; 8 experts of 4096 x 3584 in groups of 32, fp32, 384 rows 800 / 734;
// bf16, 200 371 / 343, 400 623 / 591.
int32_t gemm_tile_rows(int64_t n, int64_t experts) { return n >= 256 * experts ? 128 : 64; }

ExpertsPlan plan_experts(void* ws, int32_t dtype, int64_t T, int64_t H, int64_t W, int64_t E,
                         int64_t k) {
  ExpertsPlan p{};
  Carve c(ws);
  p.n = T * k;
  const int32_t parts = parts_of(dtype);
  // While an expert has few rows on average the weights' bytes count, not the
  // products; a workgroup of the kernel for few rows has 8 rows, and deep ones
  // are dear to split in each of them.  Few / tiles, us: 64 experts of 2048 x
  // 1024, fp32, 8 rows each 81 / 126, 14 116 / 128, 16 128 / 129, 24 175 / 136;
  // bf16 82 / 105, 109 / 105, 120 / 105, 166 / 108; 8 experts of 4096 x 3584,
  // fp32, 4 rows 73 / 147, 8 110 / 146, 16 166 / 147; bf16 61 / 127, 91 / 128,
  // 132 / 129.
  p.few = p.n <= (H <= 2048 && W <= 2048 ? 14 : 8) * E && H <= q4::kFewDepth && W <= q4::kFewDepth;
  // Few slots, mostly alone in their experts: each has workgroups, which look
  // for others of its expert, and the launch that lists the rows falls away.
  // Direct / listed, us: 64 experts, 8 slots 19.2 / 22.8, 32 37.9 / 40.2, 64
  // 55.7 / 54.1; 16 experts, 14 slots 40.8 / 42.0, 64 101 / 86.
  p.direct = p.few && p.n <= q4::kFewDirect && p.n <= E;
  // 8 rows in two parts fill the second product's operands, and rows of more than
  // 4096 share LDS by four (a token is in an expert's list once, as a rule: more
  // tiles hold the others)
  const int64_t most = H > 4096 || W > 4096 ? 4 : 8, few_rows = T < most ? T : most;
  p.tile_rows = p.few ? (int32_t)few_rows : gemm_tile_rows(p.n, E);
  p.bound = p.n ? q4::tile_bound(p.n, E, p.tile_rows) : 0;
  p.h = c.take<float>(p.n * W);
  p.y = c.take<float>(p.n * H);
  if (!p.direct) p.lists = take_lists(c, p.n, E, p.tile_rows);
  if (!p.few) {
    p.xs = take_split(c, T, H, parts);
    p.hs = take_split(c, p.n, W, 2);  // of fp32 values
  }
  p.bytes = c.at;
  return p;
}

bool experts_grid_ok(const ExpertsPlan& p, int64_t H, int64_t W) {
  const int64_t most = H > 2 * W ? H : 2 * W;
  const int64_t cols = p.few ? (most + 255) / 256 * 8 : (most + 127) / 128;
  return (double)(p.direct ? p.n : p.bound) * (double)cols <= (double)(q4::kMaxGrid / 2);
}

// ---- and backward -----------------------------------------------------------------

struct ExpertsBackPlan {
  int32_t tile_rows;
  int64_t n, bound, width_tiles, hidden_tiles, s_words;
  RowLists lists;
  uint32_t *dout_bits, *dpre_bits, *s_bits;
  float *dpre, *dw_part, *dx;
  size_t bytes;
};

// As above for the gradient, 64 / 128, us, fp32; 16-bit types alike, in two parts
// too.  One scale for a tile's columns: 32 experts of 2048 x 1408 in groups of
// 128, 128 rows each 340 / 430, 256 536 / 614, 512 940 / 1034, 1024 1791 / 1777
// (bf16 1774 / 1752); 8 experts of 4096 x 3584, 1024 rows 2085 / 2021.  Groups of
// 32, where the operand is made once a group: 128 rows 630 / 730, 192 850 / 795,
// 256 1072 / 1024, 512 1876 / 1734.
int32_t back_tile_rows(int64_t n, int64_t experts, int64_t group) {
  return n >= (group % 128 == 0 ? 1024 : 192) * experts ? 128 : 64;
}

ExpertsBackPlan plan_experts_back(void* ws, int64_t T, int64_t H, int64_t W, int64_t E, int64_t k,
                                  int64_t group) {
  ExpertsBackPlan p{};
  Carve c(ws);
  p.n = T * k;
  p.tile_rows = back_tile_rows(p.n, E, group);
  p.bound = q4::tile_bound(p.n, E, p.tile_rows);
  p.width_tiles = (W + 127) / 128;
  p.hidden_tiles = (H + 127) / 128;
  p.lists = take_lists(c, p.n, E, 64);
  p.dout_bits = c.take<uint32_t>(T);
  p.s_words = E * (q4::groups_of(W, group) + q4::groups_of(H, group));
  p.dpre_bits = c.take<uint32_t>(p.n + p.s_words);
  p.s_bits = p.dpre_bits + p.n;
  p.dpre = c.take<float>(p.n * 2 * W);
  p.dw_part = c.take<float>(p.n * 4 * p.width_tiles);  // a wave's each
  p.dx = c.take<float>(p.n * H);
  p.bytes = c.at;
  return p;
}

// ---- the head ------------------------------------------------------------------------

// Rows are taken so many at a time, which bounds the workspace.
constexpr int64_t kHeadRows = 8192;

struct HeadPlan {
  int64_t rows;  // at a time
  int32_t tile_rows;
  SplitRows xs;
  int32_t stat_parts;  // forward
  float *stats, *chosen;
  // backward
  int64_t piece;  // of the vocabulary
  int32_t splits;
  float *d, *acc;
  uint32_t *g_bits, *s_bits;
  size_t bytes;
};

// A head's rows end once: tiles of 128 where their last one is not half empty,
// or where there are many.  64 / 128, loss of 32003 x 2048, fp32, us: 96 rows
// 44 / 54, 160 59 / 71, 256 90 / 77, 320 96 / 109, 512 143 / 139; bf16 38 / 38,
// 46 / 47, 58 / 49, 67 / 62, 98 / 88.
int32_t head_tile_rows(int64_t rows) {
  return rows > 320 || (rows > 192 && rows <= 256) ? 128 : 64;
}

bool head_sizes_ok(int32_t dtype, int64_t M, int64_t V, int64_t K) {
  if (!dtype_ok(dtype) || M < 0 || M >= kMaxRows || V < 1 || V > kMaxVocab || !depth_ok(K)) return false;
  // the workgroups of a launch
  const int64_t rows = M < kHeadRows ? M : kHeadRows, tile = head_tile_rows(rows);
  return (double)((V + 127) / 128) * (double)((rows + tile - 1) / tile) <= (double)q4::kMaxGrid;
}

HeadPlan plan_head(void* ws, int32_t dtype, int64_t M, int64_t V, int64_t K, int64_t group, bool back) {
  HeadPlan p{};
  Carve c(ws);
  p.rows = M < kHeadRows ? M : kHeadRows;
  const int32_t parts = parts_of(dtype);
  p.tile_rows = head_tile_rows(p.rows);
  p.xs = take_split(c, p.rows, K, parts);
  if (!back) {
    p.stat_parts = (int32_t)((V + 127) / 128) * (p.tile_rows == 64 && parts == 1 ? 4 : 2);  // a wave's each
    p.stats = c.take<float>(p.rows * p.stat_parts * 2);
    p.chosen = c.take<float>(p.rows);
  } else {
    // A piece's gradient is to stay in the last-level cache between its two
    // products.  2048 rows of bf16 over 128257 x 2048: 64 MB a piece 3647 us, 128
    // 3343, 256 3352, 512 3417; fp32 4501, 4205, 4276, 4339.
    const int64_t most = (int64_t)(256 << 20) / 4 / p.rows;
    const int64_t pieces = (V + (most > 1024 ? most : 1024) - 1) / (most > 1024 ? most : 1024);
    p.piece = ((V + pieces - 1) / pieces + 127) / 128 * 128;
    const int64_t tiles = (p.rows + p.tile_rows - 1) / p.tile_rows * ((K + 127) / 128);
    // Splits of a piece, at least 8 steps deep, so that rounds of the workgroups
    // that fit the card (two a CU) come out even, at a hundredth each for their
    // sums.  Backward of 32003 x 4096 and 700 rows, 192 tiles, fp32, 2, 4, 5, 8, 10
    // splits 791, 759, 748, 746, 774 us; 128257 x 2048, 2048 rows, 256 tiles, bf16,
    // 1, 2, 3, 4, 6, 8 splits 4164, 3370, 3622, 3465, 3546, 3646.
    const int64_t fit = 512;
    double least = 0.0;
    for (int64_t n = 1; n <= 16 && (n == 1 || n <= p.piece / 512); ++n) {
      const double cost = (double)((tiles * n + fit - 1) / fit) / (double)n * (1.0 + 0.01 * (double)n);
      if (n == 1 || cost < least) {
        p.splits = (int32_t)n;
        least = cost;
      }
    }
    p.d = c.take<float>(p.rows * p.piece);
    p.acc = c.take<float>(p.splits * p.rows * K);
    p.g_bits = c.take<uint32_t>(p.rows);
    p.s_bits = c.take<uint32_t>(q4::groups_of(K, group));
  }
  p.bytes = c.at;
  return p;
}

}  // namespace

extern "C" {

q4_status q4_route(const void* logits, int64_t ld, int32_t dtype, int64_t T, int64_t experts,
                   int64_t top_k, int32_t score, const float* bias, int64_t groups,
                   int64_t top_groups, int32_t renormalize, float scale, int32_t* ids,
                   float* weights, void* stream) {
  if (!dtype_ok(dtype) || T < 0 || T >= kMaxRows || experts < 1 || experts > q4::kMaxExperts ||
      top_k < 1 || top_k > q4::kMaxTopK)
    return Q4_ERR_INVALID_ARG;
  if ((score != Q4_SCORE_SOFTMAX && score != Q4_SCORE_SIGMOID) ||
      (renormalize != 0 && renormalize != 1))
    return Q4_ERR_INVALID_ARG;
  if (groups < 1 || experts % groups || top_groups < 1 || top_groups > groups ||
      top_k > experts / groups * top_groups)
    return Q4_ERR_INVALID_ARG;
  if (!pitch_ok(ld, T, experts) || !(scale - scale == 0.0f)) return Q4_ERR_INVALID_ARG;
  if (T == 0) return Q4_OK;
  const int64_t e = dtype_size(dtype);
  if (!logits || !ids || !weights || !aligned(logits, e) || !aligned(bias, 4) || !aligned(ids, 4) ||
      !aligned(weights, 4))
    return Q4_ERR_INVALID_ARG;
  const Range outs[] = {flat(ids, T * top_k, 4), flat(weights, T * top_k, 4)};
  const Range ins[] = {span(logits, T, ld, experts, e), flat(bias, bias ? experts : 0, 4)};
  if (!apart(outs, ins)) return Q4_ERR_ALIAS;
  q4::RouteParams p{logits, ld, T, (int32_t)experts, (int32_t)top_k, score, (int32_t)groups,
                    (int32_t)top_groups, renormalize, bias, scale, ids, weights};
  return status_of(q4::launch_route(p, dtype, (hipStream_t)stream));
}

q4_status q4_route_backward(const void* logits, int64_t ld, int32_t dtype, int64_t T,
                            int64_t experts, int64_t top_k, const int32_t* ids, int32_t score,
                            int32_t renormalize, float scale, const float* g_weights,
                            void* dlogits, int64_t ldd, void* stream) {
  if (!dtype_ok(dtype) || T < 0 || T >= kMaxRows || experts < 1 || experts > q4::kMaxExperts ||
      top_k < 1 || top_k > q4::kMaxTopK || top_k > experts)
    return Q4_ERR_INVALID_ARG;
  if ((score != Q4_SCORE_SOFTMAX && score != Q4_SCORE_SIGMOID) ||
      (renormalize != 0 && renormalize != 1))
    return Q4_ERR_INVALID_ARG;
  if (!pitch_ok(ld, T, experts) || !pitch_ok(ldd, T, experts) || !(scale - scale == 0.0f))
    return Q4_ERR_INVALID_ARG;
  if (T == 0) return Q4_OK;
  const int64_t e = dtype_size(dtype);
  if (!logits || !ids || !g_weights || !dlogits || !aligned(logits, e) || !aligned(dlogits, e) ||
      !aligned(ids, 4) || !aligned(g_weights, 4))
    return Q4_ERR_INVALID_ARG;
  const bool in_place = dlogits == logits && (ldd == ld || T == 1);
  const Range outs[] = {span(dlogits, T, ldd, experts, e)};
  const Range ins[] = {in_place ? Range{0, 0} : span(logits, T, ld, experts, e),
                       flat(ids, T * top_k, 4), flat(g_weights, T * top_k, 4)};
  if (!apart(outs, ins)) return Q4_ERR_ALIAS;
  q4::RouteBwdParams p{logits, ld, T, (int32_t)experts, (int32_t)top_k, score, renormalize, scale,
                       ids, g_weights, dlogits, ldd};
  return status_of(q4::launch_route_backward(p, dtype, (hipStream_t)stream));
}

size_t q4_experts_workspace_bytes(int32_t dtype, int64_t T, int64_t hidden, int64_t width,
                                  int64_t experts, int64_t top_k, int64_t group_size) {
  if (!experts_sizes_ok(dtype, T, hidden, width, experts, top_k) || T == 0 ||
      group_status(group_size, hidden) != Q4_OK || group_status(group_size, width) != Q4_OK)
    return 0;
  return plan_experts(nullptr, dtype, T, hidden, width, experts, top_k).bytes;
}

q4_status q4_experts(const void* x, int64_t ldx, int32_t dtype, int64_t T, int64_t hidden,
                     int64_t width, int64_t experts, int64_t top_k, const int32_t* ids,
                     const float* weights, const uint8_t* gate_up, const float* gate_up_scales,
                     const uint8_t* down, const float* down_scales, int64_t group_size,
                     int32_t nibble_order, void* out, int64_t ldo, float* pre, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!experts_sizes_ok(dtype, T, hidden, width, experts, top_k) || !order_ok(nibble_order) ||
      !pitch_ok(ldx, T, hidden) || !pitch_ok(ldo, T, hidden))
    return Q4_ERR_INVALID_ARG;
  q4_status gst = group_status(group_size, hidden);
  if (gst == Q4_OK) gst = group_status(group_size, width);
  if (gst != Q4_OK) return gst;
  if (T == 0) return Q4_OK;
  const int64_t e = dtype_size(dtype);
  if (!x || !ids || !weights || !gate_up || !gate_up_scales || !down || !down_scales || !out)
    return Q4_ERR_INVALID_ARG;
  if (!aligned(x, e) || !aligned(out, e) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(gate_up, 4) || !aligned(down, 4) || !aligned(gate_up_scales, 4) ||
      !aligned(down_scales, 4) || !aligned(pre, 4))
    return Q4_ERR_INVALID_ARG;
  const Packed gu = q4::packed(gate_up, gate_up_scales, 2 * width, hidden, group_size);
  const Packed dn = q4::packed(down, down_scales, hidden, width, group_size);
  ExpertsPlan pl = plan_experts(workspace, dtype, T, hidden, width, experts, top_k);
  if (!experts_grid_ok(pl, hidden, width)) return Q4_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < pl.bytes || !aligned(workspace, 16)) return Q4_ERR_WORKSPACE;
  const int64_t n = pl.n;
  const Range outs[] = {span(out, T, ldo, hidden, e), flat(pre, n * 2 * width, 4),
                        flat(workspace, (int64_t)pl.bytes, 1)};
  const Range ins[] = {span(x, T, ldx, hidden, e), flat(ids, n, 4), flat(weights, n, 4),
                       flat(gate_up, experts * gu.expert_bytes, 1),
                       flat(gate_up_scales, experts * gu.expert_scales, 4),
                       flat(down, experts * dn.expert_bytes, 1),
                       flat(down_scales, experts * dn.expert_scales, 4)};
  if (!apart(outs, ins)) return Q4_ERR_ALIAS;

  hipStream_t s = (hipStream_t)stream;
  hipError_t err = hipSuccess;
  if (!pl.direct) err = q4::launch_lists(ids, n, experts, pl.tile_rows, pl.lists, s);
  if (pl.few) {
    q4::FewParams f{};
    f.nibble_order = nibble_order;
    f.n = (int32_t)n;
    f.experts = (int32_t)experts;
    if (pl.direct) {
      f.ids = ids;
    } else {
      f.slots = pl.lists.slots;
      f.tiles = pl.lists.tiles;
      f.n_tiles = pl.lists.n_tiles;
      f.row_tiles = (int32_t)pl.bound;
    }
    f.w = gu;
    f.x = x;
    f.ldx = ldx;
    f.dtype = dtype;
    f.slots_per_row = (int32_t)top_k;
    f.out = pl.h;
    f.out_ld = width;
    f.pre = pre;
    f.width = width;
    if (err == hipSuccess) err = q4::launch_few(f, pl.tile_rows, true, s);
    f.w = dn;
    f.x = pl.h;
    f.ldx = width;
    f.dtype = Q4_DTYPE_F32;
    f.slots_per_row = 1;
    f.out = pl.y;
    f.out_ld = hidden;
    f.pre = nullptr;
    if (err == hipSuccess) err = q4::launch_few(f, pl.tile_rows, false, s);
  } else {
    if (err == hipSuccess)
      err = q4::launch_split(x, ldx, dtype, hidden, nibble_order, nullptr, 0, pl.xs, s);
    q4::GemmParams g{};
    g.slots = pl.lists.slots;
    g.tiles = pl.lists.tiles;
    g.n_tiles = pl.lists.n_tiles;
    g.row_tiles = (int32_t)pl.bound;
    g.w = gu;
    g.a = pl.xs;
    g.slots_per_row = (int32_t)top_k;
    g.col_tiles = (int32_t)((width + 63) / 64);
    g.n_cols = 2 * width;
    g.out = pl.h;
    g.out_ld = width;
    g.pre = pre;
    g.width = width;
    if (err == hipSuccess) err = q4::launch_gemm(g, pl.tile_rows, q4::kGatedRows, s);
    if (err == hipSuccess)
      err = q4::launch_split(pl.h, width, Q4_DTYPE_F32, width, nibble_order, ids, experts,
                             pl.hs, s);
    g.w = dn;
    g.a = pl.hs;
    g.slots_per_row = 1;
    g.col_tiles = (int32_t)((hidden + 127) / 128);
    g.n_cols = hidden;
    g.out = pl.y;
    g.out_ld = hidden;
    g.pre = nullptr;
    if (err == hipSuccess) err = q4::launch_gemm(g, pl.tile_rows, q4::kPlainRows, s);
  }
  q4::CombineParams c{pl.y, ids, weights, T, hidden, (int32_t)top_k, (int32_t)experts, out, ldo};
  if (err == hipSuccess) err = q4::launch_combine(c, dtype, s);
  return status_of(err);
}

size_t q4_experts_backward_workspace_bytes(int32_t dtype, int64_t T, int64_t hidden, int64_t width,
                                           int64_t experts, int64_t top_k, int64_t group_size) {
  if (!experts_sizes_ok(dtype, T, hidden, width, experts, top_k) || T == 0 ||
      group_status(group_size, hidden) != Q4_OK || group_status(group_size, width) != Q4_OK)
    return 0;
  return plan_experts_back(nullptr, T, hidden, width, experts, top_k, group_size).bytes;
}

q4_status q4_experts_backward(const void* dout, int64_t lddo, int32_t dtype, int64_t T,
                              int64_t hidden, int64_t width, int64_t experts, int64_t top_k,
                              const int32_t* ids, const float* weights, const float* pre,
                              const uint8_t* gate_up, const float* gate_up_scales,
                              const uint8_t* down, const float* down_scales, int64_t group_size,
                              int32_t nibble_order, void* dx, int64_t lddx, float* dweights,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!experts_sizes_ok(dtype, T, hidden, width, experts, top_k) || !order_ok(nibble_order) ||
      !pitch_ok(lddo, T, hidden) || !pitch_ok(lddx, T, hidden))
    return Q4_ERR_INVALID_ARG;
  q4_status gst = group_status(group_size, hidden);
  if (gst == Q4_OK) gst = group_status(group_size, width);
  if (gst != Q4_OK) return gst;
  if (T == 0) return Q4_OK;
  const int64_t e = dtype_size(dtype);
  if (!dout || !ids || !weights || !pre || !gate_up || !gate_up_scales || !down || !down_scales ||
      !dx || !dweights)
    return Q4_ERR_INVALID_ARG;
  if (!aligned(dout, e) || !aligned(dx, e) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(pre, 4) || !aligned(dweights, 4) || !aligned(gate_up, 4) || !aligned(down, 4) ||
      !aligned(gate_up_scales, 4) || !aligned(down_scales, 4))
    return Q4_ERR_INVALID_ARG;
  const Packed gu = q4::packed(gate_up, gate_up_scales, 2 * width, hidden, group_size);
  const Packed dn = q4::packed(down, down_scales, hidden, width, group_size);
  ExpertsBackPlan pl = plan_experts_back(workspace, T, hidden, width, experts, top_k, group_size);
  const int64_t most = pl.width_tiles > pl.hidden_tiles ? pl.width_tiles : pl.hidden_tiles;
  if ((double)pl.bound * (double)most > (double)q4::kMaxGrid) return Q4_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < pl.bytes || !aligned(workspace, 16)) return Q4_ERR_WORKSPACE;
  const int64_t n = pl.n;
  const Range outs[] = {span(dx, T, lddx, hidden, e), flat(dweights, n, 4),
                        flat(workspace, (int64_t)pl.bytes, 1)};
  const Range ins[] = {span(dout, T, lddo, hidden, e), flat(ids, n, 4), flat(weights, n, 4),
                       flat(pre, n * 2 * width, 4), flat(gate_up, experts * gu.expert_bytes, 1),
                       flat(gate_up_scales, experts * gu.expert_scales, 4),
                       flat(down, experts * dn.expert_bytes, 1),
                       flat(down_scales, experts * dn.expert_scales, 4)};
  if (!apart(outs, ins)) return Q4_ERR_ALIAS;

  hipStream_t s = (hipStream_t)stream;
  hipError_t err = q4::launch_lists(ids, n, experts, pl.tile_rows, pl.lists, s);
  if (err == hipSuccess)
    err = q4::launch_row_bits(dout, lddo, dtype, T, hidden, pl.dout_bits, pl.dpre_bits,
                              n + pl.s_words, s);
  uint32_t* gu_bits = pl.s_bits + experts * dn.G;
  if (err == hipSuccess) err = q4::launch_scale_bits(down_scales, dn.N, experts * dn.G, pl.s_bits, s);
  if (err == hipSuccess) err = q4::launch_scale_bits(gate_up_scales, gu.N, experts * gu.G, gu_bits, s);
  q4::BackParams b{};
  b.nibble_order = nibble_order;
  b.slots = pl.lists.slots;
  b.tiles = pl.lists.tiles;
  b.n_tiles = pl.lists.n_tiles;
  b.row_tiles = (int32_t)pl.bound;
  b.splits = 1;
  b.w = dn;
  b.d = dout;
  b.ldd = lddo;
  b.d_dtype = dtype;
  b.d_bits = pl.dout_bits;
  b.s_bits = pl.s_bits;
  b.slots_per_row = (int32_t)top_k;
  b.n_rows = hidden;
  b.col_tiles = (int32_t)pl.width_tiles;
  b.pre = pre;
  b.weights = weights;
  b.dpre = pl.dpre;
  b.dw_part = pl.dw_part;
  b.dpre_bits = pl.dpre_bits;
  if (err == hipSuccess) err = q4::launch_back(b, pl.tile_rows, true, s);
  if (err == hipSuccess)
    err = q4::launch_gate_sums(pl.dw_part, (int32_t)((pl.tile_rows == 64 ? 4 : 2) * pl.width_tiles), ids, n, experts, dweights, s);
  b.w = gu;
  b.d = pl.dpre;
  b.ldd = 2 * width;
  b.d_dtype = Q4_DTYPE_F32;
  b.d_bits = pl.dpre_bits;
  b.s_bits = gu_bits;
  b.slots_per_row = 1;
  b.n_rows = 2 * width;
  b.col_tiles = (int32_t)pl.hidden_tiles;
  b.out = pl.dx;
  b.out_ld = hidden;
  if (err == hipSuccess) err = q4::launch_back(b, pl.tile_rows, false, s);
  q4::CombineParams c{pl.dx, ids, nullptr, T, hidden, (int32_t)top_k, (int32_t)experts, dx, lddx};
  if (err == hipSuccess) err = q4::launch_combine(c, dtype, s);
  return status_of(err);
}

size_t q4_head_cross_entropy_workspace_bytes(int32_t dtype, int64_t M, int64_t vocab, int64_t K,
                                             int64_t group_size) {
  if (!head_sizes_ok(dtype, M, vocab, K) || M == 0 || group_status(group_size, K) != Q4_OK) return 0;
  return plan_head(nullptr, dtype, M, vocab, K, group_size, false).bytes;
}

q4_status q4_head_cross_entropy(const void* x, int64_t ldx, int32_t dtype, int64_t M,
                                int64_t vocab, int64_t K, const uint8_t* qw, const float* scales,
                                int64_t group_size, int32_t nibble_order, const int64_t* targets,
                                float* loss, float* lse, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!head_sizes_ok(dtype, M, vocab, K) || !order_ok(nibble_order) || !pitch_ok(ldx, M, K))
    return Q4_ERR_INVALID_ARG;
  const q4_status gst = group_status(group_size, K);
  if (gst != Q4_OK) return gst;
  if (M == 0) return Q4_OK;
  const int64_t e = dtype_size(dtype);
  if (!x || !qw || !scales || !targets || !loss || !lse || !aligned(x, e) || !aligned(qw, 4) ||
      !aligned(scales, 4) || !aligned(targets, 8) || !aligned(loss, 4) || !aligned(lse, 4))
    return Q4_ERR_INVALID_ARG;
  const Packed w = q4::packed(qw, scales, vocab, K, group_size);
  const HeadPlan pl = plan_head(workspace, dtype, M, vocab, K, group_size, false);
  if (!workspace || workspace_bytes < pl.bytes || !aligned(workspace, 16)) return Q4_ERR_WORKSPACE;
  const Range outs[] = {flat(loss, M, 4), flat(lse, M, 4), flat(workspace, (int64_t)pl.bytes, 1)};
  const Range ins[] = {span(x, M, ldx, K, e), flat(qw, w.expert_bytes, 1),
                       flat(scales, w.expert_scales, 4), flat(targets, M, 8)};
  if (!apart(outs, ins)) return Q4_ERR_ALIAS;

  hipStream_t s = (hipStream_t)stream;
  hipError_t err = hipSuccess;
  for (int64_t m0 = 0; m0 < M && err == hipSuccess; m0 += pl.rows) {
    SplitRows xs = pl.xs;
    xs.rows = M - m0 < pl.rows ? M - m0 : pl.rows;
    err = q4::launch_split((const uint8_t*)x + m0 * ldx * e, ldx, dtype, K, nibble_order,
                           nullptr, 0, xs, s);
    q4::GemmParams g{};
    g.w = w;
    g.a = xs;
    g.M = xs.rows;
    g.row_tiles = (int32_t)((xs.rows + pl.tile_rows - 1) / pl.tile_rows);
    g.col_tiles = (int32_t)((vocab + 127) / 128);
    g.n_cols = vocab;
    g.stats = pl.stats;
    g.chosen = pl.chosen;
    g.targets = targets + m0;
    if (err == hipSuccess) err = q4::launch_gemm(g, pl.tile_rows, q4::kHeadStats, s);
    q4::HeadFinish f{pl.stats, pl.stat_parts, pl.chosen, targets + m0, xs.rows, vocab, loss + m0,
                     lse + m0};
    if (err == hipSuccess) err = q4::launch_head_finish(f, s);
  }
  return status_of(err);
}

size_t q4_head_cross_entropy_backward_workspace_bytes(int32_t dtype, int64_t M, int64_t vocab,
                                                      int64_t K, int64_t group_size) {
  if (!head_sizes_ok(dtype, M, vocab, K) || M == 0 || group_status(group_size, K) != Q4_OK) return 0;
  return plan_head(nullptr, dtype, M, vocab, K, group_size, true).bytes;
}

q4_status q4_head_cross_entropy_backward(const void* x, int64_t ldx, int32_t dtype, int64_t M,
                                         int64_t vocab, int64_t K, const uint8_t* qw,
                                         const float* scales, int64_t group_size,
                                         int32_t nibble_order, const int64_t* targets,
                                         const float* lse, const float* g_loss, void* dx,
                                         int64_t lddx, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  if (!head_sizes_ok(dtype, M, vocab, K) || !order_ok(nibble_order) || !pitch_ok(ldx, M, K) ||
      !pitch_ok(lddx, M, K))
    return Q4_ERR_INVALID_ARG;
  const q4_status gst = group_status(group_size, K);
  if (gst != Q4_OK) return gst;
  if (M == 0) return Q4_OK;
  const int64_t e = dtype_size(dtype);
  if (!x || !qw || !scales || !targets || !lse || !g_loss || !dx || !aligned(x, e) ||
      !aligned(dx, e) || !aligned(qw, 4) || !aligned(scales, 4) || !aligned(targets, 8) ||
      !aligned(lse, 4) || !aligned(g_loss, 4))
    return Q4_ERR_INVALID_ARG;
  const Packed w = q4::packed(qw, scales, vocab, K, group_size);
  const HeadPlan pl = plan_head(workspace, dtype, M, vocab, K, group_size, true);
  if (!workspace || workspace_bytes < pl.bytes || !aligned(workspace, 16)) return Q4_ERR_WORKSPACE;
  const Range outs[] = {span(dx, M, lddx, K, e), flat(workspace, (int64_t)pl.bytes, 1)};
  const Range ins[] = {span(x, M, ldx, K, e), flat(qw, w.expert_bytes, 1),
                       flat(scales, w.expert_scales, 4), flat(targets, M, 8), flat(lse, M, 4),
                       flat(g_loss, M, 4)};
  if (!apart(outs, ins)) return Q4_ERR_ALIAS;

  hipStream_t s = (hipStream_t)stream;
  hipError_t err = hipSuccess;
  for (int64_t m0 = 0; m0 < M && err == hipSuccess; m0 += pl.rows) {
    SplitRows xs = pl.xs;
    xs.rows = M - m0 < pl.rows ? M - m0 : pl.rows;
    err = q4::launch_split((const uint8_t*)x + m0 * ldx * e, ldx, dtype, K, nibble_order,
                           nullptr, 0, xs, s);
    // no element of a row passes its g_loss: |p - 1[target]| <= 1
    if (err == hipSuccess)
      err = q4::launch_row_bits(g_loss + m0, 1, Q4_DTYPE_F32, xs.rows, 1, pl.g_bits, pl.s_bits, w.G, s);
    if (err == hipSuccess) err = q4::launch_scale_bits(scales, vocab, w.G, pl.s_bits, s);
    const int32_t row_tiles = (int32_t)((xs.rows + pl.tile_rows - 1) / pl.tile_rows);
    for (int64_t v0 = 0; v0 < vocab && err == hipSuccess; v0 += pl.piece) {
      const int64_t cols = vocab - v0 < pl.piece ? vocab - v0 : pl.piece;
      q4::GemmParams g{};
      g.w = w;
      g.a = xs;
      g.M = xs.rows;
      g.row_tiles = row_tiles;
      g.col_tiles = (int32_t)((cols + 127) / 128);
      g.n0 = v0;
      g.n_cols = cols;
      g.targets = targets + m0;
      g.lse = lse + m0;
      g.g = g_loss + m0;
      if (w.group)
        g.d = pl.d;
      else
        g.d_parts = (_Float16*)pl.d;  // (two of them take the place of a float)
      g.s_bits = pl.s_bits;
      g.out_ld = pl.piece;
      err = q4::launch_gemm(g, pl.tile_rows, q4::kHeadGrad, s);
      q4::BackParams b{};
      b.w = w;
      b.nibble_order = nibble_order;
      if (w.group)
        b.d = pl.d;
      else
        b.d_parts = g.d_parts;
      b.d_rows = xs.rows;
      b.ldd = pl.piece;
      b.d_dtype = Q4_DTYPE_F32;
      b.d_bits = pl.g_bits;
      b.s_bits = pl.s_bits;
      b.M = xs.rows;
      b.row_tiles = row_tiles;
      b.n0 = v0;
      b.n_rows = cols;
      b.splits = pl.splits;
      b.col_tiles = (int32_t)((K + 127) / 128);
      b.out = pl.acc;
      b.out_ld = K;
      b.accumulate = v0 > 0;
      if (err == hipSuccess) err = q4::launch_back(b, pl.tile_rows, false, s);
    }
    if (err == hipSuccess)
      err = q4::launch_head_store(pl.acc, pl.splits, xs.rows, K, targets + m0, vocab,
                                  (uint8_t*)dx + m0 * lddx * e, lddx, dtype, s);
  }
  return status_of(err);
}

}  // extern "C"
