// q4_serve_abi.hip -- the C ABI of include/q4serve.h: argument checks and
// launches on the caller's stream.  As in q4_abi.hip every check runs before
// anything is queued, errors are return codes and no exception can leave.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_kv.h"
#include "q4_serve.h"

namespace {

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

// Bytes that [n0][n1][n2] elements with strides s0, s1 (and 1) can touch.
Range span(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2,
           int64_t elem) {
  if (!p || n0 <= 0 || n1 <= 0 || n2 <= 0) return Range{0, 0};
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + (uintptr_t)(((n0 - 1) * s0 + (n1 - 1) * s1 + n2) * elem)};
}

Range flat(const void* p, int64_t n, int64_t elem) { return span(p, 1, 0, 1, 0, n, elem); }

bool overlap(Range a, Range b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxDim = (int64_t)1 << 31;

bool dtype_ok(int32_t d) { return d == Q4_DTYPE_F32 || d == Q4_DTYPE_F16 || d == Q4_DTYPE_BF16; }
int64_t dtype_size(int32_t d) { return d == Q4_DTYPE_F32 ? 4 : 2; }

bool size_ok(int64_t v) { return v >= 0 && v < kMaxDim; }

// strides that keep the rows of [T, heads, dim] apart, whichever of tokens
// and heads is the outer axis
bool strides_ok(int64_t ts, int64_t hs, int64_t T, int64_t heads, int64_t dim) {
  if (ts < 0 || hs < 0 || ts >= kMaxDim * 64 || hs >= kMaxDim * 64) return false;
  if (T > 1 && ts < dim) return false;
  if (heads > 1 && hs < dim) return false;
  if (T > 1 && heads > 1 && ts < (heads - 1) * hs + dim && hs < (T - 1) * ts + dim) return false;
  return true;
}

bool page_ok(int64_t page) { return page == 16 || page == 32 || page == 64 || page == 128; }

bool heads_ok(int64_t heads, int64_t kv_heads, int64_t dim) {
  return kv_heads >= 1 && heads >= kv_heads && heads % kv_heads == 0 && heads <= 65536 &&
         dim >= 16 && dim <= 256 && dim % 16 == 0;
}

// workgroups of a launch
bool grid_ok(double blocks) { return blocks <= (double)q4::kMaxGrid; }

q4_status make_cache(int8_t* k, int8_t* v, float* ks, float* vs, int64_t pages, int64_t page,
                     int64_t kv_heads, int64_t dim, const int32_t* table, int64_t table_ld,
                     int64_t max_pages, const int32_t* cu, const int32_t* lengths, int64_t batch,
                     q4::KvCache* c) {
  if (!k || !v || !ks || !vs || !table || !cu || !lengths) return Q4_ERR_INVALID_ARG;
  if (pages < 1 || pages >= kMaxDim || !page_ok(page) || max_pages < 1 || max_pages >= kMaxDim)
    return Q4_ERR_INVALID_ARG;
  if (batch > 1 && table_ld < max_pages) return Q4_ERR_INVALID_ARG;
  if (table_ld < 0 || table_ld >= kMaxDim) return Q4_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(ks, 4) || !aligned(vs, 4) ||
      !aligned(table, 4) || !aligned(cu, 4) || !aligned(lengths, 4))
    return Q4_ERR_INVALID_ARG;
  c->k = k;
  c->v = v;
  c->ks = ks;
  c->vs = vs;
  c->pages = pages;
  c->page = (int32_t)page;
  c->page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
  c->heads = (int32_t)kv_heads;
  c->dim = (int32_t)dim;
  c->table = table;
  c->table_ld = table_ld;
  c->max_pages = max_pages;
  c->cu_new = cu;
  c->lengths = lengths;
  return Q4_OK;
}

q4_status status_of(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_DEVICE; }

}  // namespace

extern "C" {

q4_status q4_kv_append(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                       int64_t v_hs, const void* q, int64_t q_ts, int64_t q_hs, void* q_out,
                       int64_t qo_ts, int64_t qo_hs, int32_t dtype, int64_t T, int64_t batch,
                       int64_t heads, int64_t kv_heads, int64_t head_dim, int8_t* k_cache,
                       int8_t* v_cache, float* k_scale, float* v_scale, int64_t pages,
                       int64_t page, const int32_t* page_table, int64_t table_ld,
                       int64_t max_pages, const int32_t* cu_new, const int32_t* lengths,
                       int64_t max_new, const float* inv_freq, int64_t rot, int32_t interleaved,
                       void* stream) {
  if (!dtype_ok(dtype) || !size_ok(T) || !size_ok(batch) || !size_ok(max_new))
    return Q4_ERR_INVALID_ARG;
  if (!heads_ok(q ? heads : kv_heads, kv_heads, head_dim)) return Q4_ERR_INVALID_ARG;
  if (rot < 0 || rot > head_dim || (rot & 1) || (rot > 0 && !inv_freq)) return Q4_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return Q4_ERR_INVALID_ARG;
  if (T == 0 || batch == 0) return Q4_OK;
  if (!k || !v || (q && !q_out)) return Q4_ERR_INVALID_ARG;
  const int64_t e = dtype_size(dtype);
  if (!strides_ok(k_ts, k_hs, T, kv_heads, head_dim) ||
      !strides_ok(v_ts, v_hs, T, kv_heads, head_dim))
    return Q4_ERR_INVALID_ARG;
  if (q && (!strides_ok(q_ts, q_hs, T, heads, head_dim) ||
            !strides_ok(qo_ts, qo_hs, T, heads, head_dim)))
    return Q4_ERR_INVALID_ARG;
  if (!aligned(k, e) || !aligned(v, e) || !aligned(q, e) || !aligned(q_out, e) ||
      !aligned(inv_freq, 4))
    return Q4_ERR_INVALID_ARG;
  q4::AppendParams p{};
  const q4_status st = make_cache(k_cache, v_cache, k_scale, v_scale, pages, page, kv_heads,
                                  head_dim, page_table, table_ld, max_pages, cu_new, lengths,
                                  batch, &p.c);
  if (st != Q4_OK) return st;
  if (max_new > T) max_new = T;
  if (max_new < 1) return Q4_ERR_INVALID_ARG;
  // a launch has workgroups for one page of each sequence at the least, and for all queries
  if (!grid_ok(2.0 * (double)batch * (double)kv_heads + (q ? (double)q4::append_turns(T) : 0.0)))
    return Q4_ERR_INVALID_ARG;

  const int64_t cache_n = pages * kv_heads * page * head_dim;
  const Range outs[] = {flat(k_cache, cache_n, 1), flat(v_cache, cache_n, 1),
                        flat(k_scale, pages * kv_heads, 4), flat(v_scale, pages * kv_heads, 4),
                        q ? span(q_out, T, qo_ts, heads, qo_hs, head_dim, e) : Range{0, 0}};
  const bool in_place = q && q_out == q && qo_ts == q_ts && qo_hs == q_hs;
  const Range ins[] = {span(k, T, k_ts, kv_heads, k_hs, head_dim, e),
                       span(v, T, v_ts, kv_heads, v_hs, head_dim, e),
                       q && !in_place ? span(q, T, q_ts, heads, q_hs, head_dim, e) : Range{0, 0},
                       span(page_table, batch, table_ld, 1, 0, max_pages, 4),
                       flat(cu_new, batch + 1, 4), flat(lengths, batch, 4),
                       rot > 0 ? flat(inv_freq, rot / 2, 4) : Range{0, 0}};
  constexpr int n_out = sizeof(outs) / sizeof(outs[0]), n_in = sizeof(ins) / sizeof(ins[0]);
  for (int i = 0; i < n_out; ++i) {
    // queries turned in place may share a fused projection's rows with k and
    // v, where the spans interleave without an element in common
    for (int j = 0; j < n_in; ++j) {
      if (!overlap(outs[i], ins[j])) continue;
      if (!(i == n_out - 1 && in_place && j < 2)) return Q4_ERR_ALIAS;
      const int64_t delta = ((intptr_t)(j == 0 ? k : v) - (intptr_t)q) / e;
      if (q4::rows_share(delta, T, head_dim, q_ts, q_hs, heads, j == 0 ? k_ts : v_ts,
                         j == 0 ? k_hs : v_hs, kv_heads))
        return Q4_ERR_ALIAS;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return Q4_ERR_ALIAS;
  }

  p.k = k;
  p.v = v;
  p.q = q;
  p.q_out = q_out;
  p.k_ts = k_ts;
  p.k_hs = k_hs;
  p.v_ts = v_ts;
  p.v_hs = v_hs;
  p.q_ts = q_ts;
  p.q_hs = q_hs;
  p.qo_ts = qo_ts;
  p.qo_hs = qo_hs;
  p.T = T;
  p.batch = (int32_t)batch;
  p.heads = (int32_t)heads;
  p.inv_freq = inv_freq;
  p.rot = (int32_t)rot;
  p.interleaved = interleaved;
  auto vec = [&](const void* x, int64_t ts, int64_t hs) {
    return aligned(x, 16) && ts * e % 16 == 0 && hs * e % 16 == 0 && rot % 8 == 0;
  };
  p.k_vec = vec(k, k_ts, k_hs);
  p.q_vec = q && vec(q, q_ts, q_hs) && vec(q_out, qo_ts, qo_hs);
  return status_of(q4::launch_kv_append(p, dtype, max_new, (hipStream_t)stream));
}

q4_status q4_kv_dequant(const int8_t* k_cache, const int8_t* v_cache, const float* k_scale,
                        const float* v_scale, int64_t pages, int64_t kv_heads, int64_t page,
                        int64_t head_dim, int32_t dtype, void* k, void* v, void* stream) {
  if (!dtype_ok(dtype) || !size_ok(pages) || !page_ok(page) ||
      !heads_ok(kv_heads, kv_heads, head_dim))
    return Q4_ERR_INVALID_ARG;
  if (pages == 0) return Q4_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !k || !v) return Q4_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return Q4_ERR_INVALID_ARG;
  const int64_t n = pages * kv_heads * page * head_dim, e = dtype_size(dtype);
  const Range ko = flat(k, n, e), vo = flat(v, n, e);
  const Range ins[] = {flat(k_cache, n, 1), flat(v_cache, n, 1),
                       flat(k_scale, pages * kv_heads, 4), flat(v_scale, pages * kv_heads, 4)};
  for (const Range& r : ins)
    if (overlap(ko, r) || overlap(vo, r)) return Q4_ERR_ALIAS;
  if (overlap(ko, vo)) return Q4_ERR_ALIAS;
  q4::KvCache c{};
  c.k = const_cast<int8_t*>(k_cache);
  c.v = const_cast<int8_t*>(v_cache);
  c.ks = const_cast<float*>(k_scale);
  c.vs = const_cast<float*>(v_scale);
  c.pages = pages;
  c.page = (int32_t)page;
  c.page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
  c.heads = (int32_t)kv_heads;
  c.dim = (int32_t)head_dim;
  return status_of(q4::launch_kv_dequant(c, dtype, k, v, (hipStream_t)stream));
}

static bool attention_sizes_ok(int32_t dtype, int64_t T, int64_t batch, int64_t heads,
                               int64_t kv_heads, int64_t head_dim, int64_t page, int64_t max_new,
                               int64_t max_len, int64_t window) {
  return dtype_ok(dtype) && size_ok(T) && size_ok(batch) && heads_ok(heads, kv_heads, head_dim) &&
         page_ok(page) && size_ok(max_new) && size_ok(max_len) && size_ok(window) &&
         (double)T * (double)heads < 2147483648.0;
}

// An upper bound of the new tokens beyond T is T.
static int64_t rows_bound(int64_t max_new, int64_t T) { return max_new < T ? max_new : T; }

size_t q4_attention_workspace_bytes(int32_t dtype, int64_t T, int64_t batch, int64_t heads,
                                    int64_t kv_heads, int64_t head_dim, int64_t page,
                                    int64_t max_new, int64_t max_len, int64_t window) {
  if (!attention_sizes_ok(dtype, T, batch, heads, kv_heads, head_dim, page, max_new, max_len,
                          window) ||
      T == 0 || batch == 0 || max_new == 0)
    return 0;
  return q4::plan_attention(dtype, T, batch, heads, kv_heads, head_dim, page,
                            rows_bound(max_new, T), max_len, window)
      .workspace;
}

q4_status q4_attention(const void* q, int64_t q_ts, int64_t q_hs, void* out, int64_t o_ts,
                       int64_t o_hs, int32_t dtype, int64_t T, int64_t batch, int64_t heads,
                       int64_t kv_heads, int64_t head_dim, const int8_t* k_cache,
                       const int8_t* v_cache, const float* k_scale, const float* v_scale,
                       int64_t pages, int64_t page, const int32_t* page_table, int64_t table_ld,
                       int64_t max_pages, const int32_t* cu_new, const int32_t* lengths,
                       int64_t max_new, int64_t max_len, float scale, int64_t window,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!attention_sizes_ok(dtype, T, batch, heads, kv_heads, head_dim, page, max_new, max_len,
                          window))
    return Q4_ERR_INVALID_ARG;
  if (T == 0 || batch == 0) return Q4_OK;
  if (!q || !out || max_new < 1) return Q4_ERR_INVALID_ARG;
  if (!(scale - scale == 0.0f)) return Q4_ERR_INVALID_ARG;  // finite
  const int64_t e = dtype_size(dtype);
  if (!strides_ok(q_ts, q_hs, T, heads, head_dim) || !strides_ok(o_ts, o_hs, T, heads, head_dim) ||
      !aligned(q, e) || !aligned(out, e))
    return Q4_ERR_INVALID_ARG;
  q4::AttnParams p{};
  const q4_status st = make_cache(
      const_cast<int8_t*>(k_cache), const_cast<int8_t*>(v_cache), const_cast<float*>(k_scale),
      const_cast<float*>(v_scale), pages, page, kv_heads, head_dim, page_table, table_ld,
      max_pages, cu_new, lengths, batch, &p.c);
  if (st != Q4_OK) return st;
  max_new = rows_bound(max_new, T);
  const q4::AttnPlan pl = q4::plan_attention(dtype, T, batch, heads, kv_heads, head_dim, page,
                                             max_new, max_len, window);
  if (!grid_ok((double)batch * (double)kv_heads * (double)pl.row_blocks * (double)pl.splits) ||
      (pl.splits > 1 && !grid_ok((double)batch * (double)kv_heads * (double)pl.max_rows)))
    return Q4_ERR_INVALID_ARG;

  const int64_t cache_n = pages * kv_heads * page * head_dim;
  const Range ins[] = {span(q, T, q_ts, heads, q_hs, head_dim, e),
                       flat(k_cache, cache_n, 1), flat(v_cache, cache_n, 1),
                       flat(k_scale, pages * kv_heads, 4), flat(v_scale, pages * kv_heads, 4),
                       span(page_table, batch, table_ld, 1, 0, max_pages, 4),
                       flat(cu_new, batch + 1, 4), flat(lengths, batch, 4)};
  const Range ro = span(out, T, o_ts, heads, o_hs, head_dim, e);
  Range ws{0, 0};
  if (pl.workspace > 0) {
    if (!workspace || workspace_bytes < pl.workspace || !aligned(workspace, 16))
      return Q4_ERR_WORKSPACE;
    ws = flat(workspace, (int64_t)pl.workspace, 1);
  }
  for (const Range& r : ins)
    if (overlap(ro, r) || overlap(ws, r)) return Q4_ERR_ALIAS;
  if (overlap(ro, ws)) return Q4_ERR_ALIAS;

  p.q = q;
  p.out = out;
  p.q_ts = q_ts;
  p.q_hs = q_hs;
  p.o_ts = o_ts;
  p.o_hs = o_hs;
  p.T = T;
  p.dtype = dtype;
  p.batch = (int32_t)batch;
  p.heads = (int32_t)heads;
  p.group = (int32_t)(heads / kv_heads);
  p.max_len = max_len;
  p.window = window;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q_vec = aligned(q, 16) && q_ts * e % 16 == 0 && q_hs * e % 16 == 0;
  p.max_rows = pl.max_rows;
  p.block_rows = pl.block_rows;
  p.row_blocks = pl.row_blocks;
  p.few = pl.few;
  p.splits = pl.splits;
  p.split_tiles = pl.split_tiles;
  p.part_o = (float*)workspace;
  p.part_ml = p.part_o + pl.parts * head_dim;
  return status_of(q4::launch_attention(p, (hipStream_t)stream));
}

// indices within a row, a step past its end included, are 32-bit
constexpr int64_t kMaxVocab = (int64_t)1 << 30;

static bool logprob_sizes_ok(int64_t M, int64_t vocab, int64_t top_k, int32_t dtype) {
  return dtype_ok(dtype) && size_ok(M) && vocab >= 1 && vocab <= kMaxVocab && top_k >= 0 &&
         top_k <= 32 && top_k <= vocab;
}

size_t q4_token_logprobs_workspace_bytes(int64_t M, int64_t vocab, int64_t top_k, int32_t dtype) {
  if (!logprob_sizes_ok(M, vocab, top_k, dtype) || M == 0) return 0;
  return q4::plan_logprobs(M, vocab, top_k, dtype).workspace;
}

q4_status q4_token_logprobs(const void* logits, int64_t ld, int32_t dtype, int64_t M,
                            int64_t vocab, const int64_t* targets, int64_t top_k, float* logprob,
                            float* entropy, float* lse, int64_t* top_ids, float* top_logprobs,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!logprob_sizes_ok(M, vocab, top_k, dtype) || ld < 0 || ld >= kMaxDim * 64)
    return Q4_ERR_INVALID_ARG;
  if (M == 0) return Q4_OK;
  const int64_t e = dtype_size(dtype);
  if (!logits || !entropy || !lse || (targets && !logprob) ||
      (top_k > 0 && (!top_ids || !top_logprobs)) || (M > 1 && ld < vocab))
    return Q4_ERR_INVALID_ARG;
  if (!aligned(logits, e) || !aligned(targets, 8) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(top_ids, 8) || !aligned(top_logprobs, 4))
    return Q4_ERR_INVALID_ARG;
  const q4::LogprobPlan pl = q4::plan_logprobs(M, vocab, top_k, dtype);
  Range outs[6] = {targets ? flat(logprob, M, 4) : Range{0, 0}, flat(entropy, M, 4),
                   flat(lse, M, 4), flat(top_ids, M * top_k, 8), flat(top_logprobs, M * top_k, 4),
                   Range{0, 0}};
  if (pl.workspace > 0) {
    if (!workspace || workspace_bytes < pl.workspace || !aligned(workspace, 16))
      return Q4_ERR_WORKSPACE;
    outs[5] = flat(workspace, (int64_t)pl.workspace, 1);
  }
  const Range ins[] = {span(logits, M, ld, 1, 0, vocab, e), flat(targets, M, 8)};
  for (int i = 0; i < 6; ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return Q4_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return Q4_ERR_ALIAS;
  }
  q4::LogprobParams p{};
  p.x = logits;
  p.ld = ld;
  p.M = M;
  p.V = vocab;
  p.targets = targets;
  p.top_k = (int32_t)top_k;
  p.logprob = logprob;
  p.entropy = entropy;
  p.lse = lse;
  p.top_lp = top_logprobs;
  p.top_ids = top_ids;
  p.splits = pl.splits;
  p.split_len = pl.split_len;
  if (pl.workspace) {
    p.part = (float*)workspace;
    p.part_val = p.part + M * pl.splits * 4;
    p.part_id = (int32_t*)(p.part_val + M * pl.splits * top_k);
  }
  return status_of(q4::launch_logprobs(p, dtype, (hipStream_t)stream));
}

q4_status q4_token_logprobs_backward(const void* logits, int64_t ld, int32_t dtype, int64_t M,
                                     int64_t vocab, const int64_t* targets, const float* lse,
                                     const float* entropy, const float* g_logprob,
                                     const float* g_entropy, void* dlogits, int64_t ldd,
                                     void* stream) {
  if (!logprob_sizes_ok(M, vocab, 0, dtype) || ld < 0 || ldd < 0 || ld >= kMaxDim * 64 ||
      ldd >= kMaxDim * 64)
    return Q4_ERR_INVALID_ARG;
  if (M == 0) return Q4_OK;
  const int64_t e = dtype_size(dtype);
  if (!logits || !lse || !entropy || !dlogits || (!g_logprob && !g_entropy) ||
      (g_logprob && !targets) || (M > 1 && (ld < vocab || ldd < vocab)))
    return Q4_ERR_INVALID_ARG;
  if (!aligned(logits, e) || !aligned(dlogits, e) || !aligned(targets, 8) || !aligned(lse, 4) ||
      !aligned(entropy, 4) || !aligned(g_logprob, 4) || !aligned(g_entropy, 4))
    return Q4_ERR_INVALID_ARG;
  const Range out = span(dlogits, M, ldd, 1, 0, vocab, e);
  const bool in_place = dlogits == logits && (ldd == ld || M == 1);
  const Range ins[] = {in_place ? Range{0, 0} : span(logits, M, ld, 1, 0, vocab, e),
                       flat(targets, M, 8), flat(lse, M, 4), flat(entropy, M, 4),
                       flat(g_logprob, M, 4), flat(g_entropy, M, 4)};
  for (const Range& r : ins)
    if (overlap(out, r)) return Q4_ERR_ALIAS;
  q4::LogprobBwdParams p{logits, ld, M, vocab, targets, lse, entropy, g_logprob, g_entropy,
                         dlogits, ldd};
  return status_of(q4::launch_logprobs_backward(p, dtype, (hipStream_t)stream));
}

}  // extern "C"
