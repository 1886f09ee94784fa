// q4_serve.h -- host-side interface between the C ABI of the decode-side
// operators (q4_serve_abi.hip) and their kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "q4serve.h"

namespace q4 {

// Workgroups that one launch may have: a grid holds fewer than 2^32 threads,
// and one of more is taken without an error and run in part (an append of 4200
// sequences with the default max_new left most of them out).  In workgroups of
// 256 threads; launches of more threads each have few of them.
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;

struct KvCache {
  int8_t* k;
  int8_t* v;
  float* ks;
  float* vs;
  int64_t pages;
  int32_t page;       // 16, 32, 64 or 128
  int32_t page_log2;
  int32_t heads;      // kv heads
  int32_t dim;        // multiple of 16, <= 256
  const int32_t* table;
  int64_t table_ld, max_pages;
  const int32_t* cu_new;
  const int32_t* lengths;
};

struct AppendParams {
  const void *k, *v, *q;
  void* q_out;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, qo_ts, qo_hs;
  KvCache c;
  int64_t T, max_new;
  int32_t batch, heads;
  const float* inv_freq;
  int32_t rot, interleaved;
  int32_t first, touched;  // pages of one sequence that the launch covers
  int32_t cache_blocks;  // workgroups that store; the rest turn queries,
  int32_t turn;          // so many tokens each
  int32_t k_vec, q_vec;  // rows of k, and of q and q_out, allow vector accesses
};

// Tokens of a workgroup that turns queries (one while that leaves CUs without
// work), and such workgroups.
inline int32_t append_turn(int64_t T) { return T >= 2048 ? 4 : 1; }
inline int64_t append_turns(int64_t T) { return (T + append_turn(T) - 1) / append_turn(T); }
hipError_t launch_kv_append(const AppendParams& p, int32_t dtype, int64_t max_new, hipStream_t s);
hipError_t launch_kv_dequant(const KvCache& c, int32_t dtype, void* k, void* v, hipStream_t s);

struct AttnParams {
  const void* q;
  void* out;
  int64_t q_ts, q_hs, o_ts, o_hs;
  KvCache c;
  int64_t T;
  int32_t dtype, batch, heads, group;  // group = heads / kv heads
  int64_t max_len, window;
  float scale_log2;             // scale * log2(e)
  int32_t q_vec;                // 16-byte aligned query rows
  int32_t max_rows;             // per sequence and kv head
  int32_t block_rows;           // query rows of a workgroup: 16, or 64 or 128 (attention_wide_kernel)
  int32_t row_blocks;           // per sequence and kv head
  int32_t splits;               // workgroups along the keys (grid)
  int32_t few;                  // few workgroups: eight waves in each
  int32_t split_tiles;          // tiles of 64 keys each of them takes
  float* part_o;                // [splits][T * heads][dim]
  float* part_ml;               // [splits][T * heads][2]: maximum (log2), sum
};

struct AttnPlan {
  int32_t max_rows, block_rows, row_blocks, splits, split_tiles, few;
  size_t parts;  // rows of partial outputs in the workspace
  size_t workspace;
};
AttnPlan plan_attention(int32_t dtype, int64_t T, int64_t batch, int64_t heads, int64_t kv_heads,
                        int64_t dim, int64_t page, int64_t max_new, int64_t max_len,
                        int64_t window);
hipError_t launch_attention(const AttnParams& p, hipStream_t s);
template <int ND>
hipError_t launch_attention_digits(const AttnParams& p, hipStream_t s);
// (instantiated for 3 and 4 digits in q4_attention_d3.hip / q4_attention_d4.hip)

struct LogprobParams {
  const void* x;
  int64_t ld, M, V;
  const int64_t* targets;
  int32_t top_k;
  float *logprob, *entropy, *lse, *top_lp;
  int64_t* top_ids;
  int32_t splits;
  int64_t split_len;
  float* part;       // [M][splits][kPartStats]
  float* part_val;   // [M][splits][top_k]
  int32_t* part_id;  // [M][splits][top_k]
};
struct LogprobPlan {
  int32_t splits;
  int64_t split_len;
  size_t workspace;
};
LogprobPlan plan_logprobs(int64_t M, int64_t V, int64_t top_k, int32_t dtype);
hipError_t launch_logprobs(const LogprobParams& p, int32_t dtype, hipStream_t s);

struct LogprobBwdParams {
  const void* x;
  int64_t ld, M, V;
  const int64_t* targets;
  const float *lse, *entropy, *g_lp, *g_ent;
  void* dx;
  int64_t ldd;
};
hipError_t launch_logprobs_backward(const LogprobBwdParams& p, int32_t dtype, hipStream_t s);

}  // namespace q4
