// q4_logprobs.hip -- token log probabilities, entropy and top alternatives of
// a row of logits in one pass, and their gradient.
//
// With m the running maximum, y = x - m:  S = sum e^y,  W = sum e^y y.  When m
// grows by d, S and W become  S e^-d  and  (W - d S) e^-d.  Then
//   lse = m + log S,  logprob = (x_t - m) - log S,  entropy = log S - W / S
// (all of W's terms are <= 0, so nothing cancels).  Each thread keeps its own
// (m, S, W), joined by the same rule.
//
// The top_k largest are kept per wave as a sorted list, entry i in lane i.  A
// value enters only if it beats the last entry, which few do: for values in
// random order the expected number is top_k (1 + log(n / top_k)).
//
// Bound by HBM reads for many rows; for a few rows, whose parts go to several
// workgroups and are joined by a second launch, by latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_serve.h"
#include "q4_serve_device.h"

namespace q4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxTop = 32;
constexpr int32_t kNone = 0x7fffffff;  // index of an empty list entry
constexpr int kPartStats = 4;          // m, S, W of a part (padded)

struct Stats {
  float m, s, w;
};

__device__ __forceinline__ Stats stats_empty() { return Stats{-__builtin_inff(), 0.0f, 0.0f}; }

// Joins two; an empty side (m = -inf) leaves the other as it is.
__device__ __forceinline__ Stats stats_join(const Stats& a, const Stats& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -__builtin_inff()) return Stats{m, a.s + b.s, a.w + b.w};
  const float da = a.m - m, db = b.m - m;  // <= 0
  const float fa = exp2_fast(da * kLog2e), fb = exp2_fast(db * kLog2e);
  // a side too far below to count may overflow in d S (a NaN shows in its S)
  const float wa = fa > 0.0f ? fa * (a.w + da * a.s) : 0.0f;
  const float wb = fb > 0.0f ? fb * (b.w + db * b.s) : 0.0f;
  const float sa = a.s == 0.0f ? 0.0f : fa * a.s, sb = b.s == 0.0f ? 0.0f : fb * b.s;
  return Stats{m, sa + sb, wa + wb};
}

__device__ __forceinline__ Stats stats_shfl(const Stats& a, int mask) {
  return Stats{__shfl_xor(a.m, mask, 64), __shfl_xor(a.s, mask, 64), __shfl_xor(a.w, mask, 64)};
}

// (value, index) before (v, i) in the order of alternatives
__device__ __forceinline__ bool before(float value, int32_t index, float v, int32_t i) {
  return value > v || (value == v && index < i);
}

// A wave's sorted list: entry i in lane i (lanes past top_k hold nothing of
// use), the last entry's value and index known to every lane.
struct TopList {
  float value, last_value;
  int32_t index, last_index;
};

__device__ __forceinline__ TopList top_empty() {
  return TopList{-__builtin_inff(), -__builtin_inff(), kNone, kNone};
}

// Every lane passes the same (v, i).
__device__ __forceinline__ void top_insert(TopList& t, float v, int32_t i, int k, int lane) {
  const uint64_t ahead = __ballot(before(t.value, t.index, v, i));
  const int at = __popcll(ahead);
  if (at >= k) return;
  const float pv = __shfl_up(t.value, 1, 64);
  const int32_t pi = __shfl_up(t.index, 1, 64);
  if (lane > at) {
    t.value = pv;
    t.index = pi;
  } else if (lane == at) {
    t.value = v;
    t.index = i;
  }
  t.last_value = __shfl(t.value, k - 1, 64);
  t.last_index = __shfl(t.index, k - 1, 64);
}

// The lanes' values x (index i), each entering if it belongs.
__device__ __forceinline__ void top_offer(TopList& t, float x, int32_t i, bool on, int k, int lane) {
  uint64_t todo = __ballot(on && before(x, i, t.last_value, t.last_index));
  while (todo) {
    const int from = __builtin_ctzll(todo);
    todo &= todo - 1;
    top_insert(t, __shfl(x, from, 64), __shfl(i, from, 64), k, lane);
  }
}

struct Result {
  float lse, entropy;
};

__device__ __forceinline__ Result finish(const Stats& a) {
  if (a.s == 0.0f) return Result{-__builtin_inff(), 0.0f};  // nothing but -inf
  const float log_s = log2_fast(a.s) * kLn2;
  return Result{a.m + log_s, log_s - a.w / a.s};
}

// Log probability of x given the statistics: x - m first, as both may be large.
__device__ __forceinline__ float logprob_of(float x, const Stats& a) {
  if (a.s == 0.0f) return -__builtin_inff();
  return (x - a.m) - log2_fast(a.s) * kLn2;
}

template <typename T>
__device__ __forceinline__ void write_row(const LogprobParams& p, int64_t row, const Stats& a) {
  const Result r = finish(a);
  p.lse[row] = r.lse;
  p.entropy[row] = r.entropy;
  if (p.targets) {
    const int64_t t = p.targets[row];
    float lp = 0.0f;
    if (t >= p.V) lp = bits_f32(0x7fc00000u);
    else if (t >= 0) lp = logprob_of(to_f32(((const T*)p.x)[row * p.ld + t]), a);
    p.logprob[row] = lp;
  }
}

// Ranks the n entries of (vals, ids) in LDS and gives the first k to `out`
// (called with the entry's rank, value and index).  Indices differ, but for
// empty entries, which come last in any order.
template <typename F>
__device__ __forceinline__ void rank_entries(const float* vals, const int32_t* ids, int n, int k,
                                             F out) {
  for (int e = threadIdx.x; e < n; e += kThreads) {
    const float v = vals[e];
    const int32_t i = ids[e];
    int rank = 0;
    for (int o = 0; o < n; ++o) {
      const bool b = before(vals[o], ids[o], v, i) || (ids[o] == i && vals[o] == v && o < e);
      rank += b ? 1 : 0;
    }
    if (rank < k) out(rank, v, i);
  }
}

__device__ __forceinline__ void write_top(const LogprobParams& p, int64_t row, int rank, float v,
                                          int32_t i, const Stats& a) {
  const int64_t at = row * p.top_k + rank;
  p.top_ids[at] = i == kNone ? -1 : i;
  p.top_lp[at] = i == kNone ? bits_f32(0x7fc00000u) : logprob_of(v, a);
}

// One part (or all) of a row per workgroup.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobParams p) {
  constexpr int N = 16 / sizeof(T);
  __shared__ Stats wave_stats[kWaves];
  __shared__ float top_vals[kWaves * kMaxTop];
  __shared__ int32_t top_ids[kWaves * kMaxTop];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x / p.splits;
  const int split = (int)(blockIdx.x - row * p.splits);
  const int64_t from = split * p.split_len;
  const int64_t to = from + p.split_len < p.V ? from + p.split_len : p.V;
  const T* x = (const T*)p.x + row * p.ld;
  const int k = p.top_k;

  Stats st = stats_empty();
  TopList top = top_empty();
  auto take = [&](const float (&v)[N], int n, int64_t at) {
    float vm = v[0];
#pragma unroll
    for (int e = 1; e < N; ++e) vm = fmaxf(vm, v[e]);
    const float m = fmaxf(st.m, vm);
    const float ref = m > -__builtin_inff() ? m : 0.0f;
    const float d = st.m - ref;
    const float f = exp2_fast(d * kLog2e);
    // an empty sum stays 0 (d is -inf), one too far below may overflow in d S
    st.w = f > 0.0f ? f * (st.w + d * st.s) : 0.0f;
    st.s = f * st.s;
    st.m = m;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float y = v[e] - ref;
      const float ex = exp2_fast(y * kLog2e);
      st.s += ex;
      st.w += ex == 0.0f ? 0.0f : ex * y;  // y may be -inf
    }
    if (k > 0 && __any(vm >= top.last_value)) {
#pragma unroll
      for (int e = 0; e < N; ++e) top_offer(top, v[e], (int32_t)(at + e), e < n, k, lane);
    }
  };
  // elements up to the first 16-byte boundary, whole vectors, the rest
  const int64_t mis = ((uintptr_t)(x + from) & 15) / sizeof(T);
  int64_t head = mis ? N - mis : 0;
  if (head > to - from) head = to - from;
  const int64_t vecs = (to - from - head) / N;
  const int64_t tail = from + head + vecs * N;
  {
    float v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = -__builtin_inff();
    // lane l of wave 0 takes element l of the head, then of the tail
    if (wave == 0) {
      if (lane < head) v[0] = to_f32(x[from + lane]);
      take(v, lane < head ? 1 : 0, from + lane);
      v[0] = tail + lane < to ? to_f32(x[tail + lane]) : -__builtin_inff();
      take(v, tail + lane < to ? 1 : 0, tail + lane);
    }
  }
  const T* body = x + from + head;
  // whole waves step together: a lane past the end offers nothing
  for (int64_t i0 = (int64_t)wave * 64; i0 < vecs; i0 += kThreads) {
    const int64_t i = i0 + lane;
    float v[N];
    if (i < vecs) {
      const u32x4v w = *(const u32x4v*)(body + i * N);
      const T* t = (const T*)&w;
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = to_f32(t[e]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = -__builtin_inff();
    }
    take(v, i < vecs ? N : 0, from + head + i * N);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) st = stats_join(st, stats_shfl(st, m));
  if (lane == 0) wave_stats[wave] = st;
  if (lane < k) {
    top_vals[wave * k + lane] = top.value;
    top_ids[wave * k + lane] = top.index;
  }
  __syncthreads();
  st = wave_stats[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) st = stats_join(st, wave_stats[w]);
  if (p.splits == 1) {
    if (threadIdx.x == 0) write_row<T>(p, row, st);
    rank_entries(top_vals, top_ids, kWaves * k, k,
                 [&](int rank, float v, int32_t i) { write_top(p, row, rank, v, i, st); });
  } else {
    const int64_t part = blockIdx.x;
    if (threadIdx.x == 0) {
      p.part[part * kPartStats] = st.m;
      p.part[part * kPartStats + 1] = st.s;
      p.part[part * kPartStats + 2] = st.w;
    }
    rank_entries(top_vals, top_ids, kWaves * k, k, [&](int rank, float v, int32_t i) {
      p.part_val[part * k + rank] = v;
      p.part_id[part * k + rank] = i;
    });
  }
}

// Joins the parts of a row.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_join_kernel(LogprobParams p) {
  extern __shared__ float vals[];  // [splits * k], then the indices
  const int64_t row = blockIdx.x;
  const int k = p.top_k, n = p.splits * k;
  int32_t* ids = (int32_t*)(vals + n);
  for (int e = threadIdx.x; e < n; e += kThreads) {
    vals[e] = p.part_val[row * n + e];
    ids[e] = p.part_id[row * n + e];
  }
  Stats st = stats_empty();
  for (int s = 0; s < p.splits; ++s) {
    const float* q = p.part + (row * p.splits + s) * kPartStats;
    st = stats_join(st, Stats{q[0], q[1], q[2]});
  }
  __syncthreads();
  if (threadIdx.x == 0) write_row<T>(p, row, st);
  rank_entries(vals, ids, n, k,
               [&](int rank, float v, int32_t i) { write_top(p, row, rank, v, i, st); });
}

// dx_v = g (1[v = t] - p_v) - h p_v (log p_v + H), 16 bytes a thread.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_backward_kernel(LogprobBwdParams p,
                                                                     int64_t blocks_per_row) {
  constexpr int N = 16 / sizeof(T);
  const int64_t row = blockIdx.x / blocks_per_row;
  const int64_t blk = blockIdx.x - row * blocks_per_row;
  const T* x = (const T*)p.x + row * p.ld;
  T* dx = (T*)p.dx + row * p.ldd;
  const float lse = p.lse[row], ent = p.entropy[row];
  const int64_t t = p.targets ? p.targets[row] : -1;
  float g = p.g_lp && t >= 0 ? p.g_lp[row] : 0.0f;
  const float h = p.g_ent ? p.g_ent[row] : 0.0f;
  if (p.g_lp && t >= p.V) g = bits_f32(0x7fc00000u);
  const bool empty = lse == -__builtin_inff();
  auto grad = [&](float v, int64_t at) {
    const float lp = v - lse;
    const float pr = exp2_fast(lp * kLog2e);
    float r = -pr * (g + h * (lp + ent));
    if (pr == 0.0f) r = 0.0f * (g + h);  // lp may be -inf; NaN gradients still show
    if (at == t) r += g;
    return empty && g == g ? 0.0f : r;
  };
  const int64_t mis = ((uintptr_t)x & 15) / sizeof(T);
  int64_t head = mis ? N - mis : 0;
  if (head > p.V) head = p.V;
  const int64_t vecs = (p.V - head) / N;
  const int64_t tail = head + vecs * N;
  if (blk == 0) {
    const int64_t i = threadIdx.x;
    if (i < head) dx[i] = from_f32<T>(grad(to_f32(x[i]), i));
    if (tail + i < p.V) dx[tail + i] = from_f32<T>(grad(to_f32(x[tail + i]), tail + i));
  }
  for (int64_t i = blk * kThreads + threadIdx.x; i < vecs; i += blocks_per_row * kThreads) {
    const int64_t at = head + i * N;
    const u32x4v w = *(const u32x4v*)(x + at);
    const T* v = (const T*)&w;
    T o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = from_f32<T>(grad(to_f32(v[e]), at + e));
    __builtin_memcpy(dx + at, o, 16);  // dx need not share x's alignment
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// Rows go to several workgroups while rows alone leave the chip without work.
LogprobPlan plan_logprobs(int64_t M, int64_t V, int64_t top_k, int32_t dtype) {
  (void)dtype;
  constexpr int64_t kTargetBlocks = 1024, kMinLen = 4096;
  LogprobPlan pl;
  int64_t splits = ceil_div(kTargetBlocks, M > 0 ? M : 1);
  if (splits > ceil_div(V, kMinLen)) splits = ceil_div(V, kMinLen);
  if (M >= 256) splits = 1;
  if (splits < 1) splits = 1;
  if (splits > 64) splits = 64;
  pl.split_len = ceil_div(ceil_div(V, splits), 64) * 64;
  pl.splits = (int32_t)ceil_div(V, pl.split_len);
  const size_t n = pl.splits > 1 ? (size_t)M * pl.splits : 0;
  pl.workspace = n * (kPartStats * sizeof(float) + (size_t)top_k * (sizeof(float) + sizeof(int32_t)));
  return pl;
}

hipError_t launch_logprobs(const LogprobParams& p, int32_t dtype, hipStream_t s) {
  const dim3 grid((unsigned)(p.M * p.splits));
  const size_t lds = (size_t)p.splits * p.top_k * (sizeof(float) + sizeof(int32_t));
#define Q4_LOGPROBS(T)                                                                       \
  do {                                                                                       \
    hipLaunchKernelGGL((logprobs_kernel<T>), grid, dim3(kThreads), 0, s, p);                 \
    if (p.splits > 1)                                                                        \
      hipLaunchKernelGGL((logprobs_join_kernel<T>), dim3((unsigned)p.M), dim3(kThreads), lds, \
                         s, p);                                                              \
  } while (0)
  if (dtype == Q4_DTYPE_F32) Q4_LOGPROBS(float);
  else if (dtype == Q4_DTYPE_F16) Q4_LOGPROBS(_Float16);
  else Q4_LOGPROBS(bf16);
#undef Q4_LOGPROBS
  return hipGetLastError();
}

hipError_t launch_logprobs_backward(const LogprobBwdParams& p, int32_t dtype, hipStream_t s) {
  const int64_t bytes = dtype == Q4_DTYPE_F32 ? 4 : 2;
  const int64_t per_row = ceil_div(ceil_div(p.V * bytes, 16), kThreads * 4);
  const dim3 grid((unsigned)(p.M * per_row));
  if (dtype == Q4_DTYPE_F32)
    hipLaunchKernelGGL(logprobs_backward_kernel<float>, grid, dim3(kThreads), 0, s, p, per_row);
  else if (dtype == Q4_DTYPE_F16)
    hipLaunchKernelGGL(logprobs_backward_kernel<_Float16>, grid, dim3(kThreads), 0, s, p, per_row);
  else
    hipLaunchKernelGGL(logprobs_backward_kernel<bf16>, grid, dim3(kThreads), 0, s, p, per_row);
  return hipGetLastError();
}

}  // namespace q4
