// q4_logprobs.hip -- token log probabilities, entropy and top alternatives of
// a row of logits in one pass, and their gradient.
//
// With m the running maximum, y = (x - m) log2 e:  S = sum 2^y,  W = sum 2^y y.
// When m grows, so that every y falls by d, they become 2^-d S and
// 2^-d (W - d S).  Then, with ln 2 for the base,
//   lse = m + ln S,  logprob = (x_t - m) - ln S,  entropy = ln S - ln 2 W / S
// (all of W's terms are <= 0, so nothing cancels).  Each thread keeps its own
// (m, S, W), joined by the same rule.
//
// The top_k largest: the lanes' largest so far, in 64 groups, give a bar, their
// top_k-th largest, that the top_k-th of the row cannot be below.  Every wave
// collects in LDS what reaches the bar, in any order; it is raised after 1, 2,
// 4, ... steps, between which about 1.2 top_k more values pass in all for
// values in random order.  What reaches the last bar is ranked by counting.  A
// full buffer is cut to its top_k best.  (A sorted list in the lanes, an entry
// inserted at a time through ballots, took 75 us for 512 rows of 128257 and
// top_k 5, where this took 61; now 55, and none at all 49.)
//
// Bound by HBM reads for many rows; for a few rows, whose parts go to several
// workgroups and are joined by a second launch, by latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "q4_serve.h"
#include "q4_serve_device.h"

namespace q4 {

namespace {

constexpr int kMaxTop = 32;
constexpr int kChunk = 16;             // elements of a thread's step
constexpr int32_t kNone = 0x7fffffff;  // index of an empty list entry
constexpr int kPartStats = 4;          // m, s, W, c of a part
constexpr int kMaxParts = 64;          // of a row: a lane each in the join

// S is s + c, c what the additions to s have rounded off: a row whose largest
// logit holds nearly all has S = 1 + r with a small r that its entropy and log
// probabilities hang on.
struct Stats {
  float m, s, w, c;
};

// Adds to S.
__device__ __forceinline__ void add_sum(float& s, float& c, float x) {
  const float t = s + x, part = t - s;
  c += (s - (t - part)) + (x - part);
  s = t;
}

// Joins two; an empty side (m = -inf) leaves the other as it is.
__device__ __forceinline__ Stats stats_join(const Stats& a, const Stats& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -__builtin_inff()) return Stats{m, a.s + b.s, a.w + b.w, 0.0f};
  const float da = (a.m - m) * kLog2e, db = (b.m - m) * kLog2e;  // <= 0
  const float fa = exp2_fast(da), fb = exp2_fast(db);
  // a side too far below to count may overflow in d S (a NaN shows in its S)
  const float wa = fa > 0.0f ? fa * (a.w + da * a.s) : 0.0f;
  const float wb = fb > 0.0f ? fb * (b.w + db * b.s) : 0.0f;
  const float sa = a.s == 0.0f ? 0.0f : fa * a.s, sb = b.s == 0.0f ? 0.0f : fb * b.s;
  Stats r{m, sa, wa + wb, fa * a.c + fb * b.c};
  add_sum(r.s, r.c, sb);
  return r;
}

__device__ __forceinline__ Stats stats_wave(Stats a) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1)
    a = stats_join(a, Stats{__shfl_xor(a.m, m, 64), __shfl_xor(a.s, m, 64), __shfl_xor(a.w, m, 64),
                            __shfl_xor(a.c, m, 64)});
  return a;
}

// (value, index) before (v, i) in the order of alternatives
__device__ __forceinline__ bool before(float value, int32_t index, float v, int32_t i) {
  return (value > v) | ((value == v) & (index < i));
}

// Bits of a number as an integer that orders like it (NaN below all, 0).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = f32_bits(v);
  return v != v ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return bits_f32((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// Other lanes' LDS accesses of the same wave are done and seen.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The key of group i's largest value, different for every group: the low bits
// give way to its number.
__device__ __forceinline__ uint32_t group_key(float v, int i) {
  return (order_key(v) & ~63u) | (uint32_t)i;
}

// A number that the k-th largest of 64 groups' values is not below, and not
// more than 2^-17 of it less (-inf if fewer are numbers): every lane counts
// the groups above its own.  Groups are different elements, and a group's key
// only grows, so the result stands whatever mix of old and new keys is read.
__device__ __forceinline__ float kth_of_groups(const uint32_t* keys, int k, int lane) {
  const uint32_t key = keys[lane];
  int above = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const u32x4v q = ((const u32x4v*)keys)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) above += q[e] > key ? 1 : 0;
  }
  // a key that grows meanwhile can leave no lane at k - 1: no bar this time
  const uint64_t at = __ballot(above == k - 1);
  if (at == 0) return -__builtin_inff();
  const uint32_t kth = (uint32_t)__builtin_amdgcn_readlane((int)key, __builtin_ctzll(at)) & ~63u;
  return kth < 0x00800000u ? -__builtin_inff() : key_value(kth);  // -inf's key and below
}

// The largest of each W neighbouring lanes (W = 4 or 8), in every one of them.
template <int W>
__device__ __forceinline__ float group_max(float v) {
  auto dpp = [&](auto ctrl) {
    return bits_f32((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f32_bits(v), decltype(ctrl)::value,
                                                          0xf, 0xf, true));
  };
  v = fmaxf(v, dpp(std::integral_constant<int, 0xb1>{}));   // quad_perm 1 0 3 2
  v = fmaxf(v, dpp(std::integral_constant<int, 0x4e>{}));   // quad_perm 2 3 0 1
  if (W == 8) v = fmaxf(v, dpp(std::integral_constant<int, 0x141>{}));  // row_half_mirror
  return v;
}

constexpr int kBuffer = 256;  // of a wave's candidates, a multiple of 64
constexpr int kFinal = 64;    // of them at the end

// A wave's candidates: values and indices in LDS, how many, and what the next
// ones have to be before.
struct Best {
  float* val;
  int32_t* id;
  int count;
  float bar;
  int32_t bar_id;
};

// Leaves the k best of more than k candidates, and raises the bar to the last.
__device__ __forceinline__ void best_cut(Best& t, int k, int lane) {
  constexpr int J = kBuffer / 64;
  float v[J];
  uint32_t key[J];
  int32_t id[J];
  wave_lds_fence();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = 64 * j + lane;
    const bool on = e < t.count;
    v[j] = on ? t.val[e] : 0.0f;
    id[j] = on ? t.id[e] : kNone;
    key[j] = on ? order_key(v[j] + 0.0f) : 0u;  // -0 and 0 are equal: both 0
  }
  wave_lds_fence();
  uint32_t at = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t next = at | (1u << bit);
    int c = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) c += __popcll(__ballot(key[j] >= next));
    if (c >= k) at = next;
  }
  int above = 0, ties = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    above += __popcll(__ballot(key[j] > at));
    ties += __popcll(__ballot(key[j] == at));
  }
  int32_t last = kNone;  // of equal ones, the lowest indices stay
  if (above + ties > k) {
    last = 0;
#pragma unroll 1
    for (int bit = 30; bit >= 0; --bit) {
      const int32_t next = last | (1 << bit);
      int c = above;
#pragma unroll
      for (int j = 0; j < J; ++j) c += __popcll(__ballot(key[j] == at && id[j] < next));
      if (c < k) last = next;
    }
  }
  t.count = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const bool keep = key[j] > at || (key[j] == at && id[j] <= last);
    const uint64_t mask = __ballot(keep);
    if (keep) {
      const int to = t.count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                         __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
      t.val[to] = v[j];
      t.id[to] = id[j];
    }
    t.count += __popcll(mask);
  }
  wave_lds_fence();
  t.bar = key_value(at);
  t.bar_id = last;
}

// The lanes' values x (number i), each kept if it is before the bar.
__device__ __forceinline__ void best_offer(Best& t, float x, int32_t i, bool on, int k, int lane) {
  const bool keep = on && before(x, i, t.bar, t.bar_id);
  const uint64_t mask = __ballot(keep);
  if (!mask) return;
  if (t.count > kBuffer - 64) best_cut(t, k, lane);
  if (keep) {
    const int to = t.count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                       __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
    t.val[to] = x;
    t.id[to] = i;
  }
  t.count += __popcll(mask);
}

// Sum over the lanes up to and with this one.
__device__ __forceinline__ int lane_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);  // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast 15, 31
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return x;
}

struct Result {
  float lse, entropy;
};

// ln (s + c), to a few roundings of itself also where S is close to 1.
__device__ __forceinline__ float log_sum(const Stats& a) {
  return __builtin_fmaf(a.c, __builtin_amdgcn_rcpf(a.s), log2_fast(a.s) * kLn2);
}

__device__ __forceinline__ Result finish(const Stats& a) {
  if (a.s == 0.0f) return Result{-__builtin_inff(), 0.0f};  // nothing but -inf
  const float log_s = log_sum(a);
  return Result{a.m + log_s, log_s - kLn2 * (a.w / a.s)};
}

// Log probability of x given the statistics: x - m first, as both may be large.
__device__ __forceinline__ float logprob_of(float x, const Stats& a) {
  if (a.s == 0.0f) return -__builtin_inff();
  return (x - a.m) - log_sum(a);
}

// The target's logit, loaded before the sums are known (NaN where the target
// is past the row), and whether there is a target.
struct Target {
  float x;
  bool is;
};

template <typename T>
__device__ __forceinline__ Target target_of(const LogprobParams& p, int64_t row) {
  const int64_t t = p.targets ? p.targets[row] : -1;
  Target r{bits_f32(0x7fc00000u), t >= 0};
  if (t >= 0 && t < p.V) r.x = to_f32(((const T*)p.x)[row * p.ld + t]);
  return r;
}

__device__ __forceinline__ void write_row(const LogprobParams& p, int64_t row, const Stats& a,
                                          const Target& t) {
  const Result r = finish(a);
  p.lse[row] = r.lse;
  p.entropy[row] = r.entropy;
  if (p.targets) p.logprob[row] = !t.is ? 0.0f : t.x != t.x ? t.x : logprob_of(t.x, a);
}

// A candidate as one integer: larger for one that is before another.  -0 and 0
// are equal, and both become 0.
__device__ __forceinline__ uint64_t entry_of(float v, int32_t i) {
  return (uint64_t)order_key(v + 0.0f) << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float entry_value(uint64_t e) { return key_value((uint32_t)(e >> 32)); }
__device__ __forceinline__ int32_t entry_index(uint64_t e) { return (int32_t)~(uint32_t)e; }

// Ranks the n entries in LDS, all different and 16-byte aligned with a spare
// one at the end, and gives the first k to `out` (called with the rank, value
// and index); the ranks past n are empty.
template <typename F>
__device__ __forceinline__ void rank_entries(uint64_t* entries, int n, int k, F out) {
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  if (threadIdx.x == 0) entries[n] = 0;
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    const uint64_t mine = entries[e];
    int rank = 0;
#pragma unroll 8
    for (int o = 0; o < n; o += 2) {
      const u64x2 q = *(const u64x2*)(entries + o);
      rank += (q[0] > mine ? 1 : 0) + (q[1] > mine ? 1 : 0);
    }
    if (rank < k) out(rank, entry_value(mine), entry_index(mine));
  }
  for (int e = n + threadIdx.x; e < k; e += blockDim.x) out(e, -__builtin_inff(), kNone);
}

__device__ __forceinline__ void write_top(const LogprobParams& p, int64_t row, int rank, float v,
                                          int32_t i, const Stats& a) {
  const int64_t at = row * p.top_k + rank;
  p.top_ids[at] = i == kNone ? -1 : i;
  p.top_lp[at] = i == kNone ? bits_f32(0x7fc00000u) : logprob_of(v, a);
}

// One part (or all) of a row per workgroup of W waves.  The next step's
// elements load while this one's are summed.
template <typename T, int W>
__global__ __launch_bounds__(64 * W) void logprobs_kernel(LogprobParams p) {
  constexpr int N = 16 / sizeof(T), C = kChunk / N, kThreads = 64 * W;
  __shared__ Stats wave_stats[W];
  __shared__ float best_val[W][kBuffer];
  __shared__ int32_t best_id[W][kBuffer];
  __shared__ __attribute__((aligned(16))) uint32_t keys[64];
  __shared__ __attribute__((aligned(16))) uint64_t entries[W * kFinal + 2];
  __shared__ int32_t top_count;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t row32 = blockIdx.x / (uint32_t)p.splits;
  const int split = (int)(blockIdx.x - row32 * (uint32_t)p.splits);
  const int64_t row = row32;
  const int64_t from = split * p.split_len;
  const int64_t to = from + p.split_len < p.V ? from + p.split_len : p.V;
  const T* x = (const T*)p.x + row * p.ld;
  const int k = p.top_k;
  const float inf = __builtin_inff();

  Target target{0.0f, false};
  if (p.splits == 1 && tid == 0) target = target_of<T>(p, row);
  Stats st{-inf, 0.0f, 0.0f, 0.0f};
  Best best{best_val[wave], best_id[wave], 0, -inf, kNone};
  int step = 0;
  if (tid == 0) top_count = 0;
  // element e of v is number at + (e / N) * stride + e % N of the row, if that
  // is below limit; the first `count` are offered as alternatives
  auto take = [&](const float (&v)[kChunk], int32_t at, int32_t stride, int32_t limit, int count) {
    float vm = v[0];
#pragma unroll
    for (int e = 1; e < kChunk; ++e) vm = fmaxf(vm, v[e]);
    const float m = fmaxf(st.m, vm);
    const float ref = m > -inf ? m : 0.0f;
    const float d = (st.m - ref) * kLog2e;
    const float f = exp2_fast(d);
    // an empty sum stays 0 (d is -inf), one too far below may overflow in d S
    st.w = f > 0.0f ? f * (st.w + d * st.s) : 0.0f;
    st.s = f * st.s;
    st.c = f * st.c;
    st.m = m;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, w = 0.0f;  // four, for fewer roundings
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      const float y = (v[e] - ref) * kLog2e;
      const float ex = exp2_fast(y);
      s[e % 4] += ex;
      w = __builtin_fmaf(ex, fmaxf(y, -1e5f), w);  // y may be -inf; a NaN shows in s
    }
    add_sum(st.s, st.c, (s[0] + s[1]) + (s[2] + s[3]));
    st.w += w;
    if (k > 0) {
      if ((step & (step - 1)) == 0) {  // steps 0, 1, 2, 4, ...
        const float gm = group_max<W>(st.m);
        if (lane % W == 0) keys[tid / W] = group_key(gm, tid / W);
        if (step == 0) __syncthreads();
        else wave_lds_fence();
        const float bar = kth_of_groups(keys, k, lane);
        if (bar > best.bar) {
          best.bar = bar;
          best.bar_id = kNone;
        }
      }
      ++step;
      if (__any(vm >= best.bar)) {
        // after a cut, equal values of later steps have higher indices
        const float least =
            best.bar_id == kNone ? best.bar : key_value(order_key(best.bar + 0.0f) + 1);
        int n = 0;
#pragma unroll
        for (int e = 0; e < kChunk; ++e) n += v[e] >= least ? 1 : 0;
        const int upto = lane_scan(n);
        const int total = __builtin_amdgcn_readlane(upto, 63);
        // (places past the row hold -inf)
        if (count == kChunk && best.bar > -inf && best.count + total <= kBuffer) {
          int to = best.count + upto - n;
#pragma unroll
          for (int e = 0; e < kChunk; ++e)
            if (v[e] >= least) {
              best.val[to] = v[e];
              best.id[to] = at + (e / N) * stride + e % N;
              ++to;
            }
          best.count += total;
        } else {
#pragma unroll 1
          for (int e = 0; e < count; ++e) {
            const int32_t i = at + (e / N) * stride + e % N;
            best_offer(best, v[e], i, i < limit, k, lane);
          }
        }
      }
    }
  };
  // elements up to the first 16-byte boundary, whole vectors, the rest
  const int64_t mis = ((uintptr_t)(x + from) & 15) / sizeof(T);
  int64_t head = mis ? N - mis : 0;
  if (head > to - from) head = to - from;
  const int64_t vecs = (to - from - head) / N;
  const int64_t tail = from + head + vecs * N;
  const u32x4v* body = (const u32x4v*)(x + from + head);
  u32x4v next[C];
  u32x4v none;  // -inf in every element
  {
    T t[N];
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = (T)-inf;
    __builtin_memcpy(&none, t, 16);
  }
  auto load = [&](int64_t i0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t i = i0 + c * kThreads + tid;
      next[c] = i < vecs ? body[i] : none;
    }
  };
  load(0);
  // the elements before the first and after the last whole vector are one
  // more step of the first wave: one a lane, the tail's from lane N on
  const int64_t edge = lane < N ? from + lane : tail + lane - N;
  const bool on_edge = lane < N ? lane < head : lane < 2 * N && tail + lane - N < to;
  const bool edges = wave == 0 && (head > 0 || tail < to);
  const float edge_x = edges && on_edge ? to_f32(x[edge]) : -inf;
  // (at least one, the same for all waves: the first has a barrier)
  const int64_t steps = vecs > 0 ? (vecs + C * kThreads - 1) / (C * kThreads) : 1;
  for (int64_t it = 0; it < steps + (edges ? 1 : 0); ++it) {
    const bool last = it == steps;
    float v[kChunk];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        T t[N];
        __builtin_memcpy(t, &next[c], 16);
        v[c * N + e] = last ? -inf : to_f32(t[e]);
      }
    if (last) v[0] = edge_x;
    if (it + 1 < steps) load((it + 1) * C * kThreads);
    const int32_t at = (int32_t)(last ? (on_edge ? edge : to) : from + head + (it * C * kThreads + tid) * N);
    take(v, at, kThreads * N, (int32_t)(last ? to : tail), last ? 1 : kChunk);
  }
  if (k > 0) {
    const float gm = group_max<W>(st.m);
    if (lane % W == 0) keys[tid / W] = group_key(gm, tid / W);
  }
  st = stats_wave(st);
  if (lane == 0) wave_stats[wave] = st;
  __syncthreads();
  st = wave_stats[0];
#pragma unroll
  for (int w = 1; w < W; ++w) st = stats_join(st, wave_stats[w]);
  if (k > 0) {
    const float bar = kth_of_groups(keys, k, lane);
    int n = 0;
    wave_lds_fence();
    for (int e = lane; e < best.count; e += 64) n += best.val[e] >= bar ? 1 : 0;
    if (__builtin_amdgcn_readlane(lane_scan(n), 63) > kFinal) best_cut(best, k, lane);
    for (int e = lane; e < best.count; e += 64)
      if (best.val[e] >= bar) {
        const int to = atomicAdd(&top_count, 1);  // any order: they are ranked
        entries[to] = entry_of(best.val[e], best.id[e]);
      }
    __syncthreads();
  }
  const int found = k > 0 ? top_count : 0;
  if (p.splits == 1) {
    if (tid == 0) write_row(p, row, st, target);
    rank_entries(entries, found, k,
                 [&](int rank, float v, int32_t i) { write_top(p, row, rank, v, i, st); });
  } else {
    const int64_t part = blockIdx.x;
    if (tid == 0) {
      p.part[part * kPartStats] = st.m;
      p.part[part * kPartStats + 1] = st.s;
      p.part[part * kPartStats + 2] = st.w;
      p.part[part * kPartStats + 3] = st.c;
    }
    rank_entries(entries, found, k, [&](int rank, float v, int32_t i) {
      p.part_val[part * k + rank] = v;
      p.part_id[part * k + rank] = i;
    });
  }
}

// Joins the parts of a row.  The parts' alternatives that can be the row's
// are ranked.
template <typename T>
__global__ __launch_bounds__(256) void logprobs_join_kernel(LogprobParams p) {
  __shared__ __attribute__((aligned(16))) uint64_t entries[kMaxParts * kMaxTop + 2];
  __shared__ __attribute__((aligned(16))) uint32_t keys[64];
  __shared__ int32_t count;
  const int64_t row = blockIdx.x;
  const int k = p.top_k, n = p.splits * k, tid = threadIdx.x, lane = tid & 63;
  if (tid == 0) count = 0;
  Target target{0.0f, false};
  if (tid == 0) target = target_of<T>(p, row);
  Stats st{-__builtin_inff(), 0.0f, 0.0f, 0.0f};
  if (lane < p.splits) {
    const float* q = p.part + (row * p.splits + lane) * kPartStats;
    st = Stats{q[0], q[1], q[2], q[3]};
  }
  // a group is a part's best depth + 1, and its value the least of them: k of
  // the row are no less than that of the need-th group
  const int depth = k > 0 ? (k - 1) / p.splits : 0, need = (k + depth) / (depth + 1);
  if (tid < 64)
    keys[tid] = group_key(k > 0 && tid < p.splits ? p.part_val[(row * p.splits + tid) * k + depth]
                                                  : bits_f32(0x7fc00000u), tid);
  __syncthreads();
  const float bar = k > 0 ? kth_of_groups(keys, need, lane) : 0.0f;
  for (int e = tid; e < n; e += 256) {
    const float v = p.part_val[row * n + e];
    const int32_t i = p.part_id[row * n + e];
    if (v >= bar && i != kNone) {
      const int at = atomicAdd(&count, 1);  // any order: they are ranked
      entries[at] = entry_of(v, i);
    }
  }
  st = stats_wave(st);
  __syncthreads();
  const int found = count;
  if (tid == 0) write_row(p, row, st, target);
  rank_entries(entries, found, k,
               [&](int rank, float v, int32_t i) { write_top(p, row, rank, v, i, st); });
}

// dx_v = g (1[v = t] - p_v) - h p_v (log p_v + H), 16 bytes a thread.
constexpr int kThreads = 256;  // of the gradient

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

// Rows go to several workgroups, each at least a step of a workgroup of four
// waves, while rows alone leave CUs without work.
LogprobPlan plan_logprobs(int64_t M, int64_t V, int64_t top_k, int32_t dtype) {
  (void)dtype;
  constexpr int64_t kTargetBlocks = 512, kMinLen = 4 * 64 * kChunk;
  LogprobPlan pl;
  int64_t splits = kTargetBlocks / (M > 0 ? M : 1);
  if (splits > ceil_div(V, kMinLen)) splits = ceil_div(V, kMinLen);
  if (splits > kMaxParts) splits = kMaxParts;
  if (splits < 2) splits = 1;
  pl.split_len = ceil_div(ceil_div(V, splits), 64) * 64;
  pl.splits = (int32_t)ceil_div(V, pl.split_len);
  const size_t n = pl.splits > 1 ? (size_t)M * pl.splits : 0;
  pl.workspace = n * (kPartStats * sizeof(float) + (size_t)top_k * (sizeof(float) + sizeof(int32_t)));
  return pl;
}

// Rows of one launch: of more, the rest comes in further ones.
static int64_t rows_at_once(int64_t M, int64_t blocks_a_row) {
  const int64_t most = kMaxGrid / blocks_a_row;
  return M < most ? M : most;
}

static hipError_t launch_rows(const LogprobParams& p, int32_t dtype, hipStream_t s) {
  const dim3 grid((unsigned)(p.M * p.splits));
  // A long row of its own workgroup is shared by eight waves while there are
  // few rows.  Registers leave a CU 24 waves: with 16 a row the next row could
  // not start beside it.  Waves a row, us (fp32, top_k 5): 512 x 128257 60.3
  // with 16, 55.2 with 8, 54.7 with 4 (bf16 53.4, 43.4, 52.5); 300 x 128257
  // 51.5, 42.1, 42.0; 512 x 16400 18.2 with 8, 14.1 with 4; 1024 x 128257 111,
  // 96.5, 96.2; 2000 x 20000 106, 52.4, 40.2; 4096 x 32003 217, 113, 99.9.
  const bool wide = p.splits == 1 && p.V >= 32 * 64 * kChunk && p.M < 1024;
#define Q4_LOGPROBS(T)                                                                         \
  do {                                                                                         \
    if (wide)                                                                                  \
      hipLaunchKernelGGL((logprobs_kernel<T, 8>), grid, dim3(512), 0, s, p);                   \
    else                                                                                       \
      hipLaunchKernelGGL((logprobs_kernel<T, 4>), grid, dim3(256), 0, s, p);                   \
    if (p.splits > 1)                                                                          \
      hipLaunchKernelGGL((logprobs_join_kernel<T>), dim3((unsigned)p.M), dim3(256), 0, s, p);  \
  } while (0)
  if (dtype == Q4_DTYPE_F32) Q4_LOGPROBS(float);
  else if (dtype == Q4_DTYPE_F16) Q4_LOGPROBS(_Float16);
  else Q4_LOGPROBS(bf16);
#undef Q4_LOGPROBS
  return hipGetLastError();
}

hipError_t launch_logprobs(const LogprobParams& p, int32_t dtype, hipStream_t s) {
  const int64_t e = dtype == Q4_DTYPE_F32 ? 4 : 2;
  const int64_t step = rows_at_once(p.M, p.splits);  // (all of them where rows have parts)
  for (int64_t m = 0; m < p.M; m += step) {
    LogprobParams r = p;
    r.M = p.M - m < step ? p.M - m : step;
    r.x = (const char*)p.x + m * p.ld * e;
    r.targets = p.targets ? p.targets + m : nullptr;
    r.logprob = p.logprob ? p.logprob + m : nullptr;
    r.entropy = p.entropy + m;
    r.lse = p.lse + m;
    r.top_ids = p.top_ids ? p.top_ids + m * p.top_k : nullptr;
    r.top_lp = p.top_lp ? p.top_lp + m * p.top_k : nullptr;
    const hipError_t err = launch_rows(r, dtype, s);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

static hipError_t launch_backward_rows(const LogprobBwdParams& p, int32_t dtype, int64_t per_row,
                                       hipStream_t s) {
  const dim3 grid((unsigned)(p.M * per_row));
  if (dtype == Q4_DTYPE_F32)
    hipLaunchKernelGGL(logprobs_backward_kernel<float>, grid, dim3(kThreads), 0, s, p, per_row);
  else if (dtype == Q4_DTYPE_F16)
    hipLaunchKernelGGL(logprobs_backward_kernel<_Float16>, grid, dim3(kThreads), 0, s, p, per_row);
  else
    hipLaunchKernelGGL(logprobs_backward_kernel<bf16>, grid, dim3(kThreads), 0, s, p, per_row);
  return hipGetLastError();
}

hipError_t launch_logprobs_backward(const LogprobBwdParams& p, int32_t dtype, hipStream_t s) {
  const int64_t e = dtype == Q4_DTYPE_F32 ? 4 : 2;
  const int64_t per_row = ceil_div(ceil_div(p.V * e, 16), kThreads * 4);
  const int64_t step = rows_at_once(p.M, per_row);
  for (int64_t m = 0; m < p.M; m += step) {
    LogprobBwdParams r = p;
    r.M = p.M - m < step ? p.M - m : step;
    r.x = (const char*)p.x + m * p.ld * e;
    r.dx = (char*)p.dx + m * p.ldd * e;
    r.targets = p.targets ? p.targets + m : nullptr;
    r.lse = p.lse + m;
    r.entropy = p.entropy + m;
    r.g_lp = p.g_lp ? p.g_lp + m : nullptr;
    r.g_ent = p.g_ent ? p.g_ent + m : nullptr;
    const hipError_t err = launch_backward_rows(r, dtype, per_row, s);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace q4
