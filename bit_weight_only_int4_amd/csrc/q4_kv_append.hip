// q4_kv_append.hip -- appending to the paged 8-bit cache with the rotation of
// keys and queries, and the export of a cache's values.
//
// One workgroup owns one page of one head for K or for V, since the page's
// scale covers all of its tokens: it reads the new rows once into registers
// (turning keys), takes their largest magnitude, and codes them under the
// page's new scale, together with what the page held if the scale grew.  A
// thread's share of K is 4 pairs of a token (dword stores of codes), of V 16
// tokens of a column, so that neither passes through LDS: with the rows kept
// there prompts of 6531 tokens took 103 us, the turning of their queries, in
// the rest of the grid, being held to the same 34 KB of LDS a workgroup.
// Bound by HBM for prompts (each element is read and written once), by the
// chain table -> row -> maximum -> store for decode steps.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_kv.h"
#include "q4_serve.h"
#include "q4_serve_device.h"

namespace q4 {

namespace {

constexpr int kThreads = 256;

// Cosine and sine of pos * inv_freq.  The angle in revolutions is formed in
// fp64 and its whole part dropped there (a position of 2^24 leaves 29 of 53
// bits), so the fp32 functions see at most half a turn.
__device__ __forceinline__ void turn(int32_t pos, float inv_freq, float* c, float* s) {
  const double rev = (double)pos * ((double)inv_freq * 0.15915494309189535);
  const float frac = (float)(rev - __builtin_rint(rev));  // [-1/2, 1/2]
  sincospif(2.0f * frac, s, c);
}

// Unit u of a row: pairs 4 u .. 4 u + 3.  Pair i < half turns: elements (i,
// i + half), or (2 i, 2 i + 1) if interleaved; past half (2 i, 2 i + 1) stay.
__device__ __forceinline__ void pair_elems(int i, int half, bool interleaved, int* a, int* b) {
  const bool split = i < half && !interleaved;
  *a = split ? i : 2 * i;
  *b = split ? i + half : 2 * i + 1;
}

template <typename T, int N>
__device__ __forceinline__ void load_vec(const T* p, T (&x)[N]) {
  typedef uint32_t vec __attribute__((ext_vector_type(N * sizeof(T) / 4)));
  const vec v = *(const vec*)p;
  __builtin_memcpy(x, &v, sizeof v);
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const T (&x)[N]) {
  typedef uint32_t vec __attribute__((ext_vector_type(N * sizeof(T) / 4)));
  vec v;
  __builtin_memcpy(&v, x, sizeof v);
  *(vec*)p = v;
}

// A unit's elements, x[2 i] and x[2 i + 1] of pair i.  vec: rows are 16-byte
// aligned and rot a multiple of 8, so that a unit is 4 + 4 or 8 neighbours.
template <typename T>
__device__ __forceinline__ void load_unit(const T* row, int u, int half, bool interleaved, bool vec,
                                          float (&x)[8]) {
  if (vec && 4 * u < half && !interleaved) {
    T a[4], b[4];
    load_vec(row + 4 * u, a);
    load_vec(row + 4 * u + half, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = to_f32(a[i]);
      x[2 * i + 1] = to_f32(b[i]);
    }
  } else if (vec) {
    T a[8];
    if constexpr (sizeof(T) == 2) {
      load_vec(row + 8 * u, a);
    } else {
      T lo[4], hi[4];
      load_vec(row + 8 * u, lo);
      load_vec(row + 8 * u + 4, hi);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = lo[i];
        a[i + 4] = hi[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(a[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int ea, eb;
      pair_elems(4 * u + i, half, interleaved, &ea, &eb);
      x[2 * i] = to_f32(row[ea]);
      x[2 * i + 1] = to_f32(row[eb]);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store_unit(T* row, int u, int half, bool interleaved, bool vec,
                                           const float (&x)[8]) {
  if (vec && 4 * u < half && !interleaved) {
    T a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = from_f32<T>(x[2 * i]);
      b[i] = from_f32<T>(x[2 * i + 1]);
    }
    store_vec(row + 4 * u, a);
    store_vec(row + 4 * u + half, b);
  } else if (vec) {
    T lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = from_f32<T>(x[i]);
      hi[i] = from_f32<T>(x[i + 4]);
    }
    store_vec(row + 8 * u, lo);
    store_vec(row + 8 * u + 4, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int ea, eb;
      pair_elems(4 * u + i, half, interleaved, &ea, &eb);
      row[ea] = from_f32<T>(x[2 * i]);
      row[eb] = from_f32<T>(x[2 * i + 1]);
    }
  }
}

// Turns a unit; cs, sn: cosines and sines of its four pairs.
__device__ __forceinline__ void turn_unit(float (&x)[8], const float* cs, const float* sn, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= n) break;  // the turning part may end inside a unit
    const float a = x[2 * i], b = x[2 * i + 1];
    x[2 * i] = a * cs[i] - b * sn[i];
    x[2 * i + 1] = b * cs[i] + a * sn[i];
  }
}

// Queries of tokens t0 .. t0 + kTurn - 1, all heads.
constexpr int kTurn = 4;  // append_turn at most

template <typename T>
__device__ __forceinline__ void turn_queries(const AppendParams& p, int64_t t0, int n) {
  __shared__ float cs[kTurn][128], sn[kTurn][128];
  __shared__ int32_t at[kTurn];
  const KvCache& c = p.c;
  const int half = p.rot >> 1;
  if ((int)threadIdx.x < n) {
    // the sequence of the token: the last b with cu_new[b] <= t
    const int32_t t = (int32_t)t0 + threadIdx.x;
    int32_t lo = 0, hi = p.batch - 1;
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (c.cu_new[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const SeqSpan sp = seq_span(c.cu_new, c.lengths, lo, p.T);
    at[threadIdx.x] = sp.pos0 + (t - sp.t0);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int k = i / half, f = i - k * half;
    turn(at[k], p.inv_freq[f], &cs[k][f], &sn[k][f]);
  }
  __syncthreads();
  const int units = c.dim >> 3, per_token = p.heads * units;
  const T* q = (const T*)p.q;
  T* o = (T*)p.q_out;
  for (int k = 0; k < n; ++k) {
#pragma unroll 2
    for (int i = threadIdx.x; i < per_token; i += kThreads) {
      const int h = i / units, u = i - h * units;
      float x[8];
      load_unit(q + (t0 + k) * p.q_ts + h * p.q_hs, u, half, p.interleaved, p.q_vec, x);
      if (4 * u < half) turn_unit(x, &cs[k][4 * u], &sn[k][4 * u], half - 4 * u);
      store_unit(o + (t0 + k) * p.qo_ts + h * p.qo_hs, u, half, p.interleaved, p.q_vec, x);
    }
  }
}

__device__ __forceinline__ uint32_t code_of(float x, float scale) {
  const float r = __builtin_rintf(x / scale);
  return (uint32_t)(int)fminf(fmaxf(r, -127.0f), 127.0f) & 0xffu;
}

// Four codes of a dword under a scale that grew by 1 / ratio.
__device__ __forceinline__ uint32_t recode(uint32_t w, float ratio) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = (float)(int8_t)(w >> (8 * i));
    r |= ((uint32_t)(int)__builtin_rintf(c * ratio) & 0xffu) << (8 * i);
  }
  return r;
}

// The page's scale, old and new, from the threads' largest magnitudes.
struct Scale {
  float now, ratio;
  bool grew, zero;
};

__device__ __forceinline__ Scale grow_scale(float* at, uint32_t amax, bool fresh) {
  __shared__ uint32_t wave_max[kThreads / 64];
  // (-0 is 0: magnitudes are compared as bit patterns)
  const float old = fresh ? 0.0f : __builtin_fabsf(scale_or_nan(*at));
  amax = wave_umax(amax);
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
  __syncthreads();  // and every thread has read the old scale
  amax = umax(umax(wave_max[0], wave_max[1]), umax(wave_max[2], wave_max[3]));
  Scale s;
  s.now = bits_f32(umax(f32_bits(old), f32_bits(bits_f32(amax) / 127.0f)));
  s.grew = f32_bits(s.now) != f32_bits(old);
  s.ratio = s.now > 0.0f ? old / s.now : 0.0f;
  s.zero = s.now == 0.0f;
  if (threadIdx.x == 0 && (s.grew || fresh)) *at = s.now;
  return s;
}

// U: a thread's units of K, and half of its 16-token columns of V.
template <typename T, int U>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendParams p) {
  if (blockIdx.x >= (uint32_t)p.cache_blocks) {
    const int64_t t0 = (int64_t)(blockIdx.x - p.cache_blocks) * p.turn;
    turn_queries<T>(p, t0, p.T - t0 < p.turn ? (int)(p.T - t0) : p.turn);
    return;
  }
  const KvCache& c = p.c;
  // workgroup -> (sequence, page, head, K or V)
  uint32_t id = blockIdx.x;
  const int is_v = id & 1;
  id >>= 1;
  const int h = id % c.heads;
  id /= c.heads;
  const int j = p.first + (int)(id % p.touched);
  const int b = id / p.touched;
  const SeqSpan sp = seq_span(c.cu_new, c.lengths, b, p.T);
  // new tokens of this page: slots o0 .. o1 - 1
  const int32_t first = sp.pos0 > 0 ? sp.pos0 : 0;
  const int32_t pi = (first >> c.page_log2) + j;
  const int64_t base = (int64_t)pi << c.page_log2;
  const int o0 = first > base ? (int)(first - base) : 0;
  // of a sequence the first max_new are stored, as the launch is sized
  const int64_t end = (int64_t)first + p.max_new < sp.len ? (int64_t)first + p.max_new : sp.len;
  const int64_t left = end - base;
  const int o1 = left < c.page ? (int)left : c.page;
  if (sp.n <= 0 || o1 <= o0) return;
  const int32_t pid = page_at(c.table + b * c.table_ld, c.max_pages, c.pages, pi);
  if (pid < 0) return;
  const int dim = c.dim, tid = threadIdx.x;
  const int64_t t0 = sp.t0 + (base + o0 - sp.pos0);  // token of slot o0
  const bool fresh = o0 == 0;
  const int64_t ph = (int64_t)pid * c.heads + h;
  const int64_t at = ph * ((int64_t)dim << c.page_log2);
  if (!is_v) {
    const int units = dim >> 3, half = p.rot >> 1, n = (o1 - o0) * units;
    const T* src = (const T*)p.k + h * p.k_hs;
    float x[U][8];
    int slot[U], unit[U];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int w = i * kThreads + tid;
      if (w < n) {
        const int t = w / units;
        unit[i] = w - t * units;
        slot[i] = o0 + t;
        load_unit(src + (t0 + t) * p.k_ts, unit[i], half, p.interleaved, p.k_vec, x[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (i * kThreads + tid < n) {
        const int u = unit[i];
        float cs[4], sn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * u + e < half) turn((int32_t)(base + slot[i]), p.inv_freq[4 * u + e], &cs[e], &sn[e]);
        turn_unit(x[i], cs, sn, half - 4 * u);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = umax(amax, abs_bits(x[i][e]));
      }
    }
    const Scale s = grow_scale(c.ks + ph, amax, fresh);
    int8_t* cache = c.k + at;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (i * kThreads + tid < n) {
        int8_t* row = cache + (int64_t)slot[i] * dim;
        const int u = unit[i];
        uint32_t q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = s.zero ? 0u : code_of(x[i][e], s.now);
        if (p.rot % 8 == 0 && 4 * u < half && !p.interleaved) {
          *(uint32_t*)(row + 4 * u) = q[0] | q[2] << 8 | q[4] << 16 | q[6] << 24;
          *(uint32_t*)(row + 4 * u + half) = q[1] | q[3] << 8 | q[5] << 16 | q[7] << 24;
        } else if (p.rot % 8 == 0) {
          *(u32x2*)(row + 8 * u) = u32x2{q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24,
                                         q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            int ea, eb;
            pair_elems(4 * u + e, half, p.interleaved, &ea, &eb);
            row[ea] = (int8_t)q[2 * e];
            row[eb] = (int8_t)q[2 * e + 1];
          }
        }
      }
    }
    // the rest of the page, 16 codes a step: 0 if it starts anew, coded anew
    // if the scale grew
    const int chunks = dim >> 4;
    if (fresh) {
      for (int i = o1 * chunks + tid; i < chunks << c.page_log2; i += kThreads)
        ((u32x4v*)cache)[i] = u32x4v{0, 0, 0, 0};
    } else if (s.grew) {
      // both sides of the new tokens: one that is stored again has some behind it
      for (int i = tid; i < (c.page - (o1 - o0)) * chunks; i += kThreads) {
        u32x4v* at_i = (u32x4v*)cache + (i < o0 * chunks ? i : i + (o1 - o0) * chunks);
        u32x4v w = *at_i;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = recode(w[e], s.ratio);
        *at_i = w;
      }
    }
  } else {
    // 16 slots of a column: those from o0's on; loads of a wave run along
    // the columns, a row each
    constexpr int J = (U + 1) / 2;
    const int c_lo = o0 >> 4, c_hi = (o1 + 15) >> 4, n = (c_hi - c_lo) * dim;
    const T* src = (const T*)p.v + h * p.v_hs;
    T x[J][16];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int w = i * kThreads + tid, ch = w / dim, d = w - ch * dim, s0 = 16 * (c_lo + ch);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[i][e] = (T)0.0f;
        if (w < n && s0 + e >= o0 && s0 + e < o1) x[i][e] = src[(t0 + (s0 + e - o0)) * p.v_ts + d];
      }
    }
#pragma unroll
    for (int i = 0; i < J; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) amax = umax(amax, abs_bits(to_f32(x[i][e])));
    const Scale s = grow_scale(c.vs + ph, amax, fresh);
    int8_t* cache = c.v + at;
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int w = i * kThreads + tid;
      if (w >= n) continue;
      const int ch = w / dim, d = w - ch * dim, s0 = 16 * (c_lo + ch);
      u32x4v* dst = (u32x4v*)(cache + ((int64_t)d << c.page_log2) + s0);
      u32x4v q = {0, 0, 0, 0};
      // the old slots of a column that also has new ones keep their codes
      if (s0 < o0 || (s0 + 16 > o1 && !fresh)) {
        q = *dst;
        if (s.grew) {
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = recode(q[e], s.ratio);
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (s0 + e >= o0 && s0 + e < o1) {
          const uint32_t code = s.zero ? 0u : code_of(to_f32(x[i][e]), s.now);
          q[e >> 2] = (q[e >> 2] & ~(0xffu << (8 * (e & 3)))) | code << (8 * (e & 3));
        }
      *dst = q;
    }
    if (fresh) {
      const int rest = (c.page >> 4) - c_hi;
      for (int i = tid; i < rest * dim; i += kThreads) {
        const int ch = i / dim, d = i - ch * dim;
        *(u32x4v*)(cache + ((int64_t)d << c.page_log2) + 16 * (c_hi + ch)) = u32x4v{0, 0, 0, 0};
      }
    } else if (s.grew) {
      const int old = (c.page >> 4) - (c_hi - c_lo);
      for (int i = tid; i < old * dim; i += kThreads) {
        const int k = i / dim, d = i - k * dim, ch = k < c_lo ? k : k + (c_hi - c_lo);
        u32x4v* dst = (u32x4v*)(cache + ((int64_t)d << c.page_log2) + 16 * ch);
        u32x4v q = *dst;
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = recode(q[e], s.ratio);
        *dst = q;
      }
    }
  }
}

// One page of one head: K is scaled as it lies; V is turned back to token
// order through LDS (rows padded by a dword so that both sides spread over
// the banks).
template <typename T>
__global__ __launch_bounds__(kThreads) void kv_dequant_kernel(KvCache c, T* __restrict__ ko,
                                                              T* __restrict__ vo) {
  extern __shared__ uint8_t bytes[];
  const int64_t ph = blockIdx.x;
  const int dim = c.dim, page = c.page;
  const int64_t at = ph * ((int64_t)dim << c.page_log2);
  const float sk = scale_or_nan(c.ks[ph]), sv = scale_or_nan(c.vs[ph]);
  const int n16 = (dim << c.page_log2) >> 4;
  const u32x4v* k = (const u32x4v*)(c.k + at);
  const u32x4v* v = (const u32x4v*)(c.v + at);
  const int pitch = page + 4;
  const int per_row = page >> 4;
  for (int i = threadIdx.x; i < n16; i += kThreads) {
    const u32x4v w = v[i];
    const int d = i / per_row, ch = i - d * per_row;
    uint32_t* row = (uint32_t*)(bytes + d * pitch + 16 * ch);
#pragma unroll
    for (int e = 0; e < 4; ++e) row[e] = w[e];
  }
  for (int i = threadIdx.x; i < n16; i += kThreads) {
    const u32x4v w = k[i];
    T o[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = from_f32<T>((float)(int8_t)(w[e >> 2] >> (8 * (e & 3))) * sk);
    u32x4v* dst = (u32x4v*)(ko + at + 16 * (int64_t)i);
    const u32x4v* src = (const u32x4v*)o;
#pragma unroll
    for (int e = 0; e < (int)sizeof(T); ++e) dst[e] = src[e];
  }
  __syncthreads();
  // (token, 8 columns) per step
  const int groups = dim >> 3;
  for (int i = threadIdx.x; i < page * groups; i += kThreads) {
    const int t = i / groups, g = i - t * groups;
    T o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = from_f32<T>((float)(int8_t)bytes[(8 * g + e) * pitch + t] * sv);
    u32x4v* dst = (u32x4v*)(vo + at + (int64_t)t * dim + 8 * g);
    const u32x4v* src = (const u32x4v*)o;
#pragma unroll
    for (int e = 0; e < (int)sizeof(T) / 2; ++e) dst[e] = src[e];
  }
}

}  // namespace

template <typename T>
static hipError_t launch_append(const AppendParams& p, int64_t rows, dim3 grid, hipStream_t s) {
  // K units of a page's new rows over the threads; V's 16-token columns may
  // begin and end inside the rows, so that they can be one more than the rows
  // fill: rows + 15 bounds their tokens
  const int64_t page = p.c.page;
  const int64_t k_units = rows * (p.c.dim / 8);
  const int64_t v_cols = ((rows + 15 + 15) / 16 < page / 16 ? (rows + 15 + 15) / 16 : page / 16) * p.c.dim;
  const int64_t need_k = (k_units + kThreads - 1) / kThreads;
  const int64_t need_v = 2 * ((v_cols + kThreads - 1) / kThreads);
  const int64_t u = need_k > need_v ? need_k : need_v;
  if (u <= 2)
    hipLaunchKernelGGL((kv_append_kernel<T, 2>), grid, dim3(kThreads), 0, s, p);
  else if (u <= 4)
    hipLaunchKernelGGL((kv_append_kernel<T, 4>), grid, dim3(kThreads), 0, s, p);
  else if (u <= 8)
    hipLaunchKernelGGL((kv_append_kernel<T, 8>), grid, dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL((kv_append_kernel<T, 16>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_kv_append(const AppendParams& in, int32_t dtype, int64_t max_new,
                            hipStream_t s) {
  AppendParams p = in;
  p.max_new = max_new;
  const int64_t touched = pages_touched(max_new, p.c.page);
  p.turn = append_turn(p.T);
  int64_t turns = p.q ? append_turns(p.T) : 0;
  const int64_t rows = max_new < p.c.page ? max_new : p.c.page;
  // One launch, unless a loose max_new makes more workgroups than that may have
  // (a loop over pages in the kernel costs it registers: 6531 tokens of prompts
  // 73 -> 105 us).
  const int64_t a_page = (int64_t)p.batch * p.c.heads * 2;
  for (int64_t j = 0; j < touched; j += p.touched) {
    const int64_t most = (kMaxGrid - turns) / a_page;
    p.first = (int32_t)j;
    p.touched = (int32_t)(touched - j < most ? touched - j : most);
    p.cache_blocks = (int32_t)(a_page * p.touched);
    const dim3 grid((unsigned)(p.cache_blocks + turns));
    const hipError_t e = dtype == Q4_DTYPE_F32   ? launch_append<float>(p, rows, grid, s)
                         : dtype == Q4_DTYPE_F16 ? launch_append<_Float16>(p, rows, grid, s)
                                                 : launch_append<bf16>(p, rows, grid, s);
    if (e != hipSuccess) return e;
    turns = 0;  // the queries have turned
  }
  return hipSuccess;
}

static hipError_t launch_dequant_pages(const KvCache& c, int32_t dtype, void* k, void* v,
                                       hipStream_t s) {
  const size_t lds = (size_t)c.dim * (c.page + 4);
  const dim3 grid((unsigned)(c.pages * c.heads));
  if (dtype == Q4_DTYPE_F32)
    hipLaunchKernelGGL(kv_dequant_kernel<float>, grid, dim3(kThreads), lds, s, c, (float*)k, (float*)v);
  else if (dtype == Q4_DTYPE_F16)
    hipLaunchKernelGGL(kv_dequant_kernel<_Float16>, grid, dim3(kThreads), lds, s, c, (_Float16*)k, (_Float16*)v);
  else
    hipLaunchKernelGGL(kv_dequant_kernel<bf16>, grid, dim3(kThreads), lds, s, c, (bf16*)k, (bf16*)v);
  return hipGetLastError();
}

hipError_t launch_kv_dequant(const KvCache& in, int32_t dtype, void* k, void* v, hipStream_t s) {
  const int64_t step = kMaxGrid / in.heads;  // pages of one launch
  const int64_t page = (int64_t)in.heads * in.page * in.dim, e = dtype == Q4_DTYPE_F32 ? 4 : 2;
  for (int64_t p = 0; p < in.pages; p += step) {
    KvCache c = in;
    c.pages = in.pages - p < step ? in.pages - p : step;
    c.k += p * page;
    c.v += p * page;
    c.ks += p * in.heads;
    c.vs += p * in.heads;
    const hipError_t err = launch_dequant_pages(c, dtype, (char*)k + p * page * e,
                                                (char*)v + p * page * e, s);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace q4
