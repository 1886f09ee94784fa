// q4_kv_append.hip -- appending to the paged 8-bit cache with the rotation of
// keys and queries, and the export of a cache's values.
//
// One workgroup owns one page of one head for K or for V, since the page's
// scale covers all of its tokens: it reads the new rows once (turning keys),
// keeps them in LDS as fp32, takes their largest magnitude, and codes them
// under the page's new scale, together with what the page held if the scale
// grew.  The rest of the grid turns queries, one token each.  Bound by HBM
// for prompts (each element is read once and written once), by the chain
// table -> row -> maximum -> store for decode steps.
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

// Elements of unit u (0 <= u < dim / 2): the pair that turns together, or
// two neighbours past the turning part.
__device__ __forceinline__ void unit_elems(int u, int half, bool interleaved, int* a, int* b) {
  if (u < half && !interleaved) {
    *a = u;
    *b = u + half;
  } else {
    *a = 2 * u;
    *b = 2 * u + 1;
  }
}

template <typename T>
__device__ __forceinline__ void turn_queries(const AppendParams& p, int32_t t) {
  __shared__ float cs[256];  // cosines of the token, then sines
  const KvCache& c = p.c;
  // the sequence of token t: the last b with cu_new[b] <= t
  int32_t lo = 0, hi = p.batch - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (c.cu_new[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const SeqSpan sp = seq_span(c.cu_new, c.lengths, lo, p.T);
  const int32_t pos = sp.pos0 + (t - sp.t0);
  const int half = p.rot >> 1;
  for (int i = threadIdx.x; i < half; i += kThreads) turn(pos, p.inv_freq[i], &cs[i], &cs[128 + i]);
  __syncthreads();
  const T* q = (const T*)p.q + (int64_t)t * p.q_ts;
  T* o = (T*)p.q_out + (int64_t)t * p.qo_ts;
  const int units = c.dim >> 1;
  for (int i = threadIdx.x; i < p.heads * units; i += kThreads) {
    const int h = i / units, u = i - h * units;
    int ea, eb;
    unit_elems(u, half, p.interleaved, &ea, &eb);
    const T* src = q + h * p.q_hs;
    T* dst = o + h * p.qo_hs;
    const float a = to_f32(src[ea]), b = to_f32(src[eb]);
    if (u < half) {
      const float cc = cs[u], ss = cs[128 + u];
      dst[ea] = from_f32<T>(a * cc - b * ss);
      dst[eb] = from_f32<T>(b * cc + a * ss);
    } else {
      dst[ea] = src[ea];
      dst[eb] = src[eb];
    }
  }
}

__device__ __forceinline__ int code_of(float x, float scale) {
  const float r = __builtin_rintf(x / scale);
  return (int)fminf(fmaxf(r, -127.0f), 127.0f);
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

template <typename T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendParams p) {
  if (blockIdx.x >= (uint32_t)p.cache_blocks) {
    turn_queries<T>(p, (int32_t)(blockIdx.x - p.cache_blocks));
    return;
  }
  extern __shared__ float rows[];  // new rows, fp32 [tokens][pitch]
  __shared__ uint32_t wave_max[kThreads / 64];
  const KvCache& c = p.c;
  // workgroup -> (sequence, page, head, K or V)
  uint32_t id = blockIdx.x;
  const int is_v = id & 1;
  id >>= 1;
  const int h = id % c.heads;
  id /= c.heads;
  const int j = id % p.touched;
  const int b = id / p.touched;
  const SeqSpan sp = seq_span(c.cu_new, c.lengths, b, p.T);
  // new tokens of this page: slots o0 .. o1 - 1
  const int32_t first = sp.pos0 > 0 ? sp.pos0 : 0;
  const int32_t pi = (first >> c.page_log2) + j;
  const int64_t base = (int64_t)pi << c.page_log2;
  const int o0 = first > base ? (int)(first - base) : 0;
  // the rows in LDS are sized for max_new tokens
  const int64_t end = (int64_t)first + p.max_new < sp.len ? (int64_t)first + p.max_new : sp.len;
  const int64_t left = end - base;
  const int o1 = left < c.page ? (int)left : c.page;
  if (sp.n <= 0 || o1 <= o0) return;
  const int32_t pid = page_at(c.table + b * c.table_ld, c.max_pages, c.pages, pi);
  if (pid < 0) return;
  const int dim = c.dim, nt = o1 - o0;
  // V is read from LDS along tokens: the odd pitch spreads those over banks
  const int pitch = is_v ? dim + 1 : dim + 4;
  const int32_t t0 = sp.t0 + (int32_t)(base + o0 - sp.pos0);  // token of slot o0
  const T* src = is_v ? (const T*)p.v + h * p.v_hs : (const T*)p.k + h * p.k_hs;
  const int64_t ts = is_v ? p.v_ts : p.k_ts;
  const int half = is_v ? 0 : p.rot >> 1;
  const int units = dim >> 1;
  uint32_t amax = 0;
  for (int i = threadIdx.x; i < nt * units; i += kThreads) {
    const int t = i / units, u = i - t * units;
    int ea, eb;
    unit_elems(u, half, p.interleaved, &ea, &eb);
    const T* row = src + (t0 + t) * ts;
    float a = to_f32(row[ea]), bb = to_f32(row[eb]);
    if (u < half) {
      float cc, ss;
      turn((int32_t)(base + o0 + t), p.inv_freq[u], &cc, &ss);
      const float x = a * cc - bb * ss;
      bb = bb * cc + a * ss;
      a = x;
    }
    rows[t * pitch + ea] = a;
    rows[t * pitch + eb] = bb;
    amax = umax(amax, umax(abs_bits(a), abs_bits(bb)));
  }
  amax = wave_umax(amax);
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = umax(umax(wave_max[0], wave_max[1]), umax(wave_max[2], wave_max[3]));
  float* sc = (is_v ? c.vs : c.ks) + (int64_t)pid * c.heads + h;
  const bool fresh = o0 == 0;
  const float s_old = fresh ? 0.0f : *sc;
  const float s_new = bits_f32(umax(f32_bits(s_old), f32_bits(bits_f32(amax) / 127.0f)));
  const bool grew = f32_bits(s_new) != f32_bits(s_old);
  const float ratio = s_new > 0.0f ? s_old / s_new : 0.0f;
  const bool zero = s_new == 0.0f;
  // every thread has read the old scale before one writes the new one
  __syncthreads();
  if (threadIdx.x == 0 && (grew || fresh)) *sc = s_new;
  int8_t* cache = (is_v ? c.v : c.k) + ((int64_t)pid * c.heads + h) * ((int64_t)dim << c.page_log2);
  if (!is_v) {
    // 16 codes of one token per step; old rows only if the scale grew
    const int chunks = dim >> 4;
    const int lo = grew ? 0 : o0, hi = fresh ? c.page : o1;
    for (int i = threadIdx.x; i < (hi - lo) * chunks; i += kThreads) {
      const int r = i / chunks, ch = i - r * chunks, slot = lo + r;
      u32x4v* dst = (u32x4v*)(cache + (int64_t)slot * dim + 16 * ch);
      u32x4v w = {0, 0, 0, 0};
      if (slot >= o0 && slot < o1) {
        const float* x = &rows[(slot - o0) * pitch + 16 * ch];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e >> 2] |= ((uint32_t)(zero ? 0 : code_of(x[e], s_new)) & 0xffu) << (8 * (e & 3));
      } else if (slot < o0) {
        const u32x4v old = *dst;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = recode(old[e], ratio);
      }
      *dst = w;
    }
  } else {
    // 16 tokens of one column per step; a step that mixes old and new slots
    // keeps the old ones' bytes
    const int c_lo = grew ? 0 : o0 >> 4, c_hi = fresh ? c.page >> 4 : (o1 + 15) >> 4;
    const int n = c_hi - c_lo;
    for (int i = threadIdx.x; i < n * dim; i += kThreads) {
      const int d = i / n, ch = c_lo + (i - d * n);
      u32x4v* dst = (u32x4v*)(cache + ((int64_t)d << c.page_log2) + 16 * ch);
      u32x4v w = {0, 0, 0, 0};
      if (16 * ch < o0 || (16 * ch + 16 > o1 && !fresh)) {
        w = *dst;
        if (grew) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = recode(w[e], ratio);
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int slot = 16 * ch + e;
        if (slot >= o0 && slot < o1) {
          const int code = zero ? 0 : code_of(rows[(slot - o0) * pitch + d], s_new);
          const uint32_t m = 0xffu << (8 * (e & 3));
          w[e >> 2] = (w[e >> 2] & ~m) | (((uint32_t)code << (8 * (e & 3))) & m);
        }
      }
      *dst = w;
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
  const float sk = c.ks[ph], sv = c.vs[ph];
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

hipError_t launch_kv_append(const AppendParams& in, int32_t dtype, int64_t max_new,
                            hipStream_t s) {
  AppendParams p = in;
  p.max_new = max_new;
  p.touched = (int32_t)pages_touched(max_new, p.c.page);
  p.cache_blocks = (int32_t)((int64_t)p.batch * p.touched * p.c.heads * 2);
  const int64_t rows = max_new < p.c.page ? max_new : p.c.page;
  const size_t lds = (size_t)rows * (p.c.dim + 4) * sizeof(float);
  const dim3 grid((unsigned)(p.cache_blocks + (p.q ? p.T : 0)));
#define Q4_APPEND(T)                                                                            \
  do {                                                                                          \
    if (lds > 65536) {                                                                          \
      const hipError_t e = hipFuncSetAttribute(                                                 \
          (const void*)kv_append_kernel<T>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds); \
      if (e != hipSuccess) return e;                                                            \
    }                                                                                           \
    hipLaunchKernelGGL((kv_append_kernel<T>), grid, dim3(kThreads), lds, s, p);                 \
  } while (0)
  if (dtype == Q4_DTYPE_F32) Q4_APPEND(float);
  else if (dtype == Q4_DTYPE_F16) Q4_APPEND(_Float16);
  else Q4_APPEND(bf16);
#undef Q4_APPEND
  return hipGetLastError();
}

hipError_t launch_kv_dequant(const KvCache& c, int32_t dtype, void* k, void* v, hipStream_t s) {
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

}  // namespace q4
