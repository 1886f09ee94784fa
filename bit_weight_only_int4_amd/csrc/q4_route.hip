// q4_route.hip -- the choice of experts and its gradient, for gfx950.
//
// A wave owns a token; lane l holds EPL experts from EPL l on, so that a lower
// lane has lower experts.  Choosing is top_k rounds of a maximum over the lanes.
// Values are ordered as integers: without a bias the logit's 32 bits (scores have
// their order), with one the 64 bits of score + bias formed in fp64, so that no
// rounding of a score decides between two experts (fp32 sums of 8192 tokens over
// 256 experts differ from the exact order in a few places).  An integer of 0 is an expert that is not eligible.
//
// Bound by the vector unit's issue: top_k maxima of 6 cross-lane steps one after
// the other, and with a bias exponentials in fp64.  8192 tokens, 8 of 256 experts
// in 8 groups with a bias, 19 us; 32 tokens, 8 of 64, 4.3 (an empty launch 1.7).
#include <hip/hip_runtime.h>

#include "q4_experts.h"
#include "q4_experts_device.h"

namespace q4 {
namespace {

constexpr int kWaves = 4;  // tokens of a workgroup

// Order of floats as unsigned integers: -inf is 0, NaN 1, below every number,
// so that a row of NaN still has experts for its weights to reach.
__device__ __forceinline__ uint32_t key32(float x) {
  const uint32_t b = f32_bits(x);
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return x != x ? 1u : x > -__builtin_inff() ? k : 0u;
}
__device__ __forceinline__ uint64_t key64(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint64_t k = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return x != x ? 1ull : x > -__builtin_inf() ? k : 0ull;
}
// -0 and 0 are equal values
__device__ __forceinline__ float plus_zero(float x) { return x + 0.0f; }

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const float y = __shfl_xor(x, m, 64);
    x = x > y ? x : y;
  }
  return x;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

// The largest value of the wave, in every lane.  The lanes' neighbours come
// through the vector unit's own lane moves (by 1, 2, 4, 8 within 16 lanes, then
// the rows' last lanes), a few cycles each, and not through LDS.
__device__ __forceinline__ uint32_t wave_most(uint32_t x) {
#define Q4_STEP(ctrl, rows) \
  x = umax(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, rows, 0xf, false))
  Q4_STEP(0x111, 0xf);
  Q4_STEP(0x112, 0xf);
  Q4_STEP(0x114, 0xf);
  Q4_STEP(0x118, 0xf);
  Q4_STEP(0x142, 0xa);
  Q4_STEP(0x143, 0xc);
#undef Q4_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// The largest key of the wave and the lowest expert that has it: that of the
// first lane with this key.
__device__ __forceinline__ void wave_best(uint32_t& key, int32_t& id) {
  const uint32_t top = wave_most(key);
  id = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(__ballot(key == top)));
  key = top;
}
__device__ __forceinline__ void wave_best(uint64_t& key, int32_t& id) {
  const uint32_t hi = wave_most((uint32_t)(key >> 32));
  const bool mine = (uint32_t)(key >> 32) == hi;
  uint64_t m = __ballot(mine);
  if (m & (m - 1)) {
    const uint32_t lo = wave_most(mine ? (uint32_t)key : 0u);  // by all lanes
    m = __ballot(mine & ((uint32_t)key == lo));
  }
  const int from = (int)__builtin_ctzll(m);
  id = __builtin_amdgcn_readlane(id, from);
  key = ((uint64_t)hi << 32) | (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, from);
}

__device__ __forceinline__ uint32_t shuffle_xor(uint32_t x, int d) { return __shfl_xor(x, d, 64); }
__device__ __forceinline__ uint64_t shuffle_xor(uint64_t x, int d) {
  return __shfl_xor((unsigned long long)x, d, 64);
}

// Sigmoid of a chosen logit for the share among the chosen, of which `base` is
// the largest: times e^-base where base < 0, so that scores too small for fp32
// keep their shares (the largest is then 1/2 at least).
__device__ __forceinline__ float small_sigmoid(float z, float base) {
  if (!(base < 0.0f)) return sigmoid(z);
  return exp_full(z - base) / (1.0f + exp_full(z));
}

template <bool BIAS>
struct KeyOf {
  typedef uint32_t type;
};
template <>
struct KeyOf<true> {
  typedef uint64_t type;
};

__device__ __forceinline__ double key_value(uint64_t k) {
  return __builtin_bit_cast(double, (k >> 63) ? (k & 0x7fffffffffffffffull) : ~k);
}

// EPL: experts of a lane, 64 * EPL >= E
template <typename T, int EPL, bool BIAS>
__global__ void __launch_bounds__(64 * kWaves) route_kernel(const RouteParams p) {
  typedef typename KeyOf<BIAS>::type Key;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= p.T) return;  // whole waves; no barrier follows
  const T* row = (const T*)p.x + t * p.ld;
  float z[EPL];
  Key key[EPL];
  float top = -__builtin_inff();
  bool nan = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    z[i] = e < p.E ? plus_zero(to_f32(row[e])) : -__builtin_inff();
    nan |= z[i] != z[i];
    top = z[i] > top ? z[i] : top;
  }
  nan = __any(nan);
  const bool softmax = p.score == Q4_SCORE_SOFTMAX;
  if (softmax || BIAS) top = wave_max(top);
  // a row of nothing but -inf: no expert is eligible
  nan |= softmax && top == __builtin_inff();
  if constexpr (BIAS) {
    double s[EPL], sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const double y = (double)z[i];
      if (softmax) {
        // (the largest may be infinite)
        s[i] = z[i] == top ? 1.0 : z[i] > -__builtin_inff() ? exp(y - (double)top) : 0.0;
        sum += s[i];
      } else {
        const double e = exp(y < 0.0 ? y : -y);
        s[i] = (y < 0.0 ? e : 1.0) / (1.0 + e);
      }
    }
    if (softmax) sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane * EPL + i;
      const bool in = e < p.E && z[i] != -__builtin_inff();
      const double v = (softmax ? s[i] / sum : s[i]) + (e < p.E ? (double)p.bias[e] : 0.0);
      key[i] = !in ? 0 : z[i] != z[i] ? 1 : key64(v + 0.0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = key32(z[i]);
  }

  if (p.groups > 1) {
    // a group's value: its largest key, with a bias the sum of its two largest
    const int per = p.E / p.groups;
    auto value_of = [](Key best, Key second) {
      if constexpr (BIAS) {
        if (second) best = key64(key_value(best) + key_value(second) + 0.0);
      }
      return best;
    };
    const int lanes = per / EPL;
    if (lanes * EPL == per && (lanes & (lanes - 1)) == 0) {
      // groups of whole lanes, a power of two of them: all groups join their
      // lanes' two largest keys at once, and every lane has its group's value
      Key best = 0, second = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const bool up = key[i] > best;
        const Key less = up ? best : key[i];
        best = up ? key[i] : best;
        second = less > second ? less : second;
      }
      for (int d = 1; d < lanes; d <<= 1) {
        const Key ob = shuffle_xor(best, d), os = shuffle_xor(second, d);
        const Key less = ob > best ? best : ob;
        best = ob > best ? ob : best;
        second = os > second ? os : second;
        second = less > second ? less : second;
      }
      Key value = value_of(best, second);
      bool kept = false;
      for (int r = 0; r < p.top_groups; ++r) {
        Key top = value;
        int32_t at = lane / lanes;
        wave_best(top, at);
        if (top == 0) break;
        if (lane / lanes == at) {
          value = 0;
          kept = true;
        }
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = kept ? key[i] : 0;
    } else {
      // one group after the other; lane l collects the values of groups EPL l
      // and on (groups <= E <= 64 EPL)
      Key value[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) value[i] = 0;
      for (int g = 0; g < p.groups; ++g) {
        Key best = 0, second = 0;
        int32_t at = 0, at2 = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = lane * EPL + i;
          const bool mine = e >= g * per && e < (g + 1) * per && key[i] > best;
          best = mine ? key[i] : best;
          at = mine ? e : at;
        }
        wave_best(best, at);
        if constexpr (BIAS) {
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            const int e = lane * EPL + i;
            const bool mine = e >= g * per && e < (g + 1) * per && e != at && key[i] > second;
            second = mine ? key[i] : second;
          }
          wave_best(second, at2);
        }
        best = value_of(best, second);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (g == lane * EPL + i) value[i] = best;
      }
      uint32_t kept[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) kept[i] = 0;
      for (int r = 0; r < p.top_groups; ++r) {
        Key best = 0;
        int32_t at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const bool take = value[i] > best;
          best = take ? value[i] : best;
          at = take ? lane * EPL + i : at;
        }
        wave_best(best, at);
        if (best == 0) break;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = lane * EPL + i;
          if (e == at) value[i] = 0;
          if (e >= at * per && e < (at + 1) * per) kept[i] = 1;
        }
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = kept[i] ? key[i] : 0;
    }
  }

  // lane j keeps choice j
  int32_t id = -1;
  float chosen = -__builtin_inff();
  for (int j = 0; j < p.top_k; ++j) {
    Key best = 0;
    int32_t at = 0;
    float zb = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool take = key[i] > best;
      best = take ? key[i] : best;
      at = take ? lane * EPL + i : at;
    }
    wave_best(best, at);
    if (best == 0) break;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool mine = lane * EPL + i == at;
      zb = mine ? z[i] : zb;
      key[i] = mine ? 0 : key[i];
    }
    zb = __shfl(zb, at / EPL, 64);
    if (lane == j) {
      id = at;
      chosen = zb;
    }
  }

  float w = 0.0f;
  if (softmax) {
    // renormalised, the scores' common divisor falls away: relative to the
    // largest chosen, so that none of them is lost beside an expert left out
    const float base = p.renormalize ? wave_max(chosen) : top;
    const float s = id >= 0 ? exp_full(chosen - base) : 0.0f;
    float sum = 0.0f;
    if (p.renormalize) {
      sum = wave_sum(s);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) sum += z[i] > -__builtin_inff() ? exp_full(z[i] - top) : 0.0f;
      sum = wave_sum(sum);
    }
    w = id >= 0 ? s / sum : 0.0f;
  } else {
    const float base = p.renormalize ? wave_max(chosen) : 0.0f;
    w = id >= 0 ? small_sigmoid(chosen, base) : 0.0f;
    if (p.renormalize) {
      const float sum = wave_sum(w);
      w = id >= 0 ? w / sum : 0.0f;
    }
  }
  w = id >= 0 ? w * p.scale : 0.0f;
  if (nan) w = bits_f32(0x7fc00000u);
  if (lane < p.top_k) {
    p.ids[t * p.top_k + lane] = id;
    p.weights[t * p.top_k + lane] = w;
  }
}

// With p the chosen scores' shares (renormalised) or the scores: softmax
// dz_e = s_e (ds_e - sum ds s), which is 0 off the choice when renormalised;
// sigmoid dz = ds s (1 - s).
template <typename T, int EPL>
__global__ void __launch_bounds__(64 * kWaves) route_backward_kernel(const RouteBwdParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const T* row = (const T*)p.x + t * p.ld;
  float z[EPL];
  float top = -__builtin_inff();
  bool nan = false;
  const bool softmax = p.score == Q4_SCORE_SOFTMAX;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    z[i] = e < p.E ? to_f32(row[e]) : -__builtin_inff();
    nan |= z[i] != z[i];
    top = z[i] > top ? z[i] : top;
  }
  nan = __any(nan);
  top = wave_max(top);
  nan |= softmax && top == __builtin_inff();
  int32_t id = -1;
  float g = 0.0f;
  if (lane < p.top_k) {
    id = p.ids[t * p.top_k + lane];
    g = p.g[t * p.top_k + lane] * p.scale;
  }
  nan |= __any(id >= p.E);
  if (id >= p.E) id = -1;
  if (id < 0) g = 0.0f;  // an empty slot's gradient is none, whatever stands there
  const float zc = id >= 0 ? to_f32(row[id]) : -__builtin_inff();
  // every lane's slot j: the gradient of the chosen logit
  float dz = 0.0f, share_sum = 0.0f, denom = 1.0f;
  if (p.renormalize) {
    float s, rest;
    const float base = wave_max(zc);
    if (softmax) {
      s = zc > -__builtin_inff() ? exp_full(zc - base) : 0.0f;
      rest = 1.0f;
    } else {
      s = id >= 0 ? small_sigmoid(zc, base) : 0.0f;
      rest = id >= 0 ? sigmoid(-zc) : 0.0f;  // 1 - s without its cancellation
    }
    const float sum = wave_sum(s);
    const float share = sum > 0.0f ? s / sum : 0.0f;
    const float mean = wave_sum(share != 0.0f ? g * share : 0.0f);
    dz = share != 0.0f ? share * rest * (g - mean) : 0.0f;
  } else if (softmax) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += z[i] > -__builtin_inff() ? exp_full(z[i] - top) : 0.0f;
    denom = wave_sum(sum);
    const float s = zc > -__builtin_inff() ? exp_full(zc - top) / denom : 0.0f;
    share_sum = wave_sum(s != 0.0f ? g * s : 0.0f);
  } else {
    dz = id >= 0 ? g * sigmoid(zc) * sigmoid(-zc) : 0.0f;
  }
  float out[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) out[i] = 0.0f;
  const bool spread = softmax && !p.renormalize;
  for (int j = 0; j < p.top_k; ++j) {
    const int32_t at = __shfl(id, j, 64);
    const float v = __shfl(spread ? g : dz, j, 64);
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] += at == i * 64 + lane ? v : 0.0f;
  }
  T* dst = (T*)p.dx + t * p.ldd;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    float v = out[i];
    if (spread) {
      const float s = z[i] > -__builtin_inff() ? exp_full(z[i] - top) / denom : 0.0f;
      v = s != 0.0f ? s * (v - share_sum) : 0.0f;
    }
    if (nan) v = bits_f32(0x7fc00000u);
    if (e < p.E) dst[e] = from_f32<T>(v);
  }
}

template <typename T, int EPL>
hipError_t route_of(const RouteParams& p, dim3 grid, hipStream_t s) {
  if (p.bias)
    hipLaunchKernelGGL((route_kernel<T, EPL, true>), grid, dim3(64 * kWaves), 0, s, p);
  else
    hipLaunchKernelGGL((route_kernel<T, EPL, false>), grid, dim3(64 * kWaves), 0, s, p);
  return hipGetLastError();
}
template <typename T, int EPL>
hipError_t route_of(const RouteBwdParams& p, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((route_backward_kernel<T, EPL>), grid, dim3(64 * kWaves), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename P>
hipError_t by_experts(const P& p, hipStream_t s) {
  const dim3 grid((uint32_t)((p.T + kWaves - 1) / kWaves));
  if (p.E <= 64) return route_of<T, 1>(p, grid, s);
  if (p.E <= 128) return route_of<T, 2>(p, grid, s);
  if (p.E <= 256) return route_of<T, 4>(p, grid, s);
  if (p.E <= 512) return route_of<T, 8>(p, grid, s);
  return route_of<T, 16>(p, grid, s);
}

template <typename P>
hipError_t by_type(const P& p, int32_t dtype, hipStream_t s) {
  switch (dtype) {
    case Q4_DTYPE_F32: return by_experts<float>(p, s);
    case Q4_DTYPE_F16: return by_experts<_Float16>(p, s);
    default: return by_experts<bf16>(p, s);
  }
}

}  // namespace

hipError_t launch_route(const RouteParams& p, int32_t dtype, hipStream_t s) {
  return by_type(p, dtype, s);
}
hipError_t launch_route_backward(const RouteBwdParams& p, int32_t dtype, hipStream_t s) {
  return by_type(p, dtype, s);
}

}  // namespace q4
