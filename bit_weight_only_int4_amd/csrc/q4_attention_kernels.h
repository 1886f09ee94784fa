// q4_attention_kernels.h -- attention of new tokens over the paged 8-bit
// cache, few query rows per workgroup.
//
//   out[t, h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j - max)
//
// Mathematics.  Keys and values are int8 codes with one scale per page, so
// both contractions run on the integer matrix unit without unpacking a code.
// A query row is held as X 2^-e with X an integer of ND signed 8-bit digits,
// X = sum_i d_i 256^i: ND exact int32 dot products q . k per score, joined in
// fp32.  The probabilities of a tile of 64 tokens are held the same way
// against the tile's own largest (which is 1 for the largest score): the
// tile's contribution is an exact integer sum, and running maximum, sum and
// output are fp32.
//
// Digits.  An element's own rounding is relative to itself, a digit's step to
// the row's largest element (the tile's largest probability), so digits have
// to reach past the type's bits by what elements lie apart: 16-bit queries
// take three (23 bits), fp32 ones four (31).  With one fewer, which was
// measured first, a query channel 200 times the others cost 16-bit outputs
// 3e-3 of themselves and fp32 ones 2e-5, a first token with nine tenths of the
// weight and no value 5e-3 and 2e-5; now 2e-5 and 5e-8, 2e-5 and 8e-8.  Its
// price is in the prompt chunks, which the vector unit bounds (2890 tokens
// over up to 5441: bf16 217 to 267 us, fp32 283 to 338); decode steps wait for
// memory (64 sequences of 500 to 8000: 78 to 79).
//
// Layout.  A wave holds 16 query rows as the columns of both products:
// S^T = K Q^T gives lane l the scores of column l % 16 for 4 rows of each of
// 4 key tiles, O^T = V^T P^T wants from it 16 consecutive tokens.  Reading
// key row r of tile a from token 16 (r / 4) + 4 a + r % 4 makes these the
// same 16 tokens (16 g .. 16 g + 15, g = l / 16), so the probabilities go
// from one product to the next in registers, and a lane's 16 bytes of V lie
// together because the cache keeps tokens innermost.  A column's maximum
// and sum need two exchanges between the four lane groups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "q4_kv.h"
#include "q4_serve.h"
#include "q4_serve_device.h"

namespace q4 {
namespace attn {

constexpr int kTile = 64;   // tokens per step of a wave
constexpr int kWaves = 4;   // waves of a workgroup, each over its own tiles
constexpr int kRows = 16;   // query rows of a workgroup
constexpr int kThreads = 64 * kWaves;

// largest integer that ND digits hold with the offsets of pack_digits
template <int ND>
__device__ __forceinline__ constexpr float digit_max() {
  return ND == 4 ? 2130706432.0f : 8323072.0f;  // 127 * 256^(ND - 1)
}
template <int ND>
__device__ __forceinline__ constexpr uint32_t digit_bias() {
  return ND == 4 ? 0x808080u : 0x8080u;
}

// Digits of four integers, each given as X + digit_bias: word i holds digit i
// of the four.  With the bias added, byte i of the sum is d_i + 128 for all
// but the top digit, and flipping its top bit gives d_i.
template <int ND>
__device__ __forceinline__ void pack_digits(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3,
                                            uint32_t (&w)[ND]) {
  const uint32_t lo = __builtin_amdgcn_perm(b1, b0, 0x05010400u);
  const uint32_t hi = __builtin_amdgcn_perm(b3, b2, 0x05010400u);
  w[0] = __builtin_amdgcn_perm(hi, lo, 0x05040100u) ^ 0x80808080u;
  w[1] = __builtin_amdgcn_perm(hi, lo, 0x07060302u) ^ 0x80808080u;
  const uint32_t l2 = __builtin_amdgcn_perm(b1, b0, 0x07030602u);
  const uint32_t h2 = __builtin_amdgcn_perm(b3, b2, 0x07030602u);
  w[2] = __builtin_amdgcn_perm(h2, l2, 0x05040100u);
  if constexpr (ND == 4) {
    w[2] ^= 0x80808080u;
    w[3] = __builtin_amdgcn_perm(h2, l2, 0x07060302u);
  }
}

// x (0 <= x <= digit_max + 1/2) to the nearest integer, with digit_bias added.
// Below 2^24 the sum with 2^23 and the bias holds it in the low bits.
template <int ND>
__device__ __forceinline__ uint32_t digit_bits(float p, float to_digits) {
  if constexpr (ND == 4)
    return (uint32_t)(int)__builtin_rintf(p * to_digits) + digit_bias<ND>();
  else
    return f32_bits(__builtin_fmaf(p, to_digits, 8388608.0f + (float)digit_bias<ND>()));
}

// sum_i acc_i 256^i in fp32.  The digit sums are below 2^22 in magnitude (64
// or 256 products of at most 2^14), so that two neighbours join exactly.
template <int ND>
__device__ __forceinline__ float join_digits(const int32_t (&a)[ND]) {
  const float low = (float)(a[1] * 256 + a[0]);
  if constexpr (ND == 4) return __builtin_fmaf((float)(a[3] * 256 + a[2]), 65536.0f, low);
  return __builtin_fmaf((float)a[2], 65536.0f, low);
}

// Over the four lanes that hold a column, l % 16 apart: the rows of 16 lanes
// change places in pairs, then the halves.
template <typename F>
__device__ __forceinline__ uint32_t column_fold(uint32_t x, F f) {
  auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = f(r[0], r[1]);
  r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return f(r[0], r[1]);
}
__device__ __forceinline__ float column_max(float x) {
  return bits_f32(column_fold(f32_bits(x), [](uint32_t a, uint32_t b) {
    return f32_bits(fmaxf(bits_f32(a), bits_f32(b)));
  }));
}
__device__ __forceinline__ float column_sum(float x) {
  return bits_f32(column_fold(f32_bits(x), [](uint32_t a, uint32_t b) {
    return f32_bits(bits_f32(a) + bits_f32(b));
  }));
}
__device__ __forceinline__ uint32_t column_umax(uint32_t x) {
  return column_fold(x, [](uint32_t a, uint32_t b) { return umax(a, b); });
}

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int32_t dtype) {
  if (dtype == Q4_DTYPE_F32) return ((const float*)p)[i];
  if (dtype == Q4_DTYPE_F16) return (float)((const _Float16*)p)[i];
  return (float)((const bf16*)p)[i];
}
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v, int32_t dtype) {
  if (dtype == Q4_DTYPE_F32) ((float*)p)[i] = v;
  else if (dtype == Q4_DTYPE_F16) ((_Float16*)p)[i] = (_Float16)v;
  else ((bf16*)p)[i] = (bf16)v;
}

// What a workgroup works on, the same for the attention and the join kernel.
struct Block {
  SeqSpan sp;
  int b, h;
  int64_t row0, rows;  // first query row (token * group + head) and the sequence's rows to compute
  int tile0, tiles;    // tiles of 64 positions that its queries see
  KeyRange keys;
};

// The token of a query row: rows are below 2^31 + 128, and a division of 64
// bits takes a hundred instructions on the way to the first key.
__device__ __forceinline__ int64_t row_token(const AttnParams& p, int64_t row) {
  return (uint32_t)row / (uint32_t)p.group;
}

__device__ __forceinline__ Block block_of(const AttnParams& p, int b, int h, int rb) {
  Block k;
  k.h = h;
  k.b = b;
  k.sp = seq_span(p.c.cu_new, p.c.lengths, k.b, p.T);
  // of a sequence with more than max_new tokens, its last block holds rows past it
  const int64_t rows = (int64_t)k.sp.n * p.group;
  k.rows = rows < p.max_rows ? rows : p.max_rows;
  k.row0 = (int64_t)rb * p.block_rows;
  const int64_t last = k.row0 + p.block_rows < k.rows ? k.row0 + p.block_rows : k.rows;
  k.keys = key_range(k.sp.pos0 + row_token(p, k.row0),
                     k.sp.pos0 + row_token(p, last > 0 ? last - 1 : 0), p.window, p.max_len);
  k.tile0 = (int)(k.keys.lo / kTile);
  k.tiles = k.keys.hi > k.keys.lo ? (int)((k.keys.hi + kTile - 1) / kTile) - k.tile0 : 0;
  return k;
}

// The page that holds the 16 tokens at token0 (a multiple of 16) of the
// sequence, given its table entry: -1 if it is not in the cache, -2 if no query
// sees them.
__device__ __forceinline__ int32_t segment_page(const AttnParams& p, int32_t raw,
                                                const KeyRange& keys, int64_t token0) {
  const int32_t page = page_checked(raw, p.c.max_pages, p.c.pages, token0 >> p.c.page_log2);
  return token0 + 16 <= keys.lo || token0 >= keys.hi ? -2 : page;
}

// A page's scale in its keys' scores: one that is not finite has to show, and an
// infinite one would make some of them -inf, weights of 0.
__device__ __forceinline__ float key_scale(float s) {
  return s < __builtin_inff() ? scale_or_nan(s) : bits_f32(0x7fc00000u);
}

// A lane's pages of a tile: of the keys that it loads, and of its 16 tokens
// (the same where one page covers the tile; then it has a token that is seen).
struct Pages {
  int32_t key, own;
};

template <bool UNIFORM>
__device__ __forceinline__ Pages load_pages(const AttnParams& p, const int32_t* table,
                                            int64_t token0) {
  const int lane = threadIdx.x & 63;
  Pages r;
  r.own = page_raw(table, p.c.max_pages,
                   (token0 + (UNIFORM ? 0 : 16 * (lane >> 4))) >> p.c.page_log2);
  r.key = UNIFORM ? r.own
                  : page_raw(table, p.c.max_pages,
                             (token0 + 16 * ((lane & 15) >> 2)) >> p.c.page_log2);
  return r;
}

template <bool UNIFORM>
__device__ __forceinline__ Pages check_pages(const AttnParams& p, const Pages& raw,
                                             const KeyRange& keys, int64_t token0) {
  const int lane = threadIdx.x & 63;
  Pages r;
  if (UNIFORM) {
    r.own = r.key = page_checked(__builtin_amdgcn_readfirstlane(raw.own), p.c.max_pages, p.c.pages,
                                 token0 >> p.c.page_log2);
  } else {
    r.own = segment_page(p, raw.own, keys, token0 + 16 * (lane >> 4));
    r.key = segment_page(p, raw.key, keys, token0 + 16 * ((lane & 15) >> 2));
  }
  return r;
}

// Elements d0 .. d0 + 15 of a query row as fp32, 16 bytes at a time where the
// rows allow it.
__device__ __forceinline__ void load_row16(const AttnParams& p, int64_t at, float (&x)[16]) {
  if (p.q_vec && p.dtype == Q4_DTYPE_F32) {
    const f32x4* s = (const f32x4*)((const float*)p.q + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 v = s[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * i + e] = v[e];
    }
  } else if (p.q_vec) {
    const u32x4v* s = (const u32x4v*)((const uint16_t*)p.q + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4v v = s[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t b = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        x[8 * i + e] = p.dtype == Q4_DTYPE_F16 ? (float)__builtin_bit_cast(_Float16, b)
                                               : bits_f32((uint32_t)b << 16);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = load_elem(p.q, at + e, p.dtype);
  }
}

// A query row's digits, elements 64 s + 16 g .. + 15 in the lane (zero past
// the head and for rows that do not exist), and the factor that takes a
// digit product to a score in log2 units, >= 0: a negative softmax scale goes
// into the digits, so that the largest product is the largest score.  A row
// with NaN or infinity gets a NaN factor.
template <int NS, int ND>
__device__ __forceinline__ float row_digits(const AttnParams& p, int64_t at, bool valid, int g,
                                            i32x4 (&qd)[NS][ND]) {
  const int dim = p.c.dim;
  uint32_t amax = 0;
  float x[NS][16];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int d = 64 * s + 16 * g;
    if (valid && d < dim) {
      load_row16(p, at + d, x[s]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[s][e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = umax(amax, abs_bits(x[s][e]));
  }
  amax = column_umax(amax);
  // the power of two that takes the largest element below digit_max
  const float a = bits_f32(amax);
  const int ex = __builtin_amdgcn_frexp_expf(a);  // a = m 2^ex, m in [1/2, 1)
  const float m = __builtin_amdgcn_frexp_mantf(a);
  const int up = amax == 0 ? 0 : 8 * ND - 1 - ex - (m > 127.0f / 128.0f ? 1 : 0);
  const float sign = p.scale_log2 < 0.0f ? -1.0f : 1.0f;
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t bits[4], out[ND];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        bits[e] = (uint32_t)(int)__builtin_rintf(
                      __builtin_amdgcn_ldexpf(sign * x[s][4 * w + e], up)) +
                  digit_bias<ND>();
      pack_digits<ND>(bits[0], bits[1], bits[2], bits[3], out);
#pragma unroll
      for (int i = 0; i < ND; ++i) qd[s][i][w] = (int32_t)out[i];
    }
  return amax >= 0x7f800000u ? bits_f32(0x7fc00000u)
                             : __builtin_amdgcn_ldexpf(__builtin_fabsf(p.scale_log2), -up);
}

// Running state of a column (query row): maximum in log2 units, the lane's
// part of the sum, the lane's part of the outputs (4 of every 16 elements).
template <int DT>
struct Column {
  float mx, sum;
  float o[DT][4];
};

template <int DT>
__device__ __forceinline__ void column_init(Column<DT>& c) {
  c.mx = -__builtin_inff();
  c.sum = 0.0f;
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) c.o[t][i] = 0.0f;
}

// Scores of one 64-token tile, as digit products: sc[a][i] is token
// 16 g + 4 a + i of the tile.
template <int NS, int ND>
__device__ __forceinline__ void tile_scores(const i32x4 (&kd)[4][NS], const i32x4 (&qd)[NS][ND],
                                            float (&sc)[4][4]) {
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    i32x4 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      acc[i] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < NS; ++s)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(kd[a][s], qd[s][i], acc[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int32_t part[ND];
#pragma unroll
      for (int n = 0; n < ND; ++n) part[n] = acc[n][i];
      sc[a][i] = join_digits<ND>(part);
    }
  }
}

// Scores to probability digits.  unit: score per digit product (>= 0, or
// NaN); lo, hi: first and last of the tile's tokens that the row sees,
// relative to the lane's first (MASK only); vs: the values' scale.  Updates
// maximum and sum; alpha is what the outputs so far are multiplied by, w what
// the tile's digit products are worth.
// UNIFORM: one page covers the tile.  Else its pages' scales join the
// probabilities before these become digits.
template <int ND, bool MASK, bool UNIFORM>
__device__ __forceinline__ void tile_softmax(float (&sc)[4][4], float unit, float vs, int lo, int hi,
                                             float& mx, float& sum, i32x4 (&pd)[ND], float& alpha,
                                             float& w) {
  const float inf = __builtin_inff();
  float top = -inf;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 4 * a + i;
      sc[a][i] *= unit;
      if (MASK) sc[a][i] = j >= lo && j <= hi ? sc[a][i] : -inf;
      top = fmaxf(top, sc[a][i]);
    }
  top = column_max(top);
  const bool any = top > -inf;  // not: nothing seen, or NaN scores only
  const float ref = any ? top : 0.0f;
  float part = 0.0f, big = 1.0f;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sc[a][i] = exp2_fast(sc[a][i] - ref);  // 0 where not seen
      part += sc[a][i];
    }
  uint32_t wmax = 0;
  if (!UNIFORM) {
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 4 * a + i;
        sc[a][i] = !MASK || (j >= lo && j <= hi) ? sc[a][i] * vs : 0.0f;
        wmax = umax(wmax, abs_bits(sc[a][i]));
      }
    wmax = column_umax(wmax);
    big = fmaxf(bits_f32(wmax), 1e-30f);  // below it, digits run out
  }
  const float to_digits = UNIFORM ? digit_max<ND>() : digit_max<ND>() / big;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    uint32_t bits[4], out[ND];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      bits[i] = digit_bits<ND>(sc[a][i], to_digits);
    pack_digits<ND>(bits[0], bits[1], bits[2], bits[3], out);
#pragma unroll
    for (int i = 0; i < ND; ++i) pd[i][a] = (int32_t)out[i];
  }
  const float m_new = fmaxf(mx, top);
  const float m_ref = m_new > -inf ? m_new : 0.0f;
  alpha = exp2_fast(mx - m_ref);  // 0 before the first tile with a maximum
  const float beta = any ? exp2_fast(top - m_ref) : 0.0f;
  mx = m_new;
  // a tile of NaN scores has no maximum: its sum, NaN, still has to show
  sum = sum * alpha + (any || part == part ? beta * part : part);
  // a scale that is not finite reaches the rows that see it, and no others
  const float worth = UNIFORM ? vs : wmax >= 0x7f800000u ? bits_f32(wmax) : big;
  w = any ? beta * worth * (1.0f / digit_max<ND>()) : 0.0f;
}

// Adds a tile's values: o = o alpha + w (V^T digits).
template <int DT, int ND>
__device__ __forceinline__ void tile_values(const i32x4 (&vd)[DT], const i32x4 (&pd)[ND],
                                            float alpha, float w, float (&o)[DT][4]) {
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) {
    i32x4 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
      acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vd[dt], pd[i], i32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int32_t part[ND];
#pragma unroll
      for (int n = 0; n < ND; ++n) part[n] = acc[n][i];
      o[dt][i] = __builtin_fmaf(join_digits<ND>(part), w, o[dt][i] * alpha);
    }
  }
}

// A tile's operands: keys, values, the lane's scales, and whether its page is
// in the cache (else the scales stand for NaN).
template <int NS, int DT>
struct Tile {
  i32x4 kd[4][NS], vd[DT];
  float ks, vs;
  bool k_in, v_in;
};

// A wave's tiles t, t + step, ... below t_end of a block's keys, into the
// lane's column state.  The next tile's keys and page numbers load while this
// one's scores become probabilities, its values while its scores form.  Two or
// three waves share a SIMD.  One wave per SIMD with whole tiles in two register
// buffers took 93 us where this took 84 (three digits, 64 sequences of 500 to
// 8000 tokens, 8 kv heads of 128).
template <int DT, int ND, bool UNIFORM>
__device__ __forceinline__ void attend(const AttnParams& p, const Block& k, int t, int t_end,
                                       int step, Column<DT>& st) {
  constexpr int NS = (DT + 3) / 4;  // steps of 64 elements of a head
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const KvCache& c = p.c;
  const int dim = c.dim, d16 = dim >> 4;
  const int32_t* table = c.table + (int64_t)k.b * c.table_ld;
  const int page_mask = c.page - 1;
  const float nan = bits_f32(0x7fc00000u);
  auto first_token = [&](int tile) { return (int64_t)(k.tile0 + tile) * kTile; };
  // Addresses are a 64-bit base of the page, of the wave where one page covers
  // the tile, and 32-bit offsets of the lane in it that do not change.
  uint32_t k_off[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int d = 64 * s + 16 * g;
    k_off[s] = (uint32_t)(((UNIFORM ? 16 * (col >> 2) : 0) + (col & 3)) * dim + (d < dim ? d : 0));
  }
  const uint32_t v_off = (uint32_t)((col << c.page_log2) + (UNIFORM ? 16 * g : 0));
  // What is not seen, or not in the cache, is read from page 0: its scores are
  // masked, or NaN by their scale.  Scales load first: they are needed first.
  auto load_keys = [&](int tile, const Pages& pg, Tile<NS, DT>& o) {
    const int slot = (int)((first_token(tile) + (UNIFORM ? 0 : 16 * (col >> 2))) & page_mask);
    o.k_in = pg.own >= 0;
    o.ks = c.ks[(int64_t)(pg.own > 0 ? pg.own : 0) * c.heads + k.h];
    const int8_t* base =
        c.k + ((((int64_t)(pg.key > 0 ? pg.key : 0) * c.heads + k.h) << c.page_log2) + slot) * dim;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int s = 0; s < NS; ++s) o.kd[a][s] = *(const i32x4*)(base + 4 * a * dim + k_off[s]);
  };
  auto load_values = [&](int tile, const Pages& pg, Tile<NS, DT>& o) {
    const int64_t ph = (int64_t)(pg.own > 0 ? pg.own : 0) * c.heads + k.h;
    o.v_in = pg.own >= 0;
    o.vs = c.vs[ph];
    const int8_t* v = c.v + ph * ((int64_t)dim << c.page_log2) +
                      ((first_token(tile) + (UNIFORM ? 0 : 16 * g)) & page_mask);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
      o.vd[dt] = *(const i32x4*)(v + ((dt < d16 ? 16 * dt : 0) << c.page_log2) + v_off);
  };
  Tile<NS, DT> cur;
  column_init(st);
  if (t >= t_end) return;
  // pages of the tile at hand, and the table entries of the next
  Pages pg = check_pages<UNIFORM>(p, load_pages<UNIFORM>(p, table, first_token(t)), k.keys,
                                  first_token(t));
  load_keys(t, pg, cur);
  Pages raw = load_pages<UNIFORM>(p, table, first_token(t + step));

  // the lane's query row and the positions it sees
  const int64_t r = k.row0 + col;
  const bool valid = r < k.rows;
  const int64_t tok = valid ? row_token(p, r) : 0;
  const int head = k.h * p.group + (int)(valid ? r - tok * p.group : 0);
  const int64_t pos = valid ? k.sp.pos0 + tok : -1;
  const int64_t see_lo64 = p.window > 0 ? pos - p.window + 1 : 0;
  const int64_t see_hi = pos < k.keys.hi ? pos : k.keys.hi - 1;  // last position seen
  const int64_t see_lo = see_lo64 > 0 ? see_lo64 : 0;
  // positions that every row of the block sees
  const int64_t last_row = (k.row0 + kRows < k.rows ? k.row0 + kRows : k.rows) - 1;
  const int64_t pos_first = k.sp.pos0 + row_token(p, k.row0);
  const int64_t pos_last = k.sp.pos0 + row_token(p, last_row);
  const int64_t all_hi = pos_first < k.keys.hi ? pos_first : k.keys.hi - 1;
  const int64_t all_lo = p.window > 0 ? pos_last - p.window + 1 : 0;

  i32x4 qd[NS][ND];
  const float q_unit = row_digits<NS, ND>(
      p, (k.sp.t0 + tok) * p.q_ts + (int64_t)head * p.q_hs, valid, g, qd);

  // The last tile apart: with the loads of a next tile under a condition every
  // wait for this one's values would wait for them as well.
  auto one_tile = [&](auto more) {
    const int64_t token0 = first_token(t);
    load_values(t, pg, cur);
    float sc[4][4];
    tile_scores<NS, ND>(cur.kd, qd, sc);
    const float unit = q_unit * (cur.k_in ? key_scale(cur.ks) : nan);
    const float vs = cur.v_in ? scale_or_nan(cur.vs) : nan;
    if constexpr (decltype(more)::value) {
      pg = check_pages<UNIFORM>(p, raw, k.keys, first_token(t + step));
      load_keys(t + step, pg, cur);
      raw = load_pages<UNIFORM>(p, table, first_token(t + 2 * step));
    }
    i32x4 pd[ND];
    float alpha, w;
    if (token0 >= all_lo && token0 + kTile - 1 <= all_hi) {
      tile_softmax<ND, false, UNIFORM>(sc, unit, vs, 0, 0, st.mx, st.sum, pd, alpha, w);
    } else {
      const int64_t base = token0 + 16 * g;
      const int lo = (int)(see_lo - base > 16 ? 16 : see_lo - base < 0 ? 0 : see_lo - base);
      const int hi = (int)(see_hi - base < -1 ? -1 : see_hi - base > 15 ? 15 : see_hi - base);
      tile_softmax<ND, true, UNIFORM>(sc, unit, vs, lo, hi, st.mx, st.sum, pd, alpha, w);
    }
    tile_values<DT, ND>(cur.vd, pd, alpha, w, st.o);
  };
  for (; t + step < t_end; t += step) one_tile(std::true_type{});
  one_tile(std::false_type{});
}

// Joins the parts of a workgroup's waves through LDS and writes them: finished
// (`whole`), or as partial outputs from row `first` of the workspace on, a row
// for each of token * heads + head.  lds: W * 16 (16 DT + 6) floats.
template <int DT, int W>
__device__ __forceinline__ void join_waves(const AttnParams& p, const Block& k, const Column<DT>& st,
                                           float* lds, bool whole, int64_t first) {
  const int wave = threadIdx.x >> 6, col = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
  const int dim = p.c.dim;
  // [wave][row][dim] outputs, then maxima and sums
  const float sum = column_sum(st.sum);
  constexpr int pitch = 16 * DT + 4;
  float* lo = lds;
  float* lm = lds + W * kRows * pitch;
  float* ls = lm + W * kRows;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
    *(f32x4*)&lo[(wave * kRows + col) * pitch + 16 * dt + 4 * g] =
        f32x4{st.o[dt][0], st.o[dt][1], st.o[dt][2], st.o[dt][3]};
  if (g == 0) {
    lm[wave * kRows + col] = st.mx;
    ls[wave * kRows + col] = sum;
  }
  __syncthreads();
  // 4 W threads a row, 4 elements a step
  const int row = threadIdx.x / (4 * W), sub = threadIdx.x % (4 * W);
  const int64_t rr = k.row0 + row;
  if (rr >= k.rows) return;
  float m = lm[row];
#pragma unroll
  for (int i = 1; i < W; ++i) m = fmaxf(m, lm[i * kRows + row]);
  const float ref = m > -__builtin_inff() ? m : 0.0f;
  float f[W], den = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    f[i] = exp2_fast(lm[i * kRows + row] - ref);
    // a wave without a maximum has a sum of 0, or NaN, which has to show
    const float si = ls[i * kRows + row];
    den += si != si ? si : f[i] * si;
  }
  const int64_t tk = row_token(p, rr);
  const int64_t tq = k.sp.t0 + tk, hq = k.h * p.group + (rr - tk * p.group);
  const int64_t at = first + tq * p.heads + hq;
  const float inv = den == 0.0f ? 0.0f : 1.0f / den;  // no key seen: 0
  for (int d = 4 * sub; d < dim; d += 16 * W) {
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < W; ++i)
      acc += f[i] * *(const f32x4*)&lo[(i * kRows + row) * pitch + d];
    if (whole) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        store_elem(p.out, tq * p.o_ts + hq * p.o_hs + d + e, acc[e] * inv, p.dtype);
    } else {
      *(f32x4*)&p.part_o[at * dim + d] = acc;
    }
  }
  if (!whole && sub == 0) {
    p.part_ml[2 * at] = m;
    p.part_ml[2 * at + 1] = den;
  }
}

// One workgroup: 16 query rows of one kv head, one split of their keys, the
// tiles dealt to its W waves in turn and joined through LDS.
template <int DT, int ND, int W, bool UNIFORM>
__global__ __launch_bounds__(64 * W, DT <= 4 && W == 4 ? 3 : DT <= 8 ? 2 : 1) void attention_kernel(AttnParams p) {
  extern __shared__ float lds[];
  // Heads vary fastest, then sequences, row blocks and splits: consecutive
  // workgroups go to the 8 XCDs in turn, so that neither the sequences' lengths
  // nor the splits that the short ones do not need load one XCD more than
  // another, and the row blocks of a head share an L2 where there are 8 heads.
  // The last splits, which only long sequences have, come first, so that these
  // do not end alone (32 sequences of 450 to 9000 tokens: 58 to 53 us).
  uint32_t id = blockIdx.x;
  const int h = id % p.c.heads;
  id /= p.c.heads;
  const int b = id % p.batch;
  id /= p.batch;
  const int rb = id % p.row_blocks, split = p.splits - 1 - (int)(id / p.row_blocks);
  const Block k = block_of(p, b, h, rb);
  if (k.row0 >= k.rows) return;
  // a block whose tiles fit one split writes its output itself
  const int n_splits = (k.tiles + p.split_tiles - 1) / p.split_tiles;
  if (split > 0 && split >= n_splits) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t_end = (split + 1) * p.split_tiles < k.tiles ? (split + 1) * p.split_tiles : k.tiles;
  Column<DT> st;
  attend<DT, ND, UNIFORM>(p, k, split * p.split_tiles + wave, t_end, W, st);
  join_waves<DT, W>(p, k, st, lds, n_splits <= 1, split * p.T * p.heads);
}

}  // namespace attn
}  // namespace q4
