// q4_kv.h -- index arithmetic of the paged cache, shared by the append and
// attention kernels and compiled for the host by the tests: which tokens a
// sequence has, where a position lies, and the checks that keep every access
// inside the arrays whatever the device-side tables hold.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define Q4_HD __host__ __device__ __forceinline__
#else
#define Q4_HD inline
#endif

namespace q4 {

// Sequence b's part of a call: new tokens t0 .. t0 + n - 1 of T, at positions
// pos0 .. len - 1.  A table that decreases or leaves [0, T] gives n = 0, a
// negative length is 0.  pos0 may be negative (fewer tokens than new ones):
// those tokens have no place.
struct SeqSpan {
  int32_t t0, n, len, pos0;
};

Q4_HD SeqSpan seq_span(const int32_t* cu_new, const int32_t* lengths, int64_t b, int64_t T) {
  SeqSpan s;
  const int64_t lo = cu_new[b], hi = cu_new[b + 1];
  const bool ok = lo >= 0 && hi >= lo && hi <= T;
  s.t0 = ok ? (int32_t)lo : 0;
  s.n = ok ? (int32_t)(hi - lo) : 0;
  s.len = lengths[b] > 0 ? lengths[b] : 0;
  s.pos0 = s.len - s.n;
  return s;
}

// The page number at entry `index` of a sequence's table row, or -1 if the
// entry lies past the table or its page outside the cache, in two steps: the
// load, which any index may make (max_pages >= 1), and the check, which the
// kernels put off until they need the page, as a use right after a load would
// wait for it and for every load before it.
Q4_HD int32_t page_raw(const int32_t* row, int64_t max_pages, int64_t index) {
  return row[index < 0 ? 0 : index < max_pages ? index : max_pages - 1];
}
Q4_HD int32_t page_checked(int32_t raw, int64_t max_pages, int64_t pages, int64_t index) {
  return (index >= 0 && index < max_pages && raw >= 0 && raw < pages) ? raw : -1;
}
Q4_HD int32_t page_at(const int32_t* row, int64_t max_pages, int64_t pages, int64_t index) {
  return page_checked(page_raw(row, max_pages, index), max_pages, pages, index);
}

// Pages that `n` consecutive positions can touch.
Q4_HD int64_t pages_touched(int64_t n, int64_t page) {
  return n <= 0 ? 0 : (n - 1 + page - 1) / page + 1;
}

// Whether rows of `dim` elements at a_hs * h + a_ts * t and delta + b_hs * h +
// b_ts * t (t < T, h < a_heads or b_heads; strides as the ABI admits them) have
// an element in common.  Different token strides of several tokens count as
// sharing.  Host code.
inline bool rows_share(int64_t delta, int64_t T, int64_t dim, int64_t a_ts, int64_t a_hs,
                       int64_t a_heads, int64_t b_ts, int64_t b_hs, int64_t b_heads) {
  if (T <= 0 || a_heads <= 0 || b_heads <= 0) return false;
  const int64_t a_len = (a_heads - 1) * a_hs + dim, b_len = (b_heads - 1) * b_hs + dim;
  if (T == 1) a_ts = b_ts = a_len + b_len + (delta < 0 ? -delta : delta);  // no second token in reach
  if (a_ts != b_ts) return true;
  // usually the heads of one lie between those of the other's tokens
  const int64_t in_token = ((delta % a_ts) + a_ts) % a_ts;
  if (in_token >= a_len && in_token + b_len <= a_ts) return false;
  for (int64_t a = 0; a < a_heads; ++a)
    for (int64_t b = 0; b < b_heads; ++b) {
      // tokens `near` and `near` + 1 later are the ones closest to it
      const int64_t x = delta + b * b_hs - a * a_hs;
      const int64_t near = -x / a_ts - (-x % a_ts < 0 ? 1 : 0);
      for (int64_t i = near; i <= near + 1; ++i) {
        const int64_t off = x + i * a_ts;
        if (i > -T && i < T && off > -dim && off < dim) return true;
      }
    }
  return false;
}

// Positions [lo, hi) that any of the queries at pos_min .. pos_max sees.
struct KeyRange {
  int64_t lo, hi;
};

Q4_HD KeyRange key_range(int64_t pos_min, int64_t pos_max, int64_t window, int64_t max_len) {
  KeyRange r;
  r.hi = pos_max + 1 < max_len ? pos_max + 1 : max_len;
  if (r.hi < 0) r.hi = 0;
  r.lo = window > 0 ? pos_min - window + 1 : 0;
  if (r.lo < 0) r.lo = 0;
  if (r.lo > r.hi) r.lo = r.hi;
  return r;
}

}  // namespace q4
