// rows.cuh -- which keys the rows of a tree of drafted tokens, or of a padded
// batch, see.
//
// Request b has n new tokens (own_lens[b], or q_len), the last of its L tokens;
// rows t >= n are padding and see nothing.  With a mask, new token t sees the
// keys before the new tokens, j < L - n, and of the new ones those whose bit is
// set: key L - n + i where bit i % 32 of word i / 32 of its row is.  Without one
// every own row sees every key (cross attention).
#pragma once

#include <limits.h>

#include "decode_attn.h"
#include "kernels.cuh"

namespace dattn {

// The rows of one request.
struct OwnRows {
  int n;                  // own rows; the others are padding
  int base;               // keys from here on go by the mask (INT_MAX: none does)
  const uint32_t* mask;   // this request's rows
  int words;

  // Bits of keys j .. j + 31 for row t, for j > base - 32: bit i is set where it
  // sees key j + i.  (Bits past the last new token say nothing.)
  __device__ __forceinline__ uint32_t bits(int t, int j) const {
    const uint32_t* row = mask + static_cast<int64_t>(t) * words;
    const int at = j - base;  // > -32
    const int w = at >> 5;
    const uint32_t lo = w < 0 ? 0xffffffffu : w < words ? __ldg(row + w) : 0u;
    const uint32_t hi = w + 1 < words ? __ldg(row + w + 1) : 0u;
    return __funnelshift_r(lo, hi, at & 31);
  }
  __device__ __forceinline__ bool sees(int t, int j) const {
    const int at = j - base;
    return at < 0 || ((at >> 5) < words && ((__ldg(mask + static_cast<int64_t>(t) * words + (at >> 5)) >> (at & 31)) & 1u) != 0);
  }
};

// The rows of request b of (clamped) length L and `own` rows as given; `report` (one thread per request)
// sets the status bits.
__device__ __forceinline__ OwnRows own_rows(const RowArgs& r, int q_len, int b, int L, int own, bool report,
                                            int32_t* status) {
  OwnRows o;
  o.n = own;
  uint32_t bad = 0;
  if (own < 0 || own > q_len) {
    bad |= DA_STATUS_SEQ_LEN;
    o.n = own < 0 ? 0 : q_len;
  }
  o.base = INT_MAX;
  o.mask = nullptr;
  o.words = r.words;
  if (r.mask != nullptr) {
    o.base = L - o.n;
    o.mask = r.mask + b * r.mask_sb;
    if (o.base < 0) bad |= DA_STATUS_SHORT_CAUSAL;
  }
  if (report && bad != 0 && status != nullptr) atomicOr(status, static_cast<int32_t>(bad));
  return o;
}

__device__ __forceinline__ OwnRows own_rows(const RowArgs& r, int q_len, int b, int L, bool report, int32_t* status) {
  return own_rows(r, q_len, b, L, r.own_lens != nullptr ? __ldg(r.own_lens + b) : q_len, report, status);
}

}  // namespace dattn
