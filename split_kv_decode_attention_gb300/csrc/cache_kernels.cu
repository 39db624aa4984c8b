// cache_kernels.cu -- the kernels that fill a cache and digest it: the rotary
// table, the append of new tokens (rotation, conversion to the cache's type,
// scatter through the block table) and the per-page digests that the page
// selection scores.  All of them stream their data once and are bound by HBM
// at size and by launch latency in a decode step.

#include <type_traits>

#include "cache_kernels.cuh"
#include "decode_attn.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace dattn {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------------------- rotary table
// cos / sin of pos * f.  In turns the angle is pos * f / (2 pi), and only its
// fraction counts: with F = round(2^64 frac(f / 2 pi)) as an unsigned 64-bit
// integer, pos * F modulo 2^64 is that fraction, to pos * 2^-65 turns, by one
// integer multiply; the next row of a thread is an addition away.  The nearest
// quarter turn is split off exactly, and on the remainder x of at most pi / 4
// the Taylor series through x^9 and x^10 are within 3e-9 and 2e-10 of sine and
// cosine, a twentieth of an fp32 rounding.  With the roundings of x and of the
// series an entry is within 6.5 x 2^-24 of itself, plus what the angle is off:
// pos * 2^-65 turns, and 2^-57 where a zero crossing leaves only the low word,
// which fp32 rounds.  That takes 11 fp32 multiply-adds, where an fp64 cosine is two
// orders of magnitude more work (fp64 runs at 1/64 of the fp32 rate on this GPU).  The
// F of the frequencies, the only fp64 work, are made once per CTA.  (131072
// positions x 128: 14.6 us, 4.6 TB/s written, 0.69 of a copy's rate; the integer
// and polynomial work keeps the ALU 61 % busy.)
__device__ __forceinline__ uint64_t turns_fixed(double f) {
  const double kInv2PiHi = 0.15915494309189535;      // 1 / (2 pi), rounded
  const double kInv2PiLo = -9.839338337591243e-18;   // what is left of it
  const double m = fabs(f);
  const double p = m * kInv2PiHi;
  const double e = fma(m, kInv2PiHi, -p) + m * kInv2PiLo;
  const double frac = p - floor(p);                  // exact (of a negative p it would round)
  const double hi = floor(frac * 4294967296.0);
  const double lo = (frac * 4294967296.0 - hi) * 4294967296.0 + e * 18446744073709551616.0;
  const uint64_t turns = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(static_cast<int64_t>(rint(lo)));
  return f < 0.0 ? 0 - turns : turns;
}

// cos and sin of phase / 2^64 turns, times amp.
__device__ __forceinline__ void cos_sin_turns(uint64_t phase, float amp, float& c, float& s) {
  const uint32_t hi = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  // the remainder, within 2^61: its high part signed, its low part not
  const int32_t rh = static_cast<int32_t>(hi - (quarter << 30));
  const float rest = fmaf(static_cast<float>(rh), 4294967296.f,
                          static_cast<float>(static_cast<uint32_t>(phase)));
  const float x = rest * 3.4061215800865545e-19f;  // 2 pi / 2^64
  const float z = x * x;
  const float sp = fmaf(fmaf(fmaf(fmaf(z, 1.f / 362880.f, -1.f / 5040.f), z, 1.f / 120.f), z, -1.f / 6.f), z * x, x);
  const float cp = fmaf(fmaf(fmaf(fmaf(fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), z, -1.f / 720.f), z, 1.f / 24.f), z, -0.5f), z, 1.f);
  // a quarter turn on: (c, s) -> (-s, c)
  const float cc = quarter & 1 ? sp : cp, ss = quarter & 1 ? cp : sp;
  c = cc * (((quarter + 1) & 2) ? -amp : amp);
  s = ss * ((quarter & 2) ? -amp : amp);
}

constexpr int kTableThreads = 256;

// V neighbouring frequencies per thread (4 where that divides their number).
template <int V>
__global__ void __launch_bounds__(kTableThreads)
    rope_table_kernel(const double* inv_freq, int n, int64_t first, int64_t count, float amp, float* table) {
  __shared__ uint64_t step[64];
  grid_dependency_wait();
  if (threadIdx.x < n) step[threadIdx.x] = turns_fixed(inv_freq[threadIdx.x]);
  const int cols = n / V;
  const int per = kTableThreads / cols;  // rows side by side in the CTA
  const int row = threadIdx.x / cols;
  const int i = (threadIdx.x - row * cols) * V;
  __syncthreads();
  if (row >= per) return;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * per;
  int64_t r = static_cast<int64_t>(blockIdx.x) * per + row;
  uint64_t phase[V], ahead[V];
  bool ok[V];  // (frequencies that are not finite give NaN)
#pragma unroll
  for (int v = 0; v < V; ++v) {
    phase[v] = static_cast<uint64_t>(first + r) * step[i + v];
    ahead[v] = static_cast<uint64_t>(stride) * step[i + v];
    ok[v] = fabs(inv_freq[i + v]) <= 1.7976931348623157e308;
  }
  float* out = table + r * 2 * n + i;
  const int64_t ostride = stride * 2 * n;
  for (; r < count; r += stride, out += ostride) {
    float c[V], s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      cos_sin_turns(phase[v], amp, c[v], s[v]);
      if (!ok[v]) c[v] = s[v] = __int_as_float(0x7fc00000);
      phase[v] += ahead[v];
    }
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(out) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(out + n) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
      out[0] = c[0];
      out[n] = s[0];
    }
  }
}

// ------------------------------------------------------------------- append
// 16 threads hold the 128 values of a (token, head), 8 each.  A CTA works on
// one token, eight heads a pass: passes over q's heads, then k's, then v's, each
// a pointer that steps on.  A thread keeps the cos / sin of its 8 values in
// registers for all of them, so the table is read once per CTA and row of
// threads, and the pair partners of the half layout come by shuffles (a
// thread's 8 values and their partners lie rotary_dim / 2 apart, whole threads
// when that is a multiple of 8, halves of them when it is one of 4; other sizes
// read the partner from memory).
// The first passes' rows are on their way before the token's place is known.
// Instructions bound it as much as HBM does, so values go in pairs (mul /
// add.f32x2).  (8156 tokens of 32 / 8 heads into an FP8 cache: 36.7 us, 5.1
// TB/s, 0.77 of a copy's rate; a step of 256 tokens of 64 / 8 heads into a 4-bit
// one 4.4 us, of one token 4.2: the launch.)
constexpr int kAppendThreads = 128;
constexpr int kRowsPerPass = kAppendThreads / 16;

// Two fp32 values in a register pair.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// x + y, for x a product of mul2: the assembler fuses an add.rn.f32x2 with the
// mul.rn.f32x2 before it into one rounding (it leaves the scalar forms alone),
// so the sum is x * one + y with a `one` that only the launch knows.
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y, uint64_t one) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(one), "l"(y));
  return r;
}

// Two bf16 values, exactly.
__device__ __forceinline__ uint64_t widen(uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  float lo, hi;
  unpair(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  return packed_lo(e4m3x2_to_f16x2(byte), true);
}

// Eight values to E2M1 nibbles, the first in the lowest.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// The eight values of this thread (two bf16 per word) into the cache row at
// `row` (4-bit: block scales at sf_row).  All lanes of a warp call it together.
template <int TYPE>
__device__ __forceinline__ void store_row(uint8_t* row, uint8_t* sf_row, int d16, const uint32_t (&w)[4],
                                          float inv, bool live) {
  if constexpr (TYPE == DA_CACHE_BF16) {
    if (live) *reinterpret_cast<uint4*>(row + d16 * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  [[maybe_unused]] float x[8];
  if constexpr (TYPE != DA_CACHE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(mul2(widen(w[i]), pair(inv, inv)), x[2 * i], x[2 * i + 1]);
  }
  if constexpr (TYPE == DA_CACHE_FP8_E4M3) {
    const uint2 v = make_uint2(e4m3_pair(x[0], x[1]) | (e4m3_pair(x[2], x[3]) << 16),
                               e4m3_pair(x[4], x[5]) | (e4m3_pair(x[6], x[7]) << 16));
    if (live) *reinterpret_cast<uint2*>(row + d16 * 8) = v;
  } else if constexpr (TYPE == DA_CACHE_FP4_E2M1) {
    float top = 0.f, all = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = fmaxf(top, fabsf(x[i]));  // (NaN is passed over)
      all += x[i];
    }
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
    const uint32_t code = e4m3_pair(__fdiv_rn(top, 6.f), 0.f) & 0xffu;
    const float sf = e4m3_value(code);
    // x / sf, correctly rounded: a rounded reciprocal, a product, and one
    // residual correction (Markstein 1990), three operations a value.  It needs
    // finite quotients, so NaN becomes 0 and what lies past 8 sf, and saturates
    // all the same, comes in; a block has such values only if its sum is not
    // finite or its scale saturated.
    if (!(fabsf(all) < INFINITY) || top > 6.f * 448.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -8.f * sf), 8.f * sf) : 0.f;
    }
    const float r = sf > 0.f ? __frcp_rn(sf) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __fmul_rn(x[i], r);
      x[i] = copysignf(fmaf(fmaf(-q, sf, x[i]), r, q), x[i]);  // (-0 stays -0)
    }
    if (live) {
      *reinterpret_cast<uint32_t*>(row + d16 * 4) = sf > 0.f ? e2m1x8(x) : 0u;
      if ((d16 & 1) == 0) sf_row[d16 >> 1] = static_cast<uint8_t>(code);
    }
  }
}

// ALIGN: the largest of 16, 8 and 2 that divides rotary_dim.  At 16 partners
// are whole threads' values; at 8 (72, say) halves of two threads' values, and
// table rows whole vectors all the same; else both are read value by value
// (8192 tokens, 32 / 8 heads, FP8, rotary_dim 72: 70 us that way, 41 in halves).
template <int ALIGN, int TYPE>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  constexpr bool VEC = ALIGN >= 8;
  const int d16 = threadIdx.x & 15;
  const int sub = threadIdx.x >> 4;
  const int lane = threadIdx.x & 31;
  const int token = blockIdx.x;
  const int b = token / a.g.q_len;
  const int t = token - b * a.g.q_len;
  const int d0 = 8 * d16;

  // ---- the passes of this CTA: p = blockIdx.y, + gridDim.y, ...; q's first
  const int q_passes = (a.num_q_heads + kRowsPerPass - 1) / kRowsPerPass;
  const int kv_passes = a.append ? (a.g.num_kv_heads + kRowsPerPass - 1) / kRowsPerPass : 0;
  const int passes = q_passes + 2 * kv_passes;
  const uint16_t* q0 = a.q + static_cast<int64_t>(b) * a.q_sb + static_cast<int64_t>(t) * a.q_st + d0;
  const uint16_t* k0 = a.k + static_cast<int64_t>(b) * a.k_sb + static_cast<int64_t>(t) * a.k_st + d0;
  const uint16_t* v0 = a.v + static_cast<int64_t>(b) * a.v_sb + static_cast<int64_t>(t) * a.v_st + d0;
  // this thread's row in a pass (nullptr: no such head)
  auto source = [&](int p) -> const uint16_t* {
    if (p < q_passes) {
      const int h = p * kRowsPerPass + sub;
      return h < a.num_q_heads ? q0 + h * a.q_sh : nullptr;
    }
    p -= q_passes;
    const bool is_v = p >= kv_passes;
    const int h = (is_v ? p - kv_passes : p) * kRowsPerPass + sub;
    if (p >= 2 * kv_passes || h >= a.g.num_kv_heads) return nullptr;
    return is_v ? v0 + h * a.v_sh : k0 + h * a.k_sh;
  };
  auto fetch = [&](int p) {
    const uint16_t* src = source(p);
    return src != nullptr ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
  };
  grid_dependency_wait();
  constexpr int kAhead = 3;  // passes whose rows are loaded ahead
  uint4 next[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) next[i] = fetch(blockIdx.y + i * gridDim.y);

  // ---- the token's place
  uint32_t bad = 0;
  int L = a.g.seq_lens[b];
  int n = a.new_lens != nullptr ? a.new_lens[b] : a.g.q_len;
  if (L < 0 || L > a.g.max_seq_len || n < 0 || n > a.g.q_len) {
    bad |= DA_STATUS_SEQ_LEN;
    L = min(max(L, 0), a.g.max_seq_len);
    n = min(max(n, 0), a.g.q_len);
  }
  if (L < n) bad |= DA_STATUS_SHORT_CAUSAL;
  const int at = L - n + t;                     // cache position
  bool live = t < n && at >= 0;
  int pos = at;
  if (a.positions != nullptr && live) pos = a.positions[token];
  if (live && a.rotary_dim > 0 && (pos < 0 || pos >= a.table_positions)) {
    bad |= DA_STATUS_POSITION;
    live = false;
  }
  int64_t place = 0, sf_place = 0;
  if (live && a.append) {
    int64_t group = b;
    int slot = at;
    if (a.g.block_table != nullptr) {
      const int col = at / a.g.page_size;
      slot = at - col * a.g.page_size;
      const int pg = a.g.block_table[static_cast<int64_t>(b) * a.g.bt_stride + col];
      if (pg < 0 || pg >= a.g.num_pages) bad |= DA_STATUS_BAD_PAGE;
      group = pg;
    }
    place = group * a.c.page + slot * a.c.token;
    sf_place = group * a.c.sf_page + static_cast<int64_t>(slot) * 8;
  }
  if (bad != 0 && a.g.status != nullptr && blockIdx.y == 0 && threadIdx.x == 0)
    atomicOr(a.g.status, static_cast<int32_t>(bad));
  const bool write = live && (bad & DA_STATUS_BAD_PAGE) == 0;
  if (!live) return;  // (the whole CTA: one token)

  // ---- cos and sin of this thread's values, in pairs: y = x c + partner s,
  // with s negative for the first value of a (value, partner) pair
  const int half = a.rotary_dim >> 1;
  uint64_t c[4], s[4];
  const float* row = a.table + static_cast<int64_t>(pos) * a.rotary_dim;
  const bool turned = d0 < a.rotary_dim;  // (VEC: all of the thread's values or none)
  if constexpr (VEC) {
    if (turned) {
      if (a.interleaved) {
        const float4 cc = *reinterpret_cast<const float4*>(row + (d0 >> 1));
        const float4 ss = *reinterpret_cast<const float4*>(row + half + (d0 >> 1));
        const float c4[4] = {cc.x, cc.y, cc.z, cc.w}, s4[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[i] = pair(c4[i], c4[i]);
          s[i] = pair(-s4[i], s4[i]);
        }
      } else {
#pragma unroll
        for (int v = 0; v < 2; ++v) {  // (half a multiple of 4: four values are on one side; of 8: eight)
          const bool first = (ALIGN == 8 ? d0 + 4 * v : d0) < half;
          const int f0 = first ? d0 : d0 - half;
          const float sign = first ? -1.f : 1.f;
          const float4 cc = *reinterpret_cast<const float4*>(row + f0 + 4 * v);
          const float4 ss = *reinterpret_cast<const float4*>(row + half + f0 + 4 * v);
          c[2 * v] = pair(cc.x, cc.y);
          c[2 * v + 1] = pair(cc.z, cc.w);
          s[2 * v] = pair(sign * ss.x, sign * ss.y);
          s[2 * v + 1] = pair(sign * ss.z, sign * ss.w);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float cc[2], ss[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int d = d0 + 2 * i + j;
        const bool in = d < a.rotary_dim;
        const int f = a.interleaved ? d >> 1 : (d < half ? d : d - half);
        const bool second = a.interleaved ? (d & 1) != 0 : d >= half;
        cc[j] = in ? row[f] : 1.f;
        ss[j] = in ? (second ? row[half + f] : -row[half + f]) : 0.f;
      }
      c[i] = pair(cc[0], cc[1]);
      s[i] = pair(ss[0], ss[1]);
    }
  }
  // the lanes that hold the partners of this thread's first and last four values
  // (half layout; ALIGN 8: in the other half of their words)
  int peer[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int d = ALIGN == 8 ? d0 + 4 * v : d0;
    peer[v] = (lane & 16) | (((d < half ? d + half : d - half) >> 3) & 15);
  }

  // the rotated values of a row: every product and the sum rounded, the
  // definition, and the same bytes for a token wherever it is computed again
  const uint64_t one = pair(a.one, a.one);
  auto rotate = [&](const uint4& x4, const uint16_t* src, uint32_t (&y)[4]) {
    const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
    uint64_t p[4];
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = widen(__byte_perm(x[i], 0, 0x1032));
    } else if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = widen(__shfl_sync(kFull, x[ALIGN == 8 ? (i + 2) & 3 : i], peer[i >> 1]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int d = d0 + 2 * i + j;
          if (src != nullptr && d < a.rotary_dim) o[j] = (src - d0)[d < half ? d + half : d - half];
        }
        p[i] = widen(o[0] | (o[1] << 16));
      }
      __syncwarp();  // (q_out may be q: every partner is read before any store)
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = narrow(add2(mul2(widen(x[i]), c[i]), mul2(p[i], s[i]), one));
      if constexpr (VEC) {
        y[i] = turned ? r : x[i];
      } else {
        const int d = d0 + 2 * i;
        y[i] = (d < a.rotary_dim ? r & 0xffffu : x[i] & 0xffffu) |
               (d + 1 < a.rotary_dim ? r & 0xffff0000u : x[i] & 0xffff0000u);
      }
    }
  };

  uint16_t* o0 = a.q_out + static_cast<int64_t>(b) * a.o_sb + static_cast<int64_t>(t) * a.o_st + d0;
  auto pass = [&](int p, const uint4& x) {
    uint32_t y[4];
    if (p < q_passes) {
      const int h = p * kRowsPerPass + sub;
      const bool have = h < a.num_q_heads;
      rotate(x, have ? q0 + h * a.q_sh : nullptr, y);
      if (have) *reinterpret_cast<uint4*>(o0 + h * a.o_sh) = make_uint4(y[0], y[1], y[2], y[3]);
      return;
    }
    p -= q_passes;
    const bool is_v = p >= kv_passes;  // (uniform)
    const int h = (is_v ? p - kv_passes : p) * kRowsPerPass + sub;
    const bool have = h < a.g.num_kv_heads;
    const int64_t to = place + h * a.c.head, sf_to = sf_place + h * a.c.sf_head;
    if (is_v) {
      y[0] = x.x;
      y[1] = x.y;
      y[2] = x.z;
      y[3] = x.w;
      store_row<TYPE>(a.c.v + to, a.c.vs + sf_to, d16, y, a.v_inv, have && write);
    } else {
      rotate(x, have ? k0 + h * a.k_sh : nullptr, y);
      store_row<TYPE>(a.c.k + to, a.c.ks + sf_to, d16, y, a.k_inv, have && write);
    }
  };
  for (int p = blockIdx.y; p < passes; p += kAhead * gridDim.y) {
    uint4 now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) now[i] = next[i];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) next[i] = fetch(p + (kAhead + i) * gridDim.y);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (p + i * static_cast<int>(gridDim.y) < passes) pass(p + i * gridDim.y, now[i]);
  }
}

// ------------------------------------------------------------------- digest
// A warp takes a KV head's pages, about 32 KB of them (16 ragged requests of up
// to 32K tokens in 16-token bf16 pages: one page 205 us, four 137, eight 131);
// the warps of a CTA take neighbouring heads, which a [page, slot, head, d]
// cache holds side by side.  A lane loads 16 bytes of a row (8, 16 or 32
// values; 2, 4 or 8 rows per load; 8 bytes of FP8 and 4-bit pages of 16 tokens),
// a batch of loads at work and the next on its way, and keeps packed 16-bit
// minima and maxima: bf16 as it is, FP8 and 4-bit values exactly in f16.  The
// rows' partial results meet in a reduce-scatter (each step sends half of what
// is left): 4, 12 or 28 shuffles per page, after which every lane holds 8
// channels of the minimum or of the maximum, whatever the type.  (16 ragged requests, 774 MB of bf16 keys: 126.8
// us, 6.1 TB/s, 0.91 of a copy's rate; 4-bit keys, 50 requests of 3 to 8K tokens
// in 32-token pages: 38 us, 2.2 TB/s, bound by the instructions of a page's end.)
constexpr int kDigestWarps = 8;
constexpr int64_t kWarpBytes = 32768;  // of keys that a warp walks, where there are enough
constexpr float kBf16Max = 3.3895313892515355e38f;

template <bool BF>
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y) {
  uint32_t r;
  if constexpr (BF) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

template <bool BF>
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  uint32_t r;
  if constexpr (BF) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// SHORT: batches of 16 tokens and 8 bytes a lane, for 16-token pages (16 ragged
// requests of up to 32K tokens: FP8 121 -> 99 us, 4-bit 144 -> 116; 48-token
// pages are the same either way, 64-token ones 7 % faster with 16 bytes).
template <int TYPE, bool SHORT>
struct DigestCfg {
  static constexpr bool kBf = TYPE == DA_CACHE_BF16;
  using Vec = std::conditional_t<kBf || !SHORT, uint4, uint2>;  // of a row, per lane
  static constexpr int kLanes = (TYPE == DA_CACHE_FP4_E2M1 ? 64 : kBf ? 256 : 128) / sizeof(Vec);  // of a row
  static constexpr int kRows = 32 / kLanes;                             // per load
  static constexpr int kWords = 128 / kLanes / 2;                       // packed values of a lane
  // in flight (4-bit: 4, its minima and maxima fill the registers; 8 took 95 us
  // where 4 take 72, FP8 the other way round, 90 and 75)
  static constexpr int kLoads = TYPE == DA_CACHE_FP4_E2M1 ? 4 : 8;
};

template <int TYPE, bool SHORT>
__global__ void __launch_bounds__(32 * kDigestWarps) digest_kernel(const DigestArgs a, int pages_per_warp) {
  using C = DigestCfg<TYPE, SHORT>;
  constexpr int NW = C::kWords;
  const int lane = threadIdx.x & 31;
  const int l = lane % C::kLanes, rg = lane / C::kLanes;
  const uint32_t idx = blockIdx.x * kDigestWarps + (threadIdx.x >> 5);
  const int b = blockIdx.y;
  grid_dependency_wait();
  int L = a.g.seq_lens[b];
  if (L < 0 || L > a.g.max_seq_len) {
    if (a.g.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
      atomicOr(a.g.status, static_cast<int32_t>(DA_STATUS_SEQ_LEN));
    L = L < 0 ? 0 : a.g.max_seq_len;
  }
  const int ps = a.g.page_size;
  const int first = a.max_new > 0 ? max(0, L - a.max_new) / ps : 0;
  const int cols = (L + ps - 1) / ps;                       // pages of the request
  const uint32_t group = idx / a.g.num_kv_heads;
  const int h = static_cast<int>(idx - group * a.g.num_kv_heads);
  const int64_t col0 = first + static_cast<int64_t>(group) * pages_per_warp;
  if (col0 >= cols) return;
  const int n = min(pages_per_warp, cols - static_cast<int>(col0));
  // the warp's page ids, lane i the i-th (-1: does not exist, not digested)
  int id = -1;
  if (lane < n) {
    id = a.g.block_table[static_cast<int64_t>(b) * a.g.bt_stride + col0 + lane];
    if (id < 0 || id >= a.g.num_pages) {
      if (a.g.status != nullptr) atomicOr(a.g.status, static_cast<int32_t>(DA_STATUS_BAD_PAGE));
      id = -1;
    }
  }
  constexpr int kTokens = C::kLoads * C::kRows;             // of a batch
  const int parts = (ps + kTokens - 1) / kTokens;           // batches of a page
  using Vec = typename C::Vec;
  const uint8_t* kbase = a.c.k + static_cast<int64_t>(h) * a.c.head + l * sizeof(Vec);
  const uint8_t* sbase = TYPE == DA_CACHE_FP4_E2M1 ? a.c.ks + static_cast<int64_t>(h) * a.c.sf_head + l * (SHORT ? 1 : 2) : nullptr;
  auto held = [&](int page) { return min(ps, L - (static_cast<int>(col0) + page) * ps); };  // tokens of a page

  Vec x[C::kLoads];
  uint32_t sf[TYPE == DA_CACHE_FP4_E2M1 ? C::kLoads : 1];
  auto load = [&](int page, int part) {
    const int pg = __shfl_sync(kFull, id, page);
    const int last = held(page) - 1;
    const uint8_t* p = kbase + static_cast<int64_t>(max(pg, 0)) * a.c.page;
#pragma unroll
    for (int j = 0; j < C::kLoads; ++j) {
      const int row = part * kTokens + j * C::kRows;
      if (row > last || pg < 0) continue;                   // (uniform)
      const int tok = min(row + rg, last);                  // (the last token again: no effect)
      x[j] = __ldg(reinterpret_cast<const Vec*>(p + static_cast<int64_t>(tok) * a.c.token));
      if constexpr (TYPE == DA_CACHE_FP4_E2M1)
      {
        const uint8_t* src = sbase + static_cast<int64_t>(pg) * a.c.sf_page + static_cast<int64_t>(tok) * 8;
        if constexpr (SHORT) sf[j] = __ldg(src);
        else sf[j] = __ldg(reinterpret_cast<const uint16_t*>(src));
      }
    }
  };
  load(0, 0);
  uint32_t v[2 * NW];                                       // minima, then maxima
  for (int page = 0; page < n; ++page) {
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      v[i] = C::kBf ? 0x7f807f80u : 0x7c007c00u;            // + infinity
      v[NW + i] = C::kBf ? 0xff80ff80u : 0xfc00fc00u;
    }
    const int tokens = held(page);
    for (int part = 0; part < parts; ++part) {
      Vec y[C::kLoads];
      uint32_t ys[TYPE == DA_CACHE_FP4_E2M1 ? C::kLoads : 1];
#pragma unroll
      for (int j = 0; j < C::kLoads; ++j) {
        y[j] = x[j];
        if constexpr (TYPE == DA_CACHE_FP4_E2M1) ys[j] = sf[j];
      }
      if (part + 1 < parts) load(page, part + 1);
      else if (page + 1 < n) load(page + 1, 0);
#pragma unroll
      for (int j = 0; j < C::kLoads; ++j) {
        if (part * kTokens + j * C::kRows >= tokens) break;  // (uniform)
        constexpr int kVec = sizeof(Vec) / 4;
        uint32_t w[kVec];
        w[0] = y[j].x;
        w[1] = y[j].y;
        if constexpr (kVec == 4) {
          w[2] = y[j].z;
          w[3] = y[j].w;
        }
        uint32_t u[NW];
        if constexpr (TYPE == DA_CACHE_BF16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = w[i];
        } else if constexpr (TYPE == DA_CACHE_FP8_E4M3) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) e4m3x4_to_f16x4(w[i], u[2 * i], u[2 * i + 1]);
        } else {
          const uint32_t s2 = e4m3x2_to_f16x2(ys[j]);       // the lane's block scales
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            uint32_t c4[4];
            e2m1x8_to_f16(w[i], c4);
            const uint32_t s = __byte_perm(s2, 0, i < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int q = 0; q < 4; ++q) u[4 * i + q] = mul_f16x2(c4[q], s);
          }
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) {                      // (NaN is passed over)
          v[i] = min2<C::kBf>(v[i], u[i]);
          v[NW + i] = max2<C::kBf>(v[NW + i], u[i]);
        }
      }
    }
    const int pg = __shfl_sync(kFull, id, page);
    if (pg < 0) continue;
    // ---- the row groups meet: step by step a lane keeps half of its words (by
    // its lane bit: the minima or the maxima first) and takes the other's
#pragma unroll
    for (int m = 16, left = 2 * NW; m >= C::kLanes; m >>= 1) {
      left >>= 1;
      const bool up = (lane & m) != 0;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        if (i >= left) break;
        const uint32_t mine = up ? v[left + i] : v[i], give = up ? v[i] : v[left + i];
        const uint32_t got = __shfl_xor_sync(kFull, give, m);
        v[i] = (lane & 16) != 0 ? max2<C::kBf>(mine, got) : min2<C::kBf>(mine, got);
      }
    }
    // now v[0 .. 3]: 8 channels from d0 on, of the minimum (lanes 0-15) or maximum
    float f[8];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (C::kBf) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      } else {
        f[2 * i] = packed_lo(v[i], true);
        f[2 * i + 1] = packed_hi(v[i], true);
      }
      odd |= isinf(f[2 * i]) || isinf(f[2 * i + 1]);
    }
    if (__any_sync(kFull, odd)) {
      // infinite keys, or channels with nothing but NaN (minimum above maximum)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_xor_sync(kFull, f[i], 16);
        const bool none = (lane & 16) != 0 ? f[i] < other : f[i] > other;
        f[i] = none ? 0.f : fminf(fmaxf(f[i], -kBf16Max), kBf16Max);
      }
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
    top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));  // (not negative: bits in order)
    const float inv = top > 0.f ? __fdiv_rn(127.f, top) : 0.f;
    uint32_t q[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = min(max(__float2int_rn(__fmul_rn(f[i], inv)), -127), 127);
      q[i >> 2] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (i & 3));
    }
    int d0 = l * 2 * NW;
    if constexpr (C::kRows >= 4) d0 += (lane & 8) != 0 ? NW : 0;
    if constexpr (C::kRows >= 8) d0 += (lane & 4) != 0 ? NW / 2 : 0;
    const int64_t at = static_cast<int64_t>(pg) * a.g.num_kv_heads + h;
    *reinterpret_cast<uint2*>(a.digest + at * 256 + ((lane & 16) != 0 ? 128 : 0) + d0) = make_uint2(q[0], q[1]);
    if (lane == 0) a.digest_scale[at] = __fdiv_rn(top, 127.f);
  }
}

template <class Kernel, class... Args>
cudaError_t launch(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_rope_table(const double* inv_freq, int num_freqs, int64_t first, int64_t count,
                              double amplitude, float* table, int sm_count, cudaStream_t stream) {
  if (count == 0) return cudaSuccess;
  const bool wide = num_freqs % 4 == 0;  // (and the table 16-byte aligned: the rows are then, too)
  const int per = kTableThreads / (wide ? num_freqs / 4 : num_freqs);
  // a few rows per thread at most while the CTAs fit the GPU once
  const int64_t blocks = (count + per - 1) / per;
  const int64_t most = static_cast<int64_t>(sm_count) * 8;
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
  const float amp = static_cast<float>(amplitude);
  return wide ? launch(rope_table_kernel<4>, grid, kTableThreads, 0, stream, inv_freq, num_freqs, first, count, amp, table)
              : launch(rope_table_kernel<1>, grid, kTableThreads, 0, stream, inv_freq, num_freqs, first, count, amp, table);
}

template <int ALIGN>
static cudaError_t launch_append_type(const AppendArgs& a, dim3 grid, cudaStream_t stream) {
  switch (a.c.type) {
    case DA_CACHE_BF16: return launch(append_kernel<ALIGN, DA_CACHE_BF16>, grid, kAppendThreads, 0, stream, a);
    case DA_CACHE_FP8_E4M3: return launch(append_kernel<ALIGN, DA_CACHE_FP8_E4M3>, grid, kAppendThreads, 0, stream, a);
    default: return launch(append_kernel<ALIGN, DA_CACHE_FP4_E2M1>, grid, kAppendThreads, 0, stream, a);
  }
}

cudaError_t launch_append(const AppendArgs& a, int sm_count, cudaStream_t stream) {
  const int64_t tokens = static_cast<int64_t>(a.g.batch) * a.g.q_len;
  const int64_t passes = (a.num_q_heads + kRowsPerPass - 1) / kRowsPerPass +
                         (a.append ? 2 * ((a.g.num_kv_heads + kRowsPerPass - 1) / kRowsPerPass) : 0);
  if (passes == 0 || tokens == 0) return cudaSuccess;
  // few tokens: spread a token's passes over CTAs until about four per SM exist
  const int64_t want = (4 * static_cast<int64_t>(sm_count) + tokens - 1) / tokens;
  const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(want < passes ? want : passes));
  return a.rotary_dim % 16 == 0  ? launch_append_type<16>(a, grid, stream)
         : a.rotary_dim % 8 == 0 ? launch_append_type<8>(a, grid, stream)
                                 : launch_append_type<2>(a, grid, stream);
}

cudaError_t launch_digest(const DigestArgs& a, int sm_count, cudaStream_t stream) {
  int64_t cols = (static_cast<int64_t>(a.g.max_seq_len) + a.g.page_size - 1) / a.g.page_size;
  if (a.max_new > 0) {
    const int64_t touched = (static_cast<int64_t>(a.max_new) + a.g.page_size - 2) / a.g.page_size + 1;
    if (touched < cols) cols = touched;
  }
  if (cols == 0 || a.g.batch == 0) return cudaSuccess;
  // few pages, as in a decode step: one per warp, for latency
  const int64_t row = a.c.type == DA_CACHE_BF16 ? 256 : a.c.type == DA_CACHE_FP8_E4M3 ? 128 : 72;
  const int64_t pairs = cols * a.g.num_kv_heads * a.g.batch;
  int64_t per = kWarpBytes / (row * a.g.page_size);
  if (per > pairs / (16 * static_cast<int64_t>(sm_count))) per = pairs / (16 * static_cast<int64_t>(sm_count));
  per = per < 1 ? 1 : per > 32 ? 32 : per;
  const int64_t units = (cols + per - 1) / per * a.g.num_kv_heads;
  const dim3 grid(static_cast<unsigned>((units + kDigestWarps - 1) / kDigestWarps),
                  static_cast<unsigned>(a.g.batch));
  const bool half = a.g.page_size < 32;  // (16-token batches)
  auto run = [&](auto* kernel) { return launch(kernel, grid, 32 * kDigestWarps, 0, stream, a, static_cast<int>(per)); };
  switch (a.c.type) {
    case DA_CACHE_BF16: return run(digest_kernel<DA_CACHE_BF16, false>);
    case DA_CACHE_FP8_E4M3:
      return half ? run(digest_kernel<DA_CACHE_FP8_E4M3, true>) : run(digest_kernel<DA_CACHE_FP8_E4M3, false>);
    default:
      return half ? run(digest_kernel<DA_CACHE_FP4_E2M1, true>) : run(digest_kernel<DA_CACHE_FP4_E2M1, false>);
  }
}

}  // namespace dattn
