// cache_kernels.cu -- the kernels that fill a cache and digest it: the rotary
// table, the append of new tokens (rotation, conversion to the cache's type,
// scatter through the block table) and the per-page digests that the page
// selection scores.  All of them stream their data once and are bound by HBM
// at size and by launch latency in a decode step.

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
// integer multiply.  The nearest quarter turn is split off exactly and the
// remainder, at most an eighth of a turn, goes through sincospif in fp32: full
// relative accuracy at every position, without the fp64 argument reduction
// and sine per entry (fp64 runs at 1/64 of the fp32 rate on this GPU).
__device__ __forceinline__ uint64_t turns_fixed(double f) {
  const double kInv2PiHi = 0.15915494309189535;      // 1 / (2 pi), rounded
  const double kInv2PiLo = -9.839338337591243e-18;   // what is left of it
  const double p = f * kInv2PiHi;
  const double e = fma(f, kInv2PiHi, -p) + f * kInv2PiLo;
  const double frac = p - floor(p);                  // exact
  const double hi = floor(frac * 4294967296.0);
  const double lo = (frac * 4294967296.0 - hi) * 4294967296.0 + e * 18446744073709551616.0;
  return (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(static_cast<int64_t>(rint(lo)));
}

constexpr int kTablePos = 8;  // positions per thread

__global__ void __launch_bounds__(256)
    rope_table_kernel(const double* inv_freq, int n, int64_t first, int64_t count, float amp,
                      float* table) {
  grid_dependency_wait();
  const int per = blockDim.x / n;  // positions side by side in the block
  const int i = threadIdx.x % n;
  const int row = threadIdx.x / n;
  if (row >= per) return;
  const double f = inv_freq[i];
  const bool ok = fabs(f) <= 1.7976931348623157e308;  // (not NaN or infinite)
  // frequencies of 2^31 radians and more keep no fraction worth the name in
  // fp64 terms, but stay defined: the same wrap
  const uint64_t step = ok ? turns_fixed(f) : 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * per;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * per + row; r < count; r += stride) {
    const uint64_t phase = static_cast<uint64_t>(first + r) * step;
    const uint32_t quarter = static_cast<uint32_t>((phase + (uint64_t{1} << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(phase - (static_cast<uint64_t>(quarter) << 62));
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-63f, &s, &c);  // rest turns / 2^64, in units of pi
    if (quarter & 1) {
      const float x = c;
      c = -s;
      s = x;
    }
    if (quarter & 2) {
      c = -c;
      s = -s;
    }
    if (!ok) c = s = __int_as_float(0x7fc00000);
    float* out = table + r * 2 * n;
    out[i] = c * amp;
    out[n + i] = s * amp;
  }
}

// ------------------------------------------------------------------- append
// 16 threads hold the 128 values of a (token, head), 8 each.  A CTA works on
// one token: each thread keeps the cos / sin of its 8 values in registers for
// all the heads it walks, so the table is read once per CTA and row of
// threads, and the pair partners of the half layout come by one shuffle (a
// thread's 8 values and their partners lie rotary_dim / 2 apart, whole threads
// when that is a multiple of 8; other sizes read the partner from memory).
constexpr int kAppendThreads = 128;
constexpr int kRowsPerPass = kAppendThreads / 16;

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
__device__ __forceinline__ void store_row(int type, uint8_t* row, uint8_t* sf_row, int d16,
                                          const uint32_t (&w)[4], float inv, bool live) {
  if (type == DA_CACHE_BF16) {
    if (live) *reinterpret_cast<uint4*>(row + d16 * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __fmul_rn(__uint_as_float(w[i] << 16), inv);
    x[2 * i + 1] = __fmul_rn(__uint_as_float(w[i] & 0xffff0000u), inv);
  }
  if (type == DA_CACHE_FP8_E4M3) {
    const uint2 v = make_uint2(e4m3_pair(x[0], x[1]) | (e4m3_pair(x[2], x[3]) << 16),
                               e4m3_pair(x[4], x[5]) | (e4m3_pair(x[6], x[7]) << 16));
    if (live) *reinterpret_cast<uint2*>(row + d16 * 8) = v;
    return;
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));  // (NaN is passed over)
  top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
  const uint32_t code = e4m3_pair(__fdiv_rn(top, 6.f), 0.f) & 0xffu;
  const float sf = e4m3_value(code);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = sf > 0.f && x[i] == x[i] ? __fdiv_rn(x[i], sf) : 0.f;
  if (live) {
    *reinterpret_cast<uint32_t*>(row + d16 * 4) = e2m1x8(x);
    if ((d16 & 1) == 0) sf_row[d16 >> 1] = static_cast<uint8_t>(code);
  }
}

// VEC: rotary_dim is a multiple of 16 (table and partners in whole vectors).
template <bool VEC>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  const int d16 = threadIdx.x & 15;
  const int sub = threadIdx.x >> 4;
  const int lane = threadIdx.x & 31;
  const int token = blockIdx.x;
  const int b = token / a.g.q_len;
  const int t = token - b * a.g.q_len;
  grid_dependency_wait();

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

  // ---- cos and sin of this thread's values: c[i] and the signed s[i] of value
  // 8 d16 + i, as y = x c + partner s
  const int half = a.rotary_dim >> 1;
  const int d0 = 8 * d16;
  float c[8], s[8];
  const float* row = a.table + static_cast<int64_t>(pos) * a.rotary_dim;
  if constexpr (VEC) {
    if (d0 < a.rotary_dim) {
      if (a.interleaved) {
        const float4 cc = *reinterpret_cast<const float4*>(row + (d0 >> 1));
        const float4 ss = *reinterpret_cast<const float4*>(row + half + (d0 >> 1));
        const float c4[4] = {cc.x, cc.y, cc.z, cc.w}, s4[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = c4[i >> 1];
          s[i] = i & 1 ? s4[i >> 1] : -s4[i >> 1];
        }
      } else {
        const int f0 = d0 < half ? d0 : d0 - half;
        const float sign = d0 < half ? -1.f : 1.f;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const float4 cc = *reinterpret_cast<const float4*>(row + f0 + 4 * v);
          const float4 ss = *reinterpret_cast<const float4*>(row + half + f0 + 4 * v);
          c[4 * v] = cc.x;
          c[4 * v + 1] = cc.y;
          c[4 * v + 2] = cc.z;
          c[4 * v + 3] = cc.w;
          s[4 * v] = sign * ss.x;
          s[4 * v + 1] = sign * ss.y;
          s[4 * v + 2] = sign * ss.z;
          s[4 * v + 3] = sign * ss.w;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = d0 + i;
      const bool in = d < a.rotary_dim;
      const int f = a.interleaved ? d >> 1 : (d < half ? d : d - half);
      const bool second = a.interleaved ? (d & 1) != 0 : d >= half;
      c[i] = in ? row[f] : 1.f;
      s[i] = in ? (second ? row[half + f] : -row[half + f]) : 0.f;
    }
  }
  // the lane that holds the partners of this thread's values (half layout)
  const int peer = (lane & 16) | ((d16 + (d0 < half ? (half >> 3) : -(half >> 3))) & 15);

  // ---- the heads: q, then k, then v
  const int rows = a.num_q_heads + (a.append ? 2 * a.g.num_kv_heads : 0);
  const int step = kRowsPerPass * gridDim.y;
  auto source = [&](int r) -> const uint16_t* {
    if (r < a.num_q_heads)
      return a.q + static_cast<int64_t>(b) * a.q_sb + static_cast<int64_t>(t) * a.q_st + r * a.q_sh;
    r -= a.num_q_heads;
    if (r < a.g.num_kv_heads)
      return a.k + static_cast<int64_t>(b) * a.k_sb + static_cast<int64_t>(t) * a.k_st + r * a.k_sh;
    r -= a.g.num_kv_heads;
    return a.v + static_cast<int64_t>(b) * a.v_sb + static_cast<int64_t>(t) * a.v_st + r * a.v_sh;
  };
  const int base = blockIdx.y * kRowsPerPass + (sub & ~1);  // the warp's first row of a pass
  uint4 next = make_uint4(0u, 0u, 0u, 0u);
  if (base + (sub & 1) < rows) next = *reinterpret_cast<const uint4*>(source(base + (sub & 1)) + d0);
  for (int r0 = base; r0 < rows; r0 += step) {  // (both rows of a warp together)
    const int r = r0 + (sub & 1);
    const bool have = r < rows;
    const uint4 x4 = next;
    const int rn = r + step;
    if (rn < rows) next = *reinterpret_cast<const uint4*>(source(rn) + d0);
    const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
    const int kv = r - a.num_q_heads;
    const bool is_v = kv >= a.g.num_kv_heads;
    uint32_t p[4];
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t o = __shfl_sync(kFull, x[i], peer);
        p[i] = a.interleaved ? __byte_perm(x[i], 0, 0x1032) : o;
      }
    } else {
      const uint16_t* src = have ? source(r) : nullptr;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (a.interleaved) {
          p[i] = __byte_perm(x[i], 0, 0x1032);
          continue;
        }
        uint32_t o[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int d = d0 + 2 * i + j;
          if (have && d < a.rotary_dim) o[j] = src[d < half ? d + half : d - half];
        }
        p[i] = o[0] | (o[1] << 16);
      }
      __syncwarp();  // (q_out may be q: every partner is read before any store)
    }
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = __uint_as_float(x[i] << 16), x1 = __uint_as_float(x[i] & 0xffff0000u);
      const float p0 = __uint_as_float(p[i] << 16), p1 = __uint_as_float(p[i] & 0xffff0000u);
      // every product and the sum rounded: the definition, and the same bytes
      // for a token wherever it is computed again
      const float y0 = __fadd_rn(__fmul_rn(x0, c[2 * i]), __fmul_rn(p0, s[2 * i]));
      const float y1 = __fadd_rn(__fmul_rn(x1, c[2 * i + 1]), __fmul_rn(p1, s[2 * i + 1]));
      const uint32_t lo = d0 + 2 * i < a.rotary_dim ? pack_bf16x2(y0, 0.f) & 0xffffu : x[i] & 0xffffu;
      const uint32_t hi = d0 + 2 * i + 1 < a.rotary_dim ? pack_bf16x2(0.f, y1) & 0xffff0000u
                                                        : x[i] & 0xffff0000u;
      y[i] = is_v ? x[i] : lo | hi;
    }
    if (have && kv < 0)
      *reinterpret_cast<uint4*>(a.q_out + static_cast<int64_t>(b) * a.o_sb +
                                static_cast<int64_t>(t) * a.o_st + r * a.o_sh + d0) =
          make_uint4(y[0], y[1], y[2], y[3]);
    if (r0 + 1 >= a.num_q_heads && a.append) {  // (warp-uniform: one of the two rows is k or v)
      const bool ok = have && kv >= 0 && write;
      const int h = ok ? (is_v ? kv - a.g.num_kv_heads : kv) : 0;
      store_row(a.c.type, (is_v ? a.c.v : a.c.k) + place + h * a.c.head,
                (is_v ? a.c.vs : a.c.ks) + sf_place + h * a.c.sf_head, d16, y,
                is_v ? a.v_inv : a.k_inv, ok);
    }
  }
}

// ------------------------------------------------------------------- digest
// One warp per (page, KV head): 16 lanes hold the 128 channels, 8 each, and
// the two half-warps take every other token; minima and maxima stay in
// registers.  Neighbouring warps take neighbouring heads of a page, which a
// [page, slot, head, d] cache holds side by side.
constexpr int kDigestWarps = 8;
constexpr float kBf16Max = 3.3895313892515355e38f;

template <int TYPE>
__global__ void __launch_bounds__(32 * kDigestWarps) digest_kernel(const DigestArgs a) {
  const int lane = threadIdx.x & 31;
  const int d16 = lane & 15;
  const int sub = lane >> 4;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kDigestWarps + (threadIdx.x >> 5);
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
  const int64_t c64 = first + idx / a.g.num_kv_heads;
  const int h = static_cast<int>(idx % a.g.num_kv_heads);
  if (c64 * ps >= L) return;
  const int col = static_cast<int>(c64);
  int pg = a.g.block_table[static_cast<int64_t>(b) * a.g.bt_stride + col];
  if (pg < 0 || pg >= a.g.num_pages) {
    if (a.g.status != nullptr && lane == 0)
      atomicOr(a.g.status, static_cast<int32_t>(DA_STATUS_BAD_PAGE));
    return;  // (nothing is digested for a page that does not exist)
  }
  const int held = min(ps, L - col * ps);
  const uint8_t* base = a.c.k + pg * a.c.page + h * a.c.head;
  const uint8_t* sfb = TYPE == DA_CACHE_FP4_E2M1 ? a.c.ks + pg * a.c.sf_page + h * a.c.sf_head : nullptr;
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = INFINITY;
    hi[i] = -INFINITY;
  }
  constexpr int kBatch = 8;  // 16 tokens in flight per warp
  for (int j0 = sub; j0 < held; j0 += 2 * kBatch) {
    uint4 x[kBatch];
    uint32_t sf[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int tok = min(j0 + 2 * j, held - 1);  // (the last token again: no effect)
      const uint8_t* p = base + static_cast<int64_t>(tok) * a.c.token;
      if constexpr (TYPE == DA_CACHE_BF16) {
        x[j] = __ldg(reinterpret_cast<const uint4*>(p + d16 * 16));
      } else if constexpr (TYPE == DA_CACHE_FP8_E4M3) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + d16 * 8));
        x[j].x = v.x;
        x[j].y = v.y;
      } else {
        x[j].x = __ldg(reinterpret_cast<const uint32_t*>(p + d16 * 4));
        sf[j] = __ldg(sfb + static_cast<int64_t>(tok) * 8 + (d16 >> 1));
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      float v[8];
      if constexpr (TYPE == DA_CACHE_BF16) {
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = i & 1 ? __uint_as_float(w[i >> 1] & 0xffff0000u) : __uint_as_float(w[i >> 1] << 16);
      } else if constexpr (TYPE == DA_CACHE_FP8_E4M3) {
        uint32_t w[4];
        e4m3x4_to_f16x4(x[j].x, w[0], w[1]);
        e4m3x4_to_f16x4(x[j].y, w[2], w[3]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i & 1 ? packed_hi(w[i >> 1], true) : packed_lo(w[i >> 1], true);
      } else {
        uint32_t w[4];
        e2m1x8_to_f16(x[j].x, w);
        const float s = e4m3_value(sf[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = (i & 1 ? packed_hi(w[i >> 1], true) : packed_lo(w[i >> 1], true)) * s;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // (fminf / fmaxf pass over NaN)
        lo[i] = fminf(lo[i], v[i]);
        hi[i] = fmaxf(hi[i], v[i]);
      }
    }
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = fminf(lo[i], __shfl_xor_sync(kFull, lo[i], 16));
    hi[i] = fmaxf(hi[i], __shfl_xor_sync(kFull, hi[i], 16));
    const bool none = lo[i] > hi[i];  // (nothing but NaN)
    lo[i] = none ? 0.f : fminf(fmaxf(lo[i], -kBf16Max), kBf16Max);
    hi[i] = none ? 0.f : fminf(fmaxf(hi[i], -kBf16Max), kBf16Max);
    top = fmaxf(top, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  const float inv = top > 0.f ? __fdiv_rn(127.f, top) : 0.f;
  // half-warp 0 writes the minima, 1 the maxima
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = min(max(__float2int_rn(__fmul_rn(sub == 0 ? lo[i] : hi[i], inv)), -127), 127);
    w[i >> 2] |= (static_cast<uint32_t>(q) & 0xffu) << (8 * (i & 3));
  }
  const int64_t at = static_cast<int64_t>(pg) * a.g.num_kv_heads + h;
  *reinterpret_cast<uint2*>(a.digest + at * 256 + sub * 128 + d16 * 8) = make_uint2(w[0], w[1]);
  if (lane == 0) a.digest_scale[at] = __fdiv_rn(top, 127.f);
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
  const int per = 256 / num_freqs;
  const int64_t blocks = (count + static_cast<int64_t>(per) * kTablePos - 1) / (per * kTablePos);
  const int64_t most = static_cast<int64_t>(sm_count) * 8;
  return launch(rope_table_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0,
                stream, inv_freq, num_freqs, first, count, static_cast<float>(amplitude), table);
}

cudaError_t launch_append(const AppendArgs& a, int sm_count, cudaStream_t stream) {
  const int rows = a.num_q_heads + (a.append ? 2 * a.g.num_kv_heads : 0);
  const int64_t tokens = static_cast<int64_t>(a.g.batch) * a.g.q_len;
  if (rows == 0 || tokens == 0) return cudaSuccess;
  // few tokens: spread a token's heads over CTAs until about four per SM exist
  const int64_t passes = (rows + kRowsPerPass - 1) / kRowsPerPass;
  const int64_t want = (4 * static_cast<int64_t>(sm_count) + tokens - 1) / tokens;
  const unsigned split = static_cast<unsigned>(want < passes ? want : passes);
  const dim3 grid(static_cast<unsigned>(tokens), split);
  return a.rotary_dim % 16 == 0 ? launch(append_kernel<true>, grid, kAppendThreads, 0, stream, a)
                                : launch(append_kernel<false>, grid, kAppendThreads, 0, stream, a);
}

cudaError_t launch_digest(const DigestArgs& a, cudaStream_t stream) {
  int64_t cols = (static_cast<int64_t>(a.g.max_seq_len) + a.g.page_size - 1) / a.g.page_size;
  if (a.max_new > 0) {
    const int64_t touched = (static_cast<int64_t>(a.max_new) + a.g.page_size - 2) / a.g.page_size + 1;
    if (touched < cols) cols = touched;
  }
  if (cols == 0 || a.g.batch == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((cols * a.g.num_kv_heads + kDigestWarps - 1) / kDigestWarps),
                  static_cast<unsigned>(a.g.batch));
  switch (a.c.type) {
    case DA_CACHE_BF16:
      return launch(digest_kernel<DA_CACHE_BF16>, grid, 32 * kDigestWarps, 0, stream, a);
    case DA_CACHE_FP8_E4M3:
      return launch(digest_kernel<DA_CACHE_FP8_E4M3>, grid, 32 * kDigestWarps, 0, stream, a);
    default:
      return launch(digest_kernel<DA_CACHE_FP4_E2M1>, grid, 32 * kDigestWarps, 0, stream, a);
  }
}

}  // namespace dattn
