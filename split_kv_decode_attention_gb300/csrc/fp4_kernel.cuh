// fp4_kernel.cuh -- the per-chunk kernel of split-KV decode attention over a
// 4-bit cache: E2M1 values with one E4M3 scale per 16 of them along d.
//
//     k_j[d] = k_scale * sf[j, d / 16] * e2m1(K[j, d]),   s_j = scale q . k_j,
//     o = v_scale * sum_j softmax(s)_j * sf[j, d / 16] * e2m1(V[j, d]).
//
// A token of a KV head is 2 x (64 + 8) bytes, 3.6 times fewer than in bf16, so
// the kernel is bound by HBM only while the widening stays cheap.  sf * e2m1
// has at most 6 significant bits and lies in [2^-10, 2688]: exact in f16.  The
// products therefore run on f16 operands (mma.sync m16n8k16, fp32
// accumulators) that are built in registers: one cvt widens a byte to an
// f16x2, one HMUL2 applies the block scale.  The fragment layouts are chosen
// so that no value moves between lanes:
//   * K (16 keys x 16 d per step, the MMA's A operand): a lane reads 16
//     contiguous bytes of one key, 32 values d = 32 t4 ..; step ks takes values
//     4 ks .. 4 ks + 3 of every lane, a permutation of d that Q's fragments
//     share, so the dot product is unchanged.  Those 32 values are two whole
//     scale blocks.
//   * V (16 d x 16 keys per step, the A operand of O^T = V^T P^T): a lane reads
//     8 bytes, one whole scale block d = 16 g4 .., of four keys; the two
//     nibbles of one d of two keys are brought together by two shifts and two
//     bit selects per 4 bytes, so that one cvt gives the (key, key') pair the
//     fragment wants.  Output tile mt holds d = 16 g4 + 2 mt and + 1.
//   * MMA key rows 0 .. 7 are keys 0, 3, 1, 2, 4, 7, 5, 6 (+ 8 for rows 8 and
//     up): with the TMA's 64-byte swizzle (16-byte chunk c of key j at c ^ (j /
//     2 % 4)) the lanes of every shared-memory phase, of K and of V, cover all
//     banks.
// Q is scaled per row by a power of two into f16's range (undone in fp32 on
// the scores).  P = 2^(x - m) is kept within [0, 2^15] rather than [0, 1]: m
// is the row's maximum less 6 when it was last moved, and it moves only when
// a score would pass 2^15, so most steps need no row maximum across lanes (one
// vote instead) and no rescaling, and P keeps values down to 2^-24 of 2^6.
// The LSE is summed in fp32 from unrounded values.
//
// A CTA takes HG KV heads (8, 4, 2 or 1) of a chunk; its W consumer warps take
// W / HG shares of each head's keys.  A head's 64 bytes of a token are a small
// piece of a DRAM page: boxes of one head stream at 2.9 TB/s, of two at 4.8, of
// four (256 contiguous bytes in a [page, slot, head, d] cache) and eight at
// 7.0, measured with nothing but the loads.  With HG = W a warp owns a head and
// its result needs no merge in the CTA.
//
// A producer warp keeps a ring of stages (32 keys of every consumer warp) full
// with TMA boxes (K, V and both block scales of up to 64 tokens of a page).  It
// is a warp of its own because issuing a box costs about 20 instructions: when
// the consumer that freed a stage issued its eight boxes, they took 1000 of the
// 3000 cycles of a step, always on the same, slowest warp.
// CM (HG = 1, calls of few and short chunks): the chunks of a head are a
// thread-block cluster and merge through distributed shared memory, so the
// call is one launch and writes no partials (one request of 4096 tokens, 32 / 8
// heads: 11 us replayed either way, but 7 and not 10 us of the host's time).
// Slots behind a sequence may hold anything: their scores are masked and
// their value scales replaced by zero.  More than 32 query rows per KV head run
// on the tcgen05 kernel.
//
// GB300, whole calls: 64 ragged requests of up to 32K tokens, 4 rows per head:
// 254 us, 5.4 TB/s, 0.80 of a copy's rate.  32 requests of up to 16K, 16 rows:
// 96 us, 3.5 TB/s, 0.52: there two consumer warps per scheduler (their 64
// accumulators and the widened operands fill the registers) issue 0.5
// instructions per cycle, the ALU and the tensor pipe each 39 % busy.  Twelve
// consumer warps, CTAs that stay and take item after item, V loaded before the
// softmax, and two to five stages were built and are slower or no faster.
#pragma once

#include <type_traits>

#include "decode_attn.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace dattn {
namespace fp4 {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 6.f;   // P is about 2^6 at the maximum when m moves
constexpr float kPTop = 15.f;    // m moves when P would pass 2^15
constexpr int kWarpKeys = 32;    // keys of a warp per stage

// Ring stages: 2 lose 10%, 4 and 5 cost the shared memory of a CTA and gain nothing.
constexpr int kRingStages = 3;
// Consumer warps, resident CTAs per SM and registers of a consumer thread in
// the 8-, 16- and 32-row variants.  A CTA is its consumers and a warpgroup for
// the producer, which hands its registers over: (consumers x regs + 128 x
// kProducerRegs) must not exceed the threads x the launch's registers, 65536 /
// (CTAs x threads) rounded down to 8.
constexpr int kShape[3][3] = {{4, 3, 128}, {8, 1, 232}, {8, 1, 232}};
constexpr int kProducerRegs = 32;

// NT: tiles of 8 query rows; HG: KV heads of a CTA.
template <int NT, int HG>
struct Fp4Cfg {
  static constexpr int kWarps = kShape[NT / 2][0];          // consumers
  static constexpr int kThreads = 32 * (kWarps + 4);        // and the producer's warpgroup
  static constexpr int kMinCtas = kShape[NT / 2][1];
  static constexpr int kRegs = kShape[NT / 2][2];
  static constexpr int kLaunchRegs = 65536 / (kMinCtas * kThreads) / 8 * 8;
  static_assert(kWarps % 4 == 0 && 32 * kWarps * kRegs + 128 * kProducerRegs <= kThreads * kLaunchRegs,
                "the register split would wait forever");
  static constexpr int kShares = kWarps / HG;               // warps of a head
  static_assert(kShares * HG == kWarps && (kShares & (kShares - 1)) == 0, "whole shares");
  static constexpr int kHalves = 2 * kShares;               // 16-token halves of a stage
  static constexpr int kStepTokens = 16 * kHalves;
  static constexpr int kStages = kRingStages;
  static constexpr int kRows = 8 * NT;
  // a stage: its tokens of K ([token][HG heads][64 B]), of V, then their block
  // scales (per box: [HG heads][tokens of the box][8 B])
  static constexpr int kHalfKv = HG * 16 * 64;
  static constexpr int kHalfSf = HG * 16 * 8;
  static constexpr int kOffV = kHalves * kHalfKv;
  static constexpr int kOffKs = 2 * kOffV;
  static constexpr int kOffVs = kOffKs + kHalves * kHalfSf;
  static constexpr int kStageBytes = kOffVs + kHalves * kHalfSf;
  static constexpr uint32_t kHalfBytes = 2 * (kHalfKv + kHalfSf);
  static_assert(kStageBytes % 512 == 0, "stages keep the swizzle's alignment");
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kRedStride = kHeadDim + 4;
  static constexpr int kRedBytes = kShares > 1 ? kWarps * kRows * kRedStride * 4 : 0;
  // cluster merge: the CTA's rows and their LSEs, behind the warps' in the idle ring
  static constexpr int kOutBytes = HG == 1 ? kRows * (kHeadDim + 4) * 4 : 0;
  static constexpr int kPipeBytes =
      kRingBytes > kRedBytes + kOutBytes ? kRingBytes : (kRedBytes + kOutBytes + 127) / 128 * 128;
  // Q fragments of several row tiles: [HG][4 step pairs][NT][32 lanes] of 16 B
  static constexpr bool kQSmem = NT > 1;
  static constexpr int kQBytes = kQSmem ? HG * 4 * NT * 512 : 0;
  static constexpr int kStatBytes = (2 * kWarps + HG) * kRows * 4;
  static constexpr int kBarBytes = kStages * 16;  // full and empty
  static constexpr int kSmemBytes = 1024 + kPipeBytes + kQBytes + kStatBytes + kBarBytes;
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// byte offset of 16-byte chunk c of key `key` (0 .. 15) of head hh in a half
// of K or V: 64-byte rows [key][head], in the TMA's 64-byte swizzle
template <int HG>
__device__ __forceinline__ uint32_t row_chunk(int key, int hh, int c) {
  const int r = key * HG + hh;
  return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// The page and the slot in it of the chunk's coming 16-token halves, for the
// producer warp: lane i holds those of half base + i, and of half base + 32 +
// i, loaded a window ahead.
struct HalfWindow {
  const int32_t* bt_row;  // nullptr: contiguous (page = request, slot = token)
  int b, t_begin, t_end, page_size, num_pages, lane;
  int32_t* status;
  int cur_pg, cur_sl, nxt_pg, nxt_sl, base;

  __device__ __forceinline__ void load(int first, int& pg, int& sl) const {
    const int64_t tok = static_cast<int64_t>(t_begin) + static_cast<int64_t>(first + lane) * 16;
    pg = 0;
    sl = 0;
    if (tok >= t_end) return;
    if (bt_row == nullptr) {
      pg = b;
      sl = static_cast<int>(tok);
      return;
    }
    const int col = static_cast<int>(tok) / page_size;
    sl = static_cast<int>(tok) - col * page_size;
    pg = __ldg(bt_row + col);
    if (pg < 0 || pg >= num_pages) {
      if (status != nullptr) atomicOr(status, static_cast<int32_t>(DA_STATUS_BAD_PAGE));
      pg = 0;
    }
  }
  __device__ __forceinline__ void init() {
    base = 0;
    load(0, cur_pg, cur_sl);
    load(32, nxt_pg, nxt_sl);
  }
  // (all lanes together; half rises by less than 32 from call to call)
  __device__ __forceinline__ void advance(int half) {
    if (half >= base + 32) {
      cur_pg = nxt_pg;
      cur_sl = nxt_sl;
      base += 32;
      load(base + 32, nxt_pg, nxt_sl);
    }
  }
};

// TR: the rows are a tree's or a padded batch's (rows.cuh).
template <int NT, int HG, bool CM, bool TR>
__global__ void __launch_bounds__(Fp4Cfg<NT, HG>::kThreads, Fp4Cfg<NT, HG>::kMinCtas)
    fp4_kernel(const __grid_constant__ Fp4Maps maps, const SplitArgs a) {
  using C = Fp4Cfg<NT, HG>;
  static_assert(!CM || HG == 1, "clusters are of one head's chunks");
  constexpr uint32_t kFull = 0xffffffffu;
  constexpr int W = C::kWarps;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g4 = lane >> 2;
  const int t4 = lane & 3;

  if (warp == W && lane == 0 && a.max_seq_len > 0) {
    prefetch_tensor_map(&maps.k);
    prefetch_tensor_map(&maps.v);
    prefetch_tensor_map(&maps.ks);
    prefetch_tensor_map(&maps.vs);
  }
  grid_dependency_wait();

  // ---- this CTA's work item: (chunk, KV head group, request)
  int split, unit, b, L, chunk;
  const bool listed = a.items != nullptr;
  int t0 = 0, rows = a.rows;  // first token of this CTA's rows, and their number (of a head)
  if (listed) {
    const int n_items = a.plan[1];
    const int4 itm = a.items[blockIdx.x];
    chunk = a.plan[0];
    if (static_cast<int>(blockIdx.x) >= n_items) return;
    b = itm.x;
    unit = itm.y;
    split = itm.z;
    L = itm.w;
  } else {
    split = blockIdx.x;
    unit = blockIdx.y;
    b = blockIdx.z;
    if constexpr (TR) {
      if (a.own.groups > 1) {
        t0 = b % a.own.groups * a.own.tokens;
        b /= a.own.groups;
        rows = min(rows, (a.q_len - t0) * a.group);
      }
    }
    // (a length per head only with HG = 1)
    L = a.seq_lens[static_cast<int64_t>(b) * a.len_sb + static_cast<int64_t>(unit) * a.len_sh];
    chunk = a.chunk_len;
    uint32_t bad = 0;
    if (L < 0 || L > a.max_seq_len) {
      bad |= DA_STATUS_SEQ_LEN;
      L = L < 0 ? 0 : a.max_seq_len;
    }
    if (a.causal && L > 0 && L < a.q_len) bad |= DA_STATUS_SHORT_CAUSAL;
    if (bad && a.status != nullptr && split == 0 && blockIdx.y == 0 && threadIdx.x == 0)
      atomicOr(a.status, static_cast<int32_t>(bad));
  }
  const int nsplit_b = L > 0 ? (L + chunk - 1) / chunk : 1;
  if (!CM && split >= nsplit_b) return;  // (a cluster stays whole: an empty chunk weighs nothing)
  const int t_begin = split * chunk;
  const int t_end = min(L, t_begin + chunk);
  const int n_steps = t_end > t_begin ? (t_end - t_begin + C::kStepTokens - 1) / C::kStepTokens : 0;
  const int hh = warp % HG;                              // this (consumer) warp's head of the group
  const int share = warp / HG;                           // and its share of the head's keys
  const int kvh = unit * HG + hh;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* q_smem = smem + C::kPipeBytes;
  float* stat_m = reinterpret_cast<float*>(smem + C::kPipeBytes + C::kQBytes);
  float* stat_l = stat_m + W * C::kRows;
  int* stat_e = reinterpret_cast<int*>(stat_l + W * C::kRows);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::kPipeBytes + C::kQBytes + C::kStatBytes);
  uint64_t* empty_bar = full_bar + C::kStages;
  const uint32_t ring = smem_addr(smem);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], W);
    }
    fence_mbar_init();
  }
  __syncthreads();

  const int box_halves = a.box_halves;  // 16-token halves of a box: 1, 2 or 4
  // =========================================================== producer warp
  if (warp >= W) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp > W) return;
    const int32_t* bt_row =
        a.paged ? a.block_table + static_cast<int64_t>(b) * a.bt_stride + static_cast<int64_t>(unit) * a.bt_sh
                : nullptr;
    HalfWindow win{bt_row, b, t_begin, t_end, a.page_size, a.num_pages, lane, a.status, 0, 0, 0, 0, 0};
    win.init();
    const uint64_t policy = l2_evict_first_policy();
    int stage = 0, issued = 0;
    uint32_t parity = 1;  // (the first use of a stage finds it empty)
    bool ok = true;
    for (int i = 0; i < n_steps; ++i) {
      // everything that does not need the stage, before the wait for it
      const int first = i * C::kHalves;  // half of the chunk
      win.advance(first);
      constexpr int kGroup = C::kHalves < 4 ? C::kHalves : 4;
      int pg[kGroup], sl[kGroup];
      auto place = [&](int h0) {
#pragma unroll
        for (int h = 0; h < kGroup; ++h) {
          const int src = (first - win.base + h0 + h) & 31;
          pg[h] = __shfl_sync(kFull, win.cur_pg, src);
          sl[h] = __shfl_sync(kFull, win.cur_sl, src);
        }
      };
      place(0);
      const int live = min(C::kHalves, (t_end - t_begin - first * 16 + 15) / 16);
      const uint32_t bytes = static_cast<uint32_t>((live + box_halves - 1) / box_halves * box_halves) * C::kHalfBytes;
      uint64_t* bar = &full_bar[stage];
      ok = __all_sync(kFull, mbar_wait_lazy(&empty_bar[stage], parity)) != 0;
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
#pragma unroll 1
      for (int h0 = 0; h0 < live; h0 += kGroup) {
        if (h0 > 0) place(h0);
        uint8_t* dst = smem + stage * C::kStageBytes;
        // (one thread issues, with uniform operands: lanes with maps and
        // coordinates of their own are serialised at a higher price)
        if (lane == 0) {
#pragma unroll
          for (int g = 0; g < kGroup; ++g) {
            const int h = h0 + g;
            if (h < live && (g & (box_halves - 1)) == 0) {
              tma_load_4d(dst + h * C::kHalfKv, &maps.k, bar, 0, unit * HG, sl[g], pg[g], policy);
              tma_load_4d(dst + C::kOffV + h * C::kHalfKv, &maps.v, bar, 0, unit * HG, sl[g], pg[g], policy);
              tma_load_4d(dst + C::kOffKs + h * C::kHalfSf, &maps.ks, bar, sl[g], unit * HG, 0, pg[g], policy);
              tma_load_4d(dst + C::kOffVs + h * C::kHalfSf, &maps.vs, bar, sl[g], unit * HG, 0, pg[g], policy);
            }
          }
        }
        __syncwarp();
      }
      ++issued;
      if (++stage == C::kStages) {
        stage = 0;
        parity ^= 1;
      }
    }
    if (lane == 0) {
      if (!ok && a.status != nullptr) atomicOr(a.status, static_cast<int32_t>(DA_STATUS_TIMEOUT));
      // do not leave while copies are in flight: wait (bounded) for the last ones
      for (int i = max(0, issued - C::kStages); i < issued; ++i)
        mbar_wait(&full_bar[i % C::kStages], (i / C::kStages) & 1);
    }
    return;
  }

  // ========================================================== consumer warps
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegs));
  // ---- Q fragments (B operand: row g4 of row tile nt, the lane's 32 d), and
  // the power of two that brings a row's largest value to [2^14, 2^15)
  uint32_t qf[C::kQSmem ? 1 : 8][2];
  int q_e = 0;  // (NT = 1: of row g4)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (C::kQSmem && nt % C::kShares != share) continue;  // one warp of the head prepares each row tile
    const int r = nt * 8 + g4;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      const int t = r / a.group;
      const uint16_t* qr = a.q + static_cast<int64_t>(b) * a.q_sb + static_cast<int64_t>(t0 + t) * a.q_st +
                           static_cast<int64_t>(kvh * a.group + (r - t * a.group)) * a.q_sh + 32 * t4;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(qr + 8 * i);
    }
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[4 * i] = x[i].x;
      w[4 * i + 1] = x[i].y;
      w[4 * i + 2] = x[i].z;
      w[4 * i + 3] = x[i].w;
    }
    uint32_t top = 0;  // the largest magnitude's bits (bf16 orders like integers)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    // (rows of zeros, or with infinities or NaN, as they are)
    const int e = top > 0 && top < 0x7f80u ? max(static_cast<int>(top >> 7), 1) - 127 - 14 : 0;
    // times 2^-e, in two factors since -e may exceed an exponent's range
    const float f1 = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23);
    const float f2 = __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
    uint32_t h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      h[i] = pack_f16x2(__uint_as_float(w[i] << 16) * f1 * f2,
                        __uint_as_float(w[i] & 0xffff0000u) * f1 * f2);
    if constexpr (C::kQSmem) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(q_smem + (((hh * 4 + i) * NT + nt) * 32 + lane) * 16) =
            make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
      if (t4 == 0) stat_e[hh * C::kRows + nt * 8 + g4] = e;
    } else {
      q_e = e;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qf[ks][0] = h[2 * ks];
        qf[ks][1] = h[2 * ks + 1];
      }
    }
  }
  if constexpr (C::kQSmem) named_barrier_sync(1, 32 * W);
  // per row of this thread's score columns (2 t4, 2 t4 + 1): the factor to
  // base-2 scores, and the keys it may see
  float rs[NT][2];
  int lim[NT][2];
  int lim_all = t_end;  // every row sees the keys below this
  OwnRows own;
  if constexpr (TR) {
    own = own_rows(a.own, a.q_len, b, L, split == 0 && unit == 0 && threadIdx.x == 0, a.status);
    lim_all = min(t_end, own.base);
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int row = nt * 8 + 2 * t4 + rr;
      int e;
      if constexpr (C::kQSmem) e = stat_e[hh * C::kRows + row];
      else e = __shfl_sync(kFull, q_e, (2 * t4 + rr) * 4);
      rs[nt][rr] = ldexpf(a.scale_log2, e);
      int lm = t_end;
      if constexpr (TR) {
        // (padding rows are dropped at the end and hold up nothing)
        if (t0 + row / a.group >= own.n) lm = 0;
        else lim_all = min(lim_all, lm);
      } else {
        if (a.causal && row < rows) lm = min(lm, L - a.q_len + 1 + row / a.group);
        lim_all = min(lim_all, lm);
      }
      lim[nt][rr] = lm;
    }
  lim_all = __reduce_min_sync(kFull, lim_all);

  // m: the running maximum (base 2) less kPShift, as rounded; P = 2^(x - m)
  float m[NT][2], l[NT][2], acc[8][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      m[nt][rr] = -INFINITY;
      l[nt][rr] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
  }

  const uint32_t q_addr = smem_addr(q_smem) + hh * 4 * NT * 512 + lane * 16;
  // key of MMA row g4 in a 16-key half: 0, 3, 1, 2, 4, 7, 5, 6
  const int krow = 4 * (g4 >> 2) + ((g4 & 1) ? 2 + (((g4 >> 1) & 1) ^ 1) : (g4 >> 1) & 1);
  // keys of MMA columns 2 t4 and 2 t4 + 1
  const int vkey0 = 4 * (t4 >> 1) + (t4 & 1), vkey1 = 4 * (t4 >> 1) + 2 + ((t4 & 1) ^ 1);
  // this lane's offsets in a stage; 8 keys further on everything is at a fixed
  // distance (the swizzle repeats)
  constexpr uint32_t kKeys8 = 8 * HG * 64;
  const uint32_t k_off = 2 * share * C::kHalfKv + row_chunk<HG>(krow, hh, t4);
  const uint32_t v_off0 = C::kOffV + 2 * share * C::kHalfKv + row_chunk<HG>(vkey0, hh, g4 >> 1) + (g4 & 1) * 8;
  const uint32_t v_off1 = C::kOffV + 2 * share * C::kHalfKv + row_chunk<HG>(vkey1, hh, g4 >> 1) + (g4 & 1) * 8;
  // the warp's two halves begin share * 32 tokens into the stage: the block scales' box, and the
  // place in it; the second half is 16 tokens on in the box, or the next box
  const uint32_t sf_box = (2 * share) / box_halves * box_halves;
  const uint32_t sf_off = sf_box * C::kHalfSf + hh * box_halves * 128 + (2 * share - sf_box) * 128;
  const uint32_t sf_half = box_halves > 1 ? 128 : C::kHalfSf;
  const uint32_t ks_off = C::kOffKs + sf_off + krow * 8 + 2 * t4;
  const uint32_t vs_off0 = C::kOffVs + sf_off + vkey0 * 8 + g4;
  const uint32_t vs_off1 = C::kOffVs + sf_off + vkey1 * 8 + g4;
  // One warp's 32 keys of a stage at st, the first of them token tok0 (FULL:
  // every row sees all of them).
  auto consume = [&](auto full_tag, uint32_t st, int tok0, auto&& release) {
    constexpr bool FULL = decltype(full_tag)::value;
    // ---- S^T[32 keys x 8 NT rows] = K . Q^T
    float sc[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[h][nt][j] = 0.f;
      const uint4 w0 = lds128(st + k_off + h * C::kHalfKv);
      const uint4 w1 = lds128(st + k_off + h * C::kHalfKv + kKeys8);
      const uint32_t s0 = e4m3x2_to_f16x2(lds_u16(st + ks_off + h * sf_half));
      const uint32_t s1 = e4m3x2_to_f16x2(lds_u16(st + ks_off + h * sf_half + 64));
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // the lane's two scale blocks: steps 0-3, 4-7
        const uint32_t sa = __byte_perm(s0, 0, half ? 0x3232 : 0x1010);
        const uint32_t sb = __byte_perm(s1, 0, half ? 0x3232 : 0x1010);
#pragma unroll
        for (int kp = 0; kp < 2; ++kp) {
          const uint32_t wa = half ? (kp ? w0.w : w0.z) : (kp ? w0.y : w0.x);
          const uint32_t wb = half ? (kp ? w1.w : w1.z) : (kp ? w1.y : w1.x);
          uint32_t ca[4], cb[4];
          e2m1x8_to_f16(wa, ca);
          e2m1x8_to_f16(wb, cb);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ca[j] = hmul2(ca[j], sa);
            cb[j] = hmul2(cb[j], sb);
          }
          const uint32_t a0[4] = {ca[0], cb[0], ca[1], cb[1]};
          const uint32_t a1[4] = {ca[2], cb[2], ca[3], cb[3]};
          const int ks = half * 4 + kp * 2;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (C::kQSmem) {
              const uint4 qb = lds128(q_addr + ((ks >> 1) * NT + nt) * 512);
              mma_f16_16816(sc[h][nt], a0, qb.x, qb.y);
              mma_f16_16816(sc[h][nt], a1, qb.z, qb.w);
            } else {
              mma_f16_16816(sc[h][nt], a0, qf[ks][0], qf[ks][1]);
              mma_f16_16816(sc[h][nt], a1, qf[ks + 1][0], qf[ks + 1][1]);
            }
          }
        }
      }
    }

    // ---- online softmax over the step (base 2)
    bool move = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) sc[h][nt][2 * j + rr] *= rs[nt][rr];
        if constexpr (!FULL) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (tok0 + 16 * h + 8 * j + krow >= lim[nt][rr]) sc[h][nt][2 * j + rr] = -INFINITY;
          if constexpr (TR) {
            const int t = t0 + (nt * 8 + 2 * t4 + rr) / a.group;
            if (tok0 + kWarpKeys > own.base && t < own.n) {
              const uint32_t seen = own.bits(t, tok0);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if (((seen >> (16 * h + 8 * j + krow)) & 1u) == 0) sc[h][nt][2 * j + rr] = -INFINITY;
            }
          }
        }
        const float mx = fmaxf(fmax3(sc[0][nt][rr], sc[0][nt][2 + rr], sc[1][nt][rr]), sc[1][nt][2 + rr]);
        move |= mx > m[nt][rr] + kPTop;
      }
    if (__any_sync(kFull, move)) {  // (seldom after the first step)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          float mx = fmaxf(fmax3(sc[0][nt][rr], sc[0][nt][2 + rr], sc[1][nt][rr]), sc[1][nt][2 + rr]);
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
          const float m_new = fmaxf(m[nt][rr], mx - kPShift);
          const float alpha = ex2(m[nt][rr] - (m_new == -INFINITY ? 0.f : m_new));
          m[nt][rr] = m_new;
          l[nt][rr] *= alpha;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            acc[mt][nt][rr] *= alpha;
            acc[mt][nt][2 + rr] *= alpha;
          }
        }
    }
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const float m_use = m[nt][rr] == -INFINITY ? 0.f : m[nt][rr];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) sc[h][nt][2 * j + rr] = ex2(sc[h][nt][2 * j + rr] - m_use);
        l[nt][rr] += (sc[0][nt][rr] + sc[0][nt][2 + rr]) + (sc[1][nt][rr] + sc[1][nt][2 + rr]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        pb[h][nt][0] = movmatrix_trans(pack_f16x2(sc[h][nt][0], sc[h][nt][1]));
        pb[h][nt][1] = movmatrix_trans(pack_f16x2(sc[h][nt][2], sc[h][nt][3]));
      }
    }

    // ---- O^T[128 d x 8 NT rows] += V^T . P^T
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2 v[4];
      uint32_t vs[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = lds64(st + ((j & 1) ? v_off1 : v_off0) + h * C::kHalfKv + (j >> 1) * kKeys8);
        vs[j] = lds_u8(st + ((j & 1) ? vs_off1 : vs_off0) + h * sf_half + (j >> 1) * 64);
        // slots behind the sequence may hold anything: 0 x NaN is NaN
        if constexpr (!FULL)
          if (tok0 + 16 * h + ((j & 1) ? vkey1 : vkey0) + 8 * (j >> 1) >= t_end) vs[j] = 0u;
      }
      if (h == 1) release();
      const uint32_t s01 = e4m3x2_to_f16x2(__byte_perm(vs[0], vs[1], 0x0040));
      const uint32_t s23 = e4m3x2_to_f16x2(__byte_perm(vs[2], vs[3], 0x0040));
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // bytes 0-3, 4-7 of the block: mt 0-3, 4-7
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = half ? v[j].y : v[j].x;
        constexpr uint32_t kLow = 0x0f0f0f0fu;
        // low nibbles (d even) of two keys side by side, then high ones (d odd)
        uint32_t e01[4], o01[4], e23[4], o23[4];
        e2m1x8_to_f16((x[0] & kLow) | ((x[1] << 4) & ~kLow), e01);
        e2m1x8_to_f16(((x[0] >> 4) & kLow) | (x[1] & ~kLow), o01);
        e2m1x8_to_f16((x[2] & kLow) | ((x[3] << 4) & ~kLow), e23);
        e2m1x8_to_f16(((x[2] >> 4) & kLow) | (x[3] & ~kLow), o23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t af[4] = {hmul2(e01[j], s01), hmul2(o01[j], s01), hmul2(e23[j], s23),
                                  hmul2(o23[j], s23)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16_16816(acc[half * 4 + j][nt], af, pb[h][nt][0], pb[h][nt][1]);
        }
      }
    }
  };

  bool ok = true;
  int stage = 0;
  uint32_t parity = 0;
  for (int i = 0; i < n_steps; ++i) {
    ok = __all_sync(kFull, mbar_wait_lazy(&full_bar[stage], parity)) != 0;
    if (!ok) break;
    const int tok0 = t_begin + i * C::kStepTokens + share * kWarpKeys;
    auto release = [&]() {  // this warp is done with the stage
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[stage]);
    };
    if (tok0 + kWarpKeys <= lim_all) consume(std::true_type{}, ring + stage * C::kStageBytes, tok0, release);
    else if (tok0 < t_end) consume(std::false_type{}, ring + stage * C::kStageBytes, tok0, release);
    else release();
    if (++stage == C::kStages) {
      stage = 0;
      parity ^= 1;
    }
  }
  if (!ok && lane == 0 && a.status != nullptr)
    atomicOr(a.status, static_cast<int32_t>(DA_STATUS_TIMEOUT));

  if (!CM && threadIdx.x == 0) allow_dependent_launch();

  if constexpr (TR) {
    // padding rows weigh nothing, whatever their q held, nor do rows that saw
    // nothing here, whatever the values hold
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr)
        if (t0 + (nt * 8 + 2 * t4 + rr) / a.group >= own.n || (m[nt][rr] == -INFINITY && l[nt][rr] == 0.f)) {
          m[nt][rr] = -INFINITY;
          l[nt][rr] = 0.f;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) acc[mt][nt][rr] = acc[mt][nt][2 + rr] = 0.f;
        }
  }
  // ---- the rows' sums over the lanes of the warp
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      float v = l[nt][rr];
      v += __shfl_xor_sync(kFull, v, 4);
      v += __shfl_xor_sync(kFull, v, 8);
      v += __shfl_xor_sync(kFull, v, 16);
      l[nt][rr] = v;
    }
  const bool direct = nsplit_b == 1;
  const int S = a.num_splits;
  // where a row of this head goes: its (token, head), and its partial's index
  auto place = [&](int row, int head, int& t) {
    const int tr = row / a.group;
    t = t0 + tr;
    return (unit * HG + head) * a.group + (row - tr * a.group);
  };
  auto part_index = [&](int row, int head, int t, int h) {
    return listed ? (static_cast<int64_t>(blockIdx.x) * HG + head) * a.rows + row
                  : ((static_cast<int64_t>(b) * a.q_len + t) * a.num_q_heads + h) * S + split;
  };
  auto put_lse = [&](int row, int head, float m2, float sum) {
    const float lse = sum == 0.f ? -INFINITY : (m2 + log2f(sum)) * kLn2;
    int t;
    const int h = place(row, head, t);
    if (direct) a.lse[(static_cast<int64_t>(b) * a.q_len + t) * a.num_q_heads + h] = lse;
    else st_global_hint(a.part_lse + part_index(row, head, t, h), lse, l2_evict_last_policy());
  };
  auto out_row = [&](int t, int h) {
    return a.out + static_cast<int64_t>(b) * a.o_sb + static_cast<int64_t>(t) * a.o_st +
           static_cast<int64_t>(h) * a.o_sh;
  };

  if constexpr (C::kShares == 1) {
    // ---- the warp has all of its head's keys: a lane holds d = 16 g4 .. + 15
    // of rows 2 t4 and 2 t4 + 1 of each tile
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int row = nt * 8 + 2 * t4 + rr;
        if (row >= rows) continue;
        const float sum = l[nt][rr];
        const float fac = (sum == 0.f ? 0.f : 1.f / sum) * a.v_scale;
        float o[16];
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          o[2 * mt] = acc[mt][nt][rr] * fac;
          o[2 * mt + 1] = acc[mt][nt][2 + rr] * fac;
        }
        int t;
        const int h = place(row, hh, t);
        if (direct) {
          uint4* dst = reinterpret_cast<uint4*>(out_row(t, h) + 16 * g4);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            dst[q] = make_uint4(pack_bf16x2(o[8 * q], o[8 * q + 1]), pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                                pack_bf16x2(o[8 * q + 4], o[8 * q + 5]), pack_bf16x2(o[8 * q + 6], o[8 * q + 7]));
        } else {
          float* dst = a.part_o + part_index(row, hh, t, h) * kHeadDim + 16 * g4;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            st_global_hint(dst + 4 * q, make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]),
                           l2_evict_last_policy());
        }
        if (g4 == 0) put_lse(row, hh, m[nt][rr] == -INFINITY ? 0.f : m[nt][rr], sum);
      }
    return;
  } else {
    // ---- merge the (m, l, O) of the warps that share a head
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr)
        if (g4 == 0) {
          stat_m[warp * C::kRows + nt * 8 + 2 * t4 + rr] = m[nt][rr];
          stat_l[warp * C::kRows + nt * 8 + 2 * t4 + rr] = l[nt][rr];
        }
    named_barrier_sync(1, 32 * W);  // (and every warp is past the ring)
    // the largest m of the head's warps, and the sum of weights under it
    auto row_stats = [&](int row, int head, float& Mu, float& sum) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::kShares; ++w) M = fmaxf(M, stat_m[(head + w * HG) * C::kRows + row]);
      Mu = M == -INFINITY ? 0.f : M;
      sum = 0.f;
#pragma unroll
      for (int w = 0; w < C::kShares; ++w)
        sum += stat_l[(head + w * HG) * C::kRows + row] * ex2(stat_m[(head + w * HG) * C::kRows + row] - Mu);
    };
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int row = nt * 8 + 2 * t4 + rr;
        float Mu, sum;
        row_stats(row, hh, Mu, sum);
        const float fac = (sum == 0.f ? 0.f : ex2(m[nt][rr] - Mu) / sum) * a.v_scale;
        float* dst = red + (warp * C::kRows + row) * C::kRedStride + 16 * g4;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
          *reinterpret_cast<float2*>(dst + 2 * mt) =
              make_float2(acc[mt][nt][rr] * fac, acc[mt][nt][2 + rr] * fac);
      }
    named_barrier_sync(1, 32 * W);
    if constexpr (CM) {
      // ---- publish the CTA's rows and LSEs, then each CTA of the cluster
      // merges its share of the (row, 4 d) units from all of them
      float* xo = red + C::kRedBytes / 4;
      float* xl = xo + C::kRows * kHeadDim;
      for (int idx = threadIdx.x; idx < rows * 32; idx += 32 * W) {
        const int row = idx >> 5, d = (idx & 31) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kShares; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(red + (w * C::kRows + row) * C::kRedStride + d);
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
        }
        *reinterpret_cast<float4*>(xo + row * kHeadDim + d) = v;
        if (d == 0) {
          float Mu, sum;
          row_stats(row, 0, Mu, sum);
          xl[row] = sum == 0.f ? -INFINITY : (Mu + log2f(sum)) * kLn2;
        }
      }
      cluster_sync();
      const uint32_t ao = smem_addr(xo), al = smem_addr(xl);
      for (int u = split + S * static_cast<int>(threadIdx.x); u < rows * 32; u += S * 32 * W) {
        const int row = u >> 5, d = (u & 31) * 4;
        float x[16];
        float4 v[16];
        float M = -INFINITY;
#pragma unroll
        for (int r = 0; r < 16; ++r) {  // (all peers' values on their way together)
          x[r] = -INFINITY;
          if (r < S) {
            x[r] = ld_cluster_f32(map_to_rank(al + row * 4, r));
            v[r] = ld_cluster_f32x4(map_to_rank(ao + (row * kHeadDim + d) * 4, r));
          }
          M = fmaxf(M, x[r]);
        }
        const float Mu = M == -INFINITY ? 0.f : M;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (r < S) {
            const float w = ex2((x[r] - Mu) * 1.4426950408889634f);
            sum += w;
            o.x += w * v[r].x;
            o.y += w * v[r].y;
            o.z += w * v[r].z;
            o.w += w * v[r].w;
          }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        int t;
        const int h = place(row, 0, t);
        *reinterpret_cast<uint2*>(out_row(t, h) + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (d == 0)
          a.lse[(static_cast<int64_t>(b) * a.q_len + t) * a.num_q_heads + h] =
              sum == 0.f ? -INFINITY : Mu + logf(sum);
      }
      cluster_sync();  // no CTA leaves while another may still read its shared memory
    }
    if constexpr (!CM) {
    for (int idx = threadIdx.x; idx < HG * rows * 32; idx += 32 * W) {
      const int d = (idx & 31) * 4;
      const int head = (idx >> 5) / rows;
      const int row = (idx >> 5) - head * rows;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::kShares; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(
            red + ((head + w * HG) * C::kRows + row) * C::kRedStride + d);
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
      }
      int t;
      const int h = place(row, head, t);
      if (direct)
        *reinterpret_cast<uint2*>(out_row(t, h) + d) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      else
        st_global_hint(a.part_o + part_index(row, head, t, h) * kHeadDim + d, v, l2_evict_last_policy());
    }
    for (int idx = threadIdx.x; idx < HG * rows; idx += 32 * W) {
      const int head = idx / rows;
      const int row = idx - head * rows;
      float Mu, sum;
      row_stats(row, head, Mu, sum);
      put_lse(row, head, Mu, sum);
    }
    }
  }
}

// DATTN_ROWS (translation units of their own): the instantiations for rows of a
// tree or a padded batch.
#ifndef DATTN_ROWS
#define DATTN_ROWS 0
#endif
constexpr bool kOwnRows = DATTN_ROWS != 0;

// Launch the variant of NT row tiles and HG heads.
template <int NT, int HG, bool TR, bool CM = false>
cudaError_t launch_one(const Fp4Maps& maps, const SplitArgs& a, cudaStream_t stream) {
  using C = Fp4Cfg<NT, HG>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = a.items != nullptr ? dim3(static_cast<unsigned>(a.item_slots))
                                   : dim3(a.num_splits, a.num_kv_heads / HG, a.batch);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.num_splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CM ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fp4_kernel<NT, HG, CM, TR>, maps, a);
}

// Set the variant's attributes on the current device; its resident CTAs per SM.
template <int NT, int HG, bool TR>
cudaError_t prepare_one(int* ctas) {
  using C = Fp4Cfg<NT, HG>;
  cudaError_t e = cudaFuncSetAttribute(fp4_kernel<NT, HG, false, TR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmemBytes);
  if (e != cudaSuccess) return e;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, fp4_kernel<NT, HG, false, TR>, C::kThreads, C::kSmemBytes);
}

// The same for the cluster form, and how many clusters of `splits` CTAs fit at once.
template <int NT, bool TR>
cudaError_t prepare_clusters(int splits, int* clusters) {
  using C = Fp4Cfg<NT, 1>;
  auto* kernel = fp4_kernel<NT, 1, true, TR>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(splits), 1, 1);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(clusters, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();  // (a rejected query is no error)
    *clusters = 0;
  }
  return cudaSuccess;
}

// The variants of one row-tile count (a translation unit each).
template <int NT, bool TR>
struct Variants {
  static cudaError_t launch(int hg, bool cluster, const Fp4Maps& maps, const SplitArgs& a, cudaStream_t stream);
  static cudaError_t prepare(int hg, int* ctas);
  static cudaError_t clusters(int splits, int* n);
  static int warps();  // consumer warps of a CTA
};

#define DATTN_FP4_VARIANTS(NT)                                                                          \
  template <>                                                                                           \
  cudaError_t Variants<NT, kOwnRows>::launch(int hg, bool cluster, const Fp4Maps& maps, const SplitArgs& a,\
                                   cudaStream_t st) {                                                   \
    if (cluster) return launch_one<NT, 1, kOwnRows, true>(maps, a, st);                                 \
    switch (hg) {                                                                                       \
      case 8: return launch_one<NT, kShape[NT / 2][0] == 8 ? 8 : 4, kOwnRows>(maps, a, st);             \
      case 4: return launch_one<NT, 4, kOwnRows>(maps, a, st);                                          \
      case 2: return launch_one<NT, 2, kOwnRows>(maps, a, st);                                          \
      default: return launch_one<NT, 1, kOwnRows>(maps, a, st);                                         \
    }                                                                                                   \
  }                                                                                                     \
  template <>                                                                                           \
  cudaError_t Variants<NT, kOwnRows>::prepare(int hg, int* ctas) {                                      \
    switch (hg) {                                                                                       \
      case 8: return prepare_one<NT, kShape[NT / 2][0] == 8 ? 8 : 4, kOwnRows>(ctas);                   \
      case 4: return prepare_one<NT, 4, kOwnRows>(ctas);                                                \
      case 2: return prepare_one<NT, 2, kOwnRows>(ctas);                                                \
      default: return prepare_one<NT, 1, kOwnRows>(ctas);                                               \
    }                                                                                                   \
  }                                                                                                     \
  template <>                                                                                           \
  cudaError_t Variants<NT, kOwnRows>::clusters(int splits, int* n) {                                    \
    return prepare_clusters<NT, kOwnRows>(splits, n);                                                   \
  }                                                                                                     \
  template <>                                                                                           \
  int Variants<NT, kOwnRows>::warps() {                                                                 \
    return kShape[NT / 2][0];                                                                           \
  }

}  // namespace fp4
}  // namespace dattn
