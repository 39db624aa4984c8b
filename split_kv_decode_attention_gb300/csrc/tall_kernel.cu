// tall_kernel.cu -- attention of more than 128 query rows per KV head (prompts
// over an encoder's states, large trees of drafts) over bf16 keys and values, on
// the fifth-generation tensor cores.
//
// For the rows r = (t, g) of a (request, kv head), t a token and g a head of the
// group, over the keys j that rows.cuh says they see:
//     s_rj = scale q_r . k_j,   o_r = sum_j softmax(s_r)_j v_j,
// in one pass with the running maximum m and sum l: when m grows, l and o are
// scaled by 2^(m - m').  With 256 rows a key is used 256 times per read, so the
// tensor pipe bounds the kernel and not HBM: per 128 keys and 256 rows it is busy
// for 4 x 128^3 x 2 multiply-adds, and everything else has to fit beside that.
//
// A CTA takes 256 rows as two tiles of 128, one per softmax warpgroup, over a
// chunk of the keys, 128 at a time.  Per key tile and row tile the tensor core
// makes S = Q K^T (Q, K from shared memory) and O += P V (P from TMEM): while it
// works for one row tile, the other's warpgroup turns its scores into P, so that
// neither waits for long.  TMEM holds S of both tiles (128 columns each; P, in
// bf16, replaces the first 64 of them) and both O: all 512 columns.  The MMAs of
// one thread run in the order of their issue, so the next S of a tile is issued
// behind the P V that reads the P it overwrites, and its completion also says
// that O may be touched.
// O is rescaled only when a row's maximum has grown by more than 2^8 (P stays
// below 2^8 and is exact in the end's division), which is rare after the first
// tiles.  P is rounded to bf16; O is divided by the sum of the rounded weights,
// the log-sum-exp takes the sum of the fp32 ones.
// Three producer warps fill a ring of five 32 KB slots (128 keys of K or of V)
// with TMA boxes of up to 128 tokens (what divides a page).
// Values of keys behind a sequence may be anything: they are zeroed in shared
// memory (0 x NaN is NaN).  Every wait is bounded.

#include <mutex>

#include "decode_attn.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rows.cuh"
#include "tcgen05.cuh"

namespace dattn {
namespace {

constexpr float kLn2t = 0.6931471805599453f;
constexpr int kTRows = 128;                       // rows of a tile (MMA M)
constexpr int kTKeys = 128;                       // keys of a tile (MMA N of S, K of P V)
constexpr int kTHalf = kTKeys * 128;              // [128 tokens][64 d] bf16 = 16 KB
constexpr int kTSlot = 2 * kTHalf;                // K or V of a key tile
constexpr int kTSlots = 5;
constexpr int kTProducers = 3;
constexpr int kTMmaWarp = 8;
constexpr int kTThreads = 32 * (kTMmaWarp + 1 + kTProducers);
constexpr int kTOffRing = 2 * kTSlot;             // behind the two Q tiles
constexpr int kTOffBar = kTOffRing + kTSlots * kTSlot;
constexpr int kTBars = 2 * kTSlots + 1 + 2 + 2 + 2 + 1;
constexpr int kTSmem = 1024 + kTOffBar + kTBars * 8 + 16;
static_assert(kTSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kTTmemCols = 512;
constexpr uint32_t kTColO = 256;
constexpr float kTRescale = 8.f;                  // log2 units
// registers: 65536 / 384 threads, rounded down to 8, is what the launch gives
constexpr int kTLaunchRegs = 65536 / kTThreads / 8 * 8;
constexpr int kTSoftmaxRegs = 208;
constexpr int kTOtherRegs = 80;
static_assert(256 * kTSoftmaxRegs + 128 * kTOtherRegs <= kTThreads * kTLaunchRegs,
              "the register split would wait forever");

struct TallMaps {
  CUtensorMap k, v;
};

__global__ void __launch_bounds__(kTThreads, 1)
    tall_kernel(const __grid_constant__ TallMaps maps, const SplitArgs a, const int box_tokens) {
  constexpr uint32_t kFull = 0xffffffffu;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  grid_dependency_wait();

  // ---- this CTA's item: chunk `split` of request b, KV head kvh, rows r0 ..
  const int S = a.num_splits;
  const int pair = blockIdx.x / S;
  const int split = blockIdx.x - pair * S;
  const int kvh = blockIdx.y;
  const int b = blockIdx.z;
  const int chunk = a.chunk_len;
  int L = a.seq_lens[b];
  const bool report = blockIdx.x == 0 && kvh == 0 && tid == 0;
  if (L < 0 || L > a.max_seq_len) {
    if (report && a.status != nullptr) atomicOr(a.status, static_cast<int32_t>(DA_STATUS_SEQ_LEN));
    L = L < 0 ? 0 : a.max_seq_len;
  }
  const OwnRows own = own_rows(a.own, a.q_len, b, L, report, a.status);
  const int nsplit_b = L > 0 ? (L + chunk - 1) / chunk : 1;
  if (split >= nsplit_b) return;
  const int t_begin = split * chunk;
  const int t_end = min(L, t_begin + chunk);
  const int n_iters = t_end > t_begin ? (t_end - t_begin + kTKeys - 1) / kTKeys : 0;
  const int r0 = pair * 2 * kTRows;
  const int own_rows_n = min(a.rows, own.n * a.group);  // (rows are (t, g), t slowest)
  // row tiles with rows of the request's own; none without keys
  const int tiles = n_iters == 0 ? 0 : r0 + kTRows < own_rows_n ? 2 : r0 < own_rows_n ? 1 : 0;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + kTOffBar);  // [slots] bytes landed
  uint64_t* empty_bar = full_bar + kTSlots;                           // [slots] read by the MMAs
  uint64_t* q_full = empty_bar + kTSlots;                             // Q in shared memory
  uint64_t* s_full = q_full + 1;                                      // [2] scores in TMEM
  uint64_t* p_full = s_full + 2;                                      // [2] P in TMEM
  uint64_t* o_done = p_full + 2;                                      // [2] the last P V
  uint64_t* tmem_done = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tmem_done + 1);

  if (tiles > 0) {  // (the same for the whole CTA)
    if (tid == 0) {
      for (int s = 0; s < kTSlots; ++s) {
        mbar_init(&full_bar[s], 1);
        mbar_init(&empty_bar[s], 1);
      }
      mbar_init(q_full, 8);
      for (int g = 0; g < 2; ++g) {
        mbar_init(&s_full[g], 1);
        mbar_init(&p_full[g], 4);
        mbar_init(&o_done[g], 1);
      }
      mbar_init(tmem_done, 8);
      fence_mbar_init();
    }
    if (warp == kTMmaWarp) {
      tmem_alloc(tmem_slot, kTTmemCols);
      tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
  }
  const uint32_t smem_base = smem_addr(smem);

  if (warp >= kTMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTOtherRegs));
    if (tiles == 0) return;
    const uint32_t tmem = *tmem_slot;
    if (warp > kTMmaWarp) {
      // ========================================================== TMA producers
      // unit u: K (even) or V (odd) of key tile u / 2, in slot u % kTSlots; each
      // producer warp takes every third.  A lane issues one box.
      const int pw = warp - kTMmaWarp - 1;
      if (lane == 0 && pw == 0) {
        prefetch_tensor_map(&maps.k);
        prefetch_tensor_map(&maps.v);
      }
      const int boxes = 2 * (kTKeys / box_tokens);  // of a unit: [token box][d half]
      const int half = lane & 1;
      const int box_tok = (lane >> 1) * box_tokens;  // of the lane's box in the tile
      const uint32_t box_bytes = static_cast<uint32_t>(box_tokens) * 128u;
      const int32_t* bt_row = a.paged ? a.block_table + static_cast<int64_t>(b) * a.bt_stride : nullptr;
      auto page_of = [&](int u) {
        const int64_t tok = static_cast<int64_t>(t_begin) + static_cast<int64_t>(u >> 1) * kTKeys + box_tok;
        return bt_row != nullptr && lane < boxes && tok < t_end ? __ldg(bt_row + tok / a.page_size) : 0;
      };
      const int units = 2 * n_iters;
      int last = -1;
      bool ok = true;
      int pg_next = page_of(pw);
      for (int u = pw; u < units; u += kTProducers) {
        const int s = u % kTSlots, use = u / kTSlots;
        int pg = pg_next;
        pg_next = page_of(u + kTProducers);
        if (use > 0) ok = __all_sync(kFull, mbar_wait_lazy(&empty_bar[s], (use - 1) & 1)) != 0;
        if (!ok) break;
        const int tok0 = t_begin + (u >> 1) * kTKeys;
        const int live = min(kTKeys / box_tokens, (t_end - tok0 + box_tokens - 1) / box_tokens);
        if (lane == 0) mbar_arrive_expect_tx(&full_bar[s], 2u * live * box_bytes);
        __syncwarp();
        if (lane < 2 * live) {
          if (a.paged && static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
            if (a.status != nullptr) atomicOr(a.status, static_cast<int32_t>(DA_STATUS_BAD_PAGE));
            pg = 0;
          }
          const int tok = tok0 + box_tok;
          uint8_t* dst = smem + kTOffRing + s * kTSlot + half * kTHalf + box_tok * 128;
          // (other CTAs read the same keys: no eviction hint)
          tma_load_4d_plain(dst, (u & 1) ? &maps.v : &maps.k, &full_bar[s], half * 64, kvh,
                            a.paged ? tok % a.page_size : tok, a.paged ? pg : b);
        }
        __syncwarp();
        last = u;
      }
      if (lane == 0) {
        if (!ok && a.status != nullptr) atomicOr(a.status, static_cast<int32_t>(DA_STATUS_TIMEOUT));
        // no copy of this warp may still be landing when the CTA exits: wait
        // (bounded) for its units whose slots no later unit uses
        const int first = ok ? units - kTSlots : last - kTSlots + 1;
        for (int u = last; u >= max(0, first); u -= kTProducers)
          mbar_wait(&full_bar[u % kTSlots], (u / kTSlots) & 1);
      }
      return;
    }

    // ============================================================== MMA issuer
    constexpr uint32_t kIdescS = umma_idesc_bf16(kTRows, kTKeys, false, false);
    constexpr uint32_t kIdescO = umma_idesc_bf16(kTRows, kHeadDim, false, true);
    const uint64_t q_desc = umma_smem_desc(smem_base, 16, 1024);
    const uint64_t k_desc = umma_smem_desc(smem_base + kTOffRing, 16, 1024);
    // V [128 keys][2 x 64 d], MN-major: d halves kTHalf apart, 8-key groups 1 KB
    const uint64_t v_desc = umma_smem_desc(smem_base + kTOffRing, kTHalf, 1024);
    auto issue_s = [&](int g, int slot) {
      const uint64_t qd = q_desc + static_cast<uint64_t>(g * (kTSlot >> 4));
      const uint64_t kd = k_desc + static_cast<uint64_t>(slot * (kTSlot >> 4));
      const uint32_t d = tmem + g * kTKeys;
#pragma unroll
      for (int kk = 0; kk < kHeadDim / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kTHalf + (kk & 3) * 32) >> 4;
        umma_bf16_ss_warp(d, qd + off, kd + off, kIdescS, kk > 0 ? 1u : 0u);
      }
      umma_commit_warp(&s_full[g]);
    };
    auto issue_o = [&](int g, int slot, bool first) {
      const uint64_t vd = v_desc + static_cast<uint64_t>(slot * (kTSlot >> 4));
      const uint32_t d = tmem + kTColO + g * kHeadDim;
#pragma unroll
      for (int kk = 0; kk < kTKeys / 16; ++kk)
        umma_bf16_ts_warp(d, tmem + g * kTKeys + kk * 8, vd + kk * (2048 >> 4), kIdescO,
                          (!first || kk > 0) ? 1u : 0u);
    };
    auto landed = [&](int u) {
      return __all_sync(kFull, mbar_wait_lazy(&full_bar[u % kTSlots], (u / kTSlots) & 1)) != 0;
    };
    bool ok = __all_sync(kFull, mbar_wait_lazy(q_full, 0)) != 0 && landed(0);
    if (ok) {
      tc_fence_after_sync();
      for (int g = 0; g < tiles; ++g) issue_s(g, 0);
      umma_commit_warp(&empty_bar[0]);
    }
    for (int j = 0; ok && j < n_iters; ++j) {
      const int uv = 2 * j + 1, uk = 2 * j + 2;
      const bool more = j + 1 < n_iters;
      ok = landed(uv);
      for (int g = 0; ok && g < tiles; ++g) {
        ok = __all_sync(kFull, mbar_wait_lazy(&p_full[g], j & 1)) != 0;
        if (!ok) break;
        tc_fence_after_sync();
        issue_o(g, uv % kTSlots, j == 0);
        if (g == tiles - 1) umma_commit_warp(&empty_bar[uv % kTSlots]);
        if (more) {
          if (g == 0) ok = landed(uk);
          if (!ok) break;
          issue_s(g, uk % kTSlots);
          if (g == tiles - 1) umma_commit_warp(&empty_bar[uk % kTSlots]);
        } else {
          umma_commit_warp(&o_done[g]);
        }
      }
    }
    // TMEM is released once the softmax warps are done with it.  After a wait
    // that ran out a softmax warp passes at most one more (o_done) before it
    // arrives here; five limits cover it, and past them TMEM is released anyway.
    ok = (__all_sync(kFull, mbar_wait_for(tmem_done, 0, 5 * kWaitLimitNs + n_iters * 100000ull)) != 0) && ok;
    if (!ok && lane == 0 && a.status != nullptr)
      atomicOr(a.status, static_cast<int32_t>(DA_STATUS_TIMEOUT));
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTTmemCols);
    return;
  }

  // =================================================== softmax warpgroups (0-7)
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTSoftmaxRegs));
  const int g = warp >> 2;         // row tile
  const int row = r0 + tid;        // (tid = 128 g + the lane of TMEM)
  const bool direct = nsplit_b == 1;
  const int t = row < a.rows ? row / a.group : 0;
  const int h = kvh * a.group + (row - t * a.group);
  const int64_t prow = (static_cast<int64_t>(b) * a.q_len + t) * a.num_q_heads + h;
  const bool mine = row < own_rows_n;
  bool ok = true;
  float m_used = -INFINITY;  // reference maximum of P (log2 domain), raised lazily
  float l = 0.f, lq = 0.f;   // sums of the fp32 weights, and of the rounded ones
  uint32_t tmem = 0;
  if (tiles > 0) {
    tmem = *tmem_slot + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // ---- the row of Q into shared memory, in the layout of a TMA tile
    if (g < tiles) {
      uint4 v[16];
      if (mine) {
        const uint4* q = reinterpret_cast<const uint4*>(
            a.q + static_cast<int64_t>(b) * a.q_sb + static_cast<int64_t>(t) * a.q_st +
            static_cast<int64_t>(h) * a.q_sh);
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = __ldg(q + c);
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = make_uint4(0u, 0u, 0u, 0u);
      }
      const int r = tid & 127;
      uint8_t* dst = smem + g * kTSlot + r * 128;
#pragma unroll
      for (int c = 0; c < 16; ++c)
        *reinterpret_cast<uint4*>(dst + (c >> 3) * kTHalf + (((c & 7) ^ (r & 7)) << 4)) = v[c];
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
  }
  if (g < tiles) {
    const uint32_t s_col = tmem + g * kTKeys;
    const uint32_t o_col = tmem + kTColO + g * kHeadDim;
    const float sc = a.scale_log2;
    const bool raw = sc > 0.f;  // (the scores stay unscaled; the exponent's multiply-add scales)
    const float s_fma = raw ? sc : 1.f;
    const int lim = mine ? min(t_end, own.base) : 0;  // keys below are all seen
    for (int j = 0; j < n_iters; ++j) {
      ok = __all_sync(kFull, mbar_wait_lazy(&s_full[g], j & 1)) != 0;
      if (!ok) break;
      tc_fence_after_sync();
      float x[kTKeys];
      {
        float y[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, y[c]);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < kTKeys; ++i) x[i] = y[i / 32][i % 32];
      }
      const int tok0 = t_begin + j * kTKeys;
      if (tok0 + kTKeys > lim) {
        // some key is hidden from this row: behind the chunk's end, or by the mask
        const int end = mine ? t_end : 0;
#pragma unroll
        for (int w = 0; w < kTKeys / 32; ++w) {
          const int left = end - (tok0 + 32 * w);
          uint32_t seen = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
          if (seen != 0 && tok0 + 32 * w + 32 > own.base) seen &= own.bits(t, tok0 + 32 * w);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[32 * w + i] = (seen >> i) & 1u ? x[32 * w + i] * (raw ? 1.f : sc) : -INFINITY;
        }
      } else if (!raw) {
#pragma unroll
        for (int i = 0; i < kTKeys; ++i) x[i] *= sc;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kTKeys; i += 8)
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = fmax3(mx[c], x[i + 2 * c], x[i + 2 * c + 1]);
      float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (raw) mt *= sc;
      const bool raise = mt != -INFINITY && (m_used == -INFINITY || mt > m_used + kTRescale);
      const float alpha = raise ? (m_used == -INFINITY ? 0.f : ex2(m_used - mt)) : 1.f;
      if (raise) m_used = mt;
      const float mref = m_used == -INFINITY ? 0.f : m_used;  // (nothing seen yet: P = 0)
      if (j > 0 && __any_sync(kFull, raise && alpha != 1.f)) {
        // (S of this tile was complete, so was the P V issued before it)
#pragma unroll 1
        for (int c = 0; c < kHeadDim / 32; ++c) {
          float o[32];
          tmem_ld32(o_col + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= alpha;
          tmem_st32(o_col + c * 32, o);
        }
        tmem_wait_st();
      }
      float2 ps = make_float2(0.f, 0.f), qs = make_float2(0.f, 0.f);
      const float2 s2 = make_float2(s_fma, s_fma);
      const float2 nm2 = make_float2(-mref, -mref);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 e = __ffma2_rn(make_float2(x[64 * c + 2 * i], x[64 * c + 2 * i + 1]), s2, nm2);
          const float p0 = ex2(e.x);
          const float p1 = ex2(e.y);
          ps = __fadd2_rn(ps, make_float2(p0, p1));
          const uint32_t pk = pack_bf16x2(p0, p1);
          qs = __fadd2_rn(qs, make_float2(packed_lo(pk, false), packed_hi(pk, false)));
          w[i] = __uint_as_float(pk);
        }
        tmem_st32(s_col + 32 * c, w);
      }
      l = l * alpha + (ps.x + ps.y);
      lq = lq * alpha + (qs.x + qs.y);
      // values of keys behind the chunk's end (P V of both tiles follows p_full[0])
      const int n_valid = t_end - tok0;
      if (g == 0 && n_valid < kTKeys) {
        const int u = 2 * j + 1;
        ok = __all_sync(kFull, mbar_wait_lazy(&full_bar[u % kTSlots], (u / kTSlots) & 1)) != 0;
        if (!ok) break;
        uint8_t* vs = smem + kTOffRing + (u % kTSlots) * kTSlot;
        for (int idx = tid; idx < (kTKeys - n_valid) * 16; idx += 128)
          *reinterpret_cast<uint4*>(vs + ((idx >> 3) & 1) * kTHalf + (n_valid + (idx >> 4)) * 128 + (idx & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[g]);
    }
    if (ok) {
      ok = __all_sync(kFull, mbar_wait_lazy(&o_done[g], 0)) != 0;
      tc_fence_after_sync();
    }
  }
  if (tid == 0) allow_dependent_launch();

  // ---- the row's output
  const float inv = (lq == 0.f ? 0.f : 1.f / lq) * a.v_scale;  // (NaN stays NaN)
  const bool have = ok && g < tiles;
  const int64_t pidx = prow * S + split;
#pragma unroll 1
  for (int c = 0; c < kHeadDim / 32; ++c) {
    float o[32];
    if (g < tiles) {
      tmem_ld32(tmem + kTColO + g * kHeadDim + c * 32, o);
      tmem_wait_ld();
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = have && l != 0.f ? o[i] * inv : 0.f;
    if (row < a.rows) {
      if (direct) {
        uint16_t* dst = a.out + static_cast<int64_t>(b) * a.o_sb + static_cast<int64_t>(t) * a.o_st +
                        static_cast<int64_t>(h) * a.o_sh + c * 32;
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          *reinterpret_cast<uint4*>(dst + i) =
              make_uint4(pack_bf16x2(o[i], o[i + 1]), pack_bf16x2(o[i + 2], o[i + 3]),
                         pack_bf16x2(o[i + 4], o[i + 5]), pack_bf16x2(o[i + 6], o[i + 7]));
      } else {
        float* dst = a.part_o + pidx * kHeadDim + c * 32;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      }
    }
  }
  if (row < a.rows) {
    const float lse = l == 0.f ? -INFINITY : (m_used == -INFINITY ? 0.f : m_used) * kLn2t + logf(l);
    if (direct) a.lse[prow] = lse;
    else a.part_lse[pidx] = lse;
  }
  if (!ok && lane == 0 && a.status != nullptr)
    atomicOr(a.status, static_cast<int32_t>(DA_STATUS_TIMEOUT));
  if (tiles > 0) {
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(tmem_done);
  }
}

std::mutex g_tall_mu;
bool g_tall_attr[64];

}  // namespace

cudaError_t launch_tall(const CUtensorMap& k_map, const CUtensorMap& v_map, const SplitArgs& a,
                        int box_tokens, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_tall_mu);
    if (!g_tall_attr[dev]) {
      e = cudaFuncSetAttribute(tall_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTSmem);
      if (e != cudaSuccess) return e;
      g_tall_attr[dev] = true;
    }
  }
  const int pairs = (a.rows + 2 * kTRows - 1) / (2 * kTRows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs) * a.num_splits, a.num_kv_heads, a.batch);
  cfg.blockDim = dim3(kTThreads);
  cfg.dynamicSmemBytes = kTSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tall_kernel, TallMaps{k_map, v_map}, a, box_tokens);
}

}  // namespace dattn
