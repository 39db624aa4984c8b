// fp4_kernel.cu -- the per-chunk kernel of split-KV decode attention over a
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
//   * MMA key row 2 p is key p and row 2 p + 1 key 4 + (p ^ 1) (+ 8 for rows 8
//     and up), and the 16-byte chunks of a key are XOR-ed by its bit 1: the
//     lanes of every shared-memory phase, of K and of V, then cover all banks.
// Q is scaled per row by a power of two into f16's range (undone in fp32 on
// the scores), P is held times 2^12, so that neither loses values that bf16
// or fp32 would have kept (P's subnormals begin at 2^-26 of the row's maximum
// and the LSE is summed in fp32 from unrounded values).
//
// Each warp streams its own 32-key steps through a private ring of stages with
// cp.async (rows past the end are zero-filled, so nothing behind a sequence is
// read), with no block-wide barrier until the warps' (m, l, O) are merged.
// More than 32 query rows per KV head run as groups of 32 in the grid's y.

#include <mutex>

#include "decode_attn.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace dattn {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 12.f;  // P is held times 2^12
constexpr int kStepKeys = 32;

#ifndef DATTN_F4_WARPS
#define DATTN_F4_WARPS 4
#endif
#ifndef DATTN_F4_STAGES
#define DATTN_F4_STAGES 3
#endif

template <int NT>
struct Fp4Cfg {
  static constexpr int kWarps = DATTN_F4_WARPS;
  static constexpr int kStages = DATTN_F4_STAGES;
  static constexpr int kRows = 8 * NT;
  // a stage: 32 keys of K (64 B each), of V, then their block scales (8 B each)
  static constexpr int kOffV = kStepKeys * 64;
  static constexpr int kOffKs = 2 * kStepKeys * 64;
  static constexpr int kOffVs = kOffKs + kStepKeys * 8;
  static constexpr int kStageBytes = kOffVs + kStepKeys * 8;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kRedStride = kHeadDim + 4;
  static constexpr int kRedBytes = kWarps * kRows * kRedStride * 4;
  static constexpr int kPipeBytes = kRingBytes > kRedBytes ? kRingBytes : kRedBytes;
  static constexpr bool kQSmem = NT > 1;  // Q fragments [4 step pairs][NT][32 lanes] of 16 B
  static constexpr int kQBytes = kQSmem ? 4 * NT * 512 : 0;
  static constexpr int kStatBytes = (2 * kWarps + 1) * kRows * 4;
  static constexpr int kSmemBytes = kPipeBytes + kQBytes + kStatBytes;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src, bool live) {
  const int n = live ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// byte address of 16-byte chunk c of key row `key` of a K or V step
__device__ __forceinline__ uint32_t row_chunk(int key, int c) {
  return static_cast<uint32_t>(key * 64 + ((c ^ (key & 2)) << 4));
}

// The page and the slot in it of the 16-token halves of this warp's next 16
// steps: lane 2 i + h holds those of half h of step i of the current window
// (and of the next one, loaded a window ahead).
struct HalfWindow {
  const int32_t* bt_row;  // nullptr: contiguous (page = request, slot = token)
  int b, t_begin, t_end, page_size, num_pages, warp, warps, lane;
  int32_t* status;
  int cur_pg, cur_sl, nxt_pg, nxt_sl, base;

  __device__ __forceinline__ void load(int first, int& pg, int& sl) const {
    const int step = (first + (lane >> 1)) * warps + warp;
    const int64_t tok = static_cast<int64_t>(t_begin) + static_cast<int64_t>(step) * kStepKeys +
                        (lane & 1) * 16;
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
    load(16, nxt_pg, nxt_sl);
  }
  // (all lanes together, with i rising by one from 0)
  __device__ __forceinline__ void advance(int i) {
    if (i >= base + 16) {
      cur_pg = nxt_pg;
      cur_sl = nxt_sl;
      base += 16;
      load(base + 16, nxt_pg, nxt_sl);
    }
  }
};

template <int NT, bool LS>
__global__ void __launch_bounds__(32 * Fp4Cfg<NT>::kWarps) fp4_kernel(const Fp4Args f) {
  using C = Fp4Cfg<NT>;
  constexpr uint32_t kFull = 0xffffffffu;
  constexpr int W = C::kWarps;
  const SplitArgs& a = f.s;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g4 = lane >> 2;
  const int t4 = lane & 3;

  grid_dependency_wait();

  // ---- this CTA's work item: (chunk, kv head, request), row group, key range
  int split, kvh, b, L, chunk, item = 0;
  const int groups = (a.rows + C::kRows - 1) / C::kRows;
  int rgroup;
  if constexpr (LS) {
    item = blockIdx.x;
    rgroup = blockIdx.y;
    const int n_items = a.plan[1];
    const int4 itm = a.items[item];
    chunk = a.plan[0];
    if (item >= n_items) return;
    b = itm.x;
    kvh = itm.y;
    split = itm.z;
    L = itm.w;
  } else {
    split = blockIdx.x;
    kvh = blockIdx.y / groups;
    rgroup = blockIdx.y - kvh * groups;
    b = blockIdx.z;
    L = a.seq_lens[static_cast<int64_t>(b) * a.len_sb + static_cast<int64_t>(kvh) * a.len_sh];
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
  if (split >= nsplit_b) return;
  const int t_begin = split * chunk;
  const int t_end = min(L, t_begin + chunk);
  const int n_steps = t_end > t_begin ? (t_end - t_begin + kStepKeys - 1) / kStepKeys : 0;
  const int my_steps = n_steps > warp ? (n_steps - warp + W - 1) / W : 0;
  const int row0 = rgroup * C::kRows;                    // first row of the group
  const int rows = min(C::kRows, a.rows - row0);

  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* q_smem = smem + C::kPipeBytes;
  float* stat_m = reinterpret_cast<float*>(smem + C::kPipeBytes + C::kQBytes);
  float* stat_l = stat_m + W * C::kRows;
  int* stat_e = reinterpret_cast<int*>(stat_l + W * C::kRows);
  const uint32_t ring = smem_addr(smem) + warp * C::kStages * C::kStageBytes;

  // ---- the warp's loader: step i (of its own) into stage i % kStages
  const int32_t* bt_row =
      a.paged ? a.block_table + static_cast<int64_t>(b) * a.bt_stride + static_cast<int64_t>(kvh) * a.bt_sh
              : nullptr;
  HalfWindow win{bt_row, b, t_begin, t_end, a.page_size, a.num_pages, warp, W, lane, a.status,
                 0, 0, 0, 0, 0};
  win.init();
  const uint8_t* kbase = f.k + static_cast<int64_t>(kvh) * f.st_head;
  const uint8_t* vbase = f.v + static_cast<int64_t>(kvh) * f.st_head;
  const uint8_t* ksbase = f.ks + static_cast<int64_t>(kvh) * f.sf_head;
  const uint8_t* vsbase = f.vs + static_cast<int64_t>(kvh) * f.sf_head;
  auto load_step = [&](int i) {
    win.advance(i);
    const uint32_t st = ring + (i % C::kStages) * C::kStageBytes;
    const int tok0 = t_begin + (i * W + warp) * kStepKeys;
    const int src = 2 * (i - win.base);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t pg = __shfl_sync(kFull, win.cur_pg, src + h);
      const int64_t sl = __shfl_sync(kFull, win.cur_sl, src + h);
      const int64_t off = pg * f.st_page + sl * f.st_token;
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // 16 keys x 4 chunks: two per lane
        const int key = 8 * j + (lane >> 2);
        const int c = lane & 3;
        const bool live = tok0 + 16 * h + key < t_end;
        const int64_t o = live ? off + key * f.st_token + c * 16 : 0;
        const uint32_t d = st + row_chunk(16 * h + key, c);
        cp_async_16(d, kbase + o, live);
        cp_async_16(d + C::kOffV, vbase + o, live);
      }
      // block scales: 16 keys of K by lanes 0..15, of V by lanes 16..31
      const int key = lane & 15;
      const bool live = tok0 + 16 * h + key < t_end;
      const int64_t o = live ? pg * f.sf_page + (sl + key) * 8 : 0;
      cp_async_8(st + (lane < 16 ? C::kOffKs : C::kOffVs) + (16 * h + key) * 8,
                 (lane < 16 ? ksbase : vsbase) + o, live);
    }
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) {
    if (i < my_steps) load_step(i);
    cp_async_commit();
  }

  // ---- Q fragments (B operand: row g4 of row tile nt, the lane's 32 d), and
  // the power of two that brings a row's largest value to [2^14, 2^15)
  uint32_t qf[C::kQSmem ? 1 : 8][2];
  int q_e = 0;  // (NT = 1: of row g4)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (C::kQSmem && nt % W != warp) continue;  // one warp prepares each row tile
    const int r = row0 + nt * 8 + g4;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (nt * 8 + g4 < rows) {
      const int t = r / a.group;
      const uint16_t* qr = a.q + static_cast<int64_t>(b) * a.q_sb + static_cast<int64_t>(t) * a.q_st +
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
        *reinterpret_cast<uint4*>(q_smem + ((i * NT + nt) * 32 + lane) * 16) =
            make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
      if (t4 == 0) stat_e[nt * 8 + g4] = e;
    } else {
      q_e = e;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qf[ks][0] = h[2 * ks];
        qf[ks][1] = h[2 * ks + 1];
      }
    }
  }
  if constexpr (C::kQSmem) __syncthreads();
  // per row of this thread's score columns (2 t4, 2 t4 + 1): the factor to
  // base-2 scores, and the keys it may see
  float rs[NT][2];
  int lim[NT][2];
  int lim_all = t_end;  // every row sees the keys below this
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int row = nt * 8 + 2 * t4 + rr;
      int e;
      if constexpr (C::kQSmem) e = stat_e[row];
      else e = __shfl_sync(kFull, q_e, (2 * t4 + rr) * 4);
      rs[nt][rr] = ldexpf(a.scale_log2, e);
      int lm = t_end;
      if (a.causal && row < rows) lm = min(lm, L - a.q_len + 1 + (row0 + row) / a.group);
      lim[nt][rr] = lm;
      lim_all = min(lim_all, lm);
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

  const uint32_t q_addr = smem_addr(q_smem) + lane * 16;
  const int krow = (g4 & 1) ? 4 + ((g4 >> 1) ^ 1) : g4 >> 1;  // key of MMA row g4 in a 16-key half
  for (int i = 0; i < my_steps; ++i) {
    if (i + C::kStages - 1 < my_steps) load_step(i + C::kStages - 1);
    cp_async_commit();
    cp_async_wait<C::kStages - 1>();
    __syncwarp();
    const uint32_t st = ring + (i % C::kStages) * C::kStageBytes;
    const int tok0 = t_begin + (i * W + warp) * kStepKeys;

    // ---- S^T[32 keys x 8 NT rows] = K . Q^T
    float sc[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[h][nt][j] = 0.f;
      const int k0 = 16 * h + krow;
      const uint4 w0 = lds128(st + row_chunk(k0, t4));
      const uint4 w1 = lds128(st + row_chunk(k0 + 8, t4));
      const uint32_t s0 = e4m3x2_to_f16x2(lds_u16(st + C::kOffKs + k0 * 8 + 2 * t4));
      const uint32_t s1 = e4m3x2_to_f16x2(lds_u16(st + C::kOffKs + (k0 + 8) * 8 + 2 * t4));
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

    // ---- online softmax over the step (base 2; P times 2^kPShift)
    const bool full = tok0 + kStepKeys <= lim_all;
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[2][4];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        float x[4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int key = tok0 + 16 * h + 8 * j + krow;
            const float s = sc[h][nt][2 * j + rr] * rs[nt][rr];
            x[2 * h + j] = full || key < lim[nt][rr] ? s : -INFINITY;
          }
        float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
        const float m_new = fmaxf(m[nt][rr], mx - kPShift);
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        if (__any_sync(kFull, m_new != m[nt][rr])) {  // (settles after a few steps)
          const float alpha = ex2(m[nt][rr] - m_use);
          l[nt][rr] *= alpha;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            acc[mt][nt][rr] *= alpha;
            acc[mt][nt][2 + rr] *= alpha;
          }
          m[nt][rr] = m_new;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = ex2(x[j] - m_use);
        l[nt][rr] += (x[0] + x[1]) + (x[2] + x[3]);
        p[0][rr] = x[0];
        p[0][2 + rr] = x[1];
        p[1][rr] = x[2];
        p[1][2 + rr] = x[3];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        pb[h][nt][0] = movmatrix_trans(pack_f16x2(p[h][0], p[h][1]));
        pb[h][nt][1] = movmatrix_trans(pack_f16x2(p[h][2], p[h][3]));
      }
    }

    // ---- O^T[128 d x 8 NT rows] += V^T . P^T
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2 v[4];
      uint32_t s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = 16 * h + ((j & 1) ? 4 + (t4 ^ 1) : t4) + 8 * (j >> 1);
        v[j] = lds64(st + C::kOffV + row_chunk(key, g4 >> 1) + (g4 & 1) * 8);
        s[j] = lds_u8(st + C::kOffVs + key * 8 + g4);
      }
      const uint32_t s01 = e4m3x2_to_f16x2(s[0] | (s[1] << 8));
      const uint32_t s23 = e4m3x2_to_f16x2(s[2] | (s[3] << 8));
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
    __syncwarp();  // the stage is free for the load of the next iteration
  }
  cp_async_wait<0>();

  if (threadIdx.x == 0) allow_dependent_launch();

  // ---- merge the warps' (m, l, O)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      float v = l[nt][rr];
      v += __shfl_xor_sync(kFull, v, 4);
      v += __shfl_xor_sync(kFull, v, 8);
      v += __shfl_xor_sync(kFull, v, 16);
      l[nt][rr] = v;
      if (g4 == 0) {
        const int row = nt * 8 + 2 * t4 + rr;
        stat_m[warp * C::kRows + row] = m[nt][rr];
        stat_l[warp * C::kRows + row] = v;
      }
    }
  __syncthreads();  // (every warp is past its ring, too)
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int row = nt * 8 + 2 * t4 + rr;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, stat_m[w * C::kRows + row]);
      const float Mu = M == -INFINITY ? 0.f : M;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w)
        sum += stat_l[w * C::kRows + row] * ex2(stat_m[w * C::kRows + row] - Mu);
      const float fac = (sum > 0.f ? ex2(m[nt][rr] - Mu) / sum : (sum == sum ? 0.f : sum)) * a.v_scale;
      float* dst = red + (warp * C::kRows + row) * C::kRedStride + 16 * g4;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
        *reinterpret_cast<float2*>(dst + 2 * mt) =
            make_float2(acc[mt][nt][rr] * fac, acc[mt][nt][2 + rr] * fac);
    }
  __syncthreads();

  const bool direct = nsplit_b == 1;
  const int S = a.num_splits;
  auto head_of = [&](int r, int& t) {
    t = r / a.group;
    return kvh * a.group + (r - t * a.group);
  };
  for (int idx = threadIdx.x; idx < rows * 32; idx += 32 * W) {
    const int row = idx >> 5;
    const int d = (idx & 31) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(red + (w * C::kRows + row) * C::kRedStride + d);
      v.x += x.x;
      v.y += x.y;
      v.z += x.z;
      v.w += x.w;
    }
    int t;
    const int h = head_of(row0 + row, t);
    if (direct) {
      *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(b) * a.o_sb +
                                static_cast<int64_t>(t) * a.o_st + static_cast<int64_t>(h) * a.o_sh + d) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
      const int64_t pidx =
          LS ? static_cast<int64_t>(item) * a.rows + row0 + row
             : ((static_cast<int64_t>(b) * a.q_len + t) * a.num_q_heads + h) * S + split;
      st_global_hint(a.part_o + pidx * kHeadDim + d, v, l2_evict_last_policy());
    }
  }
  for (int row = threadIdx.x; row < rows; row += 32 * W) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, stat_m[w * C::kRows + row]);
    const float Mu = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w)
      sum += stat_l[w * C::kRows + row] * ex2(stat_m[w * C::kRows + row] - Mu);
    const float lse = sum == 0.f ? -INFINITY : (Mu + log2f(sum)) * kLn2;
    int t;
    const int h = head_of(row0 + row, t);
    const int64_t prow = (static_cast<int64_t>(b) * a.q_len + t) * a.num_q_heads + h;
    if (direct)
      a.lse[prow] = lse;
    else
      st_global_hint(a.part_lse + (LS ? static_cast<int64_t>(item) * a.rows + row0 + row
                                      : prow * S + split),
                     lse, l2_evict_last_policy());
  }
}

constexpr int kMaxDev = 64;
std::mutex g_mu;
int g_ctas[3][kMaxDev];  // resident CTAs per SM of the 8-, 16- and 32-row variants

int variant_of(int rows) { return rows <= 8 ? 0 : rows <= 16 ? 1 : 2; }

template <int NT>
cudaError_t ensure(int v, int dev, int* ctas) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_ctas[v][dev] == 0) {
    using C = Fp4Cfg<NT>;
    cudaError_t e = cudaFuncSetAttribute(fp4_kernel<NT, false>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(fp4_kernel<NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmemBytes);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fp4_kernel<NT, false>, 32 * C::kWarps,
                                                      C::kSmemBytes);
    if (e != cudaSuccess) return e;
    g_ctas[v][dev] = n > 0 ? n : 1;
  }
  if (ctas != nullptr) *ctas = g_ctas[v][dev];
  return cudaSuccess;
}

cudaError_t ensure_any(int rows, int* ctas) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  switch (variant_of(rows)) {
    case 0: return ensure<1>(0, dev, ctas);
    case 1: return ensure<2>(1, dev, ctas);
    default: return ensure<4>(2, dev, ctas);
  }
}

template <int NT>
cudaError_t launch_nt(const Fp4Args& f, cudaStream_t stream) {
  using C = Fp4Cfg<NT>;
  const int groups = (f.s.rows + C::kRows - 1) / C::kRows;
  cudaLaunchConfig_t cfg = {};
  const bool listed = f.s.items != nullptr;
  cfg.gridDim = listed ? dim3(static_cast<unsigned>(f.s.item_slots), groups)
                       : dim3(f.s.num_splits, f.s.num_kv_heads * groups, f.s.batch);
  cfg.blockDim = dim3(32 * C::kWarps);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return listed ? cudaLaunchKernelEx(&cfg, fp4_kernel<NT, true>, f)
                : cudaLaunchKernelEx(&cfg, fp4_kernel<NT, false>, f);
}

}  // namespace

cudaError_t launch_fp4(const Fp4Args& f, cudaStream_t stream) {
  const cudaError_t e = ensure_any(f.s.rows, nullptr);
  if (e != cudaSuccess) return e;
  switch (variant_of(f.s.rows)) {
    case 0: return launch_nt<1>(f, stream);
    case 1: return launch_nt<2>(f, stream);
    default: return launch_nt<4>(f, stream);
  }
}

int fp4_ctas_per_sm(int rows) {
  int n = 0;
  return ensure_any(rows, &n) == cudaSuccess ? n : 1;
}

}  // namespace dattn
