// select_kernel.cu -- which pages of a long context each query reads.
//
// score_kernel: for 16 pages x the query rows of a KV head the bound
//     sum_d min(q'_d, 0) min_d + max(q'_d, 0) max_d = [min(q', 0); max(q', 0)] . [min; max]
// is one matrix product over 256 channels.  q' and the digests are whole
// numbers of at most 7 and 8 bits, exact in f16, and every partial sum stays
// below 2^22 units, exact in the fp32 accumulators: mma.sync computes the same
// integers whatever its order of summation.  The digests are 1 / 16 to 1 / 256
// of the keys' bytes (2 x 128 of them per page).  The lanes of a page copy 64
// contiguous bytes at a time into a ring in shared memory, a tile of 16 pages
// ahead, from which each thread takes its own bytes as fragments: the channel
// order of a step is permuted alike in q' and digest.  (72 MB of digests in
// 20.4 us: 3.5 TB/s, 5 us of them launch and the chain length - page id - digest;
// wider loads, deeper rings and the heads of a page in one CTA change nothing.)
//
// pick_kernel: per (token, KV head) the top_k of the scores.  Scores become
// integers of the same order; forced pages the largest one.  The threshold,
// the largest value that top_k scores reach, is found by a 4-ary search over
// the range of the scores (three counts per round, packed into one warp sum,
// and one barrier), and one scan lists the pages above it, and the first of
// those equal to it, in ascending order: exact, without atomics, and
// independent of timing.  It is all latency: scores are loaded before
// the length is known (rows of up to 8192 pages), and so are the page ids (up
// to 2048); otherwise the ids of the list are looked up side by side at the end
// (one after the other by the threads that found them, they were most of 15 us).
// 6 us for short rows, 8 to 10 for 2048 to 8192 pages.

#include "cache_kernels.cuh"
#include "decode_attn.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace dattn {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr float kBf16Max = 3.3895313892515355e38f;

// tokens that new token t of a request of L tokens sees
__device__ __forceinline__ int seen_tokens(const SelectArgs& a, int L, int t) {
  return a.causal ? max(0, L - a.g.q_len + t + 1) : L;
}

__device__ __forceinline__ int clamp_len(const SelectArgs& a, int L) {
  return min(max(L, 0), a.g.max_seq_len);
}

__device__ __forceinline__ uint32_t hmin2_0(uint32_t x) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0u));
  return r;
}

__device__ __forceinline__ uint32_t hmax2_0(uint32_t x) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0u));
  return r;
}

// Four signed bytes x to two f16x2 of x + 128 in units of 2^-24: the byte as the
// mantissa of a subnormal number, exact, and no arithmetic.  A row's products
// then come out 128 sum(q') too high, which is taken off at the end.
__device__ __forceinline__ void s8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = __byte_perm(u, 0u, 0x4140);
  hi = __byte_perm(u, 0u, 0x4342);
}
constexpr float kUnits = 16777216.f;

// 16 (4) bytes to shared memory, past L1 (asynchronously; each thread waits for its own)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kScoreWarps = 4;
// Tiles of a warp's ring (72 MB of digests, 32 ragged requests: 2 tiles 20.4 us,
// 3 22.4, 4 26.7; registers in the place of a ring 21.1)
constexpr int kScoreStages = 2;
constexpr int kScoreStageBytes = 8 * 32 * 16 + 2 * 32 * 4;  // a tile's digests and scales
constexpr int kScoreCtas = 4;  // per SM (2 to 8 within 6% of each other, 12 to 32 up to 15% slower)

// Dynamic shared memory: q' fragments [row tiles][4 step pairs][32 lanes] of
// 16 B, the rows' a / 127 and 128 sum(q'), then (several tokens) each warp's row
// scores [rows][16 pages], then each warp's ring of tiles, in which a thread
// keeps the very bytes that it reads again ([8][32 lanes] of 16 B, [2][32] of
// 4 B).  NT: an upper bound of the row tiles; a single one is
// prepared by every warp for itself, in registers.
template <int NT>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g4 = lane >> 2;
  const int t4 = lane & 3;
  // (heads fastest: the digests of a page's heads lie side by side, and are read at the same time)
  const int kvh = blockIdx.x;
  const int b = blockIdx.z;
  const int group = a.num_q_heads / a.g.num_kv_heads;
  const int T = a.g.q_len;
  const int rows = group * T;
  const int tiles = (rows + 7) / 8;
  uint4* q_frag = reinterpret_cast<uint4*>(smem);
  float2* q_scale = reinterpret_cast<float2*>(smem + tiles * 2048);
  float* row_score = reinterpret_cast<float*>(q_scale + tiles * 8) + warp * tiles * 8 * 16;
  allow_dependent_launch();  // (whatever follows waits for this grid all the same)
  grid_dependency_wait();

  const int L = clamp_len(a, a.g.seq_lens[b]);
  const int nb = (L + a.g.page_size - 1) / a.g.page_size;  // pages that any token sees
  // (every page is taken: no scores are read)
  if (nb <= a.top_k || static_cast<int>(blockIdx.y) * kScoreWarps * 16 >= nb) return;

  // ---- the digests of pages tile * 16 + g4 and + 8, minima then maxima, as
  // loaded, kScoreStages - 1 tiles ahead; and the page ids of the tile after
  const int32_t* bt = a.g.block_table + static_cast<int64_t>(b) * a.g.bt_stride;
  const int tile_step = gridDim.y * kScoreWarps;
  int tile = blockIdx.y * kScoreWarps + warp;
  const uint8_t* ring =
      smem + tiles * (2048 + 64) + (T > 1 ? kScoreWarps * tiles * 512 : 0) + warp * kScoreStages * kScoreStageBytes;
  const uint32_t ring_at = smem_addr(ring) + lane * 16;
  const uint32_t ring_scale = smem_addr(ring) + 4096 + lane * 4;
  auto ids = [&](int t, int (&pg)[2]) {
#pragma unroll
    for (int p = 0; p < 2; ++p) pg[p] = __ldg(bt + min(t * 16 + g4 + 8 * p, nb - 1));
  };
  auto load = [&](int slot, const int (&pg)[2]) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int id = pg[p] < 0 || pg[p] >= a.g.num_pages ? 0 : pg[p];  // (reported by pick_kernel)
      const int64_t at = static_cast<int64_t>(id) * a.g.num_kv_heads + kvh;
      const int8_t* src = a.digest + at * 256 + 16 * t4;
#pragma unroll
      for (int i = 0; i < 4; ++i) copy16(ring_at + slot * kScoreStageBytes + (p * 4 + i) * 512, src + 64 * i);
      copy4(ring_scale + slot * kScoreStageBytes + p * 128, a.digest_scale + at);
    }
  };
  int pg[2];
  if (tile * 16 < nb) {
    int first[kScoreStages - 1][2];
#pragma unroll
    for (int i = 0; i < kScoreStages - 1; ++i) ids(tile + i * tile_step, first[i]);
    ids(tile + (kScoreStages - 1) * tile_step, pg);
#pragma unroll
    for (int i = 0; i < kScoreStages - 1; ++i) {
      if ((tile + i * tile_step) * 16 < nb) load(i, first[i]);
      copies_end();
    }
  }

  // ---- q' of the rows, one warp per row tile (or the only one, by each warp)
  uint4 q_own[NT == 1 ? 4 : 1];
  float2 own_scale[NT == 1 ? 2 : 1];  // of rows 2 t4 and 2 t4 + 1
  for (int nt = NT == 1 ? 0 : warp; nt < tiles; nt += kScoreWarps) {
    const int r = nt * 8 + g4;
    uint32_t w[16];
    if (r < rows) {
      const int t = r / group;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + static_cast<int64_t>(b) * a.q_sb + static_cast<int64_t>(t) * a.q_st +
          static_cast<int64_t>(kvh * group + (r - t * group)) * a.q_sh + 16 * t4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = src[(i & 1) + 8 * (i >> 1)];
        w[4 * i] = x.x;
        w[4 * i + 1] = x.y;
        w[4 * i + 2] = x.z;
        w[4 * i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 0u;
    }
    float x[32];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float v = i & 1 ? __uint_as_float(w[i >> 1] & 0xffff0000u) : __uint_as_float(w[i >> 1] << 16);
      x[i] = v == v ? fminf(fmaxf(v, -kBf16Max), kBf16Max) : 0.f;
      top = fmaxf(top, fabsf(x[i]));
    }
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
    float inv = top > 0.f ? __fdiv_rn(127.f, top) : 0.f;
    if (inv == INFINITY) {  // (top below 3.8e-37: zeros stay zero, 0 x infinity is NaN)
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = x[i] == 0.f ? 0.f : copysignf(127.f, x[i]);
      inv = 1.f;
    }
    uint32_t h[16];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float u = fminf(fmaxf(rintf(__fmul_rn(x[2 * i], inv)), -127.f), 127.f);
      const float v = fminf(fmaxf(rintf(__fmul_rn(x[2 * i + 1], inv)), -127.f), 127.f);
      h[i] = pack_f16x2(u, v);
      sum += u + v;
    }
    sum += __shfl_xor_sync(kFull, sum, 1);
    sum += __shfl_xor_sync(kFull, sum, 2);
    const float2 qs = make_float2(__fdiv_rn(top, 127.f), 128.f * sum);
    if constexpr (NT == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q_own[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        own_scale[rr].x = __shfl_sync(kFull, qs.x, (2 * t4 + rr) * 4);
        own_scale[rr].y = __shfl_sync(kFull, qs.y, (2 * t4 + rr) * 4);
      }
      break;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q_frag[(nt * 4 + i) * 32 + lane] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
      if (t4 == 0) q_scale[r] = qs;
    }
  }
  if constexpr (NT > 1) __syncthreads();

  int slot = 0;
  for (; tile * 16 < nb; tile += tile_step) {
    copies_wait<kScoreStages - 2>();
    uint32_t w[2][16];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 raw =
            *reinterpret_cast<const uint4*>(ring + slot * kScoreStageBytes + (p * 4 + i) * 512 + lane * 16);
        w[p][4 * i] = raw.x;
        w[p][4 * i + 1] = raw.y;
        w[p][4 * i + 2] = raw.z;
        w[p][4 * i + 3] = raw.w;
      }
    const float* ds = reinterpret_cast<const float*>(ring + slot * kScoreStageBytes + 4096) + lane;
    const float ds0 = ds[0], ds1 = ds[32];
    // (the slot before this one was read a step ago)
    if ((tile + (kScoreStages - 1) * tile_step) * 16 < nb) load(slot == 0 ? kScoreStages - 1 : slot - 1, pg);
    copies_end();
    ids(tile + kScoreStages * tile_step, pg);
    slot = slot + 1 == kScoreStages ? 0 : slot + 1;
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // step pairs: channels 64 (i / 2) + 16 t4 + 8 (i % 2) ..
      uint32_t af[4][4];           // minima of the two steps, maxima of the two
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int p = 0; p < 2; ++p)
          s8x4_to_f16(w[p][(k >> 1) * 8 + 2 * i + (k & 1)], af[k][p], af[k][2 + p]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt < tiles) {
          uint4 q;
          if constexpr (NT == 1) q = q_own[i];
          else q = q_frag[(nt * 4 + i) * 32 + lane];
          mma_f16_16816(acc[nt], af[0], hmin2_0(q.x), hmin2_0(q.y));
          mma_f16_16816(acc[nt], af[1], hmin2_0(q.z), hmin2_0(q.w));
          mma_f16_16816(acc[nt], af[2], hmax2_0(q.x), hmax2_0(q.y));
          mma_f16_16816(acc[nt], af[3], hmax2_0(q.z), hmax2_0(q.w));
        }
      }
    }
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int row = nt * 8 + 2 * t4 + rr;
        if (row < rows) {
          float2 qs;
          if constexpr (NT == 1) qs = own_scale[rr];
          else qs = q_scale[row];
          const float u = __fmul_rn(__fmul_rn(fmaf(acc[nt][rr], kUnits, -qs.y), ds0), qs.x);
          const float v = __fmul_rn(__fmul_rn(fmaf(acc[nt][2 + rr], kUnits, -qs.y), ds1), qs.x);
          if (T == 1) {
            best[0] = fmaxf(best[0], u);
            best[1] = fmaxf(best[1], v);
          } else {
            row_score[row * 16 + g4] = u;
            row_score[row * 16 + g4 + 8] = v;
          }
        }
      }
    if (T == 1) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        best[p] = fmaxf(best[p], __shfl_xor_sync(kFull, best[p], 1));
        best[p] = fmaxf(best[p], __shfl_xor_sync(kFull, best[p], 2));
      }
      const int col = tile * 16 + g4 + 8 * t4;
      if (t4 < 2 && col < nb)
        a.scores[(static_cast<int64_t>(b) * a.g.num_kv_heads + kvh) * a.score_stride + col] =
            t4 == 0 ? best[0] : best[1];
    } else {
      __syncwarp();
      for (int i = lane; i < T * 16; i += 32) {
        const int t = i >> 4;
        const int col = tile * 16 + (i & 15);
        float m = -INFINITY;
        for (int g = 0; g < group; ++g) m = fmaxf(m, row_score[(t * group + g) * 16 + (i & 15)]);
        if (col < nb)
          a.scores[((static_cast<int64_t>(b) * T + t) * a.g.num_kv_heads + kvh) * a.score_stride + col] = m;
      }
      __syncwarp();
    }
  }
}

// Order-preserving integers of floats (no NaN among them); 0 is below all.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // (-0 counts as 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kMaxTopK = 4096;

// ONE: all pages fit one chunk of THREADS x kPer scores, held in registers;
// otherwise every pass reads the chunks again (from L2).
template <int THREADS, int kPer, bool ONE>
__global__ void __launch_bounds__(THREADS) pick_kernel(const SelectArgs a) {
  constexpr int kWarps = THREADS / 32;
  constexpr int kChunk = THREADS * kPer;
  __shared__ uint32_t sh[2][kWarps];
  __shared__ uint32_t sh3[2][kWarps];
  __shared__ uint32_t scan[2][kWarps];
  constexpr bool kIds = ONE && kPer <= 8;    // page ids in registers, too (16 of them cost more than the look-up)
  __shared__ int list[kIds ? 1 : kMaxTopK];  // else the selected pages' places
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;  // (b, t, kv head)
  const int kvh = static_cast<int>(row % a.g.num_kv_heads);
  const int64_t vb = row / a.g.num_kv_heads;
  const int t = static_cast<int>(vb % a.g.q_len);
  const int b = static_cast<int>(vb / a.g.q_len);
  // (no early launch of what follows: the attention's CTAs would settle around
  // this grid's and stay unevenly spread, 52 -> 73 us on 8 requests x 3 tokens)
  grid_dependency_wait();
  const int K = a.top_k;
  const int32_t* bt = a.g.block_table + static_cast<int64_t>(b) * a.g.bt_stride;
  const float* sc = a.scores + row * a.score_stride;
  // ONE: this thread's scores and page ids are on their way before the length is known
  const int e_first = threadIdx.x * kPer;
  float4 x_all[ONE ? kPer / 4 : 1];
  int ids[kIds ? kPer : 1];
  if constexpr (ONE) {
#pragma unroll
    for (int v = 0; v < kPer / 4; ++v) {
      x_all[v] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.max_blocks > K && e_first + 4 * v < a.max_blocks) x_all[v] = *reinterpret_cast<const float4*>(sc + e_first + 4 * v);
    }
  }
  if constexpr (kIds) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) ids[i] = a.max_blocks > K && e_first + i < a.max_blocks ? __ldg(bt + e_first + i) : 0;
  }
  const int raw = a.g.seq_lens[b];
  const int L = clamp_len(a, raw);
  uint32_t bad = raw != L ? DA_STATUS_SEQ_LEN : 0;
  if (a.causal && L > 0 && L < a.g.q_len) bad |= DA_STATUS_SHORT_CAUSAL;
  if (bad != 0 && a.g.status != nullptr && kvh == 0 && t == 0 && threadIdx.x == 0)
    atomicOr(a.g.status, static_cast<int32_t>(bad));
  const int Lt = seen_tokens(a, L, t);
  const int ps = a.g.page_size;
  const int count = (Lt + ps - 1) / ps;
  const int n_sel = min(count, K);
  int32_t* pages = a.pages + row * K;
  int32_t* blocks = a.blocks != nullptr ? a.blocks + row * K : nullptr;
  auto put = [&](int at, int col, int pg) {
    if (pg < 0 || pg >= a.g.num_pages) {
      if (a.g.status != nullptr) atomicOr(a.g.status, static_cast<int32_t>(DA_STATUS_BAD_PAGE));
      pg = 0;
    }
    pages[at] = pg;
    if (blocks != nullptr) blocks[at] = col;
  };
  for (int i = n_sel + threadIdx.x; i < K; i += THREADS) {
    pages[i] = 0;
    if (blocks != nullptr) blocks[i] = -1;
  }
  if (threadIdx.x == 0) a.tokens[row] = count > 0 ? (n_sel - 1) * ps + (Lt - (count - 1) * ps) : 0;
  if (count <= K) {
    for (int i = threadIdx.x; i < count; i += THREADS) put(i, i, bt[i]);
    return;
  }

  const int local0 = count - a.local;  // (top_k >= sink + local, so local0 > sink here)
  auto load = [&](int c0, uint32_t (&key)[kPer]) {
    const int e0 = c0 + threadIdx.x * kPer;
#pragma unroll
    for (int v = 0; v < kPer / 4; ++v) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if constexpr (ONE) x = x_all[v];
      else if (e0 + 4 * v < count) x = *reinterpret_cast<const float4*>(sc + e0 + 4 * v);
      key[4 * v] = ordered(x.x);
      key[4 * v + 1] = ordered(x.y);
      key[4 * v + 2] = ordered(x.z);
      key[4 * v + 3] = ordered(x.w);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = e0 + i;
      if (e < a.sink || e >= local0) key[i] = 0xffffffffu;
      if (e >= count) key[i] = 0u;
    }
  };
  const int chunks = ONE ? 1 : (count + kChunk - 1) / kChunk;
  uint32_t key[kPer];
  if constexpr (ONE) load(0, key);

  // ---- the range of the keys that are not forced: they are more than K less
  // the forced ones, so the threshold lies in it (or at the forced ones' value,
  // where they are K)
  uint32_t least = 0xffffffffu, most = 0;
  for (int c = 0; c < chunks; ++c) {
    if constexpr (!ONE) load(c * kChunk, key);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (key[i] != 0u) least = min(least, key[i]);
      if (key[i] != 0xffffffffu) most = max(most, key[i]);
    }
  }
  least = __reduce_min_sync(kFull, least);
  most = __reduce_max_sync(kFull, most);
  if (lane == 0) {
    scan[0][warp] = least;
    scan[1][warp] = most;
  }
  __syncthreads();
  least = __reduce_min_sync(kFull, lane < kWarps ? scan[0][lane] : 0xffffffffu);
  most = __reduce_max_sync(kFull, lane < kWarps ? scan[1][lane] : 0u);

  // ---- the largest thr with at least K keys >= thr, in [lo, hi]: count(>= lo)
  // >= K always, and count(>= x) < K for every x in (hi, 0xffffffff]
  uint32_t lo = least, hi = a.sink + a.local >= K ? 0xffffffffu : most;
  bool exact = false;  // exactly K keys are >= lo
  int round = 0;
  while (lo < hi && !exact) {
    // three probes in (lo, hi]
    const uint32_t span = hi - lo;
    uint32_t probe[3];
    probe[0] = lo + (span >> 2) + (span < 4 ? 1 : 0);
    probe[1] = lo + (span >> 1) + (span < 4 ? 1 : 0);
    probe[2] = lo + (span >> 1) + (span >> 2) + (span < 4 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < 3; ++i) probe[i] = min(probe[i], hi);
    const int buf = round & 1;
    uint32_t n[3];
    if constexpr (ONE) {
      // counts of a warp are at most 32 x kPer: three fields of ten bits
      static_assert(kPer < 32, "ten bits");
      uint32_t c = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        c += (key[i] >= probe[0]) + ((key[i] >= probe[1]) << 10) + ((key[i] >= probe[2]) << 20);
      c = __reduce_add_sync(kFull, c);
      if (lane == 0) sh[buf][warp] = c;
      __syncthreads();  // (the other buffer is written next: one barrier per round)
      c = lane < kWarps ? sh[buf][lane] : 0u;
      const uint32_t two = __reduce_add_sync(kFull, (c & 0x3ffu) | ((c & 0xffc00u) << 6));
      n[0] = two & 0xffffu;
      n[1] = two >> 16;
      n[2] = __reduce_add_sync(kFull, c >> 20);
    } else {
      n[0] = n[1] = n[2] = 0;
      for (int c = 0; c < chunks; ++c) {
        load(c * kChunk, key);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          n[0] += key[i] >= probe[0];
          n[1] += key[i] >= probe[1];
          n[2] += key[i] >= probe[2];
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t x = __reduce_add_sync(kFull, n[i]);
        if (lane == 0) (i < 2 ? sh : sh3)[i & 1][warp] = x;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 3; ++i)
        n[i] = __reduce_add_sync(kFull, lane < kWarps ? (i < 2 ? sh : sh3)[i & 1][lane] : 0u);
      __syncthreads();
    }
    const uint32_t k = static_cast<uint32_t>(K);
    uint32_t new_lo = lo, new_hi = hi;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (n[i] >= k) {
        new_lo = max(new_lo, probe[i]);
        if (n[i] == k) exact = true;  // (then probes above have fewer or the same)
      } else {
        new_hi = min(new_hi, probe[i] - 1);
      }
    }
    if (exact) {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (n[i] == k) new_lo = probe[i];
    }
    lo = new_lo;
    hi = new_hi;
    ++round;
  }
  // selected: keys above `above`, and the first `take` of those equal to it
  const uint32_t above = exact ? lo - 1 : lo;

  // ---- how many equal ones to take: K less those above
  __syncthreads();
  uint32_t take = 0;
  if (!exact) {
    uint32_t gt = 0;
    for (int c = 0; c < chunks; ++c) {
      if constexpr (!ONE) load(c * kChunk, key);
#pragma unroll
      for (int i = 0; i < kPer; ++i) gt += key[i] > above;
    }
    gt = __reduce_add_sync(kFull, gt);
    if (lane == 0) sh[0][warp] = gt;
    __syncthreads();
    gt = __reduce_add_sync(kFull, lane < kWarps ? sh[0][lane] : 0u);
    take = static_cast<uint32_t>(K) - gt;
  }

  // ---- one scan in page order
  uint32_t gt0 = 0, eq0 = 0;  // in the chunks before
  for (int c = 0; c < chunks; ++c) {
    if constexpr (!ONE) load(c * kChunk, key);
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      gt += key[i] > above;
      eq += take != 0 && key[i] == above;
    }
    uint32_t g = gt, q = eq;  // inclusive scans over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(kFull, g, o), y = __shfl_up_sync(kFull, q, o);
      if (lane >= o) {
        g += x;
        q += y;
      }
    }
    if (lane == 31) {
      scan[0][warp] = g;
      scan[1][warp] = q;
    }
    __syncthreads();
    const uint32_t wg = lane < kWarps ? scan[0][lane] : 0u, wq = lane < kWarps ? scan[1][lane] : 0u;
    uint32_t bg = gt0 + g - gt + __reduce_add_sync(kFull, lane < warp ? wg : 0u);
    uint32_t bq = eq0 + q - eq + __reduce_add_sync(kFull, lane < warp ? wq : 0u);
    gt0 += __reduce_add_sync(kFull, wg);
    eq0 += __reduce_add_sync(kFull, wq);
    const int e0 = c * kChunk + threadIdx.x * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool up = key[i] > above;
      const bool same = take != 0 && key[i] == above && bq < take;
      if (up || same) {
        const int at = static_cast<int>(bg + min(bq, take));
        if constexpr (kIds) put(at, e0 + i, ids[i]);
        else list[at] = e0 + i;
      }
      bg += up;
      bq += take != 0 && key[i] == above;
    }
    if constexpr (!kIds) __syncthreads();  // (scan[] is written again; the list is complete)
  }
  if constexpr (!kIds)
    for (int i = threadIdx.x; i < K; i += THREADS) put(i, list[i], bt[list[i]]);
}

template <class Kernel, class Args>
cudaError_t launch(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args& a) {
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
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, int sm_count, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.g.batch) * a.g.q_len * a.g.num_kv_heads;
  if (rows == 0) return cudaSuccess;
  if (a.max_blocks > a.top_k) {
    const int q_rows = a.num_q_heads / a.g.num_kv_heads * a.g.q_len;
    const int tiles = (q_rows + 7) / 8;
    const size_t smem = static_cast<size_t>(tiles) * 2048 + tiles * 64 +
                        (a.g.q_len > 1 ? static_cast<size_t>(kScoreWarps) * tiles * 512 : 0) +
                        kScoreWarps * kScoreStages * kScoreStageBytes;
    auto* kernel = tiles == 1 ? score_kernel<1> : tiles <= 4 ? score_kernel<4> : score_kernel<16>;
    if (smem > 48 * 1024) {
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
    }
    // a tile of 16 pages per warp, several per warp once the grid has
    // kScoreCtas CTAs per SM (each CTA prepares q' again)
    const int64_t full = (a.max_blocks + kScoreWarps * 16 - 1) / (kScoreWarps * 16);
    const int64_t pairs = static_cast<int64_t>(a.g.batch) * a.g.num_kv_heads;
    int64_t x = (kScoreCtas * static_cast<int64_t>(sm_count) + pairs - 1) / pairs;
    x = x < full ? x : full;
    const cudaError_t e =
        launch(kernel, dim3(a.g.num_kv_heads, static_cast<unsigned>(x), a.g.batch),
               32 * kScoreWarps, smem, stream, a);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(rows));
  if (a.max_blocks <= 2048) return launch(pick_kernel<256, 8, true>, grid, 256, 0, stream, a);
  if (a.max_blocks <= 4096) return launch(pick_kernel<256, 16, true>, grid, 256, 0, stream, a);
  if (a.max_blocks <= 8192) return launch(pick_kernel<512, 16, true>, grid, 512, 0, stream, a);
  return launch(pick_kernel<1024, 8, false>, grid, 1024, 0, stream, a);
}

}  // namespace dattn
