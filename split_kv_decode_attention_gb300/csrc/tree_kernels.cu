// tree_kernels.cu -- what a speculative step of drafted trees needs besides its
// attention, and the way back out of a cache: the trees' masks, the kept tokens
// moved together, and a cache read as bf16.

#include "cache_kernels.cuh"
#include "decode_attn.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace dattn {
namespace {

// The length of request b and the number of its new tokens, clamped; status
// bits by the caller.
__device__ __forceinline__ uint32_t lengths_of(const int32_t* seq_lens, const int32_t* new_lens, int b,
                                               int q_len, int max_seq_len, int& L, int& n) {
  uint32_t bad = 0;
  L = seq_lens[b];
  n = new_lens != nullptr ? new_lens[b] : q_len;
  if (L < 0 || L > max_seq_len) {
    bad |= DA_STATUS_SEQ_LEN;
    L = L < 0 ? 0 : max_seq_len;
  }
  if (n < 0 || n > q_len) {
    bad |= DA_STATUS_SEQ_LEN;
    n = n < 0 ? 0 : q_len;
  }
  if (L < n) bad |= DA_STATUS_SHORT_CAUSAL;
  return bad;
}

// --------------------------------------------------------------- tree masks
// Row t of a mask has the bits of t and its ancestors, anc(t) = {t} + anc(parent
// of t); its depth is their number less one.  A thread per token walks up to the
// root through the parents in shared memory.  Parents are earlier tokens, so the
// walk meets the words of the row from the last to the first and each is stored
// once.  Latency bounds it: a load of the parents, the steps of the deepest
// token, one store.  GB300, inside a replayed graph: 1 x 16 tokens 1.4 us, 128 x 63
// 2.0 us.
constexpr int kMaskThreads = 128;

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const TreeMaskArgs a) {
  __shared__ int16_t parent[DECODE_ATTN_MAX_TREE];
  grid_dependency_wait();
  const int b = blockIdx.x;
  int L, n;
  uint32_t bad = lengths_of(a.seq_lens, a.new_lens, b, a.q_len, a.max_seq_len, L, n);
  if (threadIdx.x != 0) bad = 0;
  for (int t = threadIdx.x; t < n; t += kMaskThreads) {
    int p = a.parents[static_cast<int64_t>(b) * a.q_len + t];
    if (p < -1 || p >= t) {
      bad |= DA_STATUS_TREE;
      p = -1;
    }
    parent[t] = static_cast<int16_t>(p);
  }
  if (bad != 0 && a.status != nullptr) atomicOr(a.status, static_cast<int32_t>(bad));
  __syncthreads();
  for (int t = threadIdx.x; t < a.q_len; t += kMaskThreads) {
    const int64_t row = static_cast<int64_t>(b) * a.q_len + t;
    int p = t < n ? t : -1, steps = 0;
    for (int w = a.words - 1; w >= 0; --w) {
      uint32_t bits = 0;
      while (p >= 32 * w) {  // (p < 0 ends it)
        bits |= 1u << (p & 31);
        p = parent[p];
        ++steps;
      }
      a.mask[row * a.words + w] = bits;
    }
    if (a.positions != nullptr) a.positions[row] = t < n ? L - n + steps - 1 : 0;
  }
}

// -------------------------------------------------------------- kept tokens
// Token L - n + keep[i] moves to L - n + i, i = 0, 1, ..  As keep rises, a place
// is written only by moves that come after those that read it: keep[j] = i means
// j <= i.  So a thread that moves its 16 bytes of a token for one i after the
// other, several loads ahead of their stores, needs no other thread.  The places
// (page, slot) of all moves are looked up once per CTA.  Latency bounds it, four
// dependent loads (counts, kept tokens, pages, rows): GB300, 1 request, 16 drafts in a
// bf16 cache 2.5 us, 256 requests of 32 in a 4-bit one 4.0 us.
constexpr int kKeepThreads = 128;
constexpr int kKeepAhead = 4;

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepArgs a) {
  extern __shared__ int64_t place[];  // [moves][4]: from and to, in the cache and in the block scales
  __shared__ int cut;                 // the first entry that is out of order
  grid_dependency_wait();
  const int b = blockIdx.y;
  const int tid = threadIdx.x;
  int L, n;
  uint32_t bad = lengths_of(a.g.seq_lens, a.new_lens, b, a.g.q_len, a.g.max_seq_len, L, n);
  int m = a.counts[b];
  if (m < 0 || m > min(a.max_keep, n)) {
    bad |= DA_STATUS_TREE;
    m = m < 0 ? 0 : min(a.max_keep, n);
  }
  if (tid == 0) cut = m;
  __syncthreads();
  const int32_t* keep = a.keep + static_cast<int64_t>(b) * a.max_keep;
  for (int i = tid; i < m; i += kKeepThreads) {
    const int at = keep[i], before = i > 0 ? keep[i - 1] : -1;
    if (at <= before || at >= n || at < 0) atomicMin(&cut, i);
  }
  __syncthreads();
  if (cut < m) {
    bad |= DA_STATUS_TREE;
    m = cut;
  }
  const int base = L - n;
  const CacheView& c = a.c;
  for (int i = tid; i < m; i += kKeepThreads) {
    const int tok[2] = {base + keep[i], base + i};
    bool ok = tok[1] >= 0 && tok[0] != tok[1];
    int64_t at[4];
    for (int e = 0; e < 2 && ok; ++e) {
      int64_t group = b;
      int slot = tok[e];
      if (a.g.block_table != nullptr) {
        const int page = a.g.block_table[static_cast<int64_t>(b) * a.g.bt_stride + tok[e] / a.g.page_size];
        if (page < 0 || page >= a.g.num_pages) {
          if (a.g.status != nullptr) atomicOr(a.g.status, static_cast<int32_t>(DA_STATUS_BAD_PAGE));
          ok = false;
        }
        group = page;
        slot = tok[e] % a.g.page_size;
      }
      at[e] = group * c.page + static_cast<int64_t>(slot) * c.token;
      at[2 + e] = group * c.sf_page + static_cast<int64_t>(slot) * 8;
    }
    for (int e = 0; e < 4; ++e) place[4 * i + e] = ok ? at[e] : -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (a.out_lens != nullptr) a.out_lens[b] = max(base + m, 0);
    if (bad != 0 && a.g.status != nullptr) atomicOr(a.g.status, static_cast<int32_t>(bad));
  }
  __syncthreads();

  // columns: 16-byte pieces of K's heads, then of V's; then (4-bit caches) the 8
  // bytes of a head's block scales, K's and V's
  const int pieces = c.type == DA_CACHE_BF16 ? 16 : c.type == DA_CACHE_FP8_E4M3 ? 8 : 4;
  const int heads = a.g.num_kv_heads;
  const int sides = c.v == c.k ? 1 : 2;  // (the moves of a place are one thread's)
  const int values = sides * heads * pieces;
  const int columns = values + (c.type == DA_CACHE_FP4_E2M1 ? (c.vs == c.ks ? 1 : 2) * heads : 0);
  const int col = blockIdx.x * kKeepThreads + tid;
  if (col >= columns) return;
  if (col < values) {
    const int side = col / (heads * pieces), r = col - side * heads * pieces;
    uint8_t* at = (side ? c.v : c.k) + static_cast<int64_t>(r / pieces) * c.head + (r % pieces) * 16;
    for (int i0 = 0; i0 < m; i0 += kKeepAhead) {
      uint4 x[kKeepAhead];
#pragma unroll
      for (int j = 0; j < kKeepAhead; ++j)
        if (i0 + j < m && place[4 * (i0 + j)] >= 0)
          x[j] = *reinterpret_cast<const uint4*>(at + place[4 * (i0 + j)]);
#pragma unroll
      for (int j = 0; j < kKeepAhead; ++j)
        if (i0 + j < m && place[4 * (i0 + j)] >= 0)
          *reinterpret_cast<uint4*>(at + place[4 * (i0 + j) + 1]) = x[j];
    }
  } else {
    const int r = col - values, side = r / heads;
    uint8_t* at = (side ? c.vs : c.ks) + static_cast<int64_t>(r - side * heads) * c.sf_head;
    for (int i = 0; i < m; ++i)
      if (place[4 * i] >= 0)
        *reinterpret_cast<uint2*>(at + place[4 * i + 3]) = *reinterpret_cast<const uint2*>(at + place[4 * i + 2]);
  }
}

// ---------------------------------------------------------------- read back
// Eight values of a (token, head) per thread and step: 16, 8 or 4 bytes in, 16
// out, so a warp's loads and stores are whole lines.  A CTA takes kReadTokens
// tokens of a request, K or V; their places are looked up once, then each thread
// has kReadAhead loads in flight.  An E4M3 value, and a block scale times an
// E2M1 value, are exact in fp32 (and in bf16: at most 6 significant bits), so
// there is one rounding, that of the product with the cache's scale, and none
// where that is a power of two.  HBM bounds it at size.  GB300: 4K FP8 tokens x 8 heads
// 5.7 us; 32 requests of up to 16K tokens x 8 heads from 16-token pages, 4-bit 244 us
// (5.8 TB/s of reads and writes, 0.86 of a copy; ALU 62 % busy), 34 of 4K to 7K, bf16
// 237 us (6.9 TB/s).
constexpr int kReadThreads = 256;
constexpr int kReadTokens = 32;
constexpr int kReadAhead = 8;

// Two fp32 values of a packed f16x2, scaled and rounded to bf16x2.
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t f16x2, float scale) {
  return pack_bf16x2(packed_lo(f16x2, true) * scale, packed_hi(f16x2, true) * scale);
}

template <int TYPE>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadArgs a) {
  __shared__ int64_t src[kReadTokens], src_sf[kReadTokens];
  grid_dependency_wait();
  const int b = blockIdx.y;
  const int first = blockIdx.x * kReadTokens;  // of the tokens read
  const int tid = threadIdx.x;
  const bool is_v = blockIdx.z != 0;
  uint32_t bad = 0;
  int L = a.g.seq_lens[b];
  int start = a.starts != nullptr ? a.starts[b] : 0;
  if (L < 0 || L > a.g.max_seq_len) {
    bad |= DA_STATUS_SEQ_LEN;
    L = L < 0 ? 0 : a.g.max_seq_len;
  }
  if (start < 0 || start > L) {
    bad |= DA_STATUS_SEQ_LEN;
    start = start < 0 ? 0 : L;
  }
  int64_t n = min(L - start, a.max_tokens);
  int64_t row0 = 0;
  if (a.offsets != nullptr) {
    row0 = a.offsets[b];
    if (row0 < 0 || row0 + n > a.rows) {  // rows that the outputs do not have
      bad |= DA_STATUS_SEQ_LEN;
      n = row0 < 0 ? 0 : max(static_cast<int64_t>(0), min(n, a.rows - row0));
    }
  }
  if (bad != 0 && first == 0 && !is_v && tid == 0 && a.g.status != nullptr)
    atomicOr(a.g.status, static_cast<int32_t>(bad));
  const int count = static_cast<int>(min(n - first, static_cast<int64_t>(kReadTokens)));
  if (count <= 0) return;
  const CacheView& c = a.c;
  if (tid < count) {
    const int tok = start + first + tid;
    int64_t group = b;
    int slot = tok;
    if (a.g.block_table != nullptr) {
      int page = a.g.block_table[static_cast<int64_t>(b) * a.g.bt_stride + tok / a.g.page_size];
      if (page < 0 || page >= a.g.num_pages) {
        if (a.g.status != nullptr) atomicOr(a.g.status, static_cast<int32_t>(DA_STATUS_BAD_PAGE));
        page = 0;
      }
      group = page;
      slot = tok % a.g.page_size;
    }
    src[tid] = group * c.page + static_cast<int64_t>(slot) * c.token;
    src_sf[tid] = group * c.sf_page + static_cast<int64_t>(slot) * 8;
  }
  __syncthreads();

  const uint8_t* in = is_v ? c.v : c.k;
  const uint8_t* in_sf = is_v ? c.vs : c.ks;
  const float scale = is_v ? a.v_scale : a.k_scale;
  uint16_t* out = (is_v ? a.v : a.k) + (a.offsets != nullptr ? row0 * a.st : static_cast<int64_t>(b) * a.sb) +
                  static_cast<int64_t>(first) * a.st;
  // unit (token, head, 8 values), values fastest; a thread's units are
  // kReadThreads apart
  const int per_token = a.g.num_kv_heads * 16;
  const int step_tok = kReadThreads / per_token, step_hc = kReadThreads - step_tok * per_token;
  int tok = tid / per_token, hc = tid - tok * per_token;
  while (tok < count) {
    uint4 x[kReadAhead];
    uint32_t sf[kReadAhead];
    int64_t dst[kReadAhead];
#pragma unroll
    for (int j = 0; j < kReadAhead; ++j) {
      dst[j] = -1;
      if (tok < count) {
        const int head = hc >> 4, col = hc & 15;
        const uint8_t* p = in + src[tok] + static_cast<int64_t>(head) * c.head;
        if constexpr (TYPE == DA_CACHE_BF16) {
          x[j] = __ldg(reinterpret_cast<const uint4*>(p) + col);
        } else if constexpr (TYPE == DA_CACHE_FP8_E4M3) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(p) + col);
          x[j].x = w.x;
          x[j].y = w.y;
        } else {
          x[j].x = __ldg(reinterpret_cast<const uint32_t*>(p) + col);
          sf[j] = __ldg(in_sf + src_sf[tok] + static_cast<int64_t>(head) * c.sf_head + (col >> 1));
        }
        dst[j] = static_cast<int64_t>(tok) * a.st + static_cast<int64_t>(head) * a.sh + col * 8;
        tok += step_tok;
        hc += step_hc;
        if (hc >= per_token) {
          hc -= per_token;
          ++tok;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kReadAhead; ++j) {
      if (dst[j] < 0) continue;
      uint4 y = x[j];
      if constexpr (TYPE == DA_CACHE_FP8_E4M3) {
        uint32_t w[4];
        e4m3x4_to_f16x4(x[j].x, w[0], w[1]);
        e4m3x4_to_f16x4(x[j].y, w[2], w[3]);
        y = make_uint4(scaled_bf16x2(w[0], scale), scaled_bf16x2(w[1], scale), scaled_bf16x2(w[2], scale),
                       scaled_bf16x2(w[3], scale));
      } else if constexpr (TYPE == DA_CACHE_FP4_E2M1) {
        uint32_t w[4];
        e2m1x8_to_f16(x[j].x, w);
        const uint32_t s2 = __byte_perm(e4m3x2_to_f16x2(sf[j]), 0, 0x1010);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = scaled_bf16x2(mul_f16x2(w[i], s2), scale);
        y = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(out + dst[j]) = y;
    }
  }
}

// A launch that may begin behind the tail of the one before it.
template <typename Args>
cudaError_t launch_after(void (*kernel)(const Args), const Args& a, dim3 grid, int threads, size_t smem,
                         cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
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

cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t stream) {
  return launch_after(tree_mask_kernel, a, dim3(a.batch), kMaskThreads, 0, stream);
}

cudaError_t launch_keep(const KeepArgs& a, cudaStream_t stream) {
  const int pieces = a.c.type == DA_CACHE_BF16 ? 16 : a.c.type == DA_CACHE_FP8_E4M3 ? 8 : 4;
  const int columns = 2 * a.g.num_kv_heads * (pieces + (a.c.type == DA_CACHE_FP4_E2M1 ? 1 : 0));
  // (at most 32 KB: DECODE_ATTN_MAX_TREE moves)
  return launch_after(keep_kernel, a, dim3((columns + kKeepThreads - 1) / kKeepThreads, a.g.batch), kKeepThreads,
                      static_cast<size_t>(a.max_keep) * 32, stream);
}

cudaError_t launch_read(const ReadArgs& a, cudaStream_t stream) {
  const int64_t most = a.g.max_seq_len < a.max_tokens ? a.g.max_seq_len : a.max_tokens;
  if (most <= 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((most + kReadTokens - 1) / kReadTokens), a.g.batch, a.v != nullptr ? 2 : 1);
  switch (a.c.type) {
    case DA_CACHE_BF16: return launch_after(read_kernel<DA_CACHE_BF16>, a, grid, kReadThreads, 0, stream);
    case DA_CACHE_FP8_E4M3: return launch_after(read_kernel<DA_CACHE_FP8_E4M3>, a, grid, kReadThreads, 0, stream);
    default: return launch_after(read_kernel<DA_CACHE_FP4_E2M1>, a, grid, kReadThreads, 0, stream);
  }
}

}  // namespace dattn
