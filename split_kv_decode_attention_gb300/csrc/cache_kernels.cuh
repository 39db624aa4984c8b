// cache_kernels.cuh -- launches of the kernels around the cache (rotary table,
// append, digest, page selection), called by cache_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dattn {

// A cache as its writers and readers address it, in bytes: (group, slot, head)
// at base + group * page + slot * token + head * head_; group is the page, or
// the request of a contiguous cache.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;   // block scales (4-bit caches)
  uint8_t* vs;
  int64_t page, token, head;
  int64_t sf_page, sf_head;
  int type;      // DA_CACHE_*
};

struct PagingView {
  const int32_t* block_table;  // nullptr: contiguous
  int64_t bt_stride;
  const int32_t* seq_lens;
  int32_t* status;
  int batch, q_len, page_size, num_pages, max_seq_len, num_kv_heads;
};

cudaError_t launch_rope_table(const double* inv_freq, int num_freqs, int64_t first, int64_t count,
                              double amplitude, float* table, int sm_count, cudaStream_t stream);

struct AppendArgs {
  CacheView c;
  PagingView g;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  const float* table;
  const int32_t* positions;
  const int32_t* new_lens;
  int64_t q_sb, q_st, q_sh, o_sb, o_st, o_sh, k_sb, k_st, k_sh, v_sb, v_st, v_sh;
  int num_q_heads;      // 0: q is not rotated
  int append;           // k and v are given
  int rotary_dim, interleaved, table_positions;
  float k_inv, v_inv;   // 1 / k_scale, 1 / v_scale
  float one;            // 1
};
cudaError_t launch_append(const AppendArgs& a, int sm_count, cudaStream_t stream);

struct DigestArgs {
  CacheView c;
  PagingView g;
  int max_new;          // 0: every page
  int8_t* digest;
  float* digest_scale;
};
cudaError_t launch_digest(const DigestArgs& a, int sm_count, cudaStream_t stream);

struct SelectArgs {
  PagingView g;
  const uint16_t* q;
  int64_t q_sb, q_st, q_sh;
  const int8_t* digest;
  const float* digest_scale;
  int num_q_heads, causal;
  int top_k, sink, local;
  float* scores;        // [B * q_len * Hkv][score_stride]
  int64_t score_stride; // a multiple of 4
  int max_blocks;       // ceil(max_seq_len / page_size)
  int32_t* blocks;      // optional
  int32_t* pages;
  int32_t* tokens;
};
cudaError_t launch_select(const SelectArgs& a, int sm_count, cudaStream_t stream);

}  // namespace dattn
