// cache_kernels.cuh -- launches of the kernels around the cache (rotary table,
// append, digest, page selection), called by cache_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_attn.h"

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

// A cache and its paging as the C ABI's structs describe them.
inline CacheView cache_view(const decode_attn_params* p, const decode_attn_cache* c) {
  const int64_t eb = c->type == DA_CACHE_BF16 ? 2 : 1;
  CacheView v;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.ks = static_cast<uint8_t*>(c->k_block_scale);
  v.vs = static_cast<uint8_t*>(c->v_block_scale);
  v.page = p->kv_stride_page * eb;
  v.token = p->kv_stride_token * eb;
  v.head = p->kv_stride_head * eb;
  v.sf_page = c->bs_stride_page;
  v.sf_head = c->bs_stride_head;
  v.type = c->type;
  return v;
}

inline PagingView paging_view(const decode_attn_params* p, const int32_t* block_table,
                              const int32_t* seq_lens, int32_t* status) {
  PagingView g;
  g.block_table = block_table;
  g.bt_stride = p->block_table_stride;
  g.seq_lens = seq_lens;
  g.status = status;
  g.batch = p->batch;
  g.q_len = p->q_len;
  g.page_size = block_table != nullptr ? p->page_size : 0;
  g.num_pages = block_table != nullptr ? p->num_pages : 0;
  g.max_seq_len = p->max_seq_len;
  g.num_kv_heads = p->num_kv_heads;
  return g;
}

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

// Masks and positions of trees of drafted tokens.
struct TreeMaskArgs {
  const int32_t* parents;   // [batch][q_len]
  const int32_t* new_lens;  // optional
  const int32_t* seq_lens;
  uint32_t* mask;           // [batch][q_len][words]
  int32_t* positions;       // [batch][q_len], optional
  int32_t* status;
  int batch, q_len, words, max_seq_len;
};
cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t stream);

// Moves kept tokens together (q_len: the new tokens of a request at most).
struct KeepArgs {
  CacheView c;
  PagingView g;
  const int32_t* keep;      // [batch][max_keep]
  const int32_t* counts;
  const int32_t* new_lens;  // optional
  int32_t* out_lens;        // optional
  int max_keep;
};
cudaError_t launch_keep(const KeepArgs& a, cudaStream_t stream);

// Reads a cache back as bf16.
struct ReadArgs {
  CacheView c;
  PagingView g;
  const int32_t* starts;    // optional: first token of each request
  const int32_t* offsets;   // optional: first output row of each request
  uint16_t* k;
  uint16_t* v;
  int64_t sb, st, sh;       // element strides of both outputs
  int64_t rows;             // offsets: output rows; else unused
  int max_tokens;           // tokens of a request that the outputs hold
  float k_scale, v_scale;
};
cudaError_t launch_read(const ReadArgs& a, cudaStream_t stream);

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
