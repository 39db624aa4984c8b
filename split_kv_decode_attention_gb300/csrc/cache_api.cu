// cache_api.cu -- the C entries of the operators around the cache (declared in
// include/decode_attn.h): argument checks, workspace layouts and launches.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "cache_kernels.cuh"
#include "decode_attn.h"
#include "internal.cuh"

namespace {

using dattn::aligned16;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// element strides of 16-byte rows (bf16 tensors)
bool row_stride_ok(int64_t s) { return s > 0 && s % 8 == 0 && s < (int64_t{1} << 39); }

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int check_type(const decode_attn_params* p, const decode_attn_cache* c) {
  if (p == nullptr || c == nullptr) return DA_ERR_NULL_POINTER;
  if (c->type != DA_CACHE_BF16 && c->type != DA_CACHE_FP8_E4M3 && c->type != DA_CACHE_FP4_E2M1)
    return DA_ERR_UNSUPPORTED;
  if (c->reserved != 0) return DA_ERR_BAD_SHAPE;
  if (c->type != DA_CACHE_BF16 && (!std::isfinite(p->k_scale) || !std::isfinite(p->v_scale)))
    return DA_ERR_BAD_SHAPE;
  return DA_OK;
}

dattn::CacheView cache_view(const decode_attn_params* p, const decode_attn_cache* c) {
  const int64_t eb = c->type == DA_CACHE_BF16 ? 2 : 1;
  dattn::CacheView v;
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

dattn::PagingView paging_view(const decode_attn_params* p, const int32_t* block_table,
                              const int32_t* seq_lens, int32_t* status) {
  dattn::PagingView g;
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

int check_select(const decode_attn_params* p, const decode_attn_select* s) {
  if (s == nullptr) return DA_ERR_NULL_POINTER;
  if (s->top_k < 1 || s->top_k > 4096 || s->sink < 0 || s->local < 1 || s->reserved != 0 ||
      static_cast<int64_t>(s->sink) + s->local > s->top_k)
    return DA_ERR_BAD_SHAPE;
  int rc = dattn::check_paged(p, true);
  if (rc != DA_OK) return rc;
  const int64_t vb = static_cast<int64_t>(p->batch) * p->q_len;
  if (vb > 65535 || vb * p->num_kv_heads > 0x7fffffff ||
      (static_cast<int64_t>(p->max_seq_len) + p->page_size - 1) / p->page_size > (1 << 20) ||
      static_cast<int64_t>(s->top_k) * p->page_size > (1 << 30))
    return DA_ERR_BAD_SHAPE;
  return DA_OK;
}

int max_blocks(const decode_attn_params* p) {
  return static_cast<int>((static_cast<int64_t>(p->max_seq_len) + p->page_size - 1) / p->page_size);
}

int64_t score_stride(const decode_attn_params* p) { return (max_blocks(p) + 3) & ~int64_t{3}; }

size_t select_bytes(const decode_attn_params* p, const decode_attn_select* s) {
  if (max_blocks(p) <= s->top_k) return 0;
  return static_cast<size_t>(p->batch) * p->q_len * p->num_kv_heads * score_stride(p) * 4;
}

// The pages of a token are its whole cache: the attention of (request, token)
// pairs as requests of one token over [pairs][Hkv] page lists.
decode_attn_params selected_params(const decode_attn_params* p, const decode_attn_select* s) {
  decode_attn_params r = *p;
  r.batch = p->batch * p->q_len;
  r.q_len = 1;
  r.causal = 0;
  const int pages = std::min(s->top_k, std::max(max_blocks(p), 1));
  r.max_pages_per_seq = s->top_k;
  r.block_table_stride = static_cast<int64_t>(p->num_kv_heads) * s->top_k;
  r.max_seq_len = std::min<int64_t>(static_cast<int64_t>(pages) * p->page_size,
                                    std::max(p->max_seq_len, 0));
  r.q_stride_batch = p->q_len == 1 ? p->q_stride_batch : p->q_stride_token;
  r.o_stride_batch = p->q_len == 1 ? p->o_stride_batch : p->o_stride_token;
  return r;
}

struct SparseLayout {
  size_t scores, pages, tokens, part, total;
  int32_t splits;
};

int sparse_layout(const decode_attn_params* p, const decode_attn_cache* c,
                  const decode_attn_select* s, const decode_attn_params& sp, SparseLayout* l) {
  dattn::DecodeExt ext;
  ext.fp4 = c->type == DA_CACHE_FP4_E2M1 ? c : nullptr;
  ext.per_head = true;
  const size_t rows = static_cast<size_t>(p->batch) * p->q_len * p->num_kv_heads;
  l->scores = 0;
  l->pages = round256(select_bytes(p, s));
  l->tokens = round256(l->pages + rows * s->top_k * 4);
  l->part = round256(l->tokens + rows * 4);
  int32_t chunk = 0;
  int rc = dattn::plan_uniform(&sp, ext, &l->splits, &chunk);
  if (rc != DA_OK) return rc;
  size_t part = 0;
  rc = dattn::workspace_bytes(&sp, l->splits, ext, &part);
  if (rc != DA_OK) return rc;
  l->total = l->part + part;
  return DA_OK;
}

int select_impl(const decode_attn_params* p, const decode_attn_select* s, const void* q,
                const int8_t* digest, const float* digest_scale, const int32_t* block_table,
                const int32_t* seq_lens, int32_t* blocks, int32_t* pages, int32_t* tokens,
                void* workspace, int32_t* status, int sm_count, cudaStream_t stream) {
  dattn::SelectArgs a;
  std::memset(&a, 0, sizeof(a));
  a.g = paging_view(p, block_table, seq_lens, status);
  a.q = static_cast<const uint16_t*>(q);
  a.q_sb = p->q_stride_batch;
  a.q_st = p->q_stride_token;
  a.q_sh = p->q_stride_head;
  a.digest = digest;
  a.digest_scale = digest_scale;
  a.num_q_heads = p->num_q_heads;
  a.causal = p->causal ? 1 : 0;
  a.top_k = s->top_k;
  a.sink = s->sink;
  a.local = s->local;
  a.scores = static_cast<float*>(workspace);
  a.score_stride = score_stride(p);
  a.max_blocks = max_blocks(p);
  a.blocks = blocks;
  a.pages = pages;
  a.tokens = tokens;
  return dattn::launch_select(a, sm_count, stream) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int check_select_args(const decode_attn_params* p, const void* q, const int8_t* digest,
                      const float* digest_scale, const int32_t* block_table,
                      const int32_t* seq_lens) {
  if (q == nullptr || digest == nullptr || digest_scale == nullptr || block_table == nullptr ||
      seq_lens == nullptr)
    return DA_ERR_NULL_POINTER;
  if (!aligned16(q) || !aligned16(digest) || !aligned(digest_scale, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !row_stride_ok(p->q_stride_batch) ||
      !row_stride_ok(p->q_stride_token) || !row_stride_ok(p->q_stride_head))
    return DA_ERR_ALIGNMENT;
  return DA_OK;
}

}  // namespace

extern "C" {

int decode_attn_cached_workspace_bytes(const decode_attn_params* p, const decode_attn_cache* c,
                                       int32_t num_splits, size_t* bytes) {
  int rc = check_type(p, c);
  if (rc != DA_OK) return rc;
  const decode_attn_params cp = dattn::params_of_cache(p, c);
  rc = dattn::check_params(&cp, true);
  if (rc != DA_OK) return rc;
  dattn::DecodeExt ext;
  ext.fp4 = c->type == DA_CACHE_FP4_E2M1 ? c : nullptr;
  return dattn::workspace_bytes(&cp, num_splits, ext, bytes);
}

int decode_attn_cached(const decode_attn_params* p, const decode_attn_cache* c, const void* q,
                       const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse,
                       int32_t num_splits, void* workspace, size_t workspace_bytes,
                       int32_t* status, void* stream) {
  int rc = check_type(p, c);
  if (rc != DA_OK) return rc;
  const decode_attn_params cp = dattn::params_of_cache(p, c);
  rc = dattn::check_params(&cp, true);
  if (rc != DA_OK) return rc;
  dattn::DecodeExt ext;
  if (c->type == DA_CACHE_FP4_E2M1) {
    ext.fp4 = c;
    if (cp.batch > 0 && cp.max_seq_len > 0) {
      rc = dattn::check_cache(&cp, c, true, true);
      if (rc != DA_OK) return rc;
    }
  }
  return dattn::run_decode(&cp, q, c->k, c->v, block_table, seq_lens, out, lse, num_splits,
                           workspace, workspace_bytes, status, stream, true, ext);
}

int decode_attn_rope_table(const double* inv_freq, int32_t num_freqs, int64_t first, int64_t count,
                           double amplitude, float* table, void* stream) {
  if (num_freqs < 1 || num_freqs > DECODE_ATTN_HEAD_DIM / 2 || first < 0 || count < 0 ||
      first > (int64_t{1} << 31) || count > (int64_t{1} << 31) - first)
    return DA_ERR_BAD_SHAPE;
  if (count == 0) return DA_OK;
  if (inv_freq == nullptr || table == nullptr) return DA_ERR_NULL_POINTER;
  if (!aligned(inv_freq, 8) || !aligned16(table)) return DA_ERR_ALIGNMENT;
  int sms = 0;
  const int rc = dattn::check_device(&sms);
  if (rc != DA_OK) return rc;
  return dattn::launch_rope_table(inv_freq, num_freqs, first, count, amplitude, table, sms,
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DA_OK
             : DA_ERR_CUDA;
}

int decode_attn_rope_append(const decode_attn_params* p, const decode_attn_cache* c,
                            const decode_attn_rope* r, const void* q, const void* k, const void* v,
                            const float* table, const int32_t* positions, const int32_t* new_lens,
                            const int32_t* block_table, const int32_t* seq_lens, void* q_out,
                            int32_t* status, void* stream) {
  int rc = check_type(p, c);
  if (rc != DA_OK) return rc;
  if (r == nullptr) return DA_ERR_NULL_POINTER;
  const decode_attn_params cp = dattn::params_of_cache(p, c);
  rc = dattn::check_params(&cp, false);
  if (rc != DA_OK) return rc;
  const bool paged = block_table != nullptr;
  rc = dattn::check_paged(p, paged);
  if (rc != DA_OK) return rc;
  if (r->rotary_dim < 0 || r->rotary_dim > DECODE_ATTN_HEAD_DIM || r->rotary_dim % 2 != 0 ||
      r->table_positions < 0 || r->reserved != 0 ||
      static_cast<int64_t>(p->batch) * p->q_len > 0x7fffffff ||
      (c->type != DA_CACHE_BF16 && (!std::isfinite(1.f / p->k_scale) || !std::isfinite(1.f / p->v_scale))))
    return DA_ERR_BAD_SHAPE;
  if (p->batch == 0) return DA_OK;
  const bool rotate = q != nullptr, append = k != nullptr;
  if (seq_lens == nullptr || (q == nullptr) != (q_out == nullptr) || (k == nullptr) != (v == nullptr) ||
      (!rotate && !append) || (r->rotary_dim > 0 && table == nullptr))
    return DA_ERR_NULL_POINTER;
  if (!aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(positions, 4) ||
      !aligned(new_lens, 4) || !aligned16(table) || !aligned16(q) || !aligned16(q_out) ||
      !aligned16(k) || !aligned16(v))
    return DA_ERR_ALIGNMENT;
  if (rotate && (!row_stride_ok(p->q_stride_batch) || !row_stride_ok(p->q_stride_token) ||
                 !row_stride_ok(p->q_stride_head) || !row_stride_ok(p->o_stride_batch) ||
                 !row_stride_ok(p->o_stride_token) || !row_stride_ok(p->o_stride_head)))
    return DA_ERR_ALIGNMENT;
  if (append) {
    if (!row_stride_ok(r->k_stride_batch) || !row_stride_ok(r->k_stride_token) ||
        !row_stride_ok(r->k_stride_head) || !row_stride_ok(r->v_stride_batch) ||
        !row_stride_ok(r->v_stride_token) || !row_stride_ok(r->v_stride_head))
      return DA_ERR_ALIGNMENT;
    if (p->max_seq_len > 0) {  // (no token has a place otherwise)
      rc = dattn::check_cache(&cp, c, true, true);
      if (rc != DA_OK) return rc;
    }
  }
  int sms = 0;
  rc = dattn::check_device(&sms);
  if (rc != DA_OK) return rc;
  dattn::AppendArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = cache_view(p, c);
  a.g = paging_view(p, block_table, seq_lens, status);
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.table = table;
  a.positions = positions;
  a.new_lens = new_lens;
  a.q_sb = p->q_stride_batch;
  a.q_st = p->q_stride_token;
  a.q_sh = p->q_stride_head;
  a.o_sb = p->o_stride_batch;
  a.o_st = p->o_stride_token;
  a.o_sh = p->o_stride_head;
  a.k_sb = r->k_stride_batch;
  a.k_st = r->k_stride_token;
  a.k_sh = r->k_stride_head;
  a.v_sb = r->v_stride_batch;
  a.v_st = r->v_stride_token;
  a.v_sh = r->v_stride_head;
  a.num_q_heads = rotate ? p->num_q_heads : 0;
  a.append = append ? 1 : 0;
  a.rotary_dim = r->rotary_dim;
  a.interleaved = r->interleaved ? 1 : 0;
  a.table_positions = r->table_positions;
  a.one = 1.f;
  a.k_inv = c->type != DA_CACHE_BF16 ? 1.f / p->k_scale : 1.f;
  a.v_inv = c->type != DA_CACHE_BF16 ? 1.f / p->v_scale : 1.f;
  return dattn::launch_append(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DA_OK
             : DA_ERR_CUDA;
}

int decode_attn_block_digest(const decode_attn_params* p, const decode_attn_cache* c,
                             const int32_t* block_table, const int32_t* seq_lens, int32_t max_new,
                             int8_t* digest, float* digest_scale, int32_t* status, void* stream) {
  int rc = check_type(p, c);
  if (rc != DA_OK) return rc;
  const decode_attn_params cp = dattn::params_of_cache(p, c);
  rc = dattn::check_params(&cp, false);
  if (rc != DA_OK) return rc;
  rc = dattn::check_paged(p, true);
  if (rc != DA_OK) return rc;
  if (max_new < 0) return DA_ERR_BAD_SHAPE;
  if (p->batch == 0 || p->max_seq_len == 0) return DA_OK;
  if (block_table == nullptr || seq_lens == nullptr || digest == nullptr || digest_scale == nullptr)
    return DA_ERR_NULL_POINTER;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned16(digest) ||
      !aligned(digest_scale, 4))
    return DA_ERR_ALIGNMENT;
  rc = dattn::check_cache(&cp, c, true, false);
  if (rc != DA_OK) return rc;
  if (static_cast<int64_t>(max_blocks(p)) * p->num_kv_heads > 0x7fffffff) return DA_ERR_BAD_SHAPE;
  int sms = 0;
  rc = dattn::check_device(&sms);
  if (rc != DA_OK) return rc;
  dattn::DigestArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = cache_view(p, c);
  a.g = paging_view(p, block_table, seq_lens, status);
  a.max_new = max_new;
  a.digest = digest;
  a.digest_scale = digest_scale;
  return dattn::launch_digest(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK
                                                                                        : DA_ERR_CUDA;
}

int decode_attn_block_select_workspace_bytes(const decode_attn_params* p,
                                             const decode_attn_select* s, size_t* bytes) {
  int rc = dattn::check_params(p, true);
  if (rc != DA_OK) return rc;
  rc = check_select(p, s);
  if (rc != DA_OK) return rc;
  if (bytes == nullptr) return DA_ERR_NULL_POINTER;
  *bytes = select_bytes(p, s);
  return DA_OK;
}

int decode_attn_block_select(const decode_attn_params* p, const decode_attn_select* s,
                             const void* q, const int8_t* digest, const float* digest_scale,
                             const int32_t* block_table, const int32_t* seq_lens, int32_t* blocks,
                             int32_t* pages, int32_t* tokens, void* workspace,
                             size_t workspace_bytes, int32_t* status, void* stream) {
  int rc = dattn::check_params(p, true);
  if (rc != DA_OK) return rc;
  rc = check_select(p, s);
  if (rc != DA_OK) return rc;
  if (p->batch == 0) return DA_OK;
  rc = check_select_args(p, q, digest, digest_scale, block_table, seq_lens);
  if (rc != DA_OK) return rc;
  if (pages == nullptr || tokens == nullptr) return DA_ERR_NULL_POINTER;
  if (!aligned(pages, 4) || !aligned(tokens, 4) || !aligned(blocks, 4)) return DA_ERR_ALIGNMENT;
  const size_t need = select_bytes(p, s);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)))
    return DA_ERR_WORKSPACE;
  int sms = 0;
  rc = dattn::check_device(&sms);
  if (rc != DA_OK) return rc;
  return select_impl(p, s, q, digest, digest_scale, block_table, seq_lens, blocks, pages, tokens,
                     workspace, status, sms, static_cast<cudaStream_t>(stream));
}

int decode_attn_sparse_workspace_bytes(const decode_attn_params* p, const decode_attn_cache* c,
                                       const decode_attn_select* s, size_t* bytes) {
  int rc = check_type(p, c);
  if (rc != DA_OK) return rc;
  const decode_attn_params cp = dattn::params_of_cache(p, c);
  rc = dattn::check_params(&cp, true);
  if (rc != DA_OK) return rc;
  rc = check_select(&cp, s);
  if (rc != DA_OK) return rc;
  if (bytes == nullptr) return DA_ERR_NULL_POINTER;
  SparseLayout l;
  rc = sparse_layout(&cp, c, s, selected_params(&cp, s), &l);
  if (rc != DA_OK) return rc;
  *bytes = l.total;
  return DA_OK;
}

int decode_attn_sparse(const decode_attn_params* p, const decode_attn_cache* c,
                       const decode_attn_select* s, const void* q, const int8_t* digest,
                       const float* digest_scale, const int32_t* block_table,
                       const int32_t* seq_lens, void* out, float* lse, int32_t* blocks,
                       void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  int rc = check_type(p, c);
  if (rc != DA_OK) return rc;
  const decode_attn_params cp = dattn::params_of_cache(p, c);
  rc = dattn::check_params(&cp, true);
  if (rc != DA_OK) return rc;
  rc = check_select(&cp, s);
  if (rc != DA_OK) return rc;
  // the score bounds q . k only where both are multiplied by something positive
  if (!(cp.scale > 0.f) || (c->type != DA_CACHE_BF16 && !(cp.k_scale > 0.f)))
    return DA_ERR_BAD_SHAPE;
  if (cp.q_len > 1 && cp.batch > 1 &&
      (cp.q_stride_batch != cp.q_len * cp.q_stride_token ||
       cp.o_stride_batch != cp.q_len * cp.o_stride_token))
    return DA_ERR_BAD_SHAPE;
  if (cp.batch == 0) return DA_OK;
  rc = check_select_args(&cp, q, digest, digest_scale, block_table, seq_lens);
  if (rc != DA_OK) return rc;
  if (out == nullptr || lse == nullptr) return DA_ERR_NULL_POINTER;
  if (!aligned16(out) || !aligned(lse, 4) || !aligned(blocks, 4) ||
      !row_stride_ok(cp.o_stride_batch) || !row_stride_ok(cp.o_stride_token) ||
      !row_stride_ok(cp.o_stride_head))
    return DA_ERR_ALIGNMENT;
  if (cp.max_seq_len > 0) {
    rc = dattn::check_cache(&cp, c, true, true);
    if (rc != DA_OK) return rc;
  }
  int sms = 0;
  rc = dattn::check_device(&sms);
  if (rc != DA_OK) return rc;
  const decode_attn_params sp = selected_params(&cp, s);
  SparseLayout l;
  rc = sparse_layout(&cp, c, s, sp, &l);
  if (rc != DA_OK) return rc;
  if (workspace == nullptr || workspace_bytes < l.total || !aligned16(workspace))
    return DA_ERR_WORKSPACE;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  int32_t* pages = reinterpret_cast<int32_t*>(w + l.pages);
  int32_t* tokens = reinterpret_cast<int32_t*>(w + l.tokens);
  rc = select_impl(&cp, s, q, digest, digest_scale, block_table, seq_lens, blocks, pages, tokens,
                   w + l.scores, status, sms, static_cast<cudaStream_t>(stream));
  if (rc != DA_OK) return rc;
  dattn::DecodeExt ext;
  ext.fp4 = c->type == DA_CACHE_FP4_E2M1 ? c : nullptr;
  ext.per_head = true;
  return dattn::run_decode(&sp, q, c->k, c->v, pages, tokens, out, lse, l.splits, w + l.part,
                           workspace_bytes - l.part, status, stream, true, ext);
}

}  // extern "C"
