// tree_api.cu -- the C entries for trees of drafted tokens, cross attention and
// reading a cache back (declared in include/decode_attn.h): argument checks and
// launches.

#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "cache_kernels.cuh"
#include "decode_attn.h"
#include "internal.cuh"

namespace {

using dattn::aligned16;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether two arrays of 4-byte entries share memory.
bool overlap4(const void* x, int64_t nx, const void* y, int64_t ny) {
  if (x == nullptr || y == nullptr) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b + static_cast<uintptr_t>(ny) * 4 && b < a + static_cast<uintptr_t>(nx) * 4;
}

bool row_stride_ok(int64_t s) { return s > 0 && s % 8 == 0 && s < (int64_t{1} << 39); }

int check_type(const decode_attn_params* p, const decode_attn_cache* c) {
  if (p == nullptr || c == nullptr) return DA_ERR_NULL_POINTER;
  if (c->type != DA_CACHE_BF16 && c->type != DA_CACHE_FP8_E4M3 && c->type != DA_CACHE_FP4_E2M1)
    return DA_ERR_UNSUPPORTED;
  if (c->reserved != 0) return DA_ERR_BAD_SHAPE;
  if (c->type != DA_CACHE_BF16 && (!std::isfinite(p->k_scale) || !std::isfinite(p->v_scale)))
    return DA_ERR_BAD_SHAPE;
  return DA_OK;
}

// The params and the extension of a call whose rows see what `own` says.
int rows_call(const decode_attn_params* p, const decode_attn_cache* c, bool tree, decode_attn_params* cp,
              dattn::DecodeExt* ext) {
  int rc = check_type(p, c);
  if (rc != DA_OK) return rc;
  *cp = dattn::params_of_cache(p, c);
  cp->causal = 0;
  rc = dattn::check_params(cp, false);
  if (rc != DA_OK) return rc;
  const int64_t group = p->num_q_heads / p->num_kv_heads;
  if (group > DECODE_ATTN_MAX_ROWS) return DA_ERR_ROWS;
  if ((tree && p->q_len > DECODE_ATTN_MAX_TREE) || group * p->q_len > 0x7fffffff) return DA_ERR_BAD_SHAPE;
  ext->fp4 = c->type == DA_CACHE_FP4_E2M1 ? c : nullptr;
  ext->own.on = 1;
  return DA_OK;
}

int run_rows_call(const decode_attn_params& cp, const decode_attn_cache* c, const void* q,
                  const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse,
                  int32_t num_splits, void* workspace, size_t workspace_bytes, int32_t* status,
                  void* stream, const dattn::DecodeExt& ext) {
  if (ext.fp4 != nullptr && cp.batch > 0 && cp.max_seq_len > 0) {
    const int rc = dattn::check_cache(&cp, c, true, true);
    if (rc != DA_OK) return rc;
  }
  return dattn::run_rows(&cp, c, q, block_table, seq_lens, out, lse, num_splits, workspace,
                         workspace_bytes, status, stream, ext);
}

int rows_bytes(const decode_attn_params* p, const decode_attn_cache* c, int32_t num_splits, bool tree,
               size_t* bytes) {
  decode_attn_params cp;
  dattn::DecodeExt ext;
  const int rc = rows_call(p, c, tree, &cp, &ext);
  return rc != DA_OK ? rc : dattn::rows_workspace_bytes(&cp, c, num_splits, ext, bytes);
}

}  // namespace

extern "C" {

int decode_attn_tree_mask(int32_t batch, int32_t q_len, int32_t max_seq_len, const int32_t* parents,
                          const int32_t* new_lens, const int32_t* seq_lens, uint32_t* mask,
                          int32_t* positions, int32_t* status, void* stream) {
  if (batch < 0 || batch > 65535 || q_len < 1 || q_len > DECODE_ATTN_MAX_TREE || max_seq_len < 0)
    return DA_ERR_BAD_SHAPE;
  if (batch == 0) return DA_OK;
  if (parents == nullptr || seq_lens == nullptr || mask == nullptr) return DA_ERR_NULL_POINTER;
  if (!aligned4(parents) || !aligned4(new_lens) || !aligned4(seq_lens) || !aligned4(mask) ||
      !aligned4(positions) || !aligned4(status))
    return DA_ERR_ALIGNMENT;
  // (a request's rows are written while others' inputs are still to be read; positions
  // may take the place of parents, which are read first, row by row)
  const int64_t n = batch, tokens = n * q_len, words = tokens * ((q_len + 31) / 32);
  if (overlap4(mask, words, parents, tokens) || overlap4(mask, words, new_lens, n) || overlap4(mask, words, seq_lens, n) ||
      overlap4(mask, words, positions, tokens) || overlap4(positions, tokens, new_lens, n) ||
      overlap4(positions, tokens, seq_lens, n) || (positions != parents && overlap4(positions, tokens, parents, tokens)))
    return DA_ERR_BAD_SHAPE;
  const int rc = dattn::check_device(nullptr);
  if (rc != DA_OK) return rc;
  dattn::TreeMaskArgs a;
  std::memset(&a, 0, sizeof(a));
  a.parents = parents;
  a.new_lens = new_lens;
  a.seq_lens = seq_lens;
  a.mask = mask;
  a.positions = positions;
  a.status = status;
  a.batch = batch;
  a.q_len = q_len;
  a.words = (q_len + 31) / 32;
  a.max_seq_len = max_seq_len;
  return dattn::launch_tree_mask(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int decode_attn_tree_workspace_bytes(const decode_attn_params* p, const decode_attn_cache* c,
                                     int32_t num_splits, size_t* bytes) {
  return rows_bytes(p, c, num_splits, true, bytes);
}

int decode_attn_tree(const decode_attn_params* p, const decode_attn_cache* c, const void* q,
                     const uint32_t* mask, int64_t mask_stride_batch, const int32_t* new_lens,
                     const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse,
                     int32_t num_splits, void* workspace, size_t workspace_bytes, int32_t* status,
                     void* stream) {
  decode_attn_params cp;
  dattn::DecodeExt ext;
  const int rc = rows_call(p, c, true, &cp, &ext);
  if (rc != DA_OK) return rc;
  if (mask_stride_batch < 0) return DA_ERR_BAD_SHAPE;
  if (cp.batch == 0) return DA_OK;
  if (mask == nullptr) return DA_ERR_NULL_POINTER;
  if (!aligned4(mask) || !aligned4(new_lens) || !aligned4(status)) return DA_ERR_ALIGNMENT;
  ext.own.mask = mask;
  ext.own.mask_sb = mask_stride_batch;
  ext.own.words = (cp.q_len + 31) / 32;
  ext.own.own_lens = new_lens;
  return run_rows_call(cp, c, q, block_table, seq_lens, out, lse, num_splits, workspace, workspace_bytes,
                       status, stream, ext);
}

int decode_attn_cross_workspace_bytes(const decode_attn_params* p, const decode_attn_cache* c,
                                      int32_t num_splits, size_t* bytes) {
  return rows_bytes(p, c, num_splits, false, bytes);
}

int decode_attn_cross(const decode_attn_params* p, const decode_attn_cache* c, const void* q,
                      const int32_t* q_lens, const int32_t* block_table, const int32_t* seq_lens,
                      void* out, float* lse, int32_t num_splits, void* workspace,
                      size_t workspace_bytes, int32_t* status, void* stream) {
  decode_attn_params cp;
  dattn::DecodeExt ext;
  const int rc = rows_call(p, c, false, &cp, &ext);
  if (rc != DA_OK) return rc;
  if (!aligned4(q_lens) || !aligned4(status)) return DA_ERR_ALIGNMENT;
  ext.own.own_lens = q_lens;
  return run_rows_call(cp, c, q, block_table, seq_lens, out, lse, num_splits, workspace, workspace_bytes,
                       status, stream, ext);
}

int decode_attn_cache_keep(const decode_attn_params* p, const decode_attn_cache* c, const int32_t* keep,
                           int32_t max_keep, const int32_t* counts, const int32_t* new_lens,
                           const int32_t* block_table, const int32_t* seq_lens, int32_t* out_lens,
                           int32_t* status, void* stream) {
  int rc = check_type(p, c);
  if (rc != DA_OK) return rc;
  const decode_attn_params cp = dattn::params_of_cache(p, c);
  rc = dattn::check_params(&cp, false);
  if (rc != DA_OK) return rc;
  rc = dattn::check_paged(&cp, block_table != nullptr);
  if (rc != DA_OK) return rc;
  if (cp.q_len > DECODE_ATTN_MAX_TREE || max_keep < 0 || max_keep > cp.q_len) return DA_ERR_BAD_SHAPE;
  if (cp.batch == 0) return DA_OK;
  if ((keep == nullptr && max_keep > 0) || counts == nullptr || seq_lens == nullptr)
    return DA_ERR_NULL_POINTER;
  if (!aligned4(keep) || !aligned4(counts) || !aligned4(new_lens) || !aligned4(block_table) ||
      !aligned4(seq_lens) || !aligned4(out_lens) || !aligned4(status))
    return DA_ERR_ALIGNMENT;
  const int64_t n = cp.batch;  // (the inputs are read while out_lens is written)
  if (overlap4(out_lens, n, seq_lens, n) || overlap4(out_lens, n, counts, n) || overlap4(out_lens, n, new_lens, n) ||
      overlap4(out_lens, n, keep, n * max_keep))
    return DA_ERR_BAD_SHAPE;
  if (cp.max_seq_len > 0) {  // (no token has a place otherwise)
    rc = dattn::check_cache(&cp, c, true, true);
    if (rc != DA_OK) return rc;
  }
  rc = dattn::check_device(nullptr);
  if (rc != DA_OK) return rc;
  dattn::KeepArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = dattn::cache_view(&cp, c);
  a.g = dattn::paging_view(&cp, block_table, seq_lens, status);
  a.keep = keep;
  a.counts = counts;
  a.new_lens = new_lens;
  a.out_lens = out_lens;
  a.max_keep = max_keep;
  return dattn::launch_keep(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int decode_attn_cache_read(const decode_attn_params* p, const decode_attn_cache* c,
                           const decode_attn_read* r, const int32_t* starts, const int32_t* offsets,
                           const int32_t* block_table, const int32_t* seq_lens, void* k_out, void* v_out,
                           int32_t* status, void* stream) {
  int rc = check_type(p, c);
  if (rc != DA_OK) return rc;
  if (r == nullptr) return DA_ERR_NULL_POINTER;
  const decode_attn_params cp = dattn::params_of_cache(p, c);
  rc = dattn::check_params(&cp, false);
  if (rc != DA_OK) return rc;
  rc = dattn::check_paged(&cp, block_table != nullptr);
  if (rc != DA_OK) return rc;
  if (r->max_tokens < 0 || r->reserved != 0 || (offsets != nullptr && r->rows < 0)) return DA_ERR_BAD_SHAPE;
  if (cp.batch == 0 || cp.max_seq_len == 0 || r->max_tokens == 0 || (offsets != nullptr && r->rows == 0))
    return DA_OK;
  if (seq_lens == nullptr || k_out == nullptr) return DA_ERR_NULL_POINTER;
  if (!aligned4(starts) || !aligned4(offsets) || !aligned4(block_table) || !aligned4(seq_lens) ||
      !aligned4(status) || !aligned16(k_out) || !aligned16(v_out) ||
      (offsets == nullptr && !row_stride_ok(r->stride_batch)) || !row_stride_ok(r->stride_token) ||
      !row_stride_ok(r->stride_head))
    return DA_ERR_ALIGNMENT;
  rc = dattn::check_cache(&cp, c, true, v_out != nullptr);
  if (rc != DA_OK) return rc;
  rc = dattn::check_device(nullptr);
  if (rc != DA_OK) return rc;
  dattn::ReadArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = dattn::cache_view(&cp, c);
  a.g = dattn::paging_view(&cp, block_table, seq_lens, status);
  a.starts = starts;
  a.offsets = offsets;
  a.k = static_cast<uint16_t*>(k_out);
  a.v = static_cast<uint16_t*>(v_out);
  a.sb = r->stride_batch;
  a.st = r->stride_token;
  a.sh = r->stride_head;
  a.rows = r->rows;
  a.max_tokens = r->max_tokens;
  // (a bf16 cache has no scale)
  a.k_scale = cp.k_scale;
  a.v_scale = cp.v_scale;
  return dattn::launch_read(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

}  // extern "C"
