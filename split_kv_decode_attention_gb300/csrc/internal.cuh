// internal.cuh -- what the files of the C ABI share (api.cu implements it).
// Not part of the public header.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_attn.h"

namespace dattn {

// What a decode call needs beyond decode_attn()'s arguments.
struct DecodeExt {
  const decode_attn_cache* fp4 = nullptr;  // a 4-bit cache (else the params' flags tell)
  // lengths [batch][Hkv] and block-table rows [batch][Hkv][pages] per kv head
  bool per_head = false;
};

// The current device is usable (DA_OK) or not.
int check_device(int* sm_count);

bool aligned16(const void* p);

// Checks of the params that hold for every entry point; rows_limit: (Hq / Hkv)
// * q_len must not exceed DECODE_ATTN_MAX_ROWS (the attention calls).
int check_params(const decode_attn_params* p, bool rows_limit);
int check_paged(const decode_attn_params* p, bool paged);

// A cache described by *c under the strides of *p.
int check_cache(const decode_attn_params* p, const decode_attn_cache* c, bool need_k, bool need_v);

// p with the flags and scales that a cache of type c->type has.
decode_attn_params params_of_cache(const decode_attn_params* p, const decode_attn_cache* c);

int workspace_bytes(const decode_attn_params* p, int32_t num_splits, const DecodeExt& ext,
                    size_t* bytes);

int run_decode(const decode_attn_params* p, const void* q, const void* k_cache,
               const void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
               void* out, float* lse, int32_t num_splits, void* workspace,
               size_t workspace_bytes, int32_t* status, void* stream, bool run_combine,
               const DecodeExt& ext = {});

// The host plan for equal lengths (max_seq_len each).
int plan_uniform(const decode_attn_params* p, const DecodeExt& ext, int32_t* num_splits,
                 int32_t* chunk_len);

}  // namespace dattn
