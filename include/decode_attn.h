/*
 * decode_attn.h -- C ABI of libdecode_attn.so: split-KV decode attention
 * (Flash-Decoding) for GB300 / sm_103a.
 *
 * The operation.  For every request b < batch, new token t < q_len and query
 * head h < num_q_heads, with key/value head kvh = h / G and G = Hq / Hkv
 * (contiguous GQA groups: "Capstone FlashAttention", §4.2; the inference-engine
 * chapter "12. attention kernels", decode section):
 *
 *     s_j   = scale * q[b,t,h,:] . K[b, j, kvh, :]
 *     out   = sum_j softmax(s)_j * V[b, j, kvh, :]          (bf16)
 *     lse   = ln sum_j exp(s_j)                              (fp32)
 *
 * exact attention softmax(QK^T/sqrt(d))V ("Capstone FlashAttention", §1.1),
 * over the keys j < L = seq_lens[b]; with `causal`, token t (at position
 * L - q_len + t) only sees keys j <= L - q_len + t.  A row with no visible key
 * gives out = 0 and lse = -inf.  (So does one whose scores are all -inf, which
 * takes infinite entries or products past fp32.)  A row that meets NaN, in its
 * query or in a key that it sees, or an infinite score of +inf, gives NaN and a
 * NaN lse, whatever the number of chunks; other rows are not affected.  (Over
 * FP8 caches |q| above 65504 counts as infinite.)
 *
 * How.  The KV sequence of each (request, kv head) is cut into chunks of
 * `chunk_len` tokens that run on different SMs; each chunk keeps a running
 * max / running sum (online softmax, "Capstone FlashAttention", §1.2) and
 * writes an fp32 partial output plus its log-sum-exp; a combine kernel merges
 * the partials exactly ("Capstone FlashAttention", §2.3 FlashDecoding; the
 * per-tile LSE buffer of the CUTLASS split-KV post, §4.2).  Requests whose
 * keys fit one chunk skip the partials and the combine.  When the call needs
 * 2..16 chunks per (request, kv head) and all of them fit on the GPU at once,
 * the chunks of one head run as a thread-block cluster and merge through
 * distributed shared memory instead: one launch, no partials in memory (the
 * workspace is then unused; DA_FLAG_TWO_PASS turns this off).
 *
 * Cache layouts.  K and V share one layout; head_dim is contiguous.
 *   paged (block_table != NULL): element (page, slot, head, d) of a cache is at
 *       page*kv_stride_page + slot*kv_stride_token + head*kv_stride_head + d;
 *       logical token j of request b is page block_table[b*block_table_stride
 *       + j/page_size], slot j%page_size (PagedAttention, "Capstone
 *       FlashAttention", §4.1).
 *   contiguous (block_table == NULL): token j of request b is at
 *       b*kv_stride_page + j*kv_stride_token + head*kv_stride_head + d, for
 *       j < max_seq_len.
 * Strides are in elements; K and V base pointers must be 16-byte aligned and
 * every KV stride a multiple of 8 elements (16 bytes).
 *
 * FP8 caches (flags & DA_FLAG_KV_FP8_E4M3).  K and V hold one byte per element
 * in the OCP FP8 E4M3 format (1 sign bit, 4 exponent bits with bias 7, 3
 * mantissa bits, subnormals, no infinities, S.1111.111 = NaN) with one fp32
 * scale per cache: the keys and values are k_scale * K and v_scale * V
 * (quantisation with explicit scaling factors rather than a plain cast:
 * "Capstone FlashAttention", §2.2 FP8 with scaling; the CUTLASS split-KV post,
 * §5.8).  q, out and lse keep their types.  Strides are then in bytes and must
 * be multiples of 16.
 *
 * Ownership and errors.  The caller owns every buffer (device memory unless
 * stated otherwise), including the workspace.  The library allocates nothing
 * on the device, never synchronises the stream and may be captured in a CUDA
 * graph.  Every function returns DA_OK (0) or a negative DA_ERR_* code; an
 * argument error is detected on the host before anything is launched.  Data
 * errors found on the device (a block-table entry outside [0, num_pages), a
 * seq_len outside [0, max_seq_len], a causal request shorter than q_len) are
 * OR-ed as DA_STATUS_* bits into *status when status != NULL; the caller reads
 * it after synchronising.  Faulty entries never fault the GPU: a bad page id
 * reads page 0 instead, an out-of-range length is clamped.
 *
 * Threading: all functions are thread-safe; calls on different streams may
 * overlap.
 */
#ifndef DECODE_ATTN_H_
#define DECODE_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DECODE_ATTN_HEAD_DIM 128   /* the only supported head_dim */
#define DECODE_ATTN_MAX_ROWS 128   /* (Hq / Hkv) * q_len must not exceed this;
                                      above 16 rows the tcgen05 kernel runs */
#define DECODE_ATTN_TOKEN_TILE 16  /* chunk_len and page_size are multiples */

/* return codes */
#define DA_OK 0
#define DA_ERR_NULL_POINTER -1     /* a required pointer is NULL */
#define DA_ERR_BAD_SHAPE -2        /* negative/zero sizes, Hq % Hkv != 0, ... */
#define DA_ERR_HEAD_DIM -3         /* head_dim != 128 */
#define DA_ERR_PAGE_SIZE -4        /* page_size not a positive multiple of 16 */
#define DA_ERR_ROWS -5             /* (Hq/Hkv)*q_len > DECODE_ATTN_MAX_ROWS */
#define DA_ERR_ALIGNMENT -6        /* pointer or stride misaligned */
#define DA_ERR_WORKSPACE -7        /* workspace NULL or smaller than required */
#define DA_ERR_CUDA -8             /* a CUDA runtime call or launch failed */
#define DA_ERR_NO_DEVICE -9        /* no usable sm_103 device is current */
#define DA_ERR_SPLITS -10          /* num_splits out of range */
#define DA_ERR_STATIC_WORKSPACE_LIMIT -11 /* partials exceed the static workspace */
#define DA_ERR_UNSUPPORTED -12     /* a flag combination this library does not run
                                      (reserved: no combination returns it at present) */

/* size of the device array behind decode_attn_static_workspace() */
#define DECODE_ATTN_STATIC_WORKSPACE_BYTES (16u << 20)

/* params.flags */
#define DA_FLAG_TWO_PASS 1u        /* always write fp32 partials to the workspace and
                                      merge them with the combine kernel (no
                                      cluster merge); needed to read partials */
#define DA_FLAG_KV_FP8_E4M3 2u     /* K and V caches are FP8 E4M3 bytes scaled by
                                      k_scale / v_scale (see "FP8 caches" above) */
#define DA_FLAG_TEST_WITHHOLD_COPY 0x100u /* test hook for failure detection:
                                      block (0, 0, 0) of the split launch never
                                      fills its first pipeline stage (at most 16
                                      rows per kv head: with DA_FLAG_TWO_PASS; above
                                      16, the tcgen05 kernel: the first stage of
                                      its first work item), so the bounded waits
                                      on it run out (~2 s each) and
                                      DA_STATUS_TIMEOUT is set; no fault, the
                                      context stays usable */

/* device status bits (OR-ed into *status) */
#define DA_STATUS_BAD_PAGE 1u      /* block-table entry outside [0, num_pages) */
#define DA_STATUS_SEQ_LEN 2u       /* seq_len < 0 or > max_seq_len (clamped) */
#define DA_STATUS_SHORT_CAUSAL 4u  /* causal and 0 < seq_len < q_len */
#define DA_STATUS_TIMEOUT 8u       /* an internal pipeline wait gave up */

typedef struct decode_attn_params {
  int32_t batch;              /* B >= 0 requests */
  int32_t q_len;              /* new tokens per request, >= 1 */
  int32_t num_q_heads;        /* Hq */
  int32_t num_kv_heads;       /* Hkv; Hq % Hkv == 0 */
  int32_t head_dim;           /* must be DECODE_ATTN_HEAD_DIM */
  int32_t page_size;          /* paged: tokens per page (multiple of 16);
                                 contiguous: ignored */
  int32_t max_pages_per_seq;  /* paged: usable columns of block_table */
  int32_t num_pages;          /* paged: physical pages in each cache (>= 1) */
  int32_t max_seq_len;        /* upper bound of seq_lens in this call; the
                                 contiguous cache holds this many tokens per
                                 request; paged: <= max_pages_per_seq*page_size */
  int32_t causal;             /* nonzero: causal mask among the q_len tokens */
  float scale;                /* softmax scale, e.g. 1/sqrt(head_dim) */
  int32_t flags;              /* DA_FLAG_* bits; 0 for the default path */
  int64_t q_stride_batch;     /* q [B, q_len, Hq, D] element strides; */
  int64_t q_stride_token;     /*   D contiguous, strides multiples of 8 */
  int64_t q_stride_head;
  int64_t o_stride_batch;     /* out [B, q_len, Hq, D] element strides */
  int64_t o_stride_token;
  int64_t o_stride_head;
  int64_t kv_stride_page;     /* see "Cache layouts" above */
  int64_t kv_stride_token;
  int64_t kv_stride_head;
  int64_t block_table_stride; /* elements between rows of block_table */
  float k_scale;              /* FP8 caches: keys = k_scale * K (1 by default) */
  float v_scale;              /* FP8 caches: values = v_scale * V (1 by default) */
} decode_attn_params;

/*
 * Fill *p with the strides of densely packed tensors:
 *   q, out [B, q_len, Hq, D]; paged caches [num_pages, page_size, Hkv, D];
 *   contiguous caches [B, max_seq_len, Hkv, D]; block_table [B, max_pages].
 * scale = 1/sqrt(head_dim), k_scale = v_scale = 1, flags = 0 (bf16 caches).
 * Pass page_size = 0 for a contiguous cache.
 */
void decode_attn_params_init(decode_attn_params *p, int32_t batch, int32_t q_len,
                             int32_t num_q_heads, int32_t num_kv_heads,
                             int32_t head_dim, int32_t page_size,
                             int32_t max_pages_per_seq, int32_t num_pages,
                             int32_t max_seq_len, int32_t causal);

/*
 * Split planner (host only; reads the current device's SM count once).
 * Picks the number of KV chunks per (request, kv head) and their length from
 * batch x kv heads x sequence length against the SM count, so that the split
 * kernel fills the GPU ("Capstone FlashAttention", §2.3: too few heads leave
 * SMs idle; chunks of a few hundred tokens or more).
 *   host_seq_lens  optional host copy of seq_lens (NULL: plan for max_seq_len)
 *   *num_splits    out: chunks per request at max_seq_len (>= 1)
 *   *chunk_len     out: tokens per chunk (multiple of 16)
 */
int decode_attn_plan(const decode_attn_params *p, const int32_t *host_seq_lens,
                     int32_t *num_splits, int32_t *chunk_len);

/*
 * The same planner for an explicit device shape (host only; needs no GPU and
 * touches no CUDA state), e.g. to plan ahead for another device:
 *   resident_ctas  CTAs of the split launch resident at once: SMs x CTAs per
 *                  SM of the kernel this shape runs (decode_attn_plan takes
 *                  the current device's SM count and the CUDA occupancy of
 *                  that kernel; on GB300, 152 SMs x 4 for bf16 caches with at
 *                  most 16 query rows per kv head, x 1 above 16 rows)
 * Equal lengths (or host_seq_lens NULL): one wave of equal chunks, at most 16
 * per (request, kv head).  Ragged lengths: chunks for about eight waves of
 * the real work, at least max(256, 64 x rows) tokens (256 x rows above 16
 * rows), shrunk (not below 256) while that leaves fewer chunks than resident
 * CTAs.  Returns DA_ERR_BAD_SHAPE unless 1 <= resident_ctas <= 2^31.
 */
int decode_attn_plan_slots(const decode_attn_params *p, const int32_t *host_seq_lens,
                           int64_t resident_ctas, int32_t *num_splits, int32_t *chunk_len);

/*
 * Chunk length used for a given num_splits: the smallest multiple of 16 that
 * covers max_seq_len in num_splits chunks.  Request b uses
 * ceil(seq_lens[b] / chunk_len) chunks (at least 1).
 */
int decode_attn_chunk_len(const decode_attn_params *p, int32_t num_splits,
                          int32_t *chunk_len);

/*
 * Workspace bytes decode_attn() needs for num_splits (0 when num_splits == 1;
 * unused when the cluster merge applies, see above).
 * Layout (fp32): partial outputs [B, q_len, Hq, num_splits, D], followed by
 * partial log-sum-exps [B, q_len, Hq, num_splits] (natural log).  Partial s of
 * a row is normalised (sum of weights 1) over its chunk's keys; an empty
 * chunk has lse -inf.  Entries of requests that use a single chunk are not
 * written.
 * num_splits <= 0: the need of the planned call -- for a device-planned call
 * (see "Device planning" at decode_attn) a bound that does not depend on the
 * lengths, for one request the host plan's need.  Reads the current device.
 */
int decode_attn_workspace_bytes(const decode_attn_params *p, int32_t num_splits,
                                size_t *bytes);

/*
 * Decode attention (the whole path: split kernel, then combine when a request
 * spans more than one chunk).
 *   q            bf16 [B, q_len, Hq, 128] (strides in *p)
 *   k_cache      bf16 cache, layout per *p (16-byte aligned)
 *   v_cache      bf16 cache, same layout as k_cache
 *   block_table  int32 [B, block_table_stride] or NULL (contiguous cache)
 *   seq_lens     int32 [B]: keys per request, including the q_len new tokens
 *   out          bf16 [B, q_len, Hq, 128] (strides in *p)
 *   lse          fp32 [B, q_len, Hq], contiguous
 *   num_splits   chunks per request at max_seq_len; <= 0 asks the planner
 *   workspace    device buffer of >= decode_attn_workspace_bytes() bytes
 *                (may be NULL when that is 0)
 *   status       optional int32 device word; DA_STATUS_* bits are OR-ed in
 *   stream       cudaStream_t to launch on (NULL: legacy default stream)
 * Device pointers only.  Asynchronous with respect to the host.
 *
 * Device planning (num_splits <= 0 with two or more requests; for the
 * tcgen05 kernel, above 16 rows per kv head, at most 1024 requests).  The
 * lengths may exist only on the device -- and change between replays of a
 * captured graph -- so the call plans there: a planner kernel applies
 * decode_attn_plan()'s rule to the current seq_lens (the same plan the host
 * planner gives for those lengths), then the split kernel runs one CTA per
 * item slot of a capacity fixed by the shape (B x Hkv + 16 waves of resident
 * CTAs), then the combine kernel merges: three launches, no host
 * synchronisation, graph capturable.  If the rule's chunk would make more
 * (request, kv head, chunk) items than the capacity, the chunk grows until
 * they fit.  Workspace layout (offsets rounded up to 256 bytes): int32
 * plan[4] = {chunk_len, items, chunks of the longest request, capacity};
 * int32 pre[B + 1], the exclusive prefix over requests of their chunk
 * counts; int4 items[capacity] = (b, kv head, chunk, clamped length) in
 * (request, kv head, chunk) order; fp32 partial outputs [capacity, rows, D]
 * and partial LSEs [capacity, rows], item i = pre[b] * Hkv + kvh * n_b + s
 * holding row r = t * G + g of that (b, kvh) (n_b = max(1, ceil(L_b /
 * chunk_len)) chunks).  One request keeps the host plan (from max_seq_len)
 * and, where it fits, the cluster merge.
 */
int decode_attn(const decode_attn_params *p, const void *q, const void *k_cache,
                const void *v_cache, const int32_t *block_table,
                const int32_t *seq_lens, void *out, float *lse,
                int32_t num_splits, void *workspace, size_t workspace_bytes,
                int32_t *status, void *stream);

/*
 * The split pass alone: the same arguments and the same first launch as
 * decode_attn().  Rows of requests that fit one chunk get their final out/lse;
 * rows of longer requests get partials in `workspace` (layout above), which
 * decode_attn_combine() with the same num_splits and the chunk length from
 * decode_attn_chunk_len() then merges.  decode_attn() == decode_attn_split()
 * followed by decode_attn_combine().
 */
int decode_attn_split(const decode_attn_params *p, const void *q, const void *k_cache,
                      const void *v_cache, const int32_t *block_table,
                      const int32_t *seq_lens, void *out, float *lse,
                      int32_t num_splits, void *workspace, size_t workspace_bytes,
                      int32_t *status, void *stream);

/*
 * The combine step alone: merges the partials that a split pass left in
 * `workspace` (layout above) into out/lse, for every row whose request uses
 * two or more chunks of `chunk_len` tokens.  M = max_s lse_s,
 * w_s = exp(lse_s - M), out = sum_s w_s O_s / sum_s w_s, lse = M + ln sum w_s
 * (the two-block merge of "Capstone FlashAttention", §1.2, applied to all
 * chunks).  decode_attn() calls it itself; it is exported so that the merge
 * can be run and checked on its own.
 */
/*   num_splits / chunk_len: the values the split pass used (num_splits ==
 *   ceil(max_seq_len / chunk_len)).  Launches nothing when that split pass
 *   merged through clusters (same params, same num_splits).  num_splits <= 0:
 *   the split pass was device-planned; the chunk length, prefixes and
 *   item-indexed partials are read from `workspace` (chunk_len is ignored). */
int decode_attn_combine(const decode_attn_params *p, const int32_t *seq_lens,
                        int32_t num_splits, int32_t chunk_len,
                        const void *workspace, size_t workspace_bytes, void *out,
                        float *lse, void *stream);

/*
 * decode_attn() for callers that cannot allocate device memory.  The pages
 * have no counterpart of this entry point; it exists for callers such as
 * plugin hosts that pass only input and output buffers, runtimes whose device
 * memory is owned by another allocator, and deployments that forbid device
 * allocation after start-up.  Same arguments as decode_attn() minus the
 * workspace: the partials go to a DECODE_ATTN_STATIC_WORKSPACE_BYTES (16 MiB)
 * array in the library's own device memory, which every GPU that loads the
 * library holds until the process exits.
 *   - A call needing more than that returns DA_ERR_STATIC_WORKSPACE_LIMIT and
 *     launches nothing (decode_attn_workspace_bytes() gives the need).
 *   - All calls on a device share the array, and it keeps the last call's
 *     contents (nothing in it needs clearing).  Calls that overlap on the GPU
 *     race on it: serialise them.
 *   - The first call in each CUDA context looks up the array's address with
 *     that device current (once per device; again after cudaDeviceReset, or
 *     in another context a driver-API caller made current); make it before
 *     any stream capture in that context.
 *   - Only calls that write partials (decode_attn_launch_count() == 2) use
 *     the array and count against the limit; single-chunk and cluster-merged
 *     calls never do.
 * Allocates nothing (no cudaMalloc/cudaFree or allocating library call).
 */
int decode_attn_static_workspace(const decode_attn_params *p, const void *q,
                                 const void *k_cache, const void *v_cache,
                                 const int32_t *block_table, const int32_t *seq_lens,
                                 void *out, float *lse, int32_t num_splits,
                                 int32_t *status, void *stream);

/*
 * decode_attn() with the per-call inputs and outputs in host memory: the call
 * a serving loop makes when q, seq_lens and the block table arrive from the
 * host and out / lse go back to it, while the K/V cache stays resident on the
 * device.  It runs the same kernels as decode_attn() and returns once
 * `stream` has finished the call's work.  When q, seq_lens, the block table,
 * out and lse are all page-locked (cudaHostAlloc / cudaHostRegister), the
 * kernels read seq_lens and write out and lse in place through the GPU's
 * mapping of host memory (NVLink-C2C on Grace systems), and read q in place
 * too when there are at most 16 query rows per KV head; the block table (and
 * q above 16 rows) is first copied into `workspace` with one copy each,
 * because the kernels read them many times or late.  A page-locked status
 * word is zeroed and written in place too.  Otherwise the call copies
 * q, seq_lens and the block table into device staging buffers carved from
 * `workspace` and copies out and lse (and the status word) back.  Unlike every
 * other entry it synchronises the stream, so it cannot be captured in a CUDA
 * graph.
 *   q_host            bf16 [B, q_len, Hq, 128] in host memory, dense: the
 *                     params' q strides must be the packed ones
 *   k_cache, v_cache  the device caches, as for decode_attn()
 *   block_table_host  int32 [B, block_table_stride] in host memory, or NULL
 *                     (contiguous cache)
 *   seq_lens_host     int32 [B] in host memory
 *   out_host          bf16 [B, q_len, Hq, 128] in host memory, dense (the
 *                     params' out strides must be the packed ones)
 *   lse_host          fp32 [B, q_len, Hq] in host memory
 *   num_splits        chunks per request; <= 0 asks the planner, which here
 *                     sees the actual lengths (decode_attn_plan() with
 *                     seq_lens_host gives the same count, for sizing the
 *                     workspace)
 *   workspace         device buffer of >= decode_attn_host_workspace_bytes()
 *                     bytes for that split count (16-byte aligned): the
 *                     partials of decode_attn(), then the staging buffers
 *   status_host       optional int32 host word: the call's DA_STATUS_* bits
 *   stream            cudaStream_t (NULL: legacy default stream)
 * Page-locked host buffers (cudaHostAlloc / cudaHostRegister) take the
 * direct path above; pageable memory works through staging copies.
 * Argument errors return before anything is copied or launched; a failure
 * after the copies were queued waits for the stream, then returns the code.
 */
int decode_attn_host_workspace_bytes(const decode_attn_params *p, int32_t num_splits,
                                     size_t *bytes);
int decode_attn_host(const decode_attn_params *p, const void *q_host, const void *k_cache,
                     const void *v_cache, const int32_t *block_table_host,
                     const int32_t *seq_lens_host, void *out_host, float *lse_host,
                     int32_t num_splits, void *workspace, size_t workspace_bytes,
                     int32_t *status_host, void *stream);

/*
 * The device planner alone: writes the plan, prefixes and item list that a
 * device-planned decode_attn() call with these params would compute from
 * seq_lens (layout under "Device planning" above) into `workspace`, without
 * running the kernels that follow, so the plan can be read back and checked.
 * The params must be ones decode_attn() plans on the device (two or more
 * requests; tcgen05 shapes up to 1024 requests), else DA_ERR_BAD_SHAPE.
 * DA_STATUS_SEQ_LEN / DA_STATUS_SHORT_CAUSAL are OR-ed into *status as the
 * full call would.  Asynchronous; graph capturable.
 */
int decode_attn_device_plan(const decode_attn_params *p, const int32_t *seq_lens,
                            void *workspace, size_t workspace_bytes, int32_t *status,
                            void *stream);

/* Static description of a return code. */
const char *decode_attn_status_string(int code);

/* Number of kernel launches decode_attn() makes for these arguments (1 or 2;
 * 1 with the cluster merge; 3 for a device-planned call: planner, split,
 * combine). */
int decode_attn_launch_count(const decode_attn_params *p, int32_t num_splits);

/* ------------------------------------------------------------------------
 * The operators around the cache: rotary tables, the append that writes new
 * tokens into a cache, attention over caches held in 4 bits, and attention
 * over the pages that a cheap score selects.  They share the rules above
 * (ownership, errors, status bits, streams, graph capture, threads).
 * ------------------------------------------------------------------------ */

/* cache types */
#define DA_CACHE_BF16 0
#define DA_CACHE_FP8_E4M3 1   /* as DA_FLAG_KV_FP8_E4M3 */
#define DA_CACHE_FP4_E2M1 2   /* 4 bits per value, one E4M3 scale per 16 */

/*
 * A K/V cache of any type, under the paging and strides of a
 * decode_attn_params (strides in elements for bf16, in bytes for the others;
 * its k_scale / v_scale apply to FP8 and 4-bit caches).  The type here counts;
 * DA_FLAG_KV_FP8_E4M3 in the params is ignored by the calls that take a cache.
 *
 * 4-bit caches.  Byte i of a (token, head), 64 in all, holds value 2i in its
 * low nibble and 2i + 1 in its high one, each an OCP E2M1 code (sign, two
 * exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6).  Every 16
 * values share an E4M3 block scale: value d of token j is
 *     k_scale * block_scale[j, d / 16] * e2m1(code).
 * Block scales live beside the cache, 8 bytes per (token, head), the tokens
 * of a head one behind the other: token slot of head h in page (or, for a
 * contiguous cache, request) g is at
 *     g * bs_stride_page + h * bs_stride_head + slot * 8  (bytes).
 */
typedef struct decode_attn_cache {
  int32_t type;               /* DA_CACHE_* */
  int32_t reserved;           /* 0 */
  void *k;                    /* caches, 16-byte aligned */
  void *v;
  void *k_block_scale;        /* DA_CACHE_FP4_E2M1: 16-byte aligned; else ignored */
  void *v_block_scale;
  int64_t bs_stride_page;     /* bytes, positive multiples of 16 */
  int64_t bs_stride_head;
} decode_attn_cache;

/*
 * decode_attn() for a cache of any type: bf16 and FP8 caches run as
 * decode_attn() runs them, 4-bit ones run their own split kernel (the same
 * planner, partials, device planning and combine; every row count up to
 * DECODE_ATTN_MAX_ROWS; clusters where the call is short and has at most 32
 * rows per kv head, and the workspace is then 0 bytes).  Its chunks are
 * multiples of 64 tokens, so num_splits may come out lower, and an item of a
 * device plan may hold several KV heads.
 * k_scale and v_scale are finite.
 */
int decode_attn_cached_workspace_bytes(const decode_attn_params *p,
                                       const decode_attn_cache *c, int32_t num_splits,
                                       size_t *bytes);
int decode_attn_cached(const decode_attn_params *p, const decode_attn_cache *c, const void *q,
                       const int32_t *block_table, const int32_t *seq_lens, void *out,
                       float *lse, int32_t num_splits, void *workspace,
                       size_t workspace_bytes, int32_t *status, void *stream);

/*
 * The cos / sin table of rotary embeddings: for the positions pos = first ..
 * first + count - 1 and the frequencies f_i, i < num_freqs (radians per
 * position, fp64, device memory),
 *     table[(pos - first) * 2 num_freqs + i]             = amplitude cos(pos f_i)
 *     table[(pos - first) * 2 num_freqs + num_freqs + i] = amplitude sin(pos f_i)
 * in fp32, within 2^-21 of an entry's own size plus what the angle is off: it is
 * reduced in 64-bit fixed point, to pos * 2^-65 + 2^-56 turns (1e-9 radians at
 * the last position; entries near a zero crossing are small, but not exact to
 * their own last bits).  The table is 16-byte aligned.  Scalings for long contexts are
 * the caller's choice of f and amplitude.  1 <= num_freqs <= 64, first and first + count within 0 .. 2^31.
 * Frequencies that are not finite give NaN.
 */
int decode_attn_rope_table(const double *inv_freq, int32_t num_freqs, int64_t first,
                           int64_t count, double amplitude, float *table, void *stream);

/* Rotary embedding of the new tokens (decode_attn_rope_append). */
typedef struct decode_attn_rope {
  int32_t rotary_dim;         /* leading values of each head that are rotated: even,
                                 0 .. 128 (0: none; the table may be NULL) */
  int32_t interleaved;        /* pairs (2i, 2i + 1); else halves (i, i + rotary_dim / 2) */
  int32_t table_positions;    /* rows of the table */
  int32_t reserved;           /* 0 */
  int64_t k_stride_batch;     /* new k [B, q_len, Hkv, D] element strides, multiples */
  int64_t k_stride_token;     /*   of 8 */
  int64_t k_stride_head;
  int64_t v_stride_batch;     /* new v */
  int64_t v_stride_token;
  int64_t v_stride_head;
} decode_attn_rope;

/*
 * Rotate the new tokens' q and k and write k and v into the cache, where the
 * attention calls read them.  seq_lens counts the new tokens already: request
 * b has n_b = new_lens[b] new tokens (q_len when new_lens is NULL), at cache
 * positions L - n_b .. L - 1, in rows t = 0 .. n_b - 1 of q, k and v.  Rows t
 * >= n_b are padding: their q_out rows and the cache are left as they were.
 * The angle of a token is that of its cache position, or of positions[b *
 * q_len + t] where given.  A pair (x1, x2) becomes
 *     (x1 c - x2 s, x2 c + x1 s),
 * in fp32 with every product and sum rounded, then rounded to bf16; values
 * from rotary_dim on pass through.  From the bf16 values a cache stores
 *     FP8:   E4M3(x * (1 / k_scale)), saturated (NaN stays NaN);
 *     4-bit: z = x * (1 / k_scale); block scale E4M3(max |z| / 6), saturated;
 *            code E2M1(z / block scale), ties to even, saturated; NaN is
 *            stored as 0 and does not enter the maximum.
 * all in fp32, so the bytes are the same wherever a token is recomputed.
 *   p          the shapes, paging and strides of the attention calls; q_len
 *              may be any length here; q / o strides are those of q / q_out;
 *              scale and causal are not used; k_scale and v_scale and their
 *              reciprocals are finite
 *   q, q_out   bf16; both NULL: only the cache is written.  q_out may be q.
 *   k, v       bf16, the new tokens; both NULL: only q is rotated
 *   table      decode_attn_rope_table() from position 0
 *   positions  optional int32 [B, q_len]
 *   new_lens   optional int32 [B], 0 .. q_len
 * Status: DA_STATUS_SEQ_LEN where a length is outside [0, max_seq_len] or a
 * new_lens entry outside [0, q_len] (clamped), DA_STATUS_SHORT_CAUSAL where L
 * < n_b (the first n_b - L rows have no position and are skipped),
 * DA_STATUS_BAD_PAGE where a page is out of range (that token is not written)
 * and DA_STATUS_POSITION where a position has no row in the table (that token
 * is not rotated or written).  Two tokens of a call that map to one slot leave
 * either's values there.
 */
#define DA_STATUS_POSITION 16u
int decode_attn_rope_append(const decode_attn_params *p, const decode_attn_cache *c,
                            const decode_attn_rope *r, const void *q, const void *k,
                            const void *v, const float *table, const int32_t *positions,
                            const int32_t *new_lens, const int32_t *block_table,
                            const int32_t *seq_lens, void *q_out, int32_t *status,
                            void *stream);

/*
 * Digests of a paged K cache, for the selection of pages: per page and KV head
 * the channel-wise minimum and maximum of the page's keys (those below
 * seq_len), in 8 bits.  With amax the largest magnitude among them,
 *     digest[page, head, 0 / 1, d] = rint(min / max * (127 / amax)),
 *     digest_scale[page, head]     = amax / 127,
 * in fp32 (0 where amax is 0; below 3.8e-37, where 127 / amax overflows, zeros
 * stay 0 and the others become 127 of their sign).  Keys are the values the cache stores, without
 * k_scale; NaN values are skipped (a channel with nothing else counts as 0)
 * and infinities count as the largest finite bf16 value.
 *   digest        int8 [num_pages, Hkv, 2, 128]
 *   digest_scale  fp32 [num_pages, Hkv]
 *   max_new       > 0: only the pages that hold tokens L - max_new .. L - 1
 *                 of a request (a decode step); 0: every page it has
 * Other pages' digests are left as they were.  A page that requests of a call
 * share is digested once for each of them, at the same time: they have to see
 * the same tokens of it (whole pages of a common prefix do), else its entry may
 * be made of both.
 */
int decode_attn_block_digest(const decode_attn_params *p, const decode_attn_cache *c,
                             const int32_t *block_table, const int32_t *seq_lens,
                             int32_t max_new, int8_t *digest, float *digest_scale,
                             int32_t *status, void *stream);

/* Which pages a query reads (decode_attn_block_select, decode_attn_sparse). */
typedef struct decode_attn_select {
  int32_t top_k;              /* pages per (token, kv head), 1 .. 4096 */
  int32_t sink;               /* the first pages, always among them: >= 0 */
  int32_t local;              /* the last pages, always among them: >= 1 */
  int32_t reserved;           /* 0; sink + local <= top_k */
} decode_attn_select;

/*
 * Select pages: for every request b, new token t and KV head h, out of the n =
 * ceil(Lt / page_size) pages that the token sees (Lt = L, or L - q_len + t + 1
 * with `causal`), the first `sink`, the last `local` and, of the others, those
 * with the highest scores, top_k in all (all pages when n <= top_k; ties go to
 * the lower page).  The score of a page is the largest over the query heads of
 * the group of
 *     ((sum_d min(q'_d, 0) min_d + max(q'_d, 0) max_d) * digest_scale) * (a / 127),
 * with a = max |q_d| and q'_d = rint(q_d * (127 / a)): up to its 8 bits, a
 * bound on q . k over the page's keys, each channel at its better end.  The
 * sum is exact, the two products are fp32: the selection is the same on every
 * run.  (NaN in q counts as 0,
 * infinities as the largest finite bf16 value; a = 0 gives scores of 0; where
 * 127 / a overflows, below a = 3.8e-37, zeros stay 0 and the others become 127
 * of their sign.)
 *   blocks     int32 [B, q_len, Hkv, top_k]: the selected pages' places in
 *              the request, ascending, -1 behind the last; may be NULL
 *   pages      int32 [B, q_len, Hkv, top_k]: their page ids (0 behind the
 *              last; out-of-range entries as in decode_attn())
 *   tokens     int32 [B, q_len, Hkv]: tokens they hold up to the last one seen
 *   workspace  decode_attn_block_select_workspace_bytes() bytes
 * p as for decode_attn(), paged; max_seq_len <= 2^20 pages.
 */
int decode_attn_block_select_workspace_bytes(const decode_attn_params *p,
                                             const decode_attn_select *s, size_t *bytes);
int decode_attn_block_select(const decode_attn_params *p, const decode_attn_select *s,
                             const void *q, const int8_t *digest, const float *digest_scale,
                             const int32_t *block_table, const int32_t *seq_lens,
                             int32_t *blocks, int32_t *pages, int32_t *tokens,
                             void *workspace, size_t workspace_bytes, int32_t *status,
                             void *stream);

/*
 * Decode attention over selected pages: decode_attn_block_select(), then the
 * attention of every (token, kv head) over its own pages, exactly as
 * decode_attn() computes it for a request that holds those pages only.  Any
 * cache type.  p->scale (and k_scale, where the cache has one) must be
 * positive.  q and out hold a request's tokens at one stride: q_len == 1, B ==
 * 1, or stride_batch == q_len * stride_token.
 *   blocks      as above; may be NULL
 *   workspace   decode_attn_sparse_workspace_bytes() bytes
 */
int decode_attn_sparse_workspace_bytes(const decode_attn_params *p, const decode_attn_cache *c,
                                       const decode_attn_select *s, size_t *bytes);
int decode_attn_sparse(const decode_attn_params *p, const decode_attn_cache *c,
                       const decode_attn_select *s, const void *q, const int8_t *digest,
                       const float *digest_scale, const int32_t *block_table,
                       const int32_t *seq_lens, void *out, float *lse, int32_t *blocks,
                       void *workspace, size_t workspace_bytes, int32_t *status,
                       void *stream);

/* ------------------------------------------------------------------------
 * Trees of drafted tokens, cross attention, and reading a cache back.
 *
 * A speculative step that verifies a tree of drafts instead of one chain:
 * decode_attn_tree_mask() from each draft's parent, rope_append() at the
 * positions it gives, decode_attn_tree() instead of decode_attn(), and, once
 * the accepted path is known, decode_attn_cache_keep() for each cache.
 * ------------------------------------------------------------------------ */

#define DECODE_ATTN_MAX_TREE 1024  /* new tokens of a request in a tree */
#define DECODE_ATTN_ROWS_WORKSPACE 40162048 /* bytes of workspace in which any call of more
                                      than DECODE_ATTN_MAX_ROWS rows runs */
#define DA_STATUS_TREE 32u         /* a parent that is no earlier token, or kept tokens
                                      that do not rise */

/*
 * Masks of trees.  Request b's new tokens are the last n_b = new_lens[b] (or
 * q_len) of its seq_lens[b] tokens; parents[b * q_len + t] is the new token
 * before token t on its path, -1 where that is the sequence before the tree (a
 * request may have several such roots).
 *   parents    int32 [B, q_len], each -1 or an earlier token, parents[t] < t
 *   mask       uint32 [B, q_len, ceil(q_len / 32)]: bit i % 32 of word i / 32 of
 *              row t is set for t itself and the tokens on its path
 *   positions  int32 [B, q_len], or NULL: L - n_b + the number of tokens on t's
 *              path before it (what rope_append() takes)
 * The outputs share no memory with each other or with the inputs, but positions may
 * be the array of parents itself.
 * Rows t >= n_b get zeros.  Status: DA_STATUS_TREE for a parent that is not
 * allowed (taken as -1), DA_STATUS_SEQ_LEN for a length outside [0, max_seq_len]
 * or [0, q_len] (clamped), DA_STATUS_SHORT_CAUSAL where L < n_b.
 * 1 <= q_len <= DECODE_ATTN_MAX_TREE.
 */
int decode_attn_tree_mask(int32_t batch, int32_t q_len, int32_t max_seq_len,
                          const int32_t *parents, const int32_t *new_lens,
                          const int32_t *seq_lens, uint32_t *mask, int32_t *positions,
                          int32_t *status, void *stream);

/*
 * Decode attention of a tree's tokens: as decode_attn_cached(), where new token
 * t of request b (n_b = new_lens[b], or q_len, of them, the last of its L) sees
 *     the keys j < L - n_b, and key L - n_b + i where bit i of its row is set.
 * Rows t >= n_b are padding: their q is not used, out = 0 and lse = -inf.  So
 * for a row that sees no key.  What a hidden key holds does not matter, NaN
 * included; the values of the new tokens have to be finite, though, since a
 * hidden one enters the product with weight 0.
 * Over bf16 caches a weight may stand at up to 2^8 while the sums run, so values
 * are to stay below 2^119 / L.
 *   mask                uint32 rows as decode_attn_tree_mask() writes them (any
 *                       other pattern of bits is as good), 4-byte aligned
 *   mask_stride_batch   words from a request's rows to the next one's; 0: one
 *                       mask for all
 * p->causal is not used, nor is DA_FLAG_TEST_WITHHOLD_COPY above
 * DECODE_ATTN_MAX_ROWS.  num_splits <= 0: calls whose chunks of every request,
 * taken as max_seq_len long, are short and on the GPU together are cut so; the
 * others as decode_attn() plans them.
 * (Hq / Hkv) * q_len may exceed DECODE_ATTN_MAX_ROWS; Hq / Hkv may not, nor q_len
 * DECODE_ATTN_MAX_TREE.  Above that many rows the other calls, and all with
 * num_splits > 0 (whose value is then not used), cut their work evenly on the
 * device, and the workspace holds 40 MB of partials (DECODE_ATTN_ROWS_WORKSPACE)
 * whatever the sizes.  For FP8 and 4-bit caches and more than five pairs (one pair) of
 * tiles of 128 rows per KV head, the sizes below count K and V in bf16 besides (B *
 * max_seq_len * Hkv * 512 bytes) where those are at most 2 GB.  That copy is the
 * caller's choice: in a workspace without room for it, these calls convert K and V
 * as they go (32 pairs: FP8 17 % slower, 4-bit 36 %).  For the product with V the
 * weights are rounded to bf16 with the copy, as over bf16 caches, and to f16 without.
 * A workspace of the bytes below also serves every smaller batch of the same call,
 * with num_splits <= 0.
 * Status as decode_attn(); DA_STATUS_SHORT_CAUSAL where L < n_b (the first
 * n_b - L new tokens then have no key).
 */
int decode_attn_tree_workspace_bytes(const decode_attn_params *p, const decode_attn_cache *c,
                                     int32_t num_splits, size_t *bytes);
int decode_attn_tree(const decode_attn_params *p, const decode_attn_cache *c, const void *q,
                     const uint32_t *mask, int64_t mask_stride_batch, const int32_t *new_lens,
                     const int32_t *block_table, const int32_t *seq_lens, void *out,
                     float *lse, int32_t num_splits, void *workspace, size_t workspace_bytes,
                     int32_t *status, void *stream);

/*
 * Cross attention: as decode_attn_cached(), every row over all seq_lens[b] keys
 * (an encoder's states, of a length of their own), for any q_len: one new token
 * or a whole prompt.  Request b has q_lens[b] tokens (q_len when NULL); rows
 * behind them are padding: their q is not used, out = 0 and lse = -inf.
 * p->causal is not used.  Rows, workspace and status as decode_attn_tree(), but
 * q_len has no limit of its own (above DECODE_ATTN_MAX_ROWS rows B * Hkv *
 * ceil(q_len / (2 * floor(128 * Hkv / Hq))) * (8 * ceil(max_seq_len / 128) + 24)
 * stays below 2^32, else DA_ERR_BAD_SHAPE).
 */
int decode_attn_cross_workspace_bytes(const decode_attn_params *p, const decode_attn_cache *c,
                                      int32_t num_splits, size_t *bytes);
int decode_attn_cross(const decode_attn_params *p, const decode_attn_cache *c, const void *q,
                      const int32_t *q_lens, const int32_t *block_table,
                      const int32_t *seq_lens, void *out, float *lse, int32_t num_splits,
                      void *workspace, size_t workspace_bytes, int32_t *status, void *stream);

/*
 * Keep some of the new tokens: of request b's n_b = new_lens[b] (or p->q_len)
 * new tokens, the last of its seq_lens[b], the counts[b] tokens keep[b][0],
 * keep[b][1], .. (rising) become its first new tokens, in K, V and the block
 * scales:
 *     token L - n_b + i  <-  token L - n_b + keep[b][i],   i < counts[b],
 * and out_lens[b] = L - n_b + counts[b].  The bytes are moved as they are (a
 * key keeps the rotation it was appended with).
 *   keep      int32 [B, max_keep], 0 <= max_keep <= p->q_len
 *   out_lens  int32 [B], or NULL; shares no memory with the inputs
 * V may be K itself (c->v == c->k, with the same block scales); otherwise they
 * share no memory.
 * p->q_len <= DECODE_ATTN_MAX_TREE; of *p the shapes, paging and cache strides
 * are used.  Pages that hold new tokens belong to one request of the call.
 * Status: DA_STATUS_TREE where an entry does not rise or is no new token (it and
 * those behind it are dropped) or a count is outside [0, min(max_keep, n_b)]
 * (clamped), DA_STATUS_BAD_PAGE (that token is not moved), DA_STATUS_SEQ_LEN and
 * DA_STATUS_SHORT_CAUSAL (tokens before position 0 are not moved) as above.
 */
int decode_attn_cache_keep(const decode_attn_params *p, const decode_attn_cache *c,
                           const int32_t *keep, int32_t max_keep, const int32_t *counts,
                           const int32_t *new_lens, const int32_t *block_table,
                           const int32_t *seq_lens, int32_t *out_lens, int32_t *status,
                           void *stream);

/* Where decode_attn_cache_read() writes. */
typedef struct decode_attn_read {
  int32_t max_tokens;         /* tokens of a request at most, >= 0 */
  int32_t reserved;           /* 0 */
  int64_t rows;               /* with offsets: rows of the outputs; else not used */
  int64_t stride_batch;       /* element strides of both outputs, multiples of 8; */
  int64_t stride_token;       /*   stride_batch is not used with offsets */
  int64_t stride_head;
} decode_attn_read;

/*
 * Read a cache back: tokens starts[b] (0 when NULL) .. seq_lens[b] - 1 of every
 * request, at most max_tokens of them, as bf16,
 *     k_scale * K  and  v_scale * V   (4-bit: scale * (block_scale * e2m1)),
 * the product with the cache's scale rounded once to fp32 and once to bf16;
 * bf16 caches are copied.  NaN stays NaN.
 *   k_out, v_out  bf16, 16-byte aligned: [B, max_tokens, Hkv, 128], token
 *                 starts[b] + i in row i of request b; or, with offsets, [rows,
 *                 Hkv, 128], in row offsets[b] + i.  v_out may be NULL (with
 *                 c->v then unused).
 * Rows that no token goes to are left as they were.  Status: DA_STATUS_SEQ_LEN
 * where a length or a start is out of range (clamped) or a row of offsets is
 * (not written), DA_STATUS_BAD_PAGE as in decode_attn().  A call whose outputs
 * have no row (max_seq_len, max_tokens or, with offsets, rows 0) launches nothing
 * and looks at no length: its status stays as it was.
 */
int decode_attn_cache_read(const decode_attn_params *p, const decode_attn_cache *c,
                           const decode_attn_read *r, const int32_t *starts,
                           const int32_t *offsets, const int32_t *block_table,
                           const int32_t *seq_lens, void *k_out, void *v_out,
                           int32_t *status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_ATTN_H_ */
