/*
 * dsa.h -- C ABI of the GB300 (sm_103a) DSA sparse-MLA library.
 *
 * The library implements the data-parallel hot path of DeepSeek-style sparse
 * attention (DSA) over multi-head latent attention (MLA) with an FP8 paged KV
 * cache, as described for GLM-5.3-Flash serving:
 *
 *   scores --dsa_topk_select--> idx --dsa_sparse_mla_fwd--> (out, lse)
 *                                              \--(splits)--> partials --dsa_combine--> (out, lse)
 *
 * dsa_topk_sparse_mla_fwd runs the first two calls as two kernels (the top-k
 * also does the attention call's page lookup); dsa_sparse_mla_topk_fwd runs
 * them as one kernel.  Both give the two calls' results bit for bit.
 *
 * The rest of a serving step around them:
 *
 *   lengths --dsa_batch_layout--> block table, (req, pos, slot) of every token
 *   q, k rows --dsa_qk_norm_rope--> q, and the key rows in the FP8 cache
 *   (req, pos) --dsa_chunk_mla_fwd--> (out, lse) over every visible position
 *   probabilities --dsa_verify_draft--> tokens, the next step's lengths
 *
 * Sources (page titles):
 *  [LMSYS]  "Accelerating GLM-5.3-Flash on H200: High-Throughput Disaggregated
 *           Serving": section 1 "Architecture and workloads" (an indexer picks
 *           historical positions, DSA attends to them), section 2 "KV-only
 *           decode RadixCache" (prefix KV pages shared across requests),
 *           section 3 "Larger KV tiles for DSA Partial" and Figure 4 (the
 *           Partial step computes QK^T, online softmax and the weighted value
 *           sum over the selected positions; KV splits need a Combine step).
 *  [vLLM]   "GLM-5.3 Optimizations, Part 2: PCP, DCP, and Hybrid HiSparse on
 *           16 H200s", "Interpretation" (MLA's latent KV row is shared by all
 *           64 heads).
 *  [SGLang] GLM-5.3-Flash cookbook, "Size both memory pools" (paged KV pool)
 *           and "Keep the KV and DSA backends paired" (FP8 E4M3 KV cache on
 *           Blackwell).
 *
 * Conventions shared by every entry point:
 *  - All pointers except those documented as host pointers are DEVICE
 *    pointers.  The caller owns every buffer; the library allocates no device
 *    memory, keeps no per-call state and is reentrant.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).  Work is
 *    enqueued asynchronously; the call returns after argument checks and
 *    kernel launch.
 *  - Argument errors are reported synchronously through the return value and
 *    nothing is launched.  A failed launch returns DSA_ERR_CUDA.
 *  - Data-dependent errors (an index or page id out of range, a bad query
 *    position, an expired wait) never trap the GPU: the kernel ORs a bit
 *    (DSA_DEV_*) into `*dev_status` (an int32 in device memory, may be NULL)
 *    and the offending row contributes nothing.
 *  - Supported (heads, d_latent, d_rope): (16, 64, 16) and (64, 512, 64).
 *    A KV row is d_latent + d_rope FP8 E4M3 bytes (a multiple of 16) with one
 *    fp32 scale per token; K is the whole row, V its first d_latent bytes.
 */
#ifndef DSA_SPARSE_MLA_H_
#define DSA_SPARSE_MLA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define DSA_API __attribute__((visibility("default")))
#else
#define DSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1,       /* null pointer, negative size, bad alignment */
  DSA_ERR_UNSUPPORTED_SHAPE = 2, /* (heads, d_latent, d_rope) not compiled in, or a size past the call's limit */
  DSA_ERR_WORKSPACE_TOO_SMALL = 3,
  DSA_ERR_CUDA = 4, /* a CUDA runtime call or kernel launch failed */
  DSA_ERR_OUT_OF_PAGES = 5 /* the page pool has no free or evictable page left */
} dsa_status;

/* Bits ORed into *dev_status by the kernels. */
#define DSA_DEV_BAD_QPOS 1u  /* q_pos[i] < 0 or >= ld_scores: the row selects nothing */
#define DSA_DEV_BAD_INDEX 2u /* idx entry < -1, or its page slot is past the block table row */
#define DSA_DEV_BAD_PAGE 4u  /* block table entry < 0 or >= num_pages, or q_req out of range */
#define DSA_DEV_TIMEOUT 8u   /* a bounded wait inside a kernel expired */
#define DSA_DEV_NO_PAGES 16u /* the free list has too few pages for a request */

/* Static description of a status code (never NULL). */
DSA_API const char* dsa_status_string(int32_t status);

/* Library ABI version: major * 10000 + minor * 100 + patch (DSA_VERSION of the header
 * that the library was built with). */
#define DSA_VERSION 201
DSA_API int32_t dsa_version(void);

/*
 * dsa_topk_select -- causal top-k over fp32 indexer scores.
 * [LMSYS] section 3: the Partial step loads the KV positions the indexer
 * chose; [LMSYS] section 1: the indexer picks relevant historical positions.
 *
 * For each query row i (0 <= i < num_q) the visible positions are
 * 0..q_pos[i] (causal).  The call writes idx[i, 0:k] (int32, row-major,
 * device) = the min(k, q_pos[i] + 1) visible positions with the largest
 * scores[i, :], ranked by (score descending, position ascending) -- equal
 * scores go to the lower position and -0.0 equals +0.0 -- listed in
 * ascending position order, followed by -1 padding.  NaN scores are not
 * allowed (the result is unspecified but stays in range).
 *
 *   scores     fp32 [num_q, ld_scores], row stride ld_scores elements.
 *   q_pos      int32 [num_q]; q_pos[i] must lie in [0, ld_scores).
 *   idx        int32 [num_q, k] output.
 *   workspace  optional device scratch (caller-owned, no alignment beyond
 *              4 bytes).  Rows longer than 65,536 positions use it when
 *              dsa_topk_workspace_size() > 0: each 65,536-position slice
 *              writes its own top k there and a second pass merges them.
 *              NULL with workspace_bytes = 0 selects the slower in-place
 *              path instead; both give the same indices.
 * Errors: num_q < 0, k <= 0, ld_scores <= 0, null pointers -> INVALID_ARG;
 * 0 < workspace_bytes < dsa_topk_workspace_size() -> WORKSPACE_TOO_SMALL;
 * q_pos out of range -> dev bit DSA_DEV_BAD_QPOS and a row of -1.
 */
DSA_API dsa_status dsa_topk_select(const float* scores, int64_t ld_scores, const int32_t* q_pos, int32_t num_q,
                           int32_t k, int32_t* idx, void* workspace, size_t workspace_bytes,
                           int32_t* dev_status, void* stream);

/* Workspace bytes dsa_topk_select can use for these sizes: num_q x slices x k x 8
 * when ld_scores > 65,536 and slices x k <= 65,536 (slices = ceil(ld_scores /
 * 65,536)), else 0. */
DSA_API size_t dsa_topk_workspace_size(int32_t num_q, int64_t ld_scores, int32_t k);

/*
 * dsa_sparse_mla_fwd -- the DSA "Partial" step: sparse MLA attention of every
 * head of each query token over its selected latent-KV rows.
 * [LMSYS] section 3 "Larger KV tiles for DSA Partial": loads the selected KV
 * positions and computes QK^T, online softmax and the weighted value sum;
 * [vLLM] "Interpretation": one latent KV row serves all heads; [SGLang]: FP8
 * E4M3 paged KV.
 *
 * For query token i, request r = q_req[i], head h and every selected
 * position p = idx[i, j] != -1:
 *   slot  = block_table[r * bt_stride + p / page_size] * page_size + p % page_size
 *   x_d   = e4m3(kv[slot, d]) * kv_scale[slot]                 (d < dqk)
 *   z_p   = softmax_scale * sum_d q[i, h, d] * x_d
 *   out[i, h, :] = sum_p softmax(z)_p * x[:d_latent],   lse[i, h] = ln sum_p exp(z_p)
 * A token with no selected rows gets out = 0 and lse = -inf.
 *
 *   q            bf16 [num_q, heads, dqk] (dqk = d_latent + d_rope), 16-byte aligned.
 *   kv           e4m3 bytes [num_pages * page_size, dqk], 16-byte aligned.
 *   kv_scale     fp32 [num_pages * page_size].
 *   block_table  int32 [num_req, bt_stride] page ids; rows may share pages.
 *   q_req        int32 [num_q] request of each query token, in [0, num_req).
 *   idx          int32 [num_q, k] selected positions (-1 = none), any order.
 *   num_splits   1..64.  With 1 the call writes out (bf16 [num_q, heads,
 *                d_latent], 16-byte aligned) and lse (fp32 [num_q, heads]).  With S > 1 the k
 *                entries of each row are cut into S contiguous chunks of whole
 *                KV tiles and the call writes o_part (fp32 [S, num_q, heads,
 *                d_latent]) and lse_part (fp32 [S, num_q, heads]) instead, to
 *                be merged by dsa_combine; out and lse may then be NULL.
 *   workspace    device scratch of at least dsa_sparse_mla_workspace_size()
 *                bytes, 8-byte aligned (NULL allowed when that size is 0).
 *                Its contents are overwritten; no state survives the call.
 * Errors: see the conventions above; a workspace that is too small returns
 * DSA_ERR_WORKSPACE_TOO_SMALL; a pool of 2^31 or more token slots returns
 * DSA_ERR_UNSUPPORTED_SHAPE; page ids or indices out of range set
 * DSA_DEV_BAD_INDEX / DSA_DEV_BAD_PAGE and that row is skipped.
 * Precision, 64 heads: a weight (softmax times kv_scale) carries bits down to 2^-14 of
 * the largest kv_scale among the token's selected rows, whatever that row
 * weighs: rows whose scales are 2^6 below it lose about 2%, 2^10 14%
 * (dsa_chunk_mla_fwd goes by what rows weigh).  The 16-head kernel is fp32.
 */
DSA_API dsa_status dsa_sparse_mla_fwd(const void* q, const uint8_t* kv, const float* kv_scale, int64_t num_pages,
                                      const int32_t* block_table, int32_t num_req, int32_t bt_stride,
                                      const int32_t* q_req, const int32_t* idx, int32_t num_q, int32_t num_heads,
                                      int32_t d_latent, int32_t d_rope, int32_t page_size, int32_t k,
                                      float softmax_scale, int32_t num_splits, void* out, float* lse, float* o_part,
                                      float* lse_part, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                      void* stream);

/* Scratch bytes dsa_sparse_mla_fwd needs (8 bytes per selected entry on the
 * tensor-core path: the resolved slot and scale of each position; 0 for
 * shapes served by the CUDA-core kernel). */
DSA_API size_t dsa_sparse_mla_workspace_size(int32_t num_q, int32_t num_heads, int32_t d_latent, int32_t d_rope,
                                             int32_t k);

/*
 * dsa_sparse_mla_fwd_noalloc -- dsa_sparse_mla_fwd for callers that cannot
 * allocate device memory.  The pages describe no such call; it exists for
 * callers such as serving loops that reserve all device memory at start-up
 * and forbid later allocations (cudaMalloc can synchronise the device), or
 * plug-in hosts that offer no allocator.
 *
 * Same arguments, layouts, results and errors as dsa_sparse_mla_fwd, minus
 * the workspace: the scratch lives in a fixed 24 MiB array of device memory
 * inside the library (one per GPU, held until the process exits).  Only the
 * tensor-core shape (64, 512, 64) is accepted.  Calls needing more than 24
 * MiB of scratch (dsa_sparse_mla_workspace_size) return
 * DSA_ERR_WORKSPACE_TOO_SMALL without launching anything.  All calls share
 * the array: calls whose GPU work overlaps (unordered streams, concurrent
 * host threads) race and must be serialised by the caller.  The first call on
 * a device, made with that device current, looks up the array's device
 * address; make it before any stream capture on that device.  That address
 * is kept for the life of the process: do not call this entry point again
 * after a device reset (cudaDeviceReset, or a reset of the primary context),
 * which moves the array.  The call allocates nothing.
 */
DSA_API dsa_status dsa_sparse_mla_fwd_noalloc(const void* q, const uint8_t* kv, const float* kv_scale,
                                              int64_t num_pages, const int32_t* block_table, int32_t num_req,
                                              int32_t bt_stride, const int32_t* q_req, const int32_t* idx,
                                              int32_t num_q, int32_t num_heads, int32_t d_latent, int32_t d_rope,
                                              int32_t page_size, int32_t k, float softmax_scale, int32_t num_splits,
                                              void* out, float* lse, float* o_part, float* lse_part,
                                              int32_t* dev_status, void* stream);

/*
 * dsa_sparse_mla_topk_fwd -- dsa_topk_select followed by dsa_sparse_mla_fwd
 * with one KV split, in a single kernel: each CTA selects its own query
 * token's top k and then attends to it.  Same results, bit for bit, as the
 * two calls; [LMSYS] section 3 (the indexer's selection feeds the Partial
 * step): the selection of one token's row does not wait for every other
 * row's, and no kernel boundary separates the two steps.  Measured on GB300
 * the two calls are nevertheless faster on every decode, verify and prefill
 * shape tried: this kernel's selection and tile loop run a little slower,
 * and it cannot split the KV range, which small batches need; this call is
 * for callers that want one launch.
 *
 * Arguments are those of the two calls: scores, ld_scores, q_pos and k as
 * for dsa_topk_select (ld_scores at most 65,536), idx is written as that call
 * writes it, the rest as for dsa_sparse_mla_fwd with num_splits = 1 (out is
 * required, lse may be NULL).  Only the tensor-core shape (64, 512, 64) and
 * k <= dsa_sparse_mla_topk_max_k() are accepted; anything else returns
 * DSA_ERR_UNSUPPORTED_SHAPE.  The workspace is dsa_sparse_mla_workspace_size()
 * bytes.  A bad q_pos sets DSA_DEV_BAD_QPOS, gives a row of -1 and that
 * token out = 0, lse = -inf.
 */
DSA_API dsa_status dsa_sparse_mla_topk_fwd(const float* scores, int64_t ld_scores, const int32_t* q_pos, int32_t k,
                                           int32_t* idx, const void* q, const uint8_t* kv, const float* kv_scale,
                                           int64_t num_pages, const int32_t* block_table, int32_t num_req,
                                           int32_t bt_stride, const int32_t* q_req, int32_t num_q, int32_t num_heads,
                                           int32_t d_latent, int32_t d_rope, int32_t page_size, float softmax_scale,
                                           void* out, float* lse, void* workspace, size_t workspace_bytes,
                                           int32_t* dev_status, void* stream);

/* Largest k dsa_sparse_mla_topk_fwd accepts. */
DSA_API int32_t dsa_sparse_mla_topk_max_k(void);

/*
 * dsa_topk_sparse_mla_fwd -- dsa_topk_select followed by dsa_sparse_mla_fwd,
 * with the attention call's first step (each selected position's page and
 * dequantisation scale, looked up in the block table) done by the top-k
 * kernel as it writes its indices: two kernels instead of three, the
 * attention kernel a programmatic dependent of the top-k.  [LMSYS] section 3:
 * the indexer's selection feeds the Partial step.  Same results, bit for bit,
 * as the two calls, including dev_status: a bad q_pos sets DSA_DEV_BAD_QPOS;
 * a position past the block table row DSA_DEV_BAD_INDEX; a page id or q_req
 * out of range DSA_DEV_BAD_PAGE; such entries are attended as padding.
 *
 * Arguments are those of the two calls: scores, ld_scores, q_pos, k and idx
 * as for dsa_topk_select (ld_scores at most 65,536), the rest as for
 * dsa_sparse_mla_fwd (num_splits = 1 writes out / lse; num_splits > 1 writes
 * o_part / lse_part for dsa_combine).  The workspace is
 * dsa_sparse_mla_workspace_size() bytes (it receives the looked-up entries).
 * Only the tensor-core shape (64, 512, 64) with ld_scores <= 65,536 is
 * accepted; anything else returns DSA_ERR_UNSUPPORTED_SHAPE (the two calls
 * take every shape).
 */
DSA_API dsa_status dsa_topk_sparse_mla_fwd(const float* scores, int64_t ld_scores, const int32_t* q_pos, int32_t k,
                                           int32_t* idx, const void* q, const uint8_t* kv, const float* kv_scale,
                                           int64_t num_pages, const int32_t* block_table, int32_t num_req,
                                           int32_t bt_stride, const int32_t* q_req, int32_t num_q, int32_t num_heads,
                                           int32_t d_latent, int32_t d_rope, int32_t page_size, float softmax_scale,
                                           int32_t num_splits, void* out, float* lse, float* o_part,
                                           float* lse_part, void* workspace, size_t workspace_bytes,
                                           int32_t* dev_status, void* stream);

/*
 * dsa_combine -- the DSA "Combine" step: exact log-sum-exp merge of split-KV
 * partial results.  [LMSYS] section 3: KV splits add intermediate writes and
 * Combine work.
 *   lse[i, h] = ln sum_s exp(lse_part[s, i, h])
 *   out[i, h, :] = sum_s exp(lse_part[s, i, h] - lse[i, h]) * o_part[s, i, h, :]
 * Splits with lse_part = -inf are empty and ignored; if all are, out = 0 and
 * lse = -inf.  o_part fp32 [S, num_q, heads, d_v]; lse_part fp32 [S, num_q,
 * heads]; out bf16 [num_q, heads, d_v]; lse fp32 [num_q, heads] (may be NULL).
 * d_v must be a multiple of 4 and o_part 16-byte aligned.
 */
DSA_API dsa_status dsa_combine(const float* o_part, const float* lse_part, int32_t num_splits, int32_t num_q,
                       int32_t num_heads, int32_t d_v, void* out, float* lse, void* stream);

/*
 * dsa_kv_write -- store new latent+rope KV rows into the paged FP8 cache: the
 * write side of the rows that dsa_sparse_mla_fwd gathers.
 *
 * "Accelerating GLM-5.3-Flash on H200", section 2 "KV-only decode
 * RadixCache": rows live in a paged pool, mapped per request by a block
 * table (shared prefix pages appear in several tables).  SGLang cookbook page
 * for GLM-5.3-Flash, "Keep the KV and DSA backends paired": the cache is FP8
 * E4M3.  Row i is quantised with one fp32 scale per token: amax = max |x|,
 * scale = amax / 448, byte_j = E4M3(x_j / scale) rounded to nearest even and
 * saturated (both divisions IEEE fp32); an all-zero row stores scale 0 and
 * zero bytes.  It is stored at slot = block_table[req[i]][pos[i] / page_size]
 * * page_size + pos[i] % page_size.
 *
 *   rows         bf16 [n, d_qk] new rows (latent then rope), 16-byte aligned.
 *   req, pos     int32 [n] request (0..num_req-1) and position of each row.
 *   block_table  int32 [num_req, bt_stride] page ids (0..num_pages-1).
 *   kv           uint8 [num_pages * page_size, d_qk] the cache, 16-byte
 *                aligned; only the rows' slots are written.
 *   kv_scale     fp32 [num_pages * page_size]; only the rows' slots are written.
 *   d_qk         a multiple of 16, at most 2048.
 * Errors: DSA_ERR_INVALID_ARG for bad sizes, null or misaligned pointers
 * (nothing is launched); a request or page id out of range sets
 * DSA_DEV_BAD_PAGE, a position outside the block table row sets
 * DSA_DEV_BAD_INDEX, and that row is skipped.  Rows aimed at the same slot
 * leave an unspecified mixture of them there (scale and codes need not be of one
 * row); other slots are as written.  Asynchronous on `stream`.
 */
DSA_API dsa_status dsa_kv_write(const void* rows, int32_t n, int32_t d_qk, const int32_t* req, const int32_t* pos,
                                const int32_t* block_table, int32_t num_req, int32_t bt_stride, int32_t page_size,
                                int64_t num_pages, uint8_t* kv, float* kv_scale, int32_t* dev_status, void* stream);

/*
 * dsa_batch_layout -- block tables and slot maps of a step from its requests'
 * lengths: what dsa_kv_write, dsa_topk_select and the attention calls take as
 * req, pos and block_table, made on the GPU (no length has to reach the host;
 * a captured graph stays valid while the lengths change).  [LMSYS] section 2:
 * KV rows live in a paged pool mapped per request by a block table.
 *
 * Request r (0 <= r < num_req) has ctx_len[r] cached positions, pages_held[r]
 * pages in its block table row, and brings new_len[r] tokens.  With
 * total = ceil((ctx_len + new_len) / page_size), it needs need =
 * max(0, total - pages_held) more pages (none when new_len = 0), taken from
 * the free list in request order: block_table[r, pages_held[r] + x] =
 * free_pages[*free_used + (needs of the requests before) + x].  The call
 * writes
 *   cu_q           int32 [num_req + 1]: request r's tokens are t = cu_q[r] ..
 *                  cu_q[r + 1] - 1, cu_q the running sum of new_len.
 *   q_req, q_pos, slot  int32 [capacity]: for each token its request, its
 *                  position ctx_len[r] + t - cu_q[r] and the cache slot
 *                  block_table[r, pos / page_size] * page_size + pos % page_size;
 *                  -1 in all three for every t >= cu_q[num_req].
 *   ctx_out, held_out  int32 [num_req]: ctx_len + new_len and the pages then held.
 *   free_used_out  int32 [1]: *free_used plus the pages taken.
 * The outputs and block_table must not overlap the inputs (lengths and
 * free_used: two sets used in turn) or each other: INVALID_ARG otherwise.
 * Only new entries of block_table are written.
 *
 *   ctx_len, new_len, pages_held  int32 [num_req].
 *   block_table    int32 [num_req, bt_stride] page ids, updated in place.
 *   free_pages     int32 [num_free] page ids; free_used int32 [1]: how many of
 *                  them earlier calls have taken.  The pages have to be the list's
 *                  own: none that dsa_prefix_cache_* hands out (a cache of fewer
 *                  pages than the pool, the ids from there on in the list).  A
 *                  finished request's n pages come back by writing them over the last
 *                  taken entries, free_pages[*free_used - n ..], and lowering
 *                  *free_used by n, on the same stream between two calls.
 *   num_req        at most 8,192, capacity at most 2^30 (else UNSUPPORTED_SHAPE).
 * Data errors leave a request as it is (ctx_out = ctx_len, held_out =
 * pages_held, no pages taken, -1 for its tokens, which stay in cu_q: the
 * attention gives them 0, dsa_verify_draft_req no tokens): a negative length sets
 * DSA_DEV_BAD_QPOS (and the request has no tokens in cu_q); a block table row
 * that is too short, or a free_used outside the list, DSA_DEV_BAD_INDEX; too
 * few free pages DSA_DEV_NO_PAGES (a request's needs count against the
 * requests after it even then).  Tokens past capacity set DSA_DEV_BAD_INDEX:
 * cu_q stays at the last request that fits.  A page id out of range sets
 * DSA_DEV_BAD_PAGE and slot = -1.
 */
DSA_API dsa_status dsa_batch_layout(const int32_t* ctx_len, const int32_t* new_len, const int32_t* pages_held,
                                    int32_t num_req, int32_t* block_table, int32_t bt_stride,
                                    const int32_t* free_pages, int32_t num_free, const int32_t* free_used,
                                    int32_t page_size, int64_t num_pages, int32_t capacity, int32_t* cu_q,
                                    int32_t* q_req, int32_t* q_pos, int32_t* slot, int32_t* ctx_out,
                                    int32_t* held_out, int32_t* free_used_out, int32_t* dev_status, void* stream);

/*
 * dsa_qk_norm_rope -- norms of query and key rows for each head, and the
 * position rotation, in one pass; the key row may go straight into the paged
 * FP8 cache (the rows the attention calls gather).  [vLLM] "Interpretation":
 * one latent row serves all heads; [SGLang]: FP8 E4M3 cache.
 *
 * For a row x of token t and head h, in fp32:
 *   y_j = x_j * weight_j / sqrt(mean_{j < norm_dim} x_j^2 + eps)  (j < norm_dim),
 *   y_j = x_j (j >= norm_dim); then the last d_rope values are rotated by the
 *   angle of position pos[t]: (y_a, y_b) <- (y_a c - y_b s, y_a s + y_b c) with
 *   c = cos_sin[pos, i], s = cos_sin[pos, d_rope / 2 + i], for the pairs (a, b)
 *   = (2i, 2i + 1) of the rotated part (interleaved = 1) or (i, i + d_rope / 2)
 *   (interleaved = 0).
 * A row is rounded once, to its own type; in the cache as scale = max |y| /
 * 448 and byte_j = E4M3(y_j / scale) of the fp32 values (both divisions IEEE
 * fp32; an all-zero row stores scale 0 and zero bytes).
 *
 *   q, k      [num_tokens, heads, d] rows of `dtype` (DSA_BF16, DSA_FP16),
 *             addressed by token and head strides in elements (multiples of 8;
 *             16-byte aligned base).  q_heads or k_heads may be 0 (the side is absent).
 *   q_out, k_out  contiguous [num_tokens, heads, d], 16-byte aligned.  Each may be
 *             its own input (then contiguous); else what is written (these, kv,
 *             kv_scale) must not overlap an input or each other (INVALID_ARG).
 *             k_out may be NULL when the cache is written.
 *   q_weight, k_weight  fp32 [norm_dim], 16-byte aligned; norm_dim a multiple of 8, at
 *             most d; 0: no norm (weight may be NULL).
 *   d         a multiple of 8, at most 1024.  d_rope a multiple of 16, at most
 *             d, with d - d_rope a multiple of 8; 0: no rotation (cos_sin may be NULL).
 *   num_tokens  times the heads of both sides below 2^31 (else UNSUPPORTED_SHAPE).
 *   pos       int32 [num_tokens] (NULL allowed when d_rope = 0); -1: a padding
 *             row, whose outputs are left as they were.
 *   cos_sin   fp32 [max_pos, d_rope], 16-byte aligned.
 *   slot, kv, kv_scale  the cache write (all three or none; k_heads must be 1):
 *             slot int32 [num_tokens] (-1: not cached), kv uint8 [num_slots,
 *             d] 16-byte aligned, kv_scale fp32 [num_slots].
 * Data errors: pos outside [-1, max_pos) sets DSA_DEV_BAD_QPOS and the token
 * is skipped; slot outside [-1, num_slots) sets DSA_DEV_BAD_INDEX and the row
 * is not cached.  Rows aimed at the same slot leave an unspecified mixture of
 * them there (scale and codes need not be of one row): live slots have to be
 * different, as dsa_batch_layout's are while pages are.  Rows with NaN or
 * infinities give unspecified values.
 */
#define DSA_BF16 0
#define DSA_FP16 1
DSA_API dsa_status dsa_qk_norm_rope(const void* q, int64_t q_tok_stride, int64_t q_head_stride, int32_t q_heads,
                                    const float* q_weight, int32_t q_norm_dim, void* q_out, const void* k,
                                    int64_t k_tok_stride, int64_t k_head_stride, int32_t k_heads,
                                    const float* k_weight, int32_t k_norm_dim, void* k_out, int32_t num_tokens,
                                    int32_t d, int32_t d_rope, int32_t dtype, const int32_t* pos,
                                    const float* cos_sin, int32_t max_pos, float eps, int32_t interleaved,
                                    const int32_t* slot, uint8_t* kv, float* kv_scale, int64_t num_slots,
                                    int32_t* dev_status, void* stream);

/*
 * dsa_chunk_mla_fwd -- attention of a chunk of new tokens over the paged FP8
 * cache: dsa_sparse_mla_fwd without a selection.  Every head of token i
 * attends to all positions 0..q_pos[i] of request q_req[i] (causal: the
 * chunk's own rows are in the cache).  For prompts, decode and verify blocks
 * of contexts no longer than the top-k would be, and for layers without an
 * indexer.
 *
 * Arguments, layouts, outputs and splits are those of dsa_sparse_mla_fwd, with
 * q_pos (int32 [num_q]) in place of idx and k, and no workspace.  A split takes
 * a contiguous share of the token's own KV tiles.  With 2 to 8 splits and
 * o_part and lse_part both NULL the call merges them itself (the splits of a
 * token are one thread-block cluster) and writes out and lse; else the splits
 * write o_part and lse_part for dsa_combine.  What is written must not overlap
 * an input or each other (INVALID_ARG).  A token with q_req = -1
 * (padding) or q_pos = -1 sees nothing: out = 0 and lse = -inf.  Tokens of one
 * request next to each other share its rows in L2; any order is correct.
 * A head whose query holds a NaN or an infinity, and every head of a token that
 * sees a NaN code or a NaN scale, has out = lse = NaN, for any number of splits;
 * other heads and tokens are as without it.  (A visible row with an infinite
 * scale gives NaN in out, and an unspecified lse.)
 * Precision: logits and sums are fp32.  64 heads: of bf16 queries bits below
 * 2^-17 of the head's largest value are lost; a row's weight, softmax times
 * kv_scale, has a relative error of at most 2^-8 (0.13% root mean square) down to
 * 2^-10 of the head's largest weight, and one of 2^-18 of that below.
 * Scales are from 2^-60 (smaller ones lose bits) to 2^50.  16 heads: 2^-11, down
 * to 2^-25 of the largest kv_scale that the token sees.
 * Data errors: q_pos < -1 or past the block table row sets DSA_DEV_BAD_QPOS
 * and the token sees nothing; q_req outside [-1, num_req) or a page id out of
 * range sets DSA_DEV_BAD_PAGE; such rows are skipped.
 */
DSA_API dsa_status dsa_chunk_mla_fwd(const void* q, const uint8_t* kv, const float* kv_scale, int64_t num_pages,
                                     const int32_t* block_table, int32_t num_req, int32_t bt_stride,
                                     const int32_t* q_req, const int32_t* q_pos, int32_t num_q, int32_t num_heads,
                                     int32_t d_latent, int32_t d_rope, int32_t page_size, float softmax_scale,
                                     int32_t num_splits, void* out, float* lse, float* o_part, float* lse_part,
                                     int32_t* dev_status, void* stream);

/*
 * dsa_verify_draft -- verification of drafted tokens against the target's
 * probabilities, from given random numbers.  [LMSYS] section 3: a speculative
 * verify step runs the target over a block of drafted tokens.
 *
 * Request r has the rows t = cu_rows[r] .. cu_rows[r + 1] - 1 of the target's
 * probabilities and n = rows - 1 drafted tokens; draft i is checked by row t_i =
 * cu_rows[r] + i: it is taken while u_accept[t_i] * draft_probs[t_i, x_i] <
 * target_probs[t_i, x_i] (product exact).  At the first draft a that is not taken (a = n if all are)
 * the last token is drawn: w = max(target_probs[t_a] - draft_probs[t_a], 0)
 * (target_probs[t_n] after the last draft), token = the lowest j with
 * sum_{i <= j} w_i > u_sample[r] * sum_i w_i.  Without draft_probs a draft is
 * certain: 1 at x_i and 0 elsewhere.  If no w is positive, w =
 * target_probs[t_a].  Weights and sums are whole multiples of 2^-60: exact for
 * probabilities of 2^-37 or more, and independent of the launch.
 *
 *   num_req at most 2^24; vocab, num_rows and max_out at most 2^30 (else
 *   UNSUPPORTED_SHAPE).
 *   target_probs  fp32 [num_rows, vocab], row stride ld_target; each row in
 *                 [0, 1] with a sum below 8 (NaN and negative values count as
 *                 0, values above 1 as 1; a larger sum gives an unspecified token in range).
 *   draft_probs   fp32 [num_rows, vocab], row stride ld_draft, or NULL.
 *   draft_tokens  int32 [num_rows]: x_i of request r at cu_rows[r] + i.
 *   u_accept      fp32 [num_rows], u_sample fp32 [num_req]: uniform in [0, 1).
 *                 The entries of a request's last row in draft_probs,
 *                 draft_tokens and u_accept are not read.
 *   cu_rows       int32 [num_req + 1] (dsa_batch_layout's cu_q; after a layout use
 *                 dsa_verify_draft_req, which knows the requests it refused).
 *   tokens        int32 [num_req, max_out] output: the taken drafts, then the
 *                 drawn token, then -1.  num_out int32 [num_req] = a + 1.
 *   ctx_len, ctx_out  int32 [num_req], or both NULL: ctx_out = ctx_len + num_out,
 *                 the request's cached positions once the rejected rows are
 *                 dropped (the same buffer is allowed).  Other overlaps of outputs
 *                 with inputs or each other: INVALID_ARG.
 * A request without rows has num_out = 0 and tokens -1.  Data errors, all
 * DSA_DEV_BAD_INDEX: cu_rows decreasing or past num_rows (as a request
 * without rows); a draft outside [0, vocab) (not taken); more rows than
 * max_out (drafts past max_out - 1 are ignored).
 */
DSA_API dsa_status dsa_verify_draft(const float* target_probs, int64_t ld_target, int32_t num_rows, int32_t vocab,
                                    const float* draft_probs, int64_t ld_draft, const int32_t* draft_tokens,
                                    const float* u_accept, const float* u_sample, const int32_t* cu_rows,
                                    int32_t num_req, int32_t max_out, const int32_t* ctx_len, int32_t* tokens,
                                    int32_t* num_out, int32_t* ctx_out, int32_t* dev_status, void* stream);

/*
 * dsa_verify_draft_req -- dsa_verify_draft of a step whose rows dsa_batch_layout
 * laid out.  A request that the layout refused (no pages, a block table row too
 * short) keeps its rows in cu_q with q_req = -1: they have no positions, and
 * nothing was attended to or cached for them.  With q_req such a request ends
 * like one without rows, num_out = 0, tokens -1, ctx_out = ctx_len, so that its
 * next step starts from what is cached.
 *
 *   q_req   int32 [num_rows] (the layout's, of a capacity of num_rows or more), or
 *           NULL: dsa_verify_draft.  Only entries cu_rows[r] are read; one that is
 *           neither r nor -1 sets DSA_DEV_BAD_INDEX and counts as -1.
 */
DSA_API dsa_status dsa_verify_draft_req(const float* target_probs, int64_t ld_target, int32_t num_rows, int32_t vocab,
                                        const float* draft_probs, int64_t ld_draft, const int32_t* draft_tokens,
                                        const float* u_accept, const float* u_sample, const int32_t* cu_rows,
                                        const int32_t* q_req, int32_t num_req, int32_t max_out,
                                        const int32_t* ctx_len, int32_t* tokens, int32_t* num_out, int32_t* ctx_out,
                                        int32_t* dev_status, void* stream);

/*
 * KV-only prefix-sharing page allocator (host side, no GPU involved).
 *
 * "Accelerating GLM-5.3-Flash on H200", section 2 "KV-only decode
 * RadixCache": requests sharing a prefix share its KV pages, so N requests
 * with a common prefix of Lp tokens and private suffixes of Ls tokens occupy
 * Lp + N·Ls slots instead of N·(Lp + Ls).  The unit of sharing is a whole
 * page whose tokens, and all tokens before it, match (KV rows depend on the
 * whole causal prefix); the block tables it returns are the ones
 * dsa_kv_write and dsa_sparse_mla_fwd take.
 *
 * dsa_prefix_cache_create: a cache over a pool of num_pages pages of
 *   page_size tokens (page ids 0..num_pages-1).  NULL on bad sizes or when
 *   out of host memory.  The caller owns the handle (dsa_prefix_cache_destroy).
 * dsa_prefix_cache_acquire: pages for a request of n_tokens token ids.
 *   block_table (int32 [max_pages], host memory) receives ceil(n_tokens /
 *   page_size) page ids: the first *n_shared are cached pages of the longest
 *   matching whole-page prefix (their KV is already in the cache), the rest
 *   are fresh (the caller writes their KV rows).  The request's new full pages
 *   are cached for later requests; a partial last page stays private.  Every
 *   page returned is referenced until released.  When no page is free,
 *   unreferenced cached pages are evicted, least recently used first (leaves
 *   of the prefix tree only); if none is left the call changes nothing and
 *   returns DSA_ERR_OUT_OF_PAGES.  max_pages too small: DSA_ERR_INVALID_ARG.
 * dsa_prefix_cache_release: drops the references of a block table acquire
 *   returned (n_pages entries).  Private pages become free; cached pages stay
 *   cached (reusable) until evicted.  An entry that is not a referenced page
 *   returns DSA_ERR_INVALID_ARG and releases nothing.
 * dsa_prefix_cache_stats: pages referenced by live requests, pages cached in
 *   the prefix tree (referenced or not), free pages.
 * The calls are thread-safe (one lock per cache).
 */
typedef struct dsa_prefix_cache dsa_prefix_cache;
DSA_API dsa_prefix_cache* dsa_prefix_cache_create(int32_t page_size, int32_t num_pages);
DSA_API void dsa_prefix_cache_destroy(dsa_prefix_cache* cache);
DSA_API dsa_status dsa_prefix_cache_acquire(dsa_prefix_cache* cache, const int32_t* tokens, int64_t n_tokens,
                                            int32_t* block_table, int32_t max_pages, int32_t* n_pages,
                                            int32_t* n_shared);
DSA_API dsa_status dsa_prefix_cache_release(dsa_prefix_cache* cache, const int32_t* block_table, int32_t n_pages);
DSA_API dsa_status dsa_prefix_cache_stats(dsa_prefix_cache* cache, int32_t* pages_referenced, int32_t* pages_cached,
                                          int32_t* pages_free);

/*
 * Host-side planning helpers (no GPU needed).
 *
 * dsa_kv_tile_count: KV tiles of `tile` entries that cover an index row of
 * `width` entries; the last tile is padded virtually, the index tensor is
 * unchanged ([LMSYS] Figure 4: width 2112 -> 66 tiles of 32 or 17 of 128,
 * 2176 virtual columns of which 64 are padding).
 *
 * dsa_pick_num_splits: KV splits per query token for the given launch.  KV
 * splits are added only while query tokens alone leave SMs idle ([LMSYS]
 * section 3: splits cost intermediate writes and Combine work, so they are
 * used only when query parallelism is insufficient).  num_sms <= 0 queries
 * the current device.
 */
DSA_API int32_t dsa_kv_tile_count(int32_t width, int32_t tile);
DSA_API int32_t dsa_kv_tile_size(int32_t num_heads, int32_t d_latent, int32_t d_rope);
DSA_API int32_t dsa_pick_num_splits(int32_t num_q, int32_t num_heads, int32_t d_latent, int32_t d_rope, int32_t k,
                            int32_t num_sms);

/*
 * dsa_chunk_pick_num_splits: KV splits per token for dsa_chunk_mla_fwd over
 * contexts of about max_ctx positions: the number with the least estimated
 * time, from the tiles of a split, a CTA's fixed cost, the waves of CTAs (of clusters,
 * for the 2 to 8 splits that the call merges) and the merge or Combine.  On the
 * tensor cores a full batch and one whose second half is padding count the same;
 * a caller that knows about how many of the num_q tokens are live (num_q in a full
 * batch) asks dsa_chunk_pick_num_splits_live.
 */
DSA_API int32_t dsa_chunk_pick_num_splits(int32_t num_q, int32_t num_heads, int32_t d_latent, int32_t d_rope,
                                          int32_t max_ctx, int32_t num_sms);
DSA_API int32_t dsa_chunk_pick_num_splits_live(int32_t num_q, int32_t num_live, int32_t num_heads, int32_t d_latent,
                                               int32_t d_rope, int32_t max_ctx, int32_t num_sms);

#ifdef __cplusplus
}
#endif

#endif /* DSA_SPARSE_MLA_H_ */
