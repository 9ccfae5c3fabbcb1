// Internal declarations shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa.h"

namespace dsa {

// Kernel launchers (each returns the launch's cudaError_t).
cudaError_t launch_topk(const float* scores, int64_t ld, const int32_t* q_pos, int32_t num_q, int32_t k,
                        int32_t* idx, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                        cudaStream_t stream);
// Workspace bytes the sliced top-k of rows longer than 65,536 positions uses
// (0 when it does not apply).
size_t topk_workspace_bytes(int32_t num_q, int64_t ld, int32_t k);
// CTAs per top-k row (a thread-block cluster) for this launch.
int topk_cluster_size(int32_t num_q, int64_t ld, int num_sms);

// The page lookup of the attention call folded into the top-k's write: for
// every selected position its cache slot and dequantisation scale, as the
// attention kernel reads them (slot -1 and scale 0 for padding and for bad
// entries, which are reported as the attention call reports them).
struct TopkResolve {
  int2* res;  // [num_q, k]: (slot, scale bits)
  const int32_t* block_table;
  const int32_t* q_req;
  const float* kv_scale;
  int64_t num_pages;
  int32_t num_req, bt_stride, page_size;
};
// Top-k of rows of at most 65,536 positions (ld <= 65,536) that also writes
// rv.res; idx is written as launch_topk writes it.
cudaError_t launch_topk_resolve(const float* scores, int64_t ld, const int32_t* q_pos, int32_t num_q, int32_t k,
                                int32_t* idx, const TopkResolve& rv, int32_t* dev_status, cudaStream_t stream);

// SM count of the current device (cached per device).
int device_sm_count();

struct MlaArgs {
  const void* q;
  const uint8_t* kv;
  const float* kv_scale;
  int64_t num_pages;
  const int32_t* block_table;
  int32_t num_req;
  int32_t bt_stride;
  const int32_t* q_req;
  const int32_t* idx;
  int32_t num_q, heads, d_latent, d_rope, page_size, k;
  float softmax_scale;
  int32_t num_splits;
  void* out;
  float* lse;
  float* o_part;
  float* lse_part;
  int32_t* dev_status;
};

cudaError_t launch_mla_simt(const MlaArgs& a, cudaStream_t stream);

// Tensor-core (tcgen05) version for (heads, d_latent, d_rope) = (64, 512, 64).
// It first resolves every selected position into (slot, scale) in
// `workspace` (mla_tc_workspace_bytes), then runs the attention kernel.
bool mla_tc_supported(const MlaArgs& a);
size_t mla_tc_workspace_bytes(int32_t num_q, int32_t k);
cudaError_t launch_mla_tc(const MlaArgs& a, void* workspace, cudaStream_t stream);
// The attention kernel alone, over entries launch_topk_resolve has just
// written into `workspace` on the same stream (a programmatic dependent of
// that top-k launch).
cudaError_t launch_mla_tc_resolved(const MlaArgs& a, void* workspace, cudaStream_t stream);
// Fused decode path: top-k of each token's scores row, then attention over
// it, one CTA per token (one KV split; rows of at most 65,536 positions; k at
// most mla_tc_fused_max_k()); `workspace` as for launch_mla_tc.
int mla_tc_fused_max_k();
cudaError_t launch_mla_tc_fused(const MlaArgs& a, const float* scores, int64_t ld, const int32_t* q_pos, int32_t* idx,
                                void* workspace, cudaStream_t stream);

// KV cache write: FP8 E4M3 per-token quantisation + paged scatter (rows of up
// to kv_write_max_d() values, a multiple of 16).
int kv_write_max_d();
cudaError_t launch_kv_write(const void* rows, int32_t n, int32_t d, const int32_t* req, const int32_t* pos,
                            const int32_t* block_table, int32_t num_req, int32_t bt_stride, int32_t page_size,
                            int64_t num_pages, uint8_t* kv, float* kv_scale, int32_t* status, cudaStream_t stream);

cudaError_t launch_combine(const float* o_part, const float* lse_part, int32_t num_splits, int32_t num_q,
                           int32_t heads, int32_t d_v, void* out, float* lse, cudaStream_t stream);

// Block tables and slot maps from request lengths (dsa_batch_layout).
struct BatchLayoutArgs {
  const int32_t *ctx_len, *new_len, *pages_held;
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* free_used;
  int32_t num_req, bt_stride, page_size, num_free, capacity;
  int64_t num_pages;
  int32_t *cu_q, *q_req, *q_pos, *slot, *ctx_out, *held_out, *free_used_out;
  bool vec;  // the token arrays are 16-byte aligned
  int32_t* dev_status;
};
int batch_layout_max_requests();
cudaError_t launch_batch_layout(const BatchLayoutArgs& a, cudaStream_t stream);

// Norm and position rotation of query and key rows (dsa_qk_norm_rope).
struct NormRopeSide {
  const void* x;                    // [tokens, heads, d] through the strides, or null
  int64_t tok_stride, head_stride;  // elements
  int32_t heads, norm_dim;
  const float* weight;  // [norm_dim]
  void* out;            // [tokens, heads, d] contiguous, or null
};
struct NormRopeArgs {
  NormRopeSide q, k;
  int32_t num_tokens, d, d_rope, dtype;
  const int32_t* pos;
  const float* cos_sin;
  int32_t max_pos;
  float eps;
  bool interleaved;
  const int32_t* slot;  // FP8 cache write of the key rows (one key head), or null
  uint8_t* kv;
  float* kv_scale;
  int64_t num_slots;
  int32_t* dev_status;
};
int norm_rope_max_d();
cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, cudaStream_t stream);

// Dense attention over positions 0..q_pos[i] (dsa_chunk_mla_fwd).  MlaArgs
// without idx; k is unused.  merge: num_splits <= chunk_max_merged() CTAs of a
// cluster per token write out / lse themselves.
constexpr int chunk_max_merged() { return 8; }
cudaError_t launch_chunk_small(const MlaArgs& a, const int32_t* q_pos, bool merge, cudaStream_t stream);
// The same on the tensor cores, for (64, 512, 64).
cudaError_t launch_chunk_tc(const MlaArgs& a, const int32_t* q_pos, bool merge, cudaStream_t stream);

// Drafted tokens against the target's probabilities (dsa_verify_draft).
struct VerifyArgs {
  const float* target;  // [num_rows, ld_target]
  int64_t ld_target;
  int32_t num_rows, vocab;
  const float* draft;  // [num_rows, ld_draft] or null
  int64_t ld_draft;
  const int32_t *draft_tokens, *cu_rows;
  const int32_t* q_req;  // [num_rows] whose row it is (a request's first one counts), or null
  const float *u_accept, *u_sample;
  int32_t num_req, max_out;
  const int32_t* ctx_len;
  int32_t *tokens, *num_out, *ctx_out;
  int32_t* dev_status;
};
cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t stream);

// Latent attention's products around the cache's space (dsa_absorb_q, dsa_project_out).
struct LatentProjArgs {
  const void* x;  // bf16 [tokens, heads, d_nope + d_rope or d_latent] through the strides
  int64_t tok_stride, head_stride;  // elements
  const void* w;  // bf16 [heads, d_nope + d_v, d_latent]
  void* y;        // bf16 [tokens, heads, d_latent + d_rope or d_v]
  int32_t num_tokens, heads, d_nope, d_rope, d_v, d_latent;
  int32_t* dev_status;
};
cudaError_t launch_absorb_q(const LatentProjArgs& a, cudaStream_t stream);
cudaError_t launch_project_out(const LatentProjArgs& a, cudaStream_t stream);

// Cached latent rows to every head's keys and values (dsa_expand_kv).
struct ExpandArgs {
  const uint8_t* kv;
  const float* kv_scale;
  int64_t num_pages;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const void* w;
  int32_t num_req, bt_stride, heads, d_latent, d_rope, d_kv, page_size, capacity;
  void *kv_out, *k_rope;
  int32_t* cu_k;
  void* workspace;
  int32_t* dev_status;
};
size_t expand_kv_workspace_bytes(int32_t capacity, int32_t d_latent);
cudaError_t launch_expand_kv(const ExpandArgs& a, cudaStream_t stream);

// Attention over every head's own keys and values (dsa_prompt_mla_fwd).
struct PromptArgs {
  const void* q;  // bf16 [tokens, heads, d_nope + d_rope]
  int64_t q_tok_stride, q_head_stride;
  const void* kv;  // bf16 [rows, heads, d_nope + d_v]
  int64_t kv_tok_stride, kv_head_stride;
  const void* k_rope;  // bf16 [rows, d_rope]
  int64_t rope_stride;
  const int32_t *cu_q, *cu_k, *q_pos;
  int32_t num_rows, num_req, num_tokens, heads, d_nope, d_rope, d_v, num_splits;
  float softmax_scale;
  void* out;
  float *lse, *o_part, *lse_part;
  int32_t* dev_status;
};
cudaError_t launch_prompt_mla(const PromptArgs& a, cudaStream_t stream);

// Log probabilities, entropy, rank and alternatives of tokens (dsa_token_logprobs).
struct LogprobArgs {
  const void* logits;
  int64_t ld;
  int32_t num_rows, vocab, dtype, top;
  const int32_t* tokens;
  float *logprob, *entropy;
  int32_t *rank, *top_ids;
  float* top_logprobs;
  int32_t* dev_status;
};
constexpr int token_logprobs_max_top() { return 64; }
cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream);

// n / d for 0 <= n < 2^31: with s = ceil(log2 d) and m = ceil(2^(31 + s) / d)
// (< 2^32 or 2^31), floor(n m / 2^(31 + s)) is exact, as m d - 2^(31 + s) <= 2^s.
struct FastDiv {
  uint32_t m;
  int32_t shift;
  __device__ __forceinline__ int operator()(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> shift); }
};
inline FastDiv make_fast_div(int32_t d) {
  int s = 0;
  while ((1ll << s) < d) ++s;
  return {(uint32_t)(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}

// Report a data-dependent error without trapping.
__device__ __forceinline__ void report(int32_t* status, uint32_t bit) {
  if (status) atomicOr(reinterpret_cast<unsigned int*>(status), bit);
}

}  // namespace dsa
