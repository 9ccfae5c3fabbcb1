// C ABI of the library: argument checks, planning helpers and launches.
#include <cuda_runtime.h>
#include <math.h>

#include "dsa.h"
#include "internal.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool supported_shape(int32_t h, int32_t dl, int32_t dr) {
  return (h == 16 && dl == 64 && dr == 16) || (h == 64 && dl == 512 && dr == 64);
}

// (an error that the status tells is taken off the runtime's record, where the
// process's next, unrelated check would find it)
dsa_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return DSA_OK;
  (void)cudaGetLastError();
  return DSA_ERR_CUDA;
}

// The 64-head shape runs on the tensor cores, the 16-head shape on the CUDA
// cores; nothing else changes that choice.
bool use_tensor_cores(int32_t h, int32_t dl, int32_t dr) { return h == 64 && dl == 512 && dr == 64; }

}  // namespace

namespace dsa {
int device_sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  if (dev < 64) cached[dev] = n;
  return n;
}
}  // namespace dsa

extern "C" {

const char* dsa_status_string(int32_t status) {
  switch (status) {
    case DSA_OK: return "ok";
    case DSA_ERR_INVALID_ARG: return "invalid argument";
    case DSA_ERR_UNSUPPORTED_SHAPE: return "unsupported (heads, d_latent, d_rope) or size";
    case DSA_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case DSA_ERR_CUDA: return "CUDA error";
    case DSA_ERR_OUT_OF_PAGES: return "page pool exhausted";
    default: return "unknown status";
  }
}

int32_t dsa_version(void) { return DSA_VERSION; }

int32_t dsa_kv_tile_count(int32_t width, int32_t tile) {
  if (width < 0 || tile <= 0) return -1;
  return (int32_t)(((int64_t)width + tile - 1) / tile);
}

int32_t dsa_kv_tile_size(int32_t num_heads, int32_t d_latent, int32_t d_rope) {
  if (!supported_shape(num_heads, d_latent, d_rope)) return -1;
  return num_heads == 64 ? 64 : 32;  // tensor-core kernel: 64-row tiles; CUDA-core kernel: 32
}

int32_t dsa_pick_num_splits(int32_t num_q, int32_t num_heads, int32_t d_latent, int32_t d_rope, int32_t k,
                            int32_t num_sms) {
  const int32_t tile = dsa_kv_tile_size(num_heads, d_latent, d_rope);
  if (tile <= 0 || num_q <= 0 || k <= 0) return 1;
  if (num_sms <= 0) num_sms = dsa::device_sm_count();
  // query tokens alone fill the GPU: no split (no partials, no combine)
  if (num_q >= num_sms) return 1;
  // One CTA per SM (shared memory bound); a launch takes ceil(CTAs / SMs)
  // waves of ceil(tiles / S) tiles each, plus a fixed per-CTA cost (start-up,
  // pipeline fill, epilogue: about four 64-row tiles on the tensor-core
  // kernel, two 32-row tiles on the CUDA-core one) and one tile more for the
  // Combine when split.
  const int32_t ntiles = dsa_kv_tile_count(k, tile);
  const int64_t fixed = tile == 64 ? 4 : 2;
  int32_t best = 1;
  int64_t best_cost = -1;
  for (int32_t s = 1; s <= 64 && s <= ntiles; ++s) {
    const int64_t waves = ((int64_t)num_q * s + num_sms - 1) / num_sms;
    const int64_t per = (ntiles + s - 1) / s;
    const int64_t cost = waves * (per + fixed) + (s > 1 ? 1 : 0);
    if (best_cost < 0 || cost < best_cost) best = s, best_cost = cost;
  }
  return best;
}

}  // extern "C"

namespace {

// KV splits of dsa_chunk_mla_fwd; num_live < 0: not known.
int32_t chunk_splits(int32_t num_q, int32_t num_live, int32_t num_heads, int32_t d_latent, int32_t d_rope,
                     int32_t max_ctx, int32_t num_sms) {
  const int32_t tile = dsa_kv_tile_size(num_heads, d_latent, d_rope);
  if (tile <= 0 || num_q <= 0 || max_ctx <= 0) return 1;
  if (num_sms <= 0) num_sms = dsa::device_sm_count();
  const int64_t ntiles = dsa_kv_tile_count(max_ctx, tile);
  const bool tc = use_tensor_cores(num_heads, d_latent, d_rope);
  // Clusters of S CTAs that run at once, one CTA per SM, of 152 SMs
  // (cudaOccupancyMaxActiveClusters).
  static const int32_t clusters[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
  // (64, 512, 64), in hundredths of a tile's time (measured: 0.87 us): a CTA's start
  // and end; the merge in a cluster; the Combine, whose partials grow with tokens and
  // splits (1 x 64: 18 us, 24 x 12: 17).  Where the live rows are not known (a batch of
  // fixed capacity, as of a captured step or a verify block whose requests drafted
  // less, is padded), the cost is that of a full batch plus that of a half full one.
  // 128 rows of 4,096 positions: one split 61 us full and with 72 live rows, two 77
  // and 42.
  auto large = [&](int32_t s) {
    const int64_t fixed = 800, merge = 500, combine = 500 + s * (15 + 4 * (int64_t)num_q);
    const int64_t cap = s <= 8 ? (int64_t)clusters[s] * num_sms / 152 : num_sms / s;  // tokens that run at once
    const int64_t join = s == 1 ? 0 : s <= 8 ? merge : 2 * combine;
    // (a cluster's merge is its CTAs' work)
    const int64_t cta = 100 * ((ntiles + s - 1) / s) + fixed + (s <= 8 ? join : 0);
    auto waves = [&](int64_t n) { return cap > 0 ? (n + cap - 1) / cap : (n * s + num_sms - 1) / num_sms; };
    return (num_live >= 0 ? 2 * waves(num_live) : waves(num_q) + waves((num_q + 1) / 2)) * cta + (s <= 8 ? 0 : join);
  };
  // (16, 64, 16), in hundredths of a us: a CTA's start and end, its steps of eight
  // tiles, alone on an SM or two of them, and the merge or Combine (one token of
  // 16,384 positions: 8 splits 14 us, 16 13, 32 15; 107 of 12,733: 1 59 us, 2 55, 5 51, 8 57).
  auto small = [&](int32_t s) {
    const int64_t steps = ((ntiles + s - 1) / s + 7) / 8, ctas = (int64_t)(num_live >= 0 ? num_live : num_q) * s;
    const int64_t join = s == 1 ? 0 : s <= 8 ? 100 : 250 + 18 * s;
    return join + (ctas <= num_sms ? 400 + 108 * steps : (ctas + 2 * num_sms - 1) / (2 * num_sms) * (400 + 200 * steps));
  };
  int32_t best = 1;
  int64_t best_cost = -1;
  for (int32_t s = 1; s <= 64 && s <= ntiles; ++s) {
    const int64_t cost = tc ? large(s) : small(s);
    if (best_cost < 0 || cost < best_cost) best = s, best_cost = cost;
  }
  return best;
}

}  // namespace

extern "C" {

int32_t dsa_chunk_pick_num_splits(int32_t num_q, int32_t num_heads, int32_t d_latent, int32_t d_rope, int32_t max_ctx,
                                  int32_t num_sms) {
  return chunk_splits(num_q, -1, num_heads, d_latent, d_rope, max_ctx, num_sms);
}

int32_t dsa_chunk_pick_num_splits_live(int32_t num_q, int32_t num_live, int32_t num_heads, int32_t d_latent,
                                       int32_t d_rope, int32_t max_ctx, int32_t num_sms) {
  const int32_t live = num_live < 1 ? 1 : num_live < num_q ? num_live : num_q;
  return chunk_splits(num_q, live, num_heads, d_latent, d_rope, max_ctx, num_sms);
}

size_t dsa_sparse_mla_workspace_size(int32_t num_q, int32_t num_heads, int32_t d_latent, int32_t d_rope,
                                     int32_t k) {
  if (num_q <= 0 || k <= 0 || !use_tensor_cores(num_heads, d_latent, d_rope)) return 0;
  return dsa::mla_tc_workspace_bytes(num_q, k);
}

size_t dsa_topk_workspace_size(int32_t num_q, int64_t ld_scores, int32_t k) {
  return dsa::topk_workspace_bytes(num_q, ld_scores, k);
}

dsa_status dsa_topk_select(const float* scores, int64_t ld_scores, const int32_t* q_pos, int32_t num_q,
                           int32_t k, int32_t* idx, void* workspace, size_t workspace_bytes,
                           int32_t* dev_status, void* stream) {
  if (num_q < 0 || k <= 0 || ld_scores <= 0) return DSA_ERR_INVALID_ARG;
  if (num_q == 0) return DSA_OK;
  if (!scores || !q_pos || !idx) return DSA_ERR_INVALID_ARG;
  // the workspace is optional: none selects the in-place path; a partial one is an error
  const size_t need = dsa_topk_workspace_size(num_q, ld_scores, k);
  if (workspace_bytes > 0 && workspace_bytes < need) return DSA_ERR_WORKSPACE_TOO_SMALL;
  if (workspace_bytes > 0 && !workspace) return DSA_ERR_INVALID_ARG;
  return from_cuda(dsa::launch_topk(scores, ld_scores, q_pos, num_q, k, idx, workspace, workspace_bytes,
                                    dev_status, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// Argument checks shared by the attention entry points; fills `a` when they pass.
dsa_status check_mla_args(const void* q, const uint8_t* kv, const float* kv_scale, int64_t num_pages,
                          const int32_t* block_table, int32_t num_req, int32_t bt_stride, const int32_t* q_req,
                          const int32_t* idx, int32_t num_q, int32_t num_heads, int32_t d_latent, int32_t d_rope,
                          int32_t page_size, int32_t k, float softmax_scale, int32_t num_splits, void* out,
                          float* lse, float* o_part, float* lse_part, size_t ws_need, void* workspace,
                          size_t workspace_bytes, int32_t* dev_status, dsa::MlaArgs* a) {
  if (num_q < 0 || k <= 0 || page_size <= 0 || num_pages <= 0 || num_req <= 0 || bt_stride <= 0)
    return DSA_ERR_INVALID_ARG;
  if (num_splits < 1 || num_splits > 64 || !isfinite(softmax_scale)) return DSA_ERR_INVALID_ARG;
  if (!supported_shape(num_heads, d_latent, d_rope)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (num_pages > (int64_t)INT32_MAX / page_size) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (num_q == 0) return DSA_OK;
  if (workspace_bytes < ws_need) return DSA_ERR_WORKSPACE_TOO_SMALL;
  if (ws_need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 7u))) return DSA_ERR_INVALID_ARG;
  if (!q || !kv || !kv_scale || !block_table || !q_req || !idx) return DSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv)) return DSA_ERR_INVALID_ARG;
  if (num_splits == 1) {
    if (!out || !aligned16(out)) return DSA_ERR_INVALID_ARG;
  } else {
    if (!o_part || !lse_part || !aligned16(o_part)) return DSA_ERR_INVALID_ARG;
  }
  a->q = q;
  a->kv = kv;
  a->kv_scale = kv_scale;
  a->num_pages = num_pages;
  a->block_table = block_table;
  a->num_req = num_req;
  a->bt_stride = bt_stride;
  a->q_req = q_req;
  a->idx = idx;
  a->num_q = num_q;
  a->heads = num_heads;
  a->d_latent = d_latent;
  a->d_rope = d_rope;
  a->page_size = page_size;
  a->k = k;
  a->softmax_scale = softmax_scale;
  a->num_splits = num_splits;
  a->out = out;
  a->lse = lse;
  a->o_part = o_part;
  a->lse_part = lse_part;
  a->dev_status = dev_status;
  return DSA_OK;
}

}  // namespace

extern "C" {

dsa_status dsa_sparse_mla_fwd(const void* q, const uint8_t* kv, const float* kv_scale, int64_t num_pages,
                              const int32_t* block_table, int32_t num_req, int32_t bt_stride,
                              const int32_t* q_req, const int32_t* idx, int32_t num_q, int32_t num_heads,
                              int32_t d_latent, int32_t d_rope, int32_t page_size, int32_t k,
                              float softmax_scale, int32_t num_splits, void* out, float* lse, float* o_part,
                              float* lse_part, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                              void* stream) {
  dsa::MlaArgs a;
  const size_t ws_need = dsa_sparse_mla_workspace_size(num_q, num_heads, d_latent, d_rope, k);
  const dsa_status st = check_mla_args(q, kv, kv_scale, num_pages, block_table, num_req, bt_stride, q_req, idx,
                                       num_q, num_heads, d_latent, d_rope, page_size, k, softmax_scale, num_splits,
                                       out, lse, o_part, lse_part, ws_need, workspace, workspace_bytes, dev_status,
                                       &a);
  if (st != DSA_OK || num_q == 0) return st;
  if (use_tensor_cores(num_heads, d_latent, d_rope))
    return from_cuda(dsa::launch_mla_tc(a, workspace, static_cast<cudaStream_t>(stream)));
  return from_cuda(dsa::launch_mla_simt(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_sparse_mla_topk_fwd(const float* scores, int64_t ld_scores, const int32_t* q_pos, int32_t k,
                                   int32_t* idx, const void* q, const uint8_t* kv, const float* kv_scale,
                                   int64_t num_pages, const int32_t* block_table, int32_t num_req, int32_t bt_stride,
                                   const int32_t* q_req, int32_t num_q, int32_t num_heads, int32_t d_latent,
                                   int32_t d_rope, int32_t page_size, float softmax_scale, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (ld_scores <= 0 || k <= 0 || num_q < 0) return DSA_ERR_INVALID_ARG;
  if (!use_tensor_cores(num_heads, d_latent, d_rope)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (ld_scores > 65536 || k > dsa::mla_tc_fused_max_k()) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (num_q == 0) return DSA_OK;
  if (!scores || !q_pos || !idx) return DSA_ERR_INVALID_ARG;
  dsa::MlaArgs a;
  const size_t ws_need = dsa_sparse_mla_workspace_size(num_q, num_heads, d_latent, d_rope, k);
  const dsa_status st = check_mla_args(q, kv, kv_scale, num_pages, block_table, num_req, bt_stride, q_req, idx,
                                       num_q, num_heads, d_latent, d_rope, page_size, k, softmax_scale, 1, out, lse,
                                       nullptr, nullptr, ws_need, workspace, workspace_bytes, dev_status, &a);
  if (st != DSA_OK) return st;
  return from_cuda(dsa::launch_mla_tc_fused(a, scores, ld_scores, q_pos, idx, workspace,
                                            static_cast<cudaStream_t>(stream)));
}

int32_t dsa_sparse_mla_topk_max_k(void) { return dsa::mla_tc_fused_max_k(); }

dsa_status dsa_topk_sparse_mla_fwd(const float* scores, int64_t ld_scores, const int32_t* q_pos, int32_t k,
                                   int32_t* idx, const void* q, const uint8_t* kv, const float* kv_scale,
                                   int64_t num_pages, const int32_t* block_table, int32_t num_req, int32_t bt_stride,
                                   const int32_t* q_req, int32_t num_q, int32_t num_heads, int32_t d_latent,
                                   int32_t d_rope, int32_t page_size, float softmax_scale, int32_t num_splits,
                                   void* out, float* lse, float* o_part, float* lse_part, void* workspace,
                                   size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (ld_scores <= 0 || k <= 0 || num_q < 0) return DSA_ERR_INVALID_ARG;
  if (!use_tensor_cores(num_heads, d_latent, d_rope) || ld_scores > 65536) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (num_q == 0) return DSA_OK;
  if (!scores || !q_pos || !idx) return DSA_ERR_INVALID_ARG;
  dsa::MlaArgs a;
  const size_t ws_need = dsa_sparse_mla_workspace_size(num_q, num_heads, d_latent, d_rope, k);
  const dsa_status st = check_mla_args(q, kv, kv_scale, num_pages, block_table, num_req, bt_stride, q_req, idx,
                                       num_q, num_heads, d_latent, d_rope, page_size, k, softmax_scale, num_splits,
                                       out, lse, o_part, lse_part, ws_need, workspace, workspace_bytes, dev_status,
                                       &a);
  if (st != DSA_OK) return st;
  const dsa::TopkResolve rv{static_cast<int2*>(workspace), block_table, q_req, kv_scale, num_pages, num_req,
                            bt_stride, page_size};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dsa::launch_topk_resolve(scores, ld_scores, q_pos, num_q, k, idx, rv, dev_status, s);
  if (e != cudaSuccess) return from_cuda(e);
  return from_cuda(dsa::launch_mla_tc_resolved(a, workspace, s));
}

// Test hook, not part of include/dsa.h: the fp32 CUDA-core kernel on any
// supported shape, so that tests can cross-check it against the tensor-core
// kernel on the 64-head shape.  Same arguments as dsa_sparse_mla_fwd minus
// the workspace (the CUDA-core kernel needs none).
DSA_API dsa_status dsa_test_sparse_mla_fwd_cuda_cores(const void* q, const uint8_t* kv, const float* kv_scale,
                                                      int64_t num_pages, const int32_t* block_table, int32_t num_req,
                                                      int32_t bt_stride, const int32_t* q_req, const int32_t* idx,
                                                      int32_t num_q, int32_t num_heads, int32_t d_latent,
                                                      int32_t d_rope, int32_t page_size, int32_t k,
                                                      float softmax_scale, int32_t num_splits, void* out, float* lse,
                                                      float* o_part, float* lse_part, int32_t* dev_status,
                                                      void* stream) {
  dsa::MlaArgs a;
  const dsa_status st = check_mla_args(q, kv, kv_scale, num_pages, block_table, num_req, bt_stride, q_req, idx,
                                       num_q, num_heads, d_latent, d_rope, page_size, k, softmax_scale, num_splits,
                                       out, lse, o_part, lse_part, 0, nullptr, 0, dev_status, &a);
  if (st != DSA_OK || num_q == 0) return st;
  return from_cuda(dsa::launch_mla_simt(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_combine(const float* o_part, const float* lse_part, int32_t num_splits, int32_t num_q,
                       int32_t num_heads, int32_t d_v, void* out, float* lse, void* stream) {
  if (num_q < 0 || num_splits < 1 || num_splits > 64 || num_heads < 1 || num_heads > 64 || d_v <= 0 ||
      d_v % 4 != 0)
    return DSA_ERR_INVALID_ARG;
  if (num_q == 0) return DSA_OK;
  if (!o_part || !lse_part || !out || !aligned16(o_part) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
  return from_cuda(dsa::launch_combine(o_part, lse_part, num_splits, num_q, num_heads, d_v, out, lse,
                                       static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

dsa_status dsa_kv_write(const void* rows, int32_t n, int32_t d_qk, const int32_t* req, const int32_t* pos,
                        const int32_t* block_table, int32_t num_req, int32_t bt_stride, int32_t page_size,
                        int64_t num_pages, uint8_t* kv, float* kv_scale, int32_t* dev_status, void* stream) {
  if (n < 0 || d_qk < 16 || d_qk % 16 != 0 || d_qk > dsa::kv_write_max_d() || page_size <= 0 || num_pages <= 0 ||
      num_req <= 0 || bt_stride <= 0)
    return DSA_ERR_INVALID_ARG;
  if (num_pages > (int64_t)INT32_MAX / page_size) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (n == 0) return DSA_OK;
  if (!rows || !req || !pos || !block_table || !kv || !kv_scale) return DSA_ERR_INVALID_ARG;
  if (!aligned16(rows) || !aligned16(kv)) return DSA_ERR_INVALID_ARG;
  return from_cuda(dsa::launch_kv_write(rows, n, d_qk, req, pos, block_table, num_req, bt_stride, page_size,
                                        num_pages, kv, kv_scale, dev_status, static_cast<cudaStream_t>(stream)));
}

namespace {

// Whether [a, a + na) and [b, b + nb) bytes overlap.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + (uint64_t)nb && y < x + (uint64_t)na;
}

struct Span {
  const void* p;
  int64_t bytes;
};
// Whether a written span overlaps an input or another written one.
template <int NO, int NI>
bool outputs_overlap(const Span (&out)[NO], const Span (&in)[NI]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (overlap(out[o].p, out[o].bytes, in[i].p, in[i].bytes)) return true;
    for (int x = 0; x < o; ++x)
      if (overlap(out[o].p, out[o].bytes, out[x].p, out[x].bytes)) return true;
  }
  return false;
}

// Bytes from the first to the last value of 16-bit rows [tokens, heads, d].
int64_t row_span(int64_t tokens, int64_t heads, int64_t ts, int64_t hs, int64_t d) {
  return tokens > 0 && heads > 0 ? 2 * ((tokens - 1) * ts + (heads - 1) * hs + d) : 0;
}

// One side of dsa_qk_norm_rope.
dsa_status check_norm_side(const void* x, int64_t ts, int64_t hs, int32_t heads, const float* w, int32_t norm_dim,
                           const void* out, bool out_needed, int32_t num_tokens, int32_t d) {
  if (heads < 0 || norm_dim < 0 || norm_dim > d || norm_dim % 8 != 0) return DSA_ERR_INVALID_ARG;
  if (heads == 0 || num_tokens == 0) return DSA_OK;
  if (!x || !aligned16(x) || ts % 8 != 0 || hs % 8 != 0 || ts < 0 || hs < 0) return DSA_ERR_INVALID_ARG;
  if (norm_dim > 0 && (!w || !aligned16(w))) return DSA_ERR_INVALID_ARG;
  if ((!out && out_needed) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
  if (out == x && ((heads > 1 && hs != d) || (num_tokens > 1 && ts != (int64_t)heads * d))) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

}  // namespace

dsa_status dsa_batch_layout(const int32_t* ctx_len, const int32_t* new_len, const int32_t* pages_held, int32_t num_req,
                            int32_t* block_table, int32_t bt_stride, const int32_t* free_pages, int32_t num_free,
                            const int32_t* free_used, int32_t page_size, int64_t num_pages, int32_t capacity,
                            int32_t* cu_q, int32_t* q_req, int32_t* q_pos, int32_t* slot, int32_t* ctx_out,
                            int32_t* held_out, int32_t* free_used_out, int32_t* dev_status, void* stream) {
  if (num_req <= 0 || bt_stride <= 0 || num_free < 0 || page_size <= 0 || num_pages <= 0 || capacity < 0)
    return DSA_ERR_INVALID_ARG;
  // (the token loop counts four ahead, and one past the capacity, in 32 bits)
  if (num_req > dsa::batch_layout_max_requests() || num_pages > (int64_t)INT32_MAX / page_size || capacity > (1 << 30))
    return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!ctx_len || !new_len || !pages_held || !block_table || (num_free > 0 && !free_pages) || !free_used)
    return DSA_ERR_INVALID_ARG;
  if (!cu_q || (capacity > 0 && (!q_req || !q_pos || !slot)) || !ctx_out || !held_out || !free_used_out)
    return DSA_ERR_INVALID_ARG;
  // every CTA reads the inputs while one writes the new lengths, and others the table
  const int64_t nr = 4 * (int64_t)num_req, nt = 4 * (int64_t)capacity;
  const Span in[5] = {{ctx_len, nr}, {new_len, nr}, {pages_held, nr}, {free_used, 4}, {free_pages, 4 * (int64_t)num_free}};
  const Span out[8] = {{block_table, nr * bt_stride}, {cu_q, nr + 4}, {ctx_out, nr}, {held_out, nr}, {free_used_out, 4},
                       {q_req, nt}, {q_pos, nt}, {slot, nt}};
  if (outputs_overlap(out, in)) return DSA_ERR_INVALID_ARG;
  dsa::BatchLayoutArgs a;
  a.ctx_len = ctx_len;
  a.new_len = new_len;
  a.pages_held = pages_held;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.free_used = free_used;
  a.num_req = num_req;
  a.bt_stride = bt_stride;
  a.page_size = page_size;
  a.num_free = num_free;
  a.capacity = capacity;
  a.num_pages = num_pages;
  a.cu_q = cu_q;
  a.q_req = q_req;
  a.q_pos = q_pos;
  a.slot = slot;
  a.ctx_out = ctx_out;
  a.held_out = held_out;
  a.free_used_out = free_used_out;
  a.vec = aligned16(q_req) && aligned16(q_pos) && aligned16(slot);
  a.dev_status = dev_status;
  return from_cuda(dsa::launch_batch_layout(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_qk_norm_rope(const void* q, int64_t q_tok_stride, int64_t q_head_stride, int32_t q_heads,
                            const float* q_weight, int32_t q_norm_dim, void* q_out, const void* k,
                            int64_t k_tok_stride, int64_t k_head_stride, int32_t k_heads, const float* k_weight,
                            int32_t k_norm_dim, void* k_out, int32_t num_tokens, int32_t d, int32_t d_rope,
                            int32_t dtype, const int32_t* pos, const float* cos_sin, int32_t max_pos, float eps,
                            int32_t interleaved, const int32_t* slot, uint8_t* kv, float* kv_scale, int64_t num_slots,
                            int32_t* dev_status, void* stream) {
  if (num_tokens < 0 || d < 8 || d % 8 != 0 || d > dsa::norm_rope_max_d()) return DSA_ERR_INVALID_ARG;
  if (d_rope < 0 || d_rope > d || d_rope % 16 != 0 || (interleaved != 0 && interleaved != 1) || !(eps >= 0.f))
    return DSA_ERR_INVALID_ARG;
  if (dtype != DSA_BF16 && dtype != DSA_FP16) return DSA_ERR_INVALID_ARG;
  if (q_heads < 0 || k_heads < 0 || q_heads + (int64_t)k_heads > 65536) return DSA_ERR_INVALID_ARG;
  const bool cache = slot || kv || kv_scale;
  if (cache && (!slot || !kv || !kv_scale || k_heads != 1 || num_slots <= 0 || !aligned16(kv)))
    return DSA_ERR_INVALID_ARG;
  dsa_status st = check_norm_side(q, q_tok_stride, q_head_stride, q_heads, q_weight, q_norm_dim, q_out, true,
                                  num_tokens, d);
  if (st != DSA_OK) return st;
  st = check_norm_side(k, k_tok_stride, k_head_stride, k_heads, k_weight, k_norm_dim, k_out, !cache, num_tokens, d);
  if (st != DSA_OK) return st;
  if ((int64_t)num_tokens * (q_heads + k_heads) > INT32_MAX) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (num_tokens == 0 || q_heads + k_heads == 0) return DSA_OK;
  if (d_rope > 0 && (!pos || !cos_sin || !aligned16(cos_sin) || max_pos <= 0)) return DSA_ERR_INVALID_ARG;
  // a row may be written before another CTA has read its own: only a side in place shares
  // memory, and its input then stands for both
  const int64_t n = num_tokens, n4 = 4 * n;
  const int64_t q_in = row_span(n, q_heads, q_tok_stride, q_head_stride, d);
  const int64_t k_in = row_span(n, k_heads, k_tok_stride, k_head_stride, d);
  const bool q_own = q_heads > 0 && q_out == q, k_own = k_heads > 0 && k_out == k;
  const Span in[7] = {{q_own ? nullptr : q, q_in}, {k_own ? nullptr : k, k_in}, {q_heads > 0 ? q_weight : nullptr, 4 * (int64_t)q_norm_dim},
                      {k_heads > 0 ? k_weight : nullptr, 4 * (int64_t)k_norm_dim}, {pos, n4},
                      {d_rope > 0 ? cos_sin : nullptr, 4 * (int64_t)max_pos * d_rope}, {slot, n4}};
  const Span out[4] = {{q_out, 2 * n * q_heads * d}, {k_out, 2 * n * k_heads * d}, {kv, num_slots * d}, {kv_scale, 4 * num_slots}};
  if (outputs_overlap(out, in)) return DSA_ERR_INVALID_ARG;
  dsa::NormRopeArgs a;
  a.q = {q, q_tok_stride, q_head_stride, q_heads, q_norm_dim, q_weight, q_heads > 0 ? q_out : nullptr};
  a.k = {k, k_tok_stride, k_head_stride, k_heads, k_norm_dim, k_weight, k_heads > 0 ? k_out : nullptr};
  a.num_tokens = num_tokens;
  a.d = d;
  a.d_rope = d_rope;
  a.dtype = dtype;
  a.pos = pos;
  a.cos_sin = cos_sin;
  a.max_pos = d_rope > 0 ? max_pos : INT32_MAX;
  a.eps = eps;
  a.interleaved = interleaved != 0;
  a.slot = slot;
  a.kv = cache ? kv : nullptr;
  a.kv_scale = kv_scale;
  a.num_slots = num_slots;
  a.dev_status = dev_status;
  return from_cuda(dsa::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_chunk_mla_fwd(const void* q, const uint8_t* kv, const float* kv_scale, int64_t num_pages,
                             const int32_t* block_table, int32_t num_req, int32_t bt_stride, const int32_t* q_req,
                             const int32_t* q_pos, int32_t num_q, int32_t num_heads, int32_t d_latent, int32_t d_rope,
                             int32_t page_size, float softmax_scale, int32_t num_splits, void* out, float* lse,
                             float* o_part, float* lse_part, int32_t* dev_status, void* stream) {
  dsa::MlaArgs a;
  // splits without partials are merged by the call itself
  const bool merge = num_splits > 1 && !o_part && !lse_part;
  if (merge && num_splits > dsa::chunk_max_merged()) return DSA_ERR_INVALID_ARG;
  // q_pos stands in for idx in the checks; k is unused
  const dsa_status st = check_mla_args(q, kv, kv_scale, num_pages, block_table, num_req, bt_stride, q_req, q_pos,
                                       num_q, num_heads, d_latent, d_rope, page_size, 1, softmax_scale,
                                       merge ? 1 : num_splits, out, lse, o_part, lse_part, 0, nullptr, 0, dev_status,
                                       &a);
  if (st != DSA_OK || num_q == 0) return st;
  // a token's result may be written before another token has read what it needs
  const int64_t rows = (int64_t)num_q * num_heads, slots = num_pages * page_size, n4 = 4 * (int64_t)num_q;
  const bool whole = num_splits == 1 || merge;
  const Span in[6] = {{q, 2 * rows * (d_latent + d_rope)}, {kv, slots * (d_latent + d_rope)}, {kv_scale, 4 * slots},
                      {block_table, 4 * (int64_t)num_req * bt_stride}, {q_req, n4}, {q_pos, n4}};
  const Span out_whole[2] = {{out, 2 * rows * d_latent}, {lse, 4 * rows}};
  const Span out_part[2] = {{o_part, 4 * rows * d_latent * num_splits}, {lse_part, 4 * rows * num_splits}};
  if (outputs_overlap(whole ? out_whole : out_part, in)) return DSA_ERR_INVALID_ARG;
  a.idx = nullptr;
  a.num_splits = num_splits;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (use_tensor_cores(num_heads, d_latent, d_rope)) return from_cuda(dsa::launch_chunk_tc(a, q_pos, merge, s));
  return from_cuda(dsa::launch_chunk_small(a, q_pos, merge, s));
}

dsa_status dsa_verify_draft_req(const float* target_probs, int64_t ld_target, int32_t num_rows, int32_t vocab,
                                const float* draft_probs, int64_t ld_draft, const int32_t* draft_tokens,
                                const float* u_accept, const float* u_sample, const int32_t* cu_rows,
                                const int32_t* q_req, int32_t num_req, int32_t max_out, const int32_t* ctx_len,
                                int32_t* tokens, int32_t* num_out, int32_t* ctx_out, int32_t* dev_status,
                                void* stream) {
  if (num_rows < 0 || vocab <= 0 || num_req < 0 || max_out <= 0 || ld_target < vocab) return DSA_ERR_INVALID_ARG;
  if (draft_probs && ld_draft < vocab) return DSA_ERR_INVALID_ARG;
  if ((ctx_len == nullptr) != (ctx_out == nullptr)) return DSA_ERR_INVALID_ARG;
  // (loops over rows, columns and outputs count up to 1,024 ahead in 32 bits)
  if (num_req > (1 << 24) || vocab > (1 << 30) || num_rows > (1 << 30) || max_out > (1 << 30))
    return DSA_ERR_UNSUPPORTED_SHAPE;
  if (num_req == 0) return DSA_OK;
  if (!u_sample || !cu_rows || !tokens || !num_out) return DSA_ERR_INVALID_ARG;
  if (num_rows > 0 && (!target_probs || !draft_tokens || !u_accept)) return DSA_ERR_INVALID_ARG;
  // eight CTAs read a request's inputs while one writes its results (only ctx_len is read
  // by the thread that writes ctx_out over it)
  const int64_t nr = 4 * (int64_t)num_req, nd = 4 * (int64_t)num_rows;
  const Span in[8] = {{target_probs, num_rows > 0 ? 4 * ((num_rows - 1) * ld_target + vocab) : 0},
                      {draft_probs, num_rows > 0 ? 4 * ((num_rows - 1) * ld_draft + vocab) : 0},
                      {draft_tokens, nd}, {u_accept, nd}, {u_sample, nr}, {cu_rows, nr + 4}, {q_req, nd},
                      {ctx_out == ctx_len ? nullptr : ctx_len, nr}};
  const Span out[3] = {{tokens, nr * max_out}, {num_out, nr}, {ctx_out, nr}};
  if (outputs_overlap(out, in)) return DSA_ERR_INVALID_ARG;
  dsa::VerifyArgs a;
  a.target = target_probs;
  a.ld_target = ld_target;
  a.num_rows = num_rows;
  a.vocab = vocab;
  a.draft = draft_probs;
  a.ld_draft = ld_draft;
  a.draft_tokens = draft_tokens;
  a.cu_rows = cu_rows;
  a.q_req = q_req;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.num_req = num_req;
  a.max_out = max_out;
  a.ctx_len = ctx_len;
  a.tokens = tokens;
  a.num_out = num_out;
  a.ctx_out = ctx_out;
  a.dev_status = dev_status;
  return from_cuda(dsa::launch_verify_draft(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_verify_draft(const float* target_probs, int64_t ld_target, int32_t num_rows, int32_t vocab,
                            const float* draft_probs, int64_t ld_draft, const int32_t* draft_tokens,
                            const float* u_accept, const float* u_sample, const int32_t* cu_rows, int32_t num_req,
                            int32_t max_out, const int32_t* ctx_len, int32_t* tokens, int32_t* num_out,
                            int32_t* ctx_out, int32_t* dev_status, void* stream) {
  return dsa_verify_draft_req(target_probs, ld_target, num_rows, vocab, draft_probs, ld_draft, draft_tokens, u_accept,
                              u_sample, cu_rows, nullptr, num_req, max_out, ctx_len, tokens, num_out, ctx_out,
                              dev_status, stream);
}
