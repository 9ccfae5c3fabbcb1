// Attention of new tokens over every head's own keys and values: latent
// attention's expanded form, for prompts and their chunks.
//
//   z_j = scale (q_n . k_j + q_r . k_rope_j),  j = 0 .. q_pos of the token's request
//   out = sum_j softmax(z)_j v_j,  lse = ln sum_j exp z_j
//
// 16 tokens of a request and one head a CTA; keys and values come 32 rows at a time
// into shared memory in fp32; running maximum and sum (online softmax).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.cuh"

namespace dsa {
namespace {

constexpr int TQ = 16, TK = 32, THREADS = 128, MAX_QK = 192, MAX_V = 128;

struct Tile {
  int req, q0, rows;  // req -1: padding rows
};

__global__ void __launch_bounds__(THREADS) prompt_simple_kernel(const PromptArgs a, const int max_tiles) {
  __shared__ float qs[TQ][MAX_QK], ks[TK][MAX_QK + 1], vs[TK][MAX_V], ps[TQ][TK], alpha[TQ], mrow[TQ], lrow[TQ];
  __shared__ int last[TQ];
  const int h = blockIdx.y, split = blockIdx.z, S = gridDim.z, tid = threadIdx.x;
  const int dn = a.d_nope, dqk = a.d_nope + a.d_rope, dv = a.d_v;
  // which rows: the requests' tiles one after another, then the padding's
  Tile t = {-2, 0, 0};
  int left = blockIdx.x;
  for (int r = 0; r < a.num_req && t.req == -2; ++r) {
    const int q0 = a.cu_q[r], q1 = a.cu_q[r + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.num_tokens) {
      if (blockIdx.x == gridDim.x - 1 && tid == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);  // (it looks at all)
      continue;
    }
    const int tiles = (q1 - q0 + TQ - 1) / TQ;
    if (left < tiles) t = {r, q0 + left * TQ, min(TQ, q1 - q0 - left * TQ)};
    left -= tiles;
  }
  if (t.req == -2) {
    const int pad0 = min(max(a.num_req > 0 ? a.cu_q[a.num_req] : 0, 0), a.num_tokens);
    const int64_t q0 = pad0 + (int64_t)left * TQ;
    if (q0 >= a.num_tokens) return;
    t = {-1, (int)q0, (int)min((int64_t)TQ, a.num_tokens - q0)};
  }
  int k0 = 0, kv_len = 0;
  if (t.req >= 0) {
    k0 = a.cu_k[t.req];
    const int k1 = a.cu_k[t.req + 1];
    if (k0 < 0 || k1 < k0 || k1 > a.num_rows) {
      if (tid == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);
    } else {
      kv_len = k1 - k0;
    }
  }
  if (tid < TQ) {
    int p = -1;
    if (t.req >= 0 && tid < t.rows) {
      p = a.q_pos[t.q0 + tid];
      if (p < -1 || p >= kv_len) {
        report(a.dev_status, DSA_DEV_BAD_QPOS);
        p = -1;
      }
    }
    last[tid] = p;
    mrow[tid] = -INFINITY;
    lrow[tid] = 0.f;
  }
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
  for (int e = tid; e < TQ * dqk; e += THREADS) {
    const int i = e / dqk, d = e % dqk;
    qs[i][d] = t.req >= 0 && i < t.rows ? __bfloat162float(q[(t.q0 + i) * a.q_tok_stride + h * a.q_head_stride + d]) : 0.f;
  }
  __syncthreads();
  int end = 0;
  for (int i = 0; i < TQ; ++i) end = max(end, last[i] + 1);
  const int ntiles = (end + TK - 1) / TK;
  const int b = (int)((int64_t)ntiles * split / S), e1 = (int)((int64_t)ntiles * (split + 1) / S);
  float o[TQ];
#pragma unroll
  for (int i = 0; i < TQ; ++i) o[i] = 0.f;
  const __nv_bfloat16* kv = static_cast<const __nv_bfloat16*>(a.kv);
  for (int kt = b; kt < e1; ++kt) {
    const int j0 = kt * TK;
    for (int e = tid; e < TK * dqk; e += THREADS) {
      const int j = e / dqk, d = e % dqk;
      const int64_t n = k0 + j0 + j;
      float v = 0.f;
      if (j0 + j < end)
        v = __bfloat162float(d < dn ? kv[n * a.kv_tok_stride + h * a.kv_head_stride + d]
                                    : static_cast<const __nv_bfloat16*>(a.k_rope)[n * a.rope_stride + d - dn]);
      ks[j][d] = v;
    }
    for (int e = tid; e < TK * dv; e += THREADS) {
      const int j = e / dv, d = e % dv;
      const int64_t n = k0 + j0 + j;
      vs[j][d] = j0 + j < end ? __bfloat162float(kv[n * a.kv_tok_stride + h * a.kv_head_stride + dn + d]) : 0.f;
    }
    __syncthreads();
    for (int e = tid; e < TQ * TK; e += THREADS) {
      const int i = e / TK, j = e % TK;
      float z = -INFINITY;
      if (j0 + j <= last[i]) {
        z = 0.f;
        for (int d = 0; d < dqk; ++d) z += qs[i][d] * ks[j][d];
        z *= a.softmax_scale;
      }
      ps[i][j] = z;
    }
    __syncthreads();
    if (tid < TQ) {
      const int n = min(TK, last[tid] + 1 - j0);  // rows of the tile that this token sees
      float m = mrow[tid], l = lrow[tid];
      for (int j = 0; j < n; ++j) m = fmaxf(m, ps[tid][j]);
      const float f = n > 0 && mrow[tid] != -INFINITY ? expf(mrow[tid] - m) : n > 0 ? 0.f : 1.f;
      l *= f;
      for (int j = 0; j < n; ++j) {
        const float p = expf(ps[tid][j] - m);
        ps[tid][j] = p;
        l += p;
      }
      alpha[tid] = f;
      mrow[tid] = m;
      lrow[tid] = l;
    }
    __syncthreads();
    if (tid < dv) {
#pragma unroll
      for (int i = 0; i < TQ; ++i) {
        const int n = min(TK, last[i] + 1 - j0);
        float s = o[i] * alpha[i];
        for (int j = 0; j < n; ++j) s += ps[i][j] * vs[j][tid];
        o[i] = s;
      }
    }
    __syncthreads();
  }
  for (int i = 0; i < t.rows; ++i) {
    const float l = lrow[i];
    const int64_t row = (int64_t)(t.q0 + i) * a.heads + h, part = (int64_t)split * a.num_tokens * a.heads + row;
    const bool seen = b < e1 && mrow[i] > -INFINITY;
    const float y = l > 0.f || isnan(l) ? o[i] / l : 0.f, z = l > 0.f || isnan(l) ? mrow[i] + logf(l) : -INFINITY;
    (void)seen;
    if (tid < dv) {
      if (S == 1) static_cast<__nv_bfloat16*>(a.out)[row * dv + tid] = __float2bfloat16_rn(y);
      else a.o_part[part * dv + tid] = y;
    }
    if (tid == 0) {
      if (S > 1) a.lse_part[part] = z;
      else if (a.lse) a.lse[row] = z;
    }
  }
}

}  // namespace

cudaError_t launch_prompt_mla(const PromptArgs& a, cudaStream_t stream) {
  const int tiles = a.num_tokens / TQ + a.num_req + 1;
  prompt_simple_kernel<<<dim3((unsigned)tiles, (unsigned)a.heads, (unsigned)a.num_splits), THREADS, 0, stream>>>(a, tiles);
  return cudaGetLastError();
}

}  // namespace dsa
