// Log probabilities of given tokens, the rows' entropy, the tokens' ranks and the
// most probable alternatives.
//
// With m the row's largest logit, at column a, and d_j = z_j - m <= 0:
//   rest    = sum_{j != a} e^{d_j},  lse = m + log1p(rest)
//   logprob = d_t - log1p(rest)
//   entropy = log1p(rest) - sum_j e^{d_j} d_j / (1 + rest)     (two terms >= 0: nothing cancels)
// The largest term, 1, stays out of the sum: the logarithm of a sure token is next
// to rest, which 1 + rest in fp32 would round to 2^-24.
//
// One CTA a row, one pass for each step.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.cuh"

namespace dsa {
namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32;

template <class T>
__device__ __forceinline__ float value(const T* row, int j) {
  return (float)row[j];
}

// Whether (x, i) comes before (y, j): larger, or equal and of a lower column.
__device__ __forceinline__ bool before(float x, int i, float y, int j) { return x > y || (x == y && i < j); }

// The first of the block's (x, i) pairs in that order (NaN is never it; i = INT32_MAX: none).
__device__ __forceinline__ void block_first(float& x, int& i, float* sx, int* si) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    const int j = __shfl_xor_sync(0xffffffffu, i, o);
    if (before(y, j, x, i)) x = y, i = j;
  }
  __syncthreads();
  if (lane == 0) sx[warp] = x, si[warp] = i;
  __syncthreads();
  x = sx[0], i = si[0];
  for (int w = 1; w < WARPS; ++w)
    if (before(sx[w], si[w], x, i)) x = sx[w], i = si[w];
}

__device__ __forceinline__ float block_sum(float x, float* sx) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if (lane == 0) sx[warp] = x;
  __syncthreads();
  x = 0.f;
  for (int w = 0; w < WARPS; ++w) x += sx[w];
  return x;
}

template <class T>
__global__ void __launch_bounds__(THREADS) logprobs_kernel(const LogprobArgs a) {
  __shared__ float sx[WARPS];
  __shared__ int si[WARPS];
  const int64_t i = blockIdx.x;
  const T* row = static_cast<const T*>(a.logits) + i * a.ld;
  const int V = a.vocab, tid = threadIdx.x;
  int t = a.tokens[i];
  if (t < -1 || t >= V) {
    if (tid == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);
    t = -1;
  }
  const float zt = t >= 0 ? value(row, t) : 0.f;
  float m = -INFINITY;
  int at = INT32_MAX;
  for (int j = tid; j < V; j += THREADS) {
    const float z = value(row, j);
    if (before(z, j, m, at)) m = z, at = j;
  }
  block_first(m, at, sx, si);
  float rest = 0.f, ent = 0.f, count = 0.f, odd = m == INFINITY ? 1.f : 0.f;
  for (int j = tid; j < V; j += THREADS) {
    const float z = value(row, j);
    if (isnan(z)) odd = 1.f;
    if (t >= 0 && before(z, j, zt, t)) count += 1.f;
    if (z == -INFINITY || j == at) continue;
    const float d = z - m, e = expf(d);
    rest += e;
    ent += e * d;
  }
  rest = block_sum(rest, sx);
  ent = block_sum(ent, sx);
  count = block_sum(count, sx);
  odd = block_sum(odd, sx);
  const bool none = m == -INFINITY;
  const float log_total = log1pf(rest);
  if (tid == 0) {
    a.logprob[i] = odd > 0.f ? NAN : t < 0 || none ? -INFINITY : (zt - m) - log_total;
    a.entropy[i] = odd > 0.f ? NAN : none ? 0.f : log_total - ent / (1.f + rest);
    a.rank[i] = t < 0 ? -1 : (int)count;
  }
  float px = INFINITY;
  int pi = -1;
  for (int k = 0; k < a.top; ++k) {
    float x = -INFINITY;
    int xi = INT32_MAX;
    for (int j = tid; j < V; j += THREADS) {
      const float z = value(row, j);
      if (z > -INFINITY && before(px, pi, z, j) && before(z, j, x, xi)) x = z, xi = j;
    }
    block_first(x, xi, sx, si);
    if (tid == 0) {
      a.top_ids[i * a.top + k] = xi == INT32_MAX ? -1 : xi;
      a.top_logprobs[i * a.top + k] = odd > 0.f ? NAN : xi == INT32_MAX ? -INFINITY : (x - m) - log_total;
    }
    px = x, pi = xi;
  }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  const unsigned grid = (unsigned)a.num_rows;
  if (a.dtype == DSA_BF16) logprobs_kernel<__nv_bfloat16><<<grid, THREADS, 0, stream>>>(a);
  else if (a.dtype == DSA_FP16) logprobs_kernel<__half><<<grid, THREADS, 0, stream>>>(a);
  else logprobs_kernel<float><<<grid, THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa
