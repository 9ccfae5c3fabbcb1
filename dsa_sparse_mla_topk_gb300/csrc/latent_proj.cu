// Products of latent attention around the cache's latent space: queries into
// it (dsa_absorb_q), attention's outputs out of it (dsa_project_out), and
// cached rows to every head's keys and values (dsa_expand_kv).
//
//   absorb:   y[t, h, :] = x[t, h, :dn] W_k[h],        W_k[h] = w[h, :dn, :]   [dn, dl]
//   project:  y[t, h, :] = x[t, h, :dl] W_v[h]^T,      W_v[h] = w[h, dn:, :]   [dv, dl]
//   expand:   y[n, (h, j)] = s_n (code[n, :] . w[h, j, :])
//
// One product C = s A B per group (a head), 64 x 64 outputs a CTA on the CUDA cores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.cuh"

namespace dsa {
namespace {

struct Product {
  const __nv_bfloat16* a;  // [m, k]: row stride lda, group stride ga
  int64_t lda, ga;
  const __nv_bfloat16* b;  // b_k_major: [n, k], else [k, n]; row stride ldb, group stride gb
  int64_t ldb, gb;
  __nv_bfloat16* c;  // [m, n]
  int64_t ldc, gc;
  const float* scale;  // [m], or null
  const int32_t* rows;  // where m stands on the device, or null
  int32_t m, n, k;
};

template <bool B_K_MAJOR>
__global__ void __launch_bounds__(256) product_kernel(const Product p) {
  constexpr int TM = 64, TN = 64, TK = 16;
  __shared__ float as[TK][TM + 4], bs[TK][TN + 4];
  const int m_all = p.rows ? min(*p.rows, p.m) : p.m;
  const int m0 = blockIdx.x * TM, n0 = blockIdx.y * TN;
  if (m0 >= m_all) return;
  const __nv_bfloat16* a = p.a + blockIdx.z * p.ga;
  const __nv_bfloat16* b = p.b + blockIdx.z * p.gb;
  const int tid = threadIdx.x, tm = tid / 16 * 4, tn = tid % 16 * 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += TK) {
    for (int e = tid; e < TM * TK; e += 256) {
      const int m = e / TK, k = e % TK;
      as[k][m] = m0 + m < m_all ? __bfloat162float(a[(m0 + m) * p.lda + k0 + k]) : 0.f;
    }
    for (int e = tid; e < TN * TK; e += 256) {
      const int n = B_K_MAJOR ? e / TK : e % TN, k = B_K_MAJOR ? e % TK : e / TN;
      bs[k][n] = n0 + n < p.n ? __bfloat162float(b[B_K_MAJOR ? (n0 + n) * p.ldb + k0 + k : (k0 + k) * p.ldb + n0 + n]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += as[k][tm + i] * bs[k][tn + j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + tm + i;
    if (m >= m_all) break;
    const float s = p.scale ? p.scale[m] : 1.f;
    for (int j = 0; j < 4; ++j)
      if (n0 + tn + j < p.n) p.c[blockIdx.z * p.gc + m * p.ldc + n0 + tn + j] = __float2bfloat16_rn(acc[i][j] * s);
  }
}

// The rotated part of the queries, as it is: 16 bytes a thread.
__global__ void __launch_bounds__(256) copy_rope_kernel(const LatentProjArgs a) {
  const int per = a.d_rope / 8;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, row = e / per;
  if (row >= (int64_t)a.num_tokens * a.heads) return;
  const int64_t t = row / a.heads, h = row % a.heads;
  const int c = (int)(e % per) * 8;
  const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + t * a.tok_stride +
                                                  h * a.head_stride + a.d_nope + c);
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y) + row * (a.d_latent + a.d_rope) + a.d_latent + c) = v;
}

cudaError_t launch_product(const Product& p, bool b_k_major, int groups, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.m + 63) / 64), (unsigned)((p.n + 63) / 64), (unsigned)groups);
  if (b_k_major) product_kernel<true><<<grid, 256, 0, stream>>>(p);
  else product_kernel<false><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

// ---- cached rows: codes as bf16 numbers (exact), scales and rotated parts ----

constexpr int EX_THREADS = 256, EX_WARPS = EX_THREADS / 32, EX_ROWS = 32;  // rows a CTA

// Every CTA takes the running sum of the lengths for itself; then a warp a row.
__global__ void __launch_bounds__(EX_THREADS) expand_rows_kernel(const ExpandArgs a, __nv_bfloat16* x, float* scale) {
  extern __shared__ int32_t cu[];  // [num_req + 1]
  __shared__ int64_t wsum[EX_WARPS];
  __shared__ int64_t fit[EX_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = a.num_req;
  int64_t before = 0, most = 0;
  for (int r0 = 0; r0 < R; r0 += EX_THREADS) {
    const int r = r0 + tid;
    int64_t n = r < R ? a.ctx_len[r] : 0;
    if (n < 0 || n > (int64_t)a.bt_stride * a.page_size) {
      if (blockIdx.x == 0) report(a.dev_status, n < 0 ? DSA_DEV_BAD_QPOS : DSA_DEV_BAD_INDEX);
      n = 0;
    }
    int64_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < EX_WARPS; ++w) {
      if (w < warp) inc += wsum[w];
      all += wsum[w];
    }
    inc += before;
    before += all;
    const bool fits = inc <= a.capacity;
    if (fits) most = max(most, inc);
    if (r < R) {
      cu[r + 1] = fits ? (int32_t)inc : INT32_MAX;
      if (!fits && n > 0 && blockIdx.x == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);
    }
    __syncthreads();
  }
  // what follows the last request that fits has no rows
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) fit[warp] = most;
  if (tid == 0) cu[0] = 0;
  __syncthreads();
  for (int w = 0; w < EX_WARPS; ++w) most = max(most, fit[w]);
  const int32_t total = (int32_t)most;
  if (blockIdx.x == 0)
    for (int r = tid; r <= R; r += EX_THREADS) a.cu_k[r] = min(cu[r], total);

  const int dl = a.d_latent, row_bytes = dl + a.d_rope, chunks = row_bytes / 16;
  for (int i = warp; i < EX_ROWS; i += EX_WARPS) {
    const int n = blockIdx.x * EX_ROWS + i;
    if (n >= total) break;
    int lo = 0, hi = R - 1;  // the request with cu[r] <= n < cu[r + 1]
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (cu[mid + 1] > n) hi = mid;
      else lo = mid + 1;
    }
    const int pos = n - cu[lo];
    const int page = a.block_table[(int64_t)lo * a.bt_stride + pos / a.page_size];
    const bool good = page >= 0 && page < a.num_pages;
    if (!good && lane == 0) report(a.dev_status, DSA_DEV_BAD_PAGE);
    const int64_t slot = (int64_t)page * a.page_size + pos % a.page_size;
    const float s = good ? a.kv_scale[slot] : 0.f;
    if (lane == 0) scale[n] = s;
    for (int c = lane; c < chunks; c += 32) {
      const uint4 v = good ? *reinterpret_cast<const uint4*>(a.kv + slot * row_bytes + 16 * c) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      const bool rope = 16 * c >= dl;
      __align__(16) __nv_bfloat162 y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[e / 2] >> (16 * (e & 1))), __NV_E4M3));
        float2 f = __half22float2(h);
        if (rope) f.x *= s, f.y *= s;
        y[e] = __floats2bfloat162_rn(f.x, f.y);  // (a code is exact in bf16)
      }
      __nv_bfloat16* dst = rope ? static_cast<__nv_bfloat16*>(a.k_rope) + (int64_t)n * a.d_rope + (16 * c - dl)
                                : x + (int64_t)n * dl + 16 * c;
      *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<uint4*>(y);
      *reinterpret_cast<uint4*>(dst + 8) = *reinterpret_cast<uint4*>(y + 4);
    }
  }
}

}  // namespace

cudaError_t launch_absorb_q(const LatentProjArgs& a, cudaStream_t stream) {
  const int64_t d_out = a.d_latent + a.d_rope, d_w = a.d_nope + a.d_v;
  Product p = {static_cast<const __nv_bfloat16*>(a.x), a.tok_stride, a.head_stride,
               static_cast<const __nv_bfloat16*>(a.w), a.d_latent, d_w * a.d_latent,
               static_cast<__nv_bfloat16*>(a.y), a.heads * d_out, d_out, nullptr, nullptr,
               a.num_tokens, a.d_latent, a.d_nope};
  const cudaError_t e = launch_product(p, false, a.heads, stream);
  if (e != cudaSuccess || a.d_rope == 0) return e;
  const int64_t n = (int64_t)a.num_tokens * a.heads * (a.d_rope / 8);
  copy_rope_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_project_out(const LatentProjArgs& a, cudaStream_t stream) {
  const int64_t d_w = a.d_nope + a.d_v;
  Product p = {static_cast<const __nv_bfloat16*>(a.x), a.tok_stride, a.head_stride,
               static_cast<const __nv_bfloat16*>(a.w) + (int64_t)a.d_nope * a.d_latent, a.d_latent, d_w * a.d_latent,
               static_cast<__nv_bfloat16*>(a.y), (int64_t)a.heads * a.d_v, a.d_v, nullptr, nullptr,
               a.num_tokens, a.d_v, a.d_latent};
  return launch_product(p, true, a.heads, stream);
}

// codes as bf16 [capacity, d_latent], then a scale a row
size_t expand_kv_workspace_bytes(int32_t capacity, int32_t d_latent) {
  return (size_t)capacity * d_latent * 2 + ((size_t)capacity * 4 + 15) / 16 * 16;
}

cudaError_t launch_expand_kv(const ExpandArgs& a, cudaStream_t stream) {
  __nv_bfloat16* x = static_cast<__nv_bfloat16*>(a.workspace);
  float* scale = reinterpret_cast<float*>(x + (int64_t)a.capacity * a.d_latent);
  const int grid = max(1, (a.capacity + EX_ROWS - 1) / EX_ROWS);
  expand_rows_kernel<<<grid, EX_THREADS, 4 * (a.num_req + 1), stream>>>(a, x, scale);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.capacity == 0) return e;
  const int d_w = a.heads * a.d_kv;
  Product p = {x, a.d_latent, 0, static_cast<const __nv_bfloat16*>(a.w), a.d_latent, 0,
               static_cast<__nv_bfloat16*>(a.kv_out), d_w, 0, scale, a.cu_k + a.num_req, a.capacity, d_w, a.d_latent};
  return launch_product(p, true, 1, stream);
}

}  // namespace dsa
