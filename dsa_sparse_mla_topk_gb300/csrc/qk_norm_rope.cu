// Norms of query and key rows with the position rotation in the same pass;
// the key row may go straight into the paged FP8 cache.
//
// "GLM-5.3 Optimizations, Part 2" ("Interpretation"): a latent row of the
// cache is shared by all heads; SGLang cookbook page for GLM-5.3-Flash, "Keep
// the KV and DSA backends paired": the cache is FP8 E4M3.  For a row x of one
// (token, head), with n = norm_dim leading values normed and the last d_rope
// values rotated:
//     y_j = x_j w_j / sqrt(mean_{j < n} x_j^2 + eps)   (j < n; y_j = x_j else)
//     (y_a, y_b) <- (y_a c - y_b s, y_a s + y_b c)      (c, s) = (cos, sin)[pos]
// for the pairs (a, b) = (2i, 2i + 1) of the rotated part, or (i, i + d_rope/2)
// in the half-split form.  Everything is fp32; a row is rounded once, to its
// own type, or to E4M3 with scale = max |y| / 448 (from the fp32 values, not
// from a 16-bit copy of them).
//
// HBM-bound: each row is read once and written once.  A group of 8 lanes takes
// one row as 16-byte chunks, chunk l + 8 u in lane l: a warp holds four rows,
// so that a 576-value row has no idle lane (72 chunks, 9 a lane, all in flight
// together) and its sums take three shuffles instead of five.  In the
// half-split form the lane reads its partner chunk a second time (an L1 hit).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.cuh"

namespace dsa {
namespace {

constexpr int NR_WARPS = 4;

template <bool HALF>
__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if constexpr (HALF) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[t]));
      x[2 * t] = f.x, x[2 * t + 1] = f.y;
    } else {
      x[2 * t] = __uint_as_float(w[t] << 16), x[2 * t + 1] = __uint_as_float(w[t] & 0xffff0000u);
    }
  }
}

template <bool HALF>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if constexpr (HALF) {
      const __half2 h = __floats2half2_rn(x[2 * t], x[2 * t + 1]);
      w[t] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * t], x[2 * t + 1]);
      w[t] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t code2(float x0, float x1) {  // two E4M3 codes, x0 in the low byte
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}

// HALF: fp16 rows (else bf16).  PAIRS: the rotation's pairs are neighbours
// (else halves).  LPR lanes per row, CH chunks of 8 values per lane.
template <bool HALF, bool PAIRS, int LPR, int CH>
__global__ void __launch_bounds__(NR_WARPS * 32) qk_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int RPW = 32 / LPR;  // rows per warp
  const int lane = threadIdx.x & 31, gl = lane & (LPR - 1);
  const int heads = a.q.heads + a.k.heads;
  const int64_t row = ((int64_t)blockIdx.x * NR_WARPS + (threadIdx.x >> 5)) * RPW + lane / LPR;
  const bool in_range = row < (int64_t)a.num_tokens * heads;
  const int32_t tok = in_range ? (int32_t)(row / heads) : 0;
  const int32_t hh = in_range ? (int32_t)(row - (int64_t)tok * heads) : 0;
  const bool key = hh >= a.q.heads;
  const NormRopeSide& side = key ? a.k : a.q;
  const int32_t h = key ? hh - a.q.heads : hh;
  const int nch = a.d >> 3, rope0 = (a.d - a.d_rope) >> 3, half = a.d_rope >> 4, nn = side.norm_dim >> 3;
  const float* weight = side.weight;

  int32_t p = -1;
  if (in_range) {
    p = a.pos ? a.pos[tok] : 0;
    if (p >= a.max_pos || p < -1) {
      if (hh == 0 && gl == 0) report(a.dev_status, DSA_DEV_BAD_QPOS);
      p = -1;
    }
  }
  const bool live = p >= 0;  // a padding row, or a bad one, is left as it was

  const uint16_t* x0 = static_cast<const uint16_t*>(side.x) + (int64_t)tok * side.tok_stride + (int64_t)h * side.head_stride;
  uint4 raw[CH];
#pragma unroll
  for (int u = 0; u < CH; ++u) {
    const int c = gl + LPR * u;
    raw[u] = live && c < nch ? *reinterpret_cast<const uint4*>(x0 + 8 * c) : make_uint4(0, 0, 0, 0);
  }
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < CH; ++u) {
    if (gl + LPR * u < nn) {
      float x[8];
      unpack8<HALF>(raw[u], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    }
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float inv = nn > 0 ? rsqrtf(ss / (float)side.norm_dim + a.eps) : 1.f;

  const float* cs = a.cos_sin + (int64_t)(live ? p : 0) * a.d_rope;
  auto norm = [&](float (&v)[8], int ch) {
    if (ch >= nn) return;
    const float4 w0 = *reinterpret_cast<const float4*>(weight + 8 * ch);
    const float4 w1 = *reinterpret_cast<const float4*>(weight + 8 * ch + 4);
    const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * inv * w[e];
  };
  // the result's chunk c (of this lane's raw chunk), in fp32
  auto result = [&](const uint4 r, int c, float (&y)[8]) {
    unpack8<HALF>(r, y);
    norm(y, c);
    if (c < rope0 || a.d_rope == 0) return;
    const int rc = c - rope0;
    if constexpr (PAIRS) {
      const float4 co = *reinterpret_cast<const float4*>(cs + 4 * rc);
      const float4 si = *reinterpret_cast<const float4*>(cs + a.d_rope / 2 + 4 * rc);
      const float cc[4] = {co.x, co.y, co.z, co.w}, sn[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float va = y[2 * e], vb = y[2 * e + 1];
        y[2 * e] = va * cc[e] - vb * sn[e];
        y[2 * e + 1] = va * sn[e] + vb * cc[e];
      }
    } else {
      const bool low = rc < half;  // this chunk holds the pairs' first values
      const int pc = low ? c + half : c - half, ic = low ? rc : rc - half;
      float o[8];
      unpack8<HALF>(*reinterpret_cast<const uint4*>(x0 + 8 * pc), o);
      norm(o, pc);
#pragma unroll
      for (int e4 = 0; e4 < 2; ++e4) {
        const float4 co = *reinterpret_cast<const float4*>(cs + 8 * ic + 4 * e4);
        const float4 si = *reinterpret_cast<const float4*>(cs + a.d_rope / 2 + 8 * ic + 4 * e4);
        const float cc[4] = {co.x, co.y, co.z, co.w}, sn[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = y[4 * e4 + e], w = o[4 * e4 + e];
          y[4 * e4 + e] = low ? v * cc[e] - w * sn[e] : w * sn[e] + v * cc[e];
        }
      }
    }
  };

  // The key row into the cache: its values twice (largest, then codes) rather
  // than kept: 72 registers a lane would halve the rows in flight.
  if (a.kv) {
    const int32_t slot = live && key ? a.slot[tok] : -1;
    const bool cached = slot >= 0 && slot < a.num_slots;
    if (gl == 0 && !cached && slot != -1) report(a.dev_status, DSA_DEV_BAD_INDEX);
    float amax = 0.f;
    if (cached) {
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        const int c = gl + LPR * u;
        if (c >= nch) continue;
        float y[8];
        result(raw[u], c, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
      }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (cached) {
      const float scale = __fdiv_rn(amax, 448.0f);
      if (gl == 0) a.kv_scale[slot] = scale;
      uint8_t* dst = a.kv + (int64_t)slot * a.d;
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        const int c = gl + LPR * u;
        if (c >= nch) continue;
        uint32_t b[4] = {0u, 0u, 0u, 0u};
        if (scale > 0.f) {
          float y[8];
          result(raw[u], c, y);
#pragma unroll
          for (int t = 0; t < 4; ++t) b[t] = code2(__fdiv_rn(y[2 * t], scale), __fdiv_rn(y[2 * t + 1], scale));
        }
        *reinterpret_cast<uint2*>(dst + 8 * c) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
      }
    }
  }
  if (live && side.out) {
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int c = gl + LPR * u;
      if (c >= nch) continue;
      float y[8];
      result(raw[u], c, y);
      raw[u] = pack8<HALF>(y);
    }
  }
  __syncwarp();  // in place: every lane of the row has read its partner chunk
  if (live && side.out) {
    uint16_t* dst = static_cast<uint16_t*>(side.out) + ((int64_t)tok * side.heads + h) * a.d;
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int c = gl + LPR * u;
      if (c < nch) *reinterpret_cast<uint4*>(dst + 8 * c) = raw[u];
    }
  }
}

template <bool HALF, bool PAIRS, int LPR, int CH>
cudaError_t launch_shape(const NormRopeArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.num_tokens * (a.q.heads + a.k.heads);
  const int64_t per = NR_WARPS * (32 / LPR);
  const int64_t grid = (rows + per - 1) / per;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  qk_norm_rope_kernel<HALF, PAIRS, LPR, CH><<<(unsigned)grid, NR_WARPS * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

template <bool HALF, bool PAIRS>
cudaError_t launch_type(const NormRopeArgs& a, cudaStream_t stream) {
  const int nch = a.d / 8;
  if (nch <= 8) return launch_shape<HALF, PAIRS, 8, 1>(a, stream);
  if (nch <= 16) return launch_shape<HALF, PAIRS, 8, 2>(a, stream);
  if (nch <= 32) return launch_shape<HALF, PAIRS, 8, 4>(a, stream);
  if (nch <= 72) return launch_shape<HALF, PAIRS, 8, 9>(a, stream);
  return launch_shape<HALF, PAIRS, 32, 4>(a, stream);
}

}  // namespace

int norm_rope_max_d() { return 1024; }

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.dtype == DSA_FP16) return a.interleaved ? launch_type<true, true>(a, stream) : launch_type<true, false>(a, stream);
  return a.interleaved ? launch_type<false, true>(a, stream) : launch_type<false, false>(a, stream);
}

}  // namespace dsa
