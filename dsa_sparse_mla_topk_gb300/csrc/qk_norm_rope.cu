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
// one row as 16-byte chunks, chunk l + 8 u in lane l, so that a 576-value row has
// no idle lane (72 chunks, 9 a lane, all in flight together) and its sums take
// three shuffles instead of five; 2 to 4 heads of a token share a group's loads
// of position, rotation and weights.  Keys have CTAs of their own: no warp runs
// both sides' code.  In the half-split form a lane reads its partner chunk a
// second time (an L1 hit), unless both halves of its pairs are in the lane
// already.  Measured: 8,192 tokens of 64 x 576 + a key row into the cache 181 us,
// a copy's bandwidth; 4,099 tokens of 32 + 8 heads of 128 15.8 us, 80%, and 22 us with
// cold caches, where a plain copy of the 43 MB takes 29; 128 tokens of 64 x 576
// 6.5 us, 8.0 cold (the floor of its bytes is 2.8): latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.cuh"
#include "mla_tc_common.cuh"

namespace dsa {
namespace {

constexpr int NR_WARPS = 2;  // (8,192 tokens of 64 x 576: 4 warps a CTA 190 us, 2 184; 128 tokens 1 8.8, 2 7.8)

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
__device__ __forceinline__ void unpack8(const uint4 v, uint64_t (&x)[4]) {  // as packed pairs
  float f[8];
  unpack8<HALF>(v, f);
#pragma unroll
  for (int t = 0; t < 4; ++t) x[t] = pk2(f[2 * t], f[2 * t + 1]);
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
// (else halves).  LPR lanes per row, CH chunks of 8 values per lane, NR heads of
// one token per group of lanes: they share the loads of pos, cos_sin and the
// weights, and are in flight together.
// The first q_ctas CTAs take the queries, the rest the keys: no warp runs both
// sides' code.
template <bool HALF, bool PAIRS, int LPR, int CH, int NR>
__global__ void __launch_bounds__(NR_WARPS * 32, 16 / NR_WARPS)
    qk_norm_rope_kernel(const NormRopeArgs a, const unsigned q_ctas, const FastDiv q_div, const FastDiv k_div) {
  constexpr int GPW = 32 / LPR;  // groups per warp
  const int lane = threadIdx.x & 31, gl = lane & (LPR - 1);
  const bool key = blockIdx.x >= q_ctas;
  const NormRopeSide& side = key ? a.k : a.q;
  const int heads = side.heads;
  const int gt = (heads + NR - 1) / NR;  // groups per token
  const int64_t g64 = ((int64_t)(key ? blockIdx.x - q_ctas : blockIdx.x) * NR_WARPS + (threadIdx.x >> 5)) * GPW + lane / LPR;
  const bool in_range = g64 < (int64_t)a.num_tokens * gt;
  const int32_t g = in_range ? (int32_t)g64 : 0;
  const int32_t tok = key ? k_div(g) : q_div(g), h0 = (g - tok * gt) * NR;
  const int nch = a.d >> 3, rope0 = (a.d - a.d_rope) >> 3, half = a.d_rope >> 4, nn = side.norm_dim >> 3;
  const float* weight = side.weight;
  const uint16_t* x0 = static_cast<const uint16_t*>(side.x) + (int64_t)tok * side.tok_stride + (int64_t)h0 * side.head_stride;
  const int64_t hs = side.head_stride;

  int32_t p = -1;
  if (in_range) p = a.pos ? a.pos[tok] : 0;
  // the rows are read whatever the position turns out to be
  uint4 raw[NR][CH];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int c = gl + LPR * u;
      raw[r][u] = in_range && h0 + r < heads && c < nch ? *reinterpret_cast<const uint4*>(x0 + r * hs + 8 * c)
                                                        : make_uint4(0, 0, 0, 0);
    }
  }
  if (p >= a.max_pos || p < -1) {
    if (gl == 0) report(a.dev_status, DSA_DEV_BAD_QPOS);
    p = -1;
  }
  const bool live = p >= 0;  // a padding row, or a bad one, is left as it was
  const float* cs = a.cos_sin + (int64_t)(live ? p : 0) * a.d_rope;
  // The token's factors on their way while the rows arrive: in long calls (8,192 tokens of
  // 32 + 8 heads of 128 36.7 -> 34.3 us with cold caches, of 64 x 576 187 -> 184); in
  // short ones, a warp a row, the instructions cost more than they hide (128 tokens +0.1).
  if (LPR == 8 && live)
    for (int o = gl * 32; o < a.d_rope; o += LPR * 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(cs + o));
  float inv[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    uint64_t ss2 = pk2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      if (gl + LPR * u < nn) {
        uint64_t x[4];
        unpack8<HALF>(raw[r][u], x);
#pragma unroll
        for (int e = 0; e < 4; ++e) ss2 = fma2(x[e], x[e], ss2);
      }
    }
    float ss, s_odd;
    upk2(ss2, ss, s_odd);
    ss += s_odd;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    inv[r] = nn > 0 ? rsqrtf(ss / (float)side.norm_dim + a.eps) : 1.f;
  }

  auto load8 = [](const float* f, float (&v)[8]) {
    const float4 lo = *reinterpret_cast<const float4*>(f), hi = *reinterpret_cast<const float4*>(f + 4);
    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
  };
  // what the rows of a chunk c share: weights, and the rotation's factors
  struct Shared {
    float w[8], c[PAIRS ? 4 : 8], s[PAIRS ? 4 : 8];
    bool normed, rotated, low;
  };
  auto shared_of = [&](int c) {
    Shared t;
    t.normed = c < nn;
    t.rotated = a.d_rope > 0 && c >= rope0;
    t.low = false;
    if (t.normed) load8(weight + 8 * c, t.w);
    if (t.rotated) {
      if constexpr (PAIRS) {
        const float4 co = *reinterpret_cast<const float4*>(cs + 4 * (c - rope0));
        const float4 si = *reinterpret_cast<const float4*>(cs + a.d_rope / 2 + 4 * (c - rope0));
        t.c[0] = co.x, t.c[1] = co.y, t.c[2] = co.z, t.c[3] = co.w;
        t.s[0] = si.x, t.s[1] = si.y, t.s[2] = si.z, t.s[3] = si.w;
      } else {
        t.low = c - rope0 < half;  // this chunk holds the pairs' first values
        const int ic = t.low ? c - rope0 : c - rope0 - half;
        load8(cs + 8 * ic, t.c);
        load8(cs + a.d_rope / 2 + 8 * ic, t.s);
      }
    }
    return t;
  };
  // row r's chunk c of the result, in fp32
  auto result = [&](int r, const uint4 v, int c, const Shared& t, float (&y)[8]) {
    unpack8<HALF>(v, y);
    if (t.normed) {
      const uint64_t inv2 = pk2(inv[r], inv[r]);
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        upk2(mul2(mul2(pk2(y[e], y[e + 1]), inv2), pk2(t.w[e], t.w[e + 1])), y[e], y[e + 1]);
    }
    if (!t.rotated) return;
    if constexpr (PAIRS) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float va = y[2 * e], vb = y[2 * e + 1];
        y[2 * e] = va * t.c[e] - vb * t.s[e];
        y[2 * e + 1] = va * t.s[e] + vb * t.c[e];
      }
    } else {
      const int pc = t.low ? c + half : c - half;
      float o[8];
      unpack8<HALF>(*reinterpret_cast<const uint4*>(x0 + r * hs + 8 * pc), o);
      if (pc < nn) {
        float w[8];
        load8(weight + 8 * pc, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] * inv[r] * w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float b = o[e] * t.s[e];
        y[e] = fmaf(y[e], t.c[e], t.low ? -b : b);
      }
    }
  };

  // The key row into the cache: its values are computed twice (largest, then
  // codes) rather than kept: 72 registers a lane would halve the rows in flight.
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
        result(0, raw[0][u], c, shared_of(c), y);
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
          result(0, raw[0][u], c, shared_of(c), y);
#pragma unroll
          for (int t = 0; t < 4; ++t) b[t] = code2(__fdiv_rn(y[2 * t], scale), __fdiv_rn(y[2 * t + 1], scale));
        }
        *reinterpret_cast<uint2*>(dst + 8 * c) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
      }
    }
  }
  const bool store = live && side.out;
  // Halves that are both in this lane (the whole of a 128-value head): each pair
  // once, without reading the partner chunk again.
  bool paired = false;
  if constexpr (!PAIRS && CH == 2) paired = rope0 == 0 && half == LPR;
  if constexpr (!PAIRS && CH == 2) {
    if (store && paired) {
      Shared lo = shared_of(gl), hi;
      hi.normed = gl + LPR < nn;
      if (hi.normed) load8(weight + 8 * (gl + LPR), hi.w);
      lo.rotated = hi.rotated = false;  // result(): the norm alone
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (h0 + r >= heads) break;
        float x[8], y[8];
        result(r, raw[r][0], gl, lo, x);
        result(r, raw[r][1], gl + LPR, hi, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a0 = x[e], b0 = y[e];
          x[e] = a0 * lo.c[e] - b0 * lo.s[e];
          y[e] = a0 * lo.s[e] + b0 * lo.c[e];
        }
        raw[r][0] = pack8<HALF>(x);
        raw[r][1] = pack8<HALF>(y);
      }
    }
  }
  if (store && !paired) {
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int c = gl + LPR * u;
      if (c >= nch) continue;
      const Shared t = shared_of(c);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (h0 + r >= heads) break;
        float y[8];
        result(r, raw[r][u], c, t, y);
        raw[r][u] = pack8<HALF>(y);
      }
    }
  }
  __syncwarp();  // in place: every lane of the rows has read its partner chunks
  if (store) {
    uint16_t* dst = static_cast<uint16_t*>(side.out) + ((int64_t)tok * heads + h0) * a.d;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (h0 + r >= heads) break;
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        const int c = gl + LPR * u;
        if (c < nch) *reinterpret_cast<uint4*>(dst + (int64_t)r * a.d + 8 * c) = raw[r][u];
      }
    }
  }
}

template <bool HALF, bool PAIRS, int LPR, int CH, int NR>
cudaError_t launch_shape(const NormRopeArgs& a, cudaStream_t stream) {
  const int gq = (a.q.heads + NR - 1) / NR, gk = (a.k.heads + NR - 1) / NR;
  const int64_t per = NR_WARPS * (32 / LPR);
  const unsigned q_ctas = (unsigned)(((int64_t)a.num_tokens * gq + per - 1) / per);
  const unsigned k_ctas = (unsigned)(((int64_t)a.num_tokens * gk + per - 1) / per);
  qk_norm_rope_kernel<HALF, PAIRS, LPR, CH, NR><<<q_ctas + k_ctas, NR_WARPS * 32, 0, stream>>>(
      a, q_ctas, make_fast_div(gq > 0 ? gq : 1), make_fast_div(gk > 0 ? gk : 1));
  return cudaGetLastError();
}

template <bool HALF, bool PAIRS>
cudaError_t launch_type(const NormRopeArgs& a, cudaStream_t stream) {
  const int nch = a.d / 8;
  if (nch <= 8) return launch_shape<HALF, PAIRS, 8, 1, 4>(a, stream);
  if (nch <= 16) return launch_shape<HALF, PAIRS, 8, 2, 4>(a, stream);
  if (nch <= 32) return launch_shape<HALF, PAIRS, 8, 4, 2>(a, stream);
  if (nch <= 72) {
    // A warp a row while there are few rows, then a warp for the rows of four heads or
    // two (they share position, rotation and weights), and eight lanes a row once
    // bandwidth counts.  Tokens of 64 heads of 576, us:
    //                    1 row  4 rows  2 rows  8 lanes
    //     1 token          3.7     4.5     4.1      7.4
    //    64                5.3     5.4     5.1      7.8
    //   128                7.8     6.8     8.0      9.0
    //   320               13.4    13.6    12.5     15.2
    //   512               19.5    18.2    17.7     17.6
    // 8,192              302                      181
    const int64_t rows = (int64_t)a.num_tokens * (a.q.heads + a.k.heads), sms = device_sm_count();
    if (rows <= 32 * sms) return launch_shape<HALF, PAIRS, 32, 3, 1>(a, stream);
    if (rows <= 72 * sms) return launch_shape<HALF, PAIRS, 32, 3, 4>(a, stream);
    if (rows <= 200 * sms) return launch_shape<HALF, PAIRS, 32, 3, 2>(a, stream);
    return launch_shape<HALF, PAIRS, 8, 9, 2>(a, stream);
  }
  return launch_shape<HALF, PAIRS, 32, 4, 1>(a, stream);
}

}  // namespace

int norm_rope_max_d() { return 1024; }

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.dtype == DSA_FP16) return a.interleaved ? launch_type<true, true>(a, stream) : launch_type<true, false>(a, stream);
  return a.interleaved ? launch_type<false, true>(a, stream) : launch_type<false, false>(a, stream);
}

}  // namespace dsa
