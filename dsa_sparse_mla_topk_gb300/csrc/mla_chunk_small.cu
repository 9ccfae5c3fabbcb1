// Attention of a chunk of new tokens over every visible position of the paged
// FP8 cache, for the small head shape (16, 64, 16).
//
// "Accelerating GLM-5.3-Flash on H200", section 3: QK^T, online softmax and
// the weighted value sum one KV tile at a time, splits merged by a Combine
// step; "GLM-5.3 Optimizations, Part 2" ("Interpretation"): a latent KV row is
// shared by all heads.  For token i with request r and position p:
//   z_j = softmax_scale q . x_j,  x_j = e4m3(kv[slot_j]) s_j,  j = 0 .. p
//   out = sum_j softmax(z)_j x_j[:64],  lse = ln sum_j exp z_j
//
// 16 heads are the rows of one m16n8k16 warp MMA, a quarter of what one tcgen05
// instruction takes at least: a tile through shared memory, TMEM and their
// barriers would cost more than the products.  So each of a CTA's eight warps
// works by itself, on tiles of 32 rows that it loads straight into registers
// (one tile ahead), and the warps meet once, at the end.
// Fragments: lane (g, t) = (lane / 4, lane % 4) reads 20 bytes of row 8 u + g, the
// latent bytes 16 t .. + 15 and the rope bytes 4 t .. + 3.  The order of the
// contracted dims is free as long as Q has the same, so these bytes are the
// lane's B operands of S = Q K^T as they are (k index 2 t + e of step c is dim 16 t +
// 4 c + e, 8 + 2 t + e is dim 16 t + 4 c + 2 + e), and transposed by movmatrix those
// of O += P V; S's accumulators are P's A operands; a lane ends up with 16
// neighbouring dims of two heads.
// E4M3 is exact in fp16.  Q is too, but for values below 2^-29 of the token's largest
// (scaled to 2^14).  A weight is p s_j F in fp16 with F a power of two that puts the
// largest scale so far between 2^11 and 2^12: relative error 2^-11 down to 2^-25 of
// it.  l and both products are fp32, l from unrounded p.
// Measured: a step of the eight warps (256 rows) 1.1 us, one at a time on an SM, 2.0
// two at a time: 545 instructions a warp and tile and the waits of its chain
// (issue slots 47% busy), not the MMAs (26%).  107 tokens at the end of 12,733 positions 51 us (a CUDA-core kernel with
// the tile in shared memory: 395); 2 requests of 512 5.4 us, most of it launch.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.cuh"
#include "mla_tc_common.cuh"

namespace cg = cooperative_groups;

namespace dsa {
namespace {

constexpr int H = 16, DL = 64, DR = 16, DQK = DL + DR;
constexpr int WARPS = 8, NTHREADS = WARPS * 32;
constexpr int T = 32;                    // rows per tile, one a lane for the lookups
constexpr int NT = T / 8;                // MMA column blocks per tile
constexpr int KS = DQK / 16;             // MMA steps of a logit: 4 latent, 1 rope
constexpr int MAX_MERGED = chunk_max_merged();
constexpr int OSTR = DL + 4;             // floats per head of a warp's O (bank spread)
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // of the 8 x 8 matrix of 16-bit values in a warp
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t two) {  // the two codes in the low 16 bits
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}

// MERGE: a token's splits are the CTAs of a thread-block cluster and merge
// their results over distributed shared memory (no partials, no Combine kernel).
// PER_SM: CTAs that an SM holds, 2 at 128 registers (which spill a little), 1 without.
template <bool MERGE, int PER_SM>
__global__ void __launch_bounds__(NTHREADS, PER_SM)
    mla_chunk_small_kernel(const MlaArgs a, const int32_t* __restrict__ q_pos, const FastDiv page_div) {
  __shared__ __align__(16) float o_s[WARPS][H][OSTR];
  __shared__ float m_s[WARPS][H], l_s[WARPS][H];
  __shared__ __align__(16) float oc_s[H][DL];  // MERGE: the CTA's O, reference and l
  __shared__ float mc_s[H], lc_s[H];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  // the last tokens first: in a causal chunk they see the most
  const int i = (int)gridDim.x - 1 - (int)blockIdx.x;
  const int split = blockIdx.y, S = gridDim.y;
  const int P = a.page_size;
  const int32_t r = a.q_req[i], last = q_pos[i];
  const bool req_ok = r >= 0 && r < a.num_req;
  const bool pos_ok = last >= -1 && last <= INT32_MAX - T && page_div(max(last, 0)) < a.bt_stride;
  if (tid == 0) {
    if (!req_ok && r != -1) report(a.dev_status, DSA_DEV_BAD_PAGE);
    if (req_ok && !pos_ok) report(a.dev_status, DSA_DEV_BAD_QPOS);
  }
  const int n = req_ok && pos_ok ? last + 1 : 0;  // visible positions
  const int ntiles = (n + T - 1) / T;
  const int t_begin = (int)((int64_t)ntiles * split / S), t_end = (int)((int64_t)ntiles * (split + 1) / S);
  const int32_t* bt = a.block_table + (int64_t)(req_ok ? r : 0) * a.bt_stride;

  // a tile's rows: page ids, then slots, lane l for row l (-1: none).  Whether a row is
  // there at all goes by its position: a page id may be any number.
  auto has_row = [&](int tile) { return tile < t_end && tile * T + lane < n; };
  auto page_of = [&](int tile) -> int { return has_row(tile) ? __ldg(bt + page_div(tile * T + lane)) : -1; };
  auto slot_of = [&](int tile, int page) -> int {
    if (page >= 0 && page < a.num_pages) {
      const int pos = tile * T + lane;
      return page * P + (pos - page_div(pos) * P);
    }
    if (has_row(tile)) report(a.dev_status, DSA_DEV_BAD_PAGE);
    return -1;
  };
  struct Rows {
    uint4 lat[NT];
    uint32_t rope[NT];
  };
  auto load = [&](int slot, Rows& x) {
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int s = __shfl_sync(0xffffffffu, slot, 8 * u + g);
      x.lat[u] = make_uint4(0u, 0u, 0u, 0u);
      x.rope[u] = 0u;
      if (s >= 0) {
        const uint8_t* row = a.kv + (int64_t)s * DQK;
        x.lat[u] = __ldg(reinterpret_cast<const uint4*>(row + 16 * t));
        x.rope[u] = __ldg(reinterpret_cast<const uint32_t*>(row + DL + 4 * t));
      }
    }
  };
  const int first = t_begin + warp;
  int slot1 = slot_of(first, page_of(first));  // of the tile whose rows are loaded next
  int page2 = page_of(first + WARPS);

  // ---- Q: heads g and g + 8, this lane's dims, fp16 at 2^14 below its largest value ----
  uint32_t qa[KS][4];
  float qk_scale;
  {
    uint32_t w[2][2 * KS];  // bf16 pairs
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)i * H * DQK;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_bfloat16* row = q + (g + 8 * h) * DQK;
      const uint4 x = *reinterpret_cast<const uint4*>(row + 16 * t), y = *reinterpret_cast<const uint4*>(row + 16 * t + 8);
      const uint2 z = *reinterpret_cast<const uint2*>(row + DL + 4 * t);
      w[h][0] = x.x, w[h][1] = x.y, w[h][2] = x.z, w[h][3] = x.w, w[h][4] = y.x, w[h][5] = y.y, w[h][6] = y.z;
      w[h][7] = y.w, w[h][8] = z.x, w[h][9] = z.y;
    }
    uint32_t mx = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < 2 * KS; ++c) mx = max(mx, max((w[h][c] << 16) & 0x7fffffffu, w[h][c] & 0x7fff0000u));
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (mx >= 0x7f800000u) {  // infinities become NaN, the largest finite value counts
      mx = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2 * KS; ++c) {
          uint32_t& v = w[h][c];
          if ((v & 0x7fffu) >= 0x7f80u) v |= 0x7fffu;
          else mx = max(mx, (v << 16) & 0x7fffffffu);
          if ((v & 0x7fff0000u) >= 0x7f800000u) v |= 0x7fff0000u;
          else mx = max(mx, v & 0x7fff0000u);
        }
      mx = __reduce_max_sync(0xffffffffu, mx);
    }
    int e = 0;
    if (mx != 0) frexpf(__uint_as_float(mx), &e);  // the largest |q| < 2^e
    const int qexp = mx != 0 ? min(14 - e, 100) : 0;
    const float qs = ldexpf(1.f, qexp);
#pragma unroll
    for (int c = 0; c < KS; ++c)
#pragma unroll
      for (int x = 0; x < 4; ++x) {  // (heads g, g + 8) x (pairs 0, 1)
        const uint32_t v = w[x & 1][2 * c + (x >> 1)];
        const __half2 y = __floats2half2_rn(__uint_as_float(v << 16) * qs, __uint_as_float(v & 0xffff0000u) * qs);
        qa[c][x] = *reinterpret_cast<const uint32_t*>(&y);
      }
    qk_scale = a.softmax_scale * LOG2E * ldexpf(1.f, -qexp);
  }

  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};  // heads g, g + 8; l: this lane's share
  float o[2 * (KS - 1)][4];  // [2 c + half]: heads g, g + 8 x dims 16 t + 4 c + 2 half + {0, 1}
#pragma unroll
  for (int c = 0; c < 2 * (KS - 1); ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
  int pe = 0;           // log2 F
  float p_scale = 1.f;  // F
  bool p_set = false;

  Rows next;
  load(slot1, next);
  float sc1 = slot1 >= 0 ? __ldg(a.kv_scale + slot1) : 0.f;
  for (int tile = first; tile < t_end; tile += WARPS) {
    const Rows x = next;
    const int slot = slot1;
    const float sc = sc1;
    slot1 = slot_of(tile + WARPS, page2);
    page2 = page_of(tile + 2 * WARPS);
    load(slot1, next);
    sc1 = slot1 >= 0 ? __ldg(a.kv_scale + slot1) : 0.f;

    uint32_t kf[NT][KS][2];
    float z[NT][4];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const uint32_t w[KS] = {x.lat[u].x, x.lat[u].y, x.lat[u].z, x.lat[u].w, x.rope[u]};
      z[u][0] = z[u][1] = z[u][2] = z[u][3] = 0.f;
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        kf[u][c][0] = half2_of_e4m3(w[c] & 0xffffu);
        kf[u][c][1] = half2_of_e4m3(w[c] >> 16);
        mma16816(z[u], qa[c], kf[u][c][0], kf[u][c][1]);
      }
    }
    const unsigned valid = __ballot_sync(0xffffffffu, slot >= 0);
    const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(sc))));
    float sj[NT][2];
    float tm[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * u + 2 * t + e;
        sj[u][e] = __shfl_sync(0xffffffffu, sc, row);
        const bool in = (valid >> row) & 1u;
        z[u][e] = in ? z[u][e] * sj[u][e] * qk_scale : -INFINITY;
        z[u][2 + e] = in ? z[u][2 + e] * sj[u][e] * qk_scale : -INFINITY;
        tm[0] = fmaxf(tm[0], z[u][e]);
        tm[1] = fmaxf(tm[1], z[u][2 + e]);
      }
    }
    float alpha[2];
    bool move = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 1));
      tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 2));
      const float mn = fmaxf(m_run[h], tm[h]);
      alpha[h] = m_run[h] == -INFINITY ? 0.f : ex2(m_run[h] - mn);
      move |= mn != m_run[h];
      m_run[h] = mn;
    }
    float f = 1.f;  // (the same in every lane, as `top` is)
    if (top > 0.f && top <= 3.0e38f && (!p_set || top * p_scale >= 4096.f)) {
      int e;
      frexpf(top, &e);  // top < 2^e: top F in [2^11, 2^12)
      e = min(12 - e, 80);
      f = ldexpf(1.f, e - pe);
      pe = e;
      p_set = true;
      p_scale = ldexpf(1.f, pe);
    }
    if (__any_sync(0xffffffffu, move) || f != 1.f) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float al = alpha[h];
        l_run[h] *= al;
#pragma unroll
        for (int c = 0; c < 2 * (KS - 1); ++c) o[c][2 * h] *= al * f, o[c][2 * h + 1] *= al * f;
      }
    }
    const float ref[2] = {m_run[0] == -INFINITY ? 0.f : m_run[0], m_run[1] == -INFINITY ? 0.f : m_run[1]};
#pragma unroll
    for (int kb = 0; kb < NT / 2; ++kb) {  // 16 rows
      uint32_t pa[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {  // (heads g, g + 8) x (rows 2 t + e, 8 + 2 t + e)
        const int u = 2 * kb + (v >> 1), h = v & 1;
        const float p0 = ex2(z[u][2 * h] - ref[h]), p1 = ex2(z[u][2 * h + 1] - ref[h]);
        l_run[h] += p0 + p1;
        const __half2 y = __floats2half2_rn(p0 * (sj[u][0] * p_scale), p1 * (sj[u][1] * p_scale));
        pa[v] = *reinterpret_cast<const uint32_t*>(&y);
      }
#pragma unroll
      for (int c = 0; c < 2 * (KS - 1); ++c)
        mma16816(o[c], pa, transposed(kf[2 * kb][c >> 1][c & 1]), transposed(kf[2 * kb + 1][c >> 1][c & 1]));
    }
  }

  // ---- the warps' results together: out = sum_w 2^(m_w - m) O_w / sum_w 2^(m_w - m) l_w ----
  const float unscale = ldexpf(1.f, -pe);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 1);
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 2);
    if (t == 0) m_s[warp][g + 8 * h] = m_run[h], l_s[warp][g + 8 * h] = l_run[h];
#pragma unroll
    for (int c = 0; c < KS - 1; ++c)
      *reinterpret_cast<float4*>(&o_s[warp][g + 8 * h][16 * t + 4 * c]) =
          make_float4(o[2 * c][2 * h] * unscale, o[2 * c][2 * h + 1] * unscale, o[2 * c + 1][2 * h] * unscale,
                      o[2 * c + 1][2 * h + 1] * unscale);
  }
  __syncthreads();
  const int hh = tid >> 4, d = 4 * (tid & 15);  // four values of one head
  static_assert(NTHREADS == H * DL / 4, "one float4 of the token's result a thread");
  float m = -INFINITY, l = 0.f;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) m = fmaxf(m, m_s[w][hh]);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const float k = m_s[w][hh] == -INFINITY ? 0.f : ex2(m_s[w][hh] - m);
    const float4 v = *reinterpret_cast<const float4*>(&o_s[w][hh][d]);
    l = fmaf(k, l_s[w][hh], l);
    s.x = fmaf(k, v.x, s.x), s.y = fmaf(k, v.y, s.y), s.z = fmaf(k, v.z, s.z), s.w = fmaf(k, v.w, s.w);
  }
  if constexpr (MERGE) {
    cg::cluster_group cluster = cg::this_cluster();
    *reinterpret_cast<float4*>(&oc_s[hh][d]) = s;
    if (d == 0) mc_s[hh] = m, lc_s[hh] = l;
    cluster.sync();
    // each CTA a share of the token's values
    const int share = (NTHREADS + S - 1) / S, e = split * share + tid;
    if (tid < share && e < NTHREADS) {
      const int h = e >> 4, c = 4 * (e & 15);
      float mk[MAX_MERGED], lk[MAX_MERGED];  // (all the remote loads together)
      float4 vk[MAX_MERGED];
#pragma unroll
      for (int k = 0; k < MAX_MERGED; ++k) {
        mk[k] = k < S ? *cluster.map_shared_rank(&mc_s[h], k) : -INFINITY;
        lk[k] = k < S ? *cluster.map_shared_rank(&lc_s[h], k) : 0.f;
        vk[k] = k < S ? *reinterpret_cast<const float4*>(cluster.map_shared_rank(&oc_s[h][c], k)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      m = -INFINITY, l = 0.f, s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < MAX_MERGED; ++k) m = fmaxf(m, mk[k]);
#pragma unroll
      for (int k = 0; k < MAX_MERGED; ++k) {
        const float w = mk[k] == -INFINITY ? 0.f : ex2(mk[k] - m);
        const float4 v = vk[k];
        l = fmaf(w, lk[k], l);
        s.x = fmaf(w, v.x, s.x), s.y = fmaf(w, v.y, s.y), s.z = fmaf(w, v.z, s.z), s.w = fmaf(w, v.w, s.w);
      }
      const float inv = l != 0.f ? 1.f / l : 0.f;
      __nv_bfloat162* ob = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + ((int64_t)i * H + h) * DL + c);
      ob[0] = __floats2bfloat162_rn(s.x * inv, s.y * inv);
      ob[1] = __floats2bfloat162_rn(s.z * inv, s.w * inv);
      if (a.lse && c == 0) a.lse[(int64_t)i * H + h] = l != 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
    }
    cluster.sync();  // no CTA leaves while another reads its shared memory
  } else {
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const float lse = l != 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
    if (S == 1) {
      __nv_bfloat162* ob = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + ((int64_t)i * H + hh) * DL + d);
      ob[0] = __floats2bfloat162_rn(s.x * inv, s.y * inv);
      ob[1] = __floats2bfloat162_rn(s.z * inv, s.w * inv);
      if (a.lse && d == 0) a.lse[(int64_t)i * H + hh] = lse;
    } else {
      const int64_t row = ((int64_t)split * a.num_q + i) * H + hh;
      *reinterpret_cast<float4*>(a.o_part + row * DL + d) = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
      if (d == 0) a.lse_part[row] = lse;
    }
  }
}

}  // namespace

cudaError_t launch_chunk_small(const MlaArgs& a, const int32_t* q_pos, bool merge, cudaStream_t stream) {
  if (a.num_q == 0) return cudaSuccess;
  if (a.heads != H || a.d_latent != DL || a.d_rope != DR) return cudaErrorInvalidValue;
  auto launch = [&](auto kern) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = merge ? (unsigned)a.num_splits : 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.num_q, a.num_splits);
    cfg.blockDim = dim3(NTHREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = merge ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, q_pos, make_fast_div(a.page_size));
    return e != cudaSuccess ? e : cudaGetLastError();
  };
  // Two CTAs on an SM as soon as there is more than one each (16 x 128 tokens of 4,096
  // positions 243 us, one at a time 276); one that is alone runs faster with all the
  // registers (one token of 16,384 positions 73 us, 91 with half of them).
  if ((int64_t)a.num_q * a.num_splits > device_sm_count())
    return merge ? launch(mla_chunk_small_kernel<true, 2>) : launch(mla_chunk_small_kernel<false, 2>);
  return merge ? launch(mla_chunk_small_kernel<true, 1>) : launch(mla_chunk_small_kernel<false, 1>);
}

}  // namespace dsa
