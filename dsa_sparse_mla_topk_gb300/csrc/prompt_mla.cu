// Attention of new tokens over every head's own keys and values: latent
// attention's expanded form, for prompts and their chunks (tcgen05 + TMEM + TMA).
//
//   z_j = scale (q_n . k_j + q_r . k_rope_j),  j = 0 .. q_pos of the token's request
//   out = sum_j softmax(z)_j v_j,  lse = ln sum_j exp z_j
//
// The running maximum and sum of a softmax in one pass over the rows: with a
// reference m for each query row, p = 2^(c (s - m)), c = scale log2 e, l = sum p, O =
// sum p v; when m moves by d, l and O take the factor 2^(-c d).
//
// One CTA = one head, 256 tokens of one request (two tiles of 128 query rows) and one
// share of its rows, 128 rows a tile.  TMEM: S of both query tiles (2 x 128 columns;
// the weights P, bf16, take their place) and O (2 x 128).  Warps:
//  * 0-3 and 4-7: softmax of query tile 0 and 1, one query row a thread.  S comes into
//    registers once; a row's O is rescaled only when its maximum has risen by more
//    than 2^8 (weights stay below 2^8, sums far inside fp32).
//  * 8: TMA.  A tile's key is two 64-column chunks of the head's own and one of the
//    shared rotated part (never copied to the heads), its value two; four key chunks and
//    two value tiles in flight.
//  * 9: MMA.  P V of one query tile, then its next Q K^T, then the other's: one tile's
//    softmax runs under the other's products.
//  * 10, 11: values that are NaN or infinite are taken out of tiles that some query row
//    sees only in part (a weight of 0 would turn them into NaN); the few rows that do
//    see them look them up again at the end.
// All waits are bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.cuh"
#include "mla_tc_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int TQ = 128, QT = 2 * TQ;  // query rows of a tile, of a CTA
constexpr int TK = 128;               // rows of a key tile
constexpr int CHUNK = 128 * 128;      // 128 rows x 64 columns of bf16, 128-byte swizzle
constexpr int KSLOTS = 4, VST = 2;    // key chunks and value tiles in flight
constexpr int THREADS = 384, SM_WARPS = 8, WARP_TMA = 8, WARP_MMA = 9, WARP_FIX = 10;
// 384 threads at 168 registers: 2 x 128 x 200 + 128 x 104 = 384 x 168
constexpr int REGS_SOFTMAX = 200, REGS_OTHER = 104;
static_assert(128 * (2 * REGS_SOFTMAX + REGS_OTHER) <= THREADS * 168, "no more registers than at launch");
constexpr float LOG2E = 1.4426950408889634f;
constexpr float RISE = 8.f;  // a reference moves when a weight would pass 2^RISE

constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;  // query tile g at + 128 g

constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + 2 * 3 * CHUNK;
constexpr int OFF_V = OFF_K + KSLOTS * CHUNK;
constexpr int OFF_BAR = OFF_V + VST * 2 * CHUNK;
constexpr int B_QF = 0;              // [2] query tile g has landed
constexpr int B_KF = B_QF + 2;       // [KSLOTS] key chunk has landed
constexpr int B_KE = B_KF + KSLOTS;  // [KSLOTS] its slot is free
constexpr int B_VF = B_KE + KSLOTS;  // [VST]
constexpr int B_VE = B_VF + VST;     // [VST]
constexpr int B_VX = B_VE + VST;     // [VST] the value tile has been looked through
constexpr int B_GO = B_VX + VST;     // [VST] a value tile to look through is on its way
constexpr int B_SF = B_GO + VST;     // [2] S of query tile g is complete
constexpr int B_PF = B_SF + 2;       // [2] P is written (and O rescaled)
constexpr int B_PVD = B_PF + 2;      // [2] P V is done
constexpr int NBAR = B_PVD + 2;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
struct Misc {
  int32_t req, q0, rows, any_bad;
  int32_t wsum[12], wmax[SM_WARPS], wmin[SM_WARPS];
  uint32_t tmem;
};
constexpr int SMEM_BYTES = OFF_MISC + (int)sizeof(Misc) + 1024;  // with alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

struct PromptMaps {
  CUtensorMap q, kv, rope;  // boxes of 64 columns, one head, 128 rows
};

// The tile that this CTA takes: the requests' tiles of QT tokens one after another, then
// the padding's (req -1), in `index` order; req -2: none.
__device__ __forceinline__ void find_tile(const PromptArgs& a, int index, bool tell, Misc* misc) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.num_req + THREADS - 1) / THREADS, r0 = min(tid * per, a.num_req), r1 = min(r0 + per, a.num_req);
  auto tiles_of = [&](int r, int& q0, int& n) {
    q0 = __ldg(a.cu_q + r);
    const int q1 = __ldg(a.cu_q + r + 1);
    const bool good = q0 >= 0 && q1 >= q0 && q1 <= a.num_tokens;
    n = good ? q1 - q0 : 0;
    if (!good && tell) report(a.dev_status, DSA_DEV_BAD_INDEX);
    return (n + QT - 1) / QT;
  };
  int mine = 0, q0, n;
  for (int r = r0; r < r1; ++r) mine += tiles_of(r, q0, n);
  mine = min(mine, (int)gridDim.x);  // (ranges that overlap, an error, could add up past 32 bits)
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) misc->wsum[warp] = inc;
  if (tid == 0) misc->req = -2, misc->any_bad = 0;
  __syncthreads();
  int all = 0, first = inc - mine;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) first += misc->wsum[w];
    all += misc->wsum[w];
  }
  if (index >= first && index < first + mine) {
    int left = index - first;
    for (int r = r0; r < r1; ++r) {
      const int t = tiles_of(r, q0, n);
      if (left < t) {
        misc->req = r, misc->q0 = q0 + left * QT, misc->rows = min(QT, n - left * QT);
        break;
      }
      left -= t;
    }
  } else if (index >= all && tid == 0) {
    const int pad0 = a.num_req > 0 ? min(max(__ldg(a.cu_q + a.num_req), 0), a.num_tokens) : 0;
    const int64_t at = pad0 + (int64_t)(index - all) * QT;
    if (at < a.num_tokens) misc->req = -1, misc->q0 = (int)at, misc->rows = (int)min((int64_t)QT, a.num_tokens - at);
  }
  __syncthreads();
}

// Results of a row that sees nothing in this share.
__device__ __forceinline__ void write_nothing(const PromptArgs& a, int64_t row, int split, int lane, int lanes) {
  const int64_t part = (int64_t)split * a.num_tokens * a.heads + row;
  const bool whole = a.num_splits == 1;
  char* dst = whole ? static_cast<char*>(a.out) + row * a.d_v * 2 : reinterpret_cast<char*>(a.o_part) + part * a.d_v * 4;
  const int chunks = a.d_v * (whole ? 2 : 4) / 16;
  for (int c = lane; c < chunks; c += lanes) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
  if (lane == 0) {
    if (!whole) a.lse_part[part] = -INFINITY;
    else if (a.lse) a.lse[row] = -INFINITY;
  }
}

// STD: head widths 128 + 64 (rotated) and values of 128, known to the compiler.
template <bool STD>
__global__ void __launch_bounds__(THREADS, 1) prompt_mla_kernel(const PromptArgs a, const __grid_constant__ PromptMaps maps) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  Misc* misc = reinterpret_cast<Misc*>(smem + OFF_MISC);
  auto bar = [&](int b) { return smem_u32(bars + b); };
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int dn = STD ? 128 : a.d_nope, dr = STD ? 64 : a.d_rope, dv = STD ? 128 : a.d_v;
  const int h = blockIdx.y, split = blockIdx.z, S = a.num_splits;

  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(&misc->tmem), TM_COLS);
    tmem_relinquish();
  }
  if (tid == WARP_TMA * 32) {
    for (int b = 0; b < NBAR; ++b) mbar_init(bar(b), b >= B_PF && b < B_PF + 2 ? 4u : b >= B_VX && b < B_VX + VST ? 2u : 1u);
    fence_mbarrier_init();
    tma_prefetch_map(&maps.q);
    tma_prefetch_map(&maps.kv);
    tma_prefetch_map(&maps.rope);
  }
  // the last tiles first: in causal prompts they see the most
  const int index = (int)gridDim.x - 1 - (int)blockIdx.x;
  find_tile(a, index, blockIdx.x == 0 && h == 0 && split == 0, misc);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const int req = misc->req, q0 = misc->q0, rows = misc->rows;
  const uint32_t tmem = misc->tmem;

  // ---- what each row sees ----
  int k0 = 0, kv_len = 0;
  if (req >= 0) {
    k0 = __ldg(a.cu_k + req);
    const int k1 = __ldg(a.cu_k + req + 1);
    if (k0 >= 0 && k1 >= k0 && k1 <= a.num_rows) kv_len = k1 - k0;
    else if (tid == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);
  }
  int last = -1;  // this thread's query row (softmax warps: row tid)
  if (tid < QT) {
    if (req >= 0 && tid < rows) {
      last = __ldg(a.q_pos + q0 + tid);
      if (last < -1 || last >= kv_len) {
        report(a.dev_status, DSA_DEV_BAD_QPOS);
        last = -1;
      }
    }
    const int mx = __reduce_max_sync(0xffffffffu, last), mn = __reduce_min_sync(0xffffffffu, tid < rows ? last : INT32_MAX);
    if (lane == 0) misc->wmax[warp] = mx, misc->wmin[warp] = mn;
  }
  __syncthreads();
  int n_g[2], full_g[2];  // tiles that some row of query tile g sees, that all see whole
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    int mx = -1, mn = INT32_MAX;
#pragma unroll
    for (int w = 0; w < 4; ++w) mx = max(mx, misc->wmax[4 * g + w]), mn = min(mn, misc->wmin[4 * g + w]);
    n_g[g] = (mx + TK) / TK;  // ceil((mx + 1) / TK)
    full_g[g] = mn == INT32_MAX ? 0 : (mn + 1) / TK;
  }
  const int ntiles = max(n_g[0], n_g[1]);
  const int t_begin = (int)((int64_t)ntiles * split / S), t_end = (int)((int64_t)ntiles * (split + 1) / S);
  const int cnt0 = max(0, min(t_end, n_g[0]) - t_begin), cnt1 = max(0, min(t_end, n_g[1]) - t_begin);
  const int cnt = __reduce_max_sync(0xffffffffu, max(cnt0, cnt1));
  // local tiles from here on may be seen in part by some row
  const int fix0 = max(0, min(cnt0 > 0 ? full_g[0] : INT32_MAX, cnt1 > 0 ? full_g[1] : INT32_MAX) - t_begin);
  const int nn = (dn + 63) / 64, nk = nn + (dr > 0 ? 1 : 0), nv = (dv + 63) / 64;
  bool ok = true;

  if (cnt == 0) {
    if (req != -2)
      for (int i = warp; i < rows; i += THREADS / 32) write_nothing(a, (int64_t)(q0 + i) * a.heads + h, split, lane, 32);
  } else if (warp >= SM_WARPS) {
    reg_less<REGS_OTHER>();
    if (warp == WARP_TMA) {
      // ---------------- TMA warp ----------------
      if (lane == 0) {
        auto query = [&](int g) {
          mbar_arrive_expect_tx(bar(B_QF + g), nk * CHUNK);
          for (int c = 0; c < nk; ++c)
            tma_load_3d(smem_u32(smem + OFF_Q + (3 * g + c) * CHUNK), &maps.q, c < nn ? 64 * c : dn, h, q0 + TQ * g,
                        bar(B_QF + g));
        };
        int slot = 0, phase = 0;  // of the next key chunk
        for (int lt = 0; lt < cnt && ok; ++lt) {
          if (lt == 0 && cnt0 > 0) query(0);
          const int n0 = k0 + (t_begin + lt) * TK;
          for (int c = 0; c < nk; ++c) {
            if (!mbar_wait(bar(B_KE + slot), phase ^ 1)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(bar(B_KF + slot), CHUNK);
            const uint32_t dst = smem_u32(smem + OFF_K + slot * CHUNK);
            if (c < nn) tma_load_3d(dst, &maps.kv, 64 * c, h, n0, bar(B_KF + slot));
            else tma_load_3d(dst, &maps.rope, 0, 0, n0, bar(B_KF + slot));
            if (++slot == KSLOTS) slot = 0, phase ^= 1;
          }
          if (lt == 0 && cnt1 > 0) query(1);
          const int s = lt % VST;
          if (!ok || !mbar_wait(bar(B_VE + s), ((lt / VST) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (lt >= fix0) mbar_arrive(bar(B_GO + s));
          mbar_arrive_expect_tx(bar(B_VF + s), nv * CHUNK);
          for (int c = 0; c < nv; ++c)
            tma_load_3d(smem_u32(smem + OFF_V + (2 * s + c) * CHUNK), &maps.kv, dn + 64 * c, h, n0, bar(B_VF + s));
        }
        if (!ok) {  // no copy may land after the CTA is gone
          for (int g = 0; g < 2; ++g)
            if (g ? cnt1 > 0 : cnt0 > 0) mbar_wait(bar(B_QF + g), 0);
          for (int s = 0; s < KSLOTS; ++s) mbar_wait(bar(B_KF + s), s < slot ? phase : phase ^ 1);
        }
      }
      __syncwarp();
    } else if (warp == WARP_MMA) {
      // ---------------- MMA warp ----------------
      const uint32_t ID_QK = idesc_f16_f32(TQ, TK, 0, 0, 1);
      const uint32_t ID_PV = STD ? idesc_f16_f32(TQ, 128, 0, 1, 1) : idesc_f16_f32(TQ, dv, 0, 1, 1);
      auto wait_u = [&](int b, uint32_t parity) { return __reduce_min_sync(0xffffffffu, (uint32_t)mbar_wait(bar(b), parity)); };
      const uint64_t q_desc = smem_desc(smem_u32(smem + OFF_Q), 16, 1024, SWIZZLE_128B);
      const uint64_t k_desc = smem_desc(smem_u32(smem + OFF_K), 16, 1024, SWIZZLE_128B);
      const uint64_t v_desc = smem_desc(smem_u32(smem + OFF_V), CHUNK, 1024, SWIZZLE_128B);
      const int c0 = __reduce_max_sync(0xffffffffu, cnt0), c1 = __reduce_max_sync(0xffffffffu, cnt1);
      const int fix = __reduce_max_sync(0xffffffffu, fix0);
      uint32_t good = __reduce_min_sync(0xffffffffu, (uint32_t)(tmem == 0));
      int slot = 0, phase = 0;  // of the first key chunk of the tile to come
      // S_g = Q_g K^T; the last of the tile's users frees its chunks
      auto issue_qk = [&](int g, bool first_user, bool last_user) {
        int s = slot, ph = phase;
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (c < nk && good) {
            if (first_user) {
              good = wait_u(B_KF + s, ph);
              tc_fence_after_sync();
            }
            const uint64_t qa = q_desc + (uint32_t)((3 * g + c) * (CHUNK >> 4)), kb = k_desc + (uint32_t)(s * (CHUNK >> 4));
            const int steps = STD ? 4 : (c < nn ? min(4, (dn - 64 * c) / 16) : dr / 16);
            if (good) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (STD || kk < steps) mma_f16_ss_warp(TM_S + 128 * g, qa + 2 * kk, kb + 2 * kk, ID_QK, c | kk ? 1u : 0u);
              if (last_user) mma_commit_warp(bar(B_KE + s));
            }
            if (++s == KSLOTS) s = 0, ph ^= 1;
          }
        }
        if (good) mma_commit_warp(bar(B_SF + g));
        if (last_user) slot = s, phase = ph;
      };
      auto issue_pv = [&](int g, int lt, bool last_user) {
        const uint64_t vb = v_desc + (uint32_t)((lt % VST) * (2 * CHUNK >> 4));
#pragma unroll
        for (int kk = 0; kk < TK / 16; ++kk)
          mma_f16_ts_warp(TM_O + 128 * g, TM_S + 128 * g + 8 * kk, vb + 128 * kk, ID_PV, lt > 0 || kk > 0 ? 1u : 0u);
        mma_commit_warp(bar(B_PVD + g));
        if (last_user) mma_commit_warp(bar(B_VE + lt % VST));
      };
      if (c0 > 0 && good) {
        good = wait_u(B_QF, 0);
        issue_qk(0, true, c1 == 0);
      }
      if (c1 > 0 && good) {
        good = wait_u(B_QF + 1, 0);
        tc_fence_after_sync();
        issue_qk(1, c0 == 0, true);
      }
      for (int lt = 0; lt < cnt && good; ++lt) {
        good = wait_u(B_VF + lt % VST, (lt / VST) & 1);
        if (lt >= fix && good) good = wait_u(B_VX + lt % VST, ((lt - fix) / VST) & 1);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int mine = g ? c1 : c0, other = g ? c0 : c1;
          if (lt < mine && good) {
            good = wait_u(B_PF + g, lt & 1);
            tc_fence_after_sync();
            if (good) {
              issue_pv(g, lt, g == 1 || lt >= other);
              if (lt + 1 < mine) issue_qk(g, g == 0 || lt + 1 >= other, g == 1 || lt + 1 >= other);
            }
          }
        }
      }
      if (!good) ok = false;
    } else {
      // ---------------- values that are not finite ----------------
      const int t = tid - WARP_FIX * 32;  // rows t and t + 64 of a tile
      for (int lt = fix0; lt < cnt; ++lt) {
        const int s = lt % VST;
        // (B_VF alone would not do: a wait on a barrier whose phase before the one that is meant
        // has not ended returns at once)
        if (!__all_sync(0xffffffffu, mbar_wait(bar(B_GO + s), ((lt - fix0) / VST) & 1) &&
                                         mbar_wait(bar(B_VF + s), (lt / VST) & 1))) {
          ok = false;
          break;
        }
        for (int half = 0; half < 2; ++half) {
          unsigned char* row = smem + OFF_V + 2 * s * CHUNK + (t + 64 * half) * 128;
          uint32_t odd = 0;
          for (int c = 0; c < nv; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // (every lane at another bank; the order does not matter)
              const uint4 v = *reinterpret_cast<const uint4*>(row + c * CHUNK + 16 * ((e + lane) & 7));
              // an exponent of ones carries into the sign's place
              auto look = [&](uint32_t w) { odd |= (w & 0x7f807f80u) + 0x00800080u; };
              look(v.x), look(v.y), look(v.z), look(v.w);
            }
          if (odd & 0x80008000u) {
            for (int c = 0; c < nv; ++c)
              for (int e = 0; e < 64; ++e) {
                uint16_t* v = reinterpret_cast<uint16_t*>(row + c * CHUNK) + e;
                if ((*v & 0x7f80u) == 0x7f80u) *v = 0;
              }
            misc->any_bad = 1;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_VX + s));
      }
    }
  } else {
    // ---------------- softmax warps ----------------
    reg_more<REGS_SOFTMAX>();
    const int g = warp >> 2, mine = g ? cnt1 : cnt0;
    const int whole = max(0, (g ? full_g[1] : full_g[0]) - t_begin);  // local tiles that all rows see whole
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, ts = TM_S + 128 * g + lanes, to = TM_O + 128 * g + lanes;
    const float c = fmaxf(a.softmax_scale * LOG2E, 0x1p-120f);  // (0 would make NaN of masked logits)
    float m = -INFINITY;
    uint64_t l2 = 0;
    for (int lt = 0; lt < mine; ++lt) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_SF + g), lt & 1))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      float s[TK];
#pragma unroll
      for (int b = 0; b < 4; ++b) tmem_ld32(ts + 32 * b, *reinterpret_cast<float(*)[32]>(s + 32 * b));
      tmem_wait_ld();
      if (lt >= whole) {
        const int seen = last - (t_begin + lt) * TK;
#pragma unroll
        for (int j = 0; j < TK; ++j) s[j] = j <= seen ? s[j] : -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int j = 4; j < TK; j += 4)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[j + e]);
      const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), -INFINITY);  // (not NaN)
      const bool move = (top - m) * c > RISE;
      if (__any_sync(0xffffffffu, move)) {
        const float f = move ? ex2((m - top) * c) : 1.f;
        if (move) m = top;
        l2 = mul2(l2, pk2(f, f));
        if (lt > 0) {
          if (!__all_sync(0xffffffffu, mbar_wait(bar(B_PVD + g), (lt - 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          for (int b = 0; b < dv / 16; ++b) {
            float o[16];
            tmem_ld16(to + 16 * b, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= f;
            tmem_st16(to + 16 * b, o);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      const uint64_t ref2 = pk2(-ref, -ref), c2 = pk2(c, c);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t p[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          // (s - m first: it is exact where it matters, however large both are)
          const uint64_t x = mul2(add2(pk2(s[64 * b + 2 * j], s[64 * b + 2 * j + 1]), ref2), c2);
          float x0, x1;
          upk2(x, x0, x1);
          x0 = ex2(x0), x1 = ex2(x1);
          sum[j & 1] = add2(sum[j & 1], pk2(x0, x1));
          const __nv_bfloat162 y = __floats2bfloat162_rn(x0, x1);
          p[j] = *reinterpret_cast<const uint32_t*>(&y);
        }
        tmem_st32(ts + 32 * b, p);
      }
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PF + g));
      l2 = add2(l2, add2(sum[0], sum[1]));
    }
    if (mine > 0 && ok && !__all_sync(0xffffffffu, mbar_wait(bar(B_PVD + g), (mine - 1) & 1))) ok = false;
    tc_fence_after_sync();
    float la, lb;
    upk2(l2, la, lb);
    const float l = la + lb;
    const int64_t row = (int64_t)(q0 + tid) * a.heads + h, part = (int64_t)split * a.num_tokens * a.heads + row;
    const bool live = tid < rows && ok;
    if (mine == 0) {
      if (live) write_nothing(a, row, split, 0, 1);
    } else {
      const bool any = !(l == 0.f);  // (NaN counts)
      const float inv = any ? 1.f / l : 0.f;
      // values that were taken out, and that this row sees
      const int bad0 = misc->any_bad ? (t_begin + fix0) * TK : INT32_MAX, bad1 = min(last, t_end * TK - 1);
      for (int b = 0; b < dv / 16; ++b) {
        float o[16];
        tmem_ld16(to + 16 * b, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = any ? o[e] * inv : 0.f;
        for (int j = bad0; j <= bad1; ++j) {
          const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.kv) + (k0 + (int64_t)j) * a.kv_tok_stride +
                                   h * a.kv_head_stride + dn + 16 * b;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!isfinite(__bfloat162float(v[e]))) o[e] = NAN;
        }
        if (live) {
          if (S == 1) {
            __align__(16) __nv_bfloat162 y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * dv + 16 * b);
            dst[0] = reinterpret_cast<uint4*>(y)[0];
            dst[1] = reinterpret_cast<uint4*>(y)[1];
          } else {
            float4* dst = reinterpret_cast<float4*>(a.o_part + part * dv + 16 * b);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      }
      if (live) {
        const float z = any ? m * a.softmax_scale + __logf(l) : -INFINITY;
        if (S > 1) a.lse_part[part] = z;
        else if (a.lse) a.lse[row] = z;
      }
    }
    tc_fence_before_sync();
  }
  if (!ok && lane == 0) report(a.dev_status, DSA_DEV_TIMEOUT);
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, TM_COLS);
  }
}

template <bool STD>
cudaError_t launch(const PromptArgs& a, const PromptMaps& maps, cudaStream_t stream) {
  auto kernel = prompt_mla_kernel<STD>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  // at most so many tiles: every request has one that is not full, and the padding
  const int64_t tiles = (int64_t)a.num_tokens / QT + a.num_req + 1;
  kernel<<<dim3((unsigned)tiles, (unsigned)a.heads, (unsigned)a.num_splits), THREADS, SMEM_BYTES, stream>>>(a, maps);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_mla(const PromptArgs& a, cudaStream_t stream) {
  PromptMaps maps;
  if (!make_rows_map(&maps.q, a.q, a.num_tokens, a.heads, a.d_nope + a.d_rope, a.q_tok_stride, a.q_head_stride, 128))
    return cudaErrorInvalidValue;
  // (without rows no token sees anything, and no copy is made)
  const bool rows = a.num_rows > 0, rope = rows && a.d_rope > 0;
  if (!make_rows_map(&maps.kv, rows ? a.kv : a.q, rows ? a.num_rows : 1, rows ? a.heads : 1, rows ? a.d_nope + a.d_v : 16,
                     a.kv_tok_stride, a.kv_head_stride, 128) ||
      !make_rows_map(&maps.rope, rope ? a.k_rope : a.q, rope ? a.num_rows : 1, 1, rope ? a.d_rope : 16, a.rope_stride, 0, 128))
    return cudaErrorInvalidValue;
  const bool std = a.d_nope == 128 && a.d_rope == 64 && a.d_v == 128;
  return std ? launch<true>(a, maps, stream) : launch<false>(a, maps, stream);
}

}  // namespace dsa
