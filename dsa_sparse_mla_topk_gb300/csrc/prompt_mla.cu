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
// One item of work = one head, 256 tokens of one request (two tiles of 128 query rows)
// and one share of its rows, 128 rows a tile; one CTA each in the grid, but a CTA that is done
// takes over one that has not started (cluster launch control), whose queries and
// first keys arrive while it finishes its own.  TMEM: S of both query tiles (2 x 128
// columns; the weights P, bf16, take their place) and O (2 x 128).  Warps:
//  * 0-7 and 8-15: softmax of query tile 0 and 1, two threads a query row, 64 keys each, who
//    exchange their maxima: what lies between a tile's S and its P must be less
//    than the other tile's products take (1,280 cycles; with a thread a row, about
//    1,600).  S comes into registers once; a row's O is rescaled only when its maximum
//    has risen by more than 2^8 (weights stay below 2^8, sums far inside fp32).
//  * 16: TMA.  A tile's key is two 64-column chunks of the head's own and one of the
//    shared rotated part (never copied to the heads), its value two; four key chunks and
//    two value tiles in flight.
//  * 17: MMA.  P V of one query tile, then its next Q K^T, then the other's: one tile's
//    softmax runs under the other's products.
//  * 18: values that are NaN or infinite are taken out of tiles that some query row
//    sees only in part (a weight of 0 would turn them into NaN), and of each column the first
//    position of one is kept: a row sees a run of positions from the start, so it sees
//    a column's if and only if it sees that one.
//  * 19: the next item.
// All waits are bounded.
//
// Bound by the tensor cores, and by what keeps them waiting: 640 flop a pair and head; a tile of
// both query tiles is 2,560 cycles of MMAs and takes about 3,050.  Measured, device time back to back, 64 heads of
// 128 + 64 and 128: one prompt of 8,192 tokens 830 us (1,656 TFLOP/s), 1,024 tokens of 16,384 positions
// 408 us (256 items on 152 SMs), 8 prompts of 1,024 to 2,048 tokens on up to 1,000 positions 560 us (an
// item costs 4 us beside its tiles); 16 heads of 32 + 16, two prompts of 200: 9.7 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
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
constexpr int THREADS = 640, SM_WARPS = 16, WARP_TMA = 16, WARP_MMA = 17, WARP_FIX = 18, WARP_NEXT = 19;
constexpr int HALF = TK / 2;          // keys of a softmax thread
// 640 threads at 96 registers: 4 x 128 x 104 + 128 x 64 = 640 x 96
constexpr int REGS_SOFTMAX = 104, REGS_OTHER = 64;
static_assert(128 * (4 * REGS_SOFTMAX + REGS_OTHER) <= THREADS * 96, "no more registers than at launch");
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float RISE = 8.f;         // a reference moves when a weight would pass 2^RISE
// Waits end after this long.  Some last for an item's whole work (one query tile's warps wait out the other's): for
// 2^26 rows, the most that a call takes, 0.9 s (1.7 us a tile where all are looked through for values that are not
// finite), and 2.8 s (5.4 us) where every tile holds some.
constexpr uint64_t WAIT_NS = 6000000000ull;
constexpr float HUGE_X = 0x1p28f;   // logits (to base 2) from here on take a step more

constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;  // query tile g at + 128 g

constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + 2 * 3 * CHUNK;
constexpr int OFF_V = OFF_K + KSLOTS * CHUNK;
constexpr int OFF_BAR = OFF_V + VST * 2 * CHUNK;
constexpr int B_QF = 0;              // [2] query tile g has landed
constexpr int B_QE = B_QF + 2;       // [2] its products are done
constexpr int B_KF = B_QE + 2;       // [KSLOTS] key chunk has landed
constexpr int B_KE = B_KF + KSLOTS;  // [KSLOTS] its slot is free
constexpr int B_VF = B_KE + KSLOTS;  // [VST]
constexpr int B_VE = B_VF + VST;     // [VST]
constexpr int B_VX = B_VE + VST;     // [VST] the value tile has been looked through
constexpr int B_GO = B_VX + VST;     // [VST] a value tile to look through is on its way
constexpr int B_SF = B_GO + VST;     // [2] S of query tile g is complete
constexpr int B_PF = B_SF + 2;       // [2] P is written (and O rescaled)
constexpr int B_PVD = B_PF + 2;      // [2] P V is done
constexpr int B_IF = B_PVD + 2;      // [2] an item is described
constexpr int B_IE = B_IF + 2;       // [2] all warps are done with it
constexpr int B_CLC = B_IE + 2;      // the answer about the next CTA
constexpr int NBAR = B_CLC + 1;
constexpr int IE_COUNT = SM_WARPS + 3;  // softmax, TMA, MMA and value warps
constexpr int NCHUNK = 128;             // requests' tiles are summed in so many parts
struct Item {
  int32_t req, q0, rows, h, split;  // req -1: padding rows, -2: no more
  int32_t k0, kv_len, t_begin;
  int32_t cnt[2], whole[2];  // tiles of the share that query tile g sees, that all its rows see whole
  int32_t fix0;              // from this tile on some row may see a tile in part
  int32_t any_bad;           // a value that is not finite was taken out, and first_bad holds this item's
};
constexpr int OFF_ANSWER = OFF_BAR + (NBAR * 8 + 15) / 16 * 16;
constexpr int OFF_MISC = OFF_ANSWER + 16;
struct Misc {
  Item item[2];
  union {
    alignas(16) int32_t upto[NCHUNK];  // tiles of the requests up to the end of each part; the item warp takes them into
                                       // registers before the first item
    alignas(16) int32_t first_bad[128];  // of each column of an item's values
  };
  int32_t wsum[4];
  uint32_t tmem;
  float pair[2][2][TQ];  // what the two threads of a query row exchange: [query tile][half]
};
// (no room for alignment slack: a kernel without static shared memory gets it from a 1,024-byte boundary on)
constexpr int SMEM_BYTES = OFF_MISC + (int)sizeof(Misc);
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
static_assert(OFF_ANSWER % 16 == 0 && OFF_MISC % 16 == 0 && offsetof(Misc, upto) % 16 == 0, "16-byte accesses");

struct PromptMaps {
  CUtensorMap q, kv, rope;  // boxes of 64 columns, one head, 128 rows
};

// Tokens of request r from q0 on (0 where its range is none), in tiles of QT.
__device__ __forceinline__ int tiles_of(const PromptArgs& a, int r, int& q0, int& n) {
  q0 = __ldg(a.cu_q + r);
  const int q1 = __ldg(a.cu_q + r + 1);
  n = q0 >= 0 && q1 >= q0 && q1 <= a.num_tokens ? q1 - q0 : -1;
  return (n + QT - 1) / QT;
}

// misc->upto, by the CTA's first NCHUNK threads (a barrier follows).  Every CTA that runs tells of ranges that are
// none: which ones start, and which are taken over before they do, nothing guarantees.
__device__ __forceinline__ void sum_tiles(const PromptArgs& a, Misc* misc) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int inc = 0;
  if (tid < NCHUNK) {
    const int per = (a.num_req + NCHUNK - 1) / NCHUNK, r0 = min(tid * per, a.num_req), r1 = min(r0 + per, a.num_req);
    bool none = false;
    for (int r = r0; r < r1; ++r) {
      int q0, n;
      inc += tiles_of(a, r, q0, n);
      none |= n < 0;
    }
    if (none) report(a.dev_status, DSA_DEV_BAD_INDEX);
    inc = min(inc, (int)gridDim.x);  // (ranges that overlap, an error, could add up past 32 bits)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) misc->wsum[warp] = inc;
  }
  __syncthreads();
  if (tid < NCHUNK) {
    for (int w = 0; w < warp; ++w) inc += misc->wsum[w];
    misc->upto[tid] = inc;
  }
}

// Tile `index` of the requests' tiles one after another, then the padding's (req -1);
// req -2: none.  One warp; u: parts 4 lane .. + 3 of the sums.
__device__ __forceinline__ void find_tile(const PromptArgs& a, int index, const int4& u, int& req, int& q0, int& rows) {
  const int lane = threadIdx.x & 31;
  req = -2, q0 = 0, rows = 0;
  const int all = __shfl_sync(0xffffffffu, u.w, 31);
  if (index >= all) {
    const int pad0 = a.num_req > 0 ? min(max(__ldg(a.cu_q + a.num_req), 0), a.num_tokens) : 0;
    const int64_t at = pad0 + (int64_t)(index - all) * QT;
    if (at < a.num_tokens) req = -1, q0 = (int)at, rows = (int)min((int64_t)QT, a.num_tokens - at);
    return;
  }
  const int who = __ffs(__ballot_sync(0xffffffffu, u.w > index)) - 1;
  const int part = u.x > index ? 0 : u.y > index ? 1 : u.z > index ? 2 : 3;
  const int before = part == 0 ? 0 : part == 1 ? u.x : part == 2 ? u.y : u.z;
  const int prev = __shfl_up_sync(0xffffffffu, u.w, 1);
  const int j = 4 * who + __shfl_sync(0xffffffffu, part, who);
  int left = index - __shfl_sync(0xffffffffu, part == 0 ? (lane == 0 ? 0 : prev) : before, who);
  const int per = (a.num_req + NCHUNK - 1) / NCHUNK, r1 = min((j + 1) * per, a.num_req);
  for (int r0 = j * per; r0 < r1; r0 += 32) {
    int s = 0, n = 0, t = 0;
    if (r0 + lane < r1) t = tiles_of(a, r0 + lane, s, n);
    int inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned over = __ballot_sync(0xffffffffu, inc > left);
    if (over) {
      const int l = __ffs(over) - 1;
      const int i = left - __shfl_sync(0xffffffffu, inc - t, l);
      req = r0 + l;
      q0 = __shfl_sync(0xffffffffu, s, l) + i * QT;
      rows = min(QT, __shfl_sync(0xffffffffu, n, l) - i * QT);
      return;
    }
    left -= __shfl_sync(0xffffffffu, inc, 31);
  }
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Columns d0 .. d0 + n - 1 (16 or 32) of a row's result.
__device__ __forceinline__ void finish(const PromptArgs& a, const int32_t* first_bad, float (&o)[32], int d0, int n, int last,
                                       bool look, bool live, int64_t row, int64_t part, int dv, int S) {
  if (look) {  // values that were taken out, and that this row sees
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (4 * e < n) {
        const int4 f = reinterpret_cast<const int4*>(first_bad + d0)[e];
        if (f.x <= last) o[4 * e] = NAN;
        if (f.y <= last) o[4 * e + 1] = NAN;
        if (f.z <= last) o[4 * e + 2] = NAN;
        if (f.w <= last) o[4 * e + 3] = NAN;
      }
  }
  if (!live) return;
  if (S == 1) {
    const bool wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    uint32_t y[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
      y[e] = *reinterpret_cast<const uint32_t*>(&v);
    }
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + row * dv + d0;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (16 * e < n) {
        if (wide) {
          store32(dst + 16 * e, y + 8 * e, l2_policy(false));
        } else {
          reinterpret_cast<uint4*>(dst)[2 * e] = make_uint4(y[8 * e], y[8 * e + 1], y[8 * e + 2], y[8 * e + 3]);
          reinterpret_cast<uint4*>(dst)[2 * e + 1] = make_uint4(y[8 * e + 4], y[8 * e + 5], y[8 * e + 6], y[8 * e + 7]);
        }
      }
  } else {
    float4* dst = reinterpret_cast<float4*>(a.o_part + part * dv + d0);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (4 * e < n) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
  }
}

__device__ __forceinline__ void st_shared(uint32_t addr, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ float ld_shared(uint32_t addr) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}

// STD: head widths 128 + 64 (rotated) and values of 128, known to the compiler.
template <bool STD>
__global__ void __launch_bounds__(THREADS, 1) prompt_mla_kernel(const PromptArgs a, const __grid_constant__ PromptMaps maps) {
  extern __shared__ __align__(1024) unsigned char smem[];
  if (smem_u32(smem) % 1024 != 0) {  // (the swizzle's atoms would not be where the copies put them)
    if (threadIdx.x == 0) report(a.dev_status, DSA_DEV_TIMEOUT);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  Misc* misc = reinterpret_cast<Misc*>(smem + OFF_MISC);
  auto bar = [&](int b) { return smem_u32(bars + b); };
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int dn = STD ? 128 : a.d_nope, dr = STD ? 64 : a.d_rope, dv = STD ? 128 : a.d_v;
  const int S = a.num_splits;

  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(&misc->tmem), TM_COLS);
    tmem_relinquish();
  }
  if (tid == WARP_TMA * 32) {
    for (int b = 0; b < NBAR; ++b)
      mbar_init(bar(b), b >= B_PF && b < B_PF + 2 ? 8u : b >= B_IE && b < B_IE + 2 ? (uint32_t)IE_COUNT : 1u);
    fence_mbarrier_init();
    tma_prefetch_map(&maps.q);
    tma_prefetch_map(&maps.kv);
    tma_prefetch_map(&maps.rope);
  }
  sum_tiles(a, misc);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = misc->tmem;
  const int nn = (dn + 63) / 64, nk = nn + (dr > 0 ? 1 : 0), nv = (dv + 63) / 64;
  bool ok = true;
  auto wait_for = [](uint32_t b, uint32_t parity) { return mbar_wait(b, parity, WAIT_NS); };
  // waits for item n's description; false: no more
  auto next_item = [&](int n) -> bool {
    if (!__all_sync(0xffffffffu, wait_for(bar(B_IF + (n & 1)), (n >> 1) & 1))) {
      ok = false;
      return false;
    }
    return misc->item[n & 1].req != -2;
  };
  auto item_done = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(B_IE + (n & 1)));
  };

  if (warp >= SM_WARPS) {
    reg_less<REGS_OTHER>();
    if (warp == WARP_NEXT) {
      // ---------------- the items ----------------
      int x = blockIdx.x, y = blockIdx.y, z = blockIdx.z, n = 0, asked = 0;
      const int4 upto = reinterpret_cast<const int4*>(misc->upto)[lane];
      __syncwarp();
      bool room = true;  // item n's place is free
      for (;;) {
        int req, q0, rows;
        // the last tiles first: in causal prompts they see the most
        find_tile(a, (int)gridDim.x - 1 - x, upto, req, q0, rows);
        if (req != -2) {
          // (all loads before the first use of one)
          int k0 = 0, k1 = 0, kv_len = 0, pos[QT / 32];
          if (req >= 0) k0 = __ldg(a.cu_k + req), k1 = __ldg(a.cu_k + req + 1);
#pragma unroll
          for (int i = 0; i < QT / 32; ++i) pos[i] = req >= 0 && 32 * i + lane < rows ? __ldg(a.q_pos + q0 + 32 * i + lane) : -2;
          if (k0 >= 0 && k1 >= k0 && k1 <= a.num_rows) kv_len = k1 - k0;
          else if (lane == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);
          int n_g[2] = {0, 0}, full_g[2] = {0, 0};  // tiles that some row of query tile g sees, that all see whole
          if (req >= 0) {
            int mx[2] = {-1, -1}, mn[2] = {INT32_MAX, INT32_MAX};
#pragma unroll
            for (int i = 0; i < QT / 32; ++i)
              if (32 * i + lane < rows) {
                const int p = pos[i] < -1 || pos[i] >= kv_len ? -1 : pos[i];  // (reported by the softmax threads)
                mx[i / 4] = max(mx[i / 4], p), mn[i / 4] = min(mn[i / 4], p);
              }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int top = __reduce_max_sync(0xffffffffu, mx[g]), low = __reduce_min_sync(0xffffffffu, mn[g]);
              n_g[g] = (top + TK) / TK;  // ceil((top + 1) / TK)
              full_g[g] = low == INT32_MAX ? 0 : (low + 1) / TK;
            }
          }
          const int ntiles = max(n_g[0], n_g[1]);
          const int t_begin = (int)((int64_t)ntiles * z / S), t_end = (int)((int64_t)ntiles * (z + 1) / S);
          if (lane == 0) {
            Item& it = misc->item[n & 1];
            it.req = req, it.q0 = q0, it.rows = rows, it.h = y, it.split = z;
            it.k0 = k0, it.kv_len = kv_len, it.t_begin = t_begin, it.any_bad = 0;
            int fix0 = INT32_MAX;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              it.cnt[g] = max(0, min(t_end, n_g[g]) - t_begin);
              it.whole[g] = max(0, full_g[g] - t_begin);
              if (it.cnt[g] > 0) fix0 = min(fix0, it.whole[g]);
            }
            it.fix0 = fix0;
            mbar_arrive(bar(B_IF + (n & 1)));
          }
          __syncwarp();
          ++n;
          room = false;
        }
        // (one item ahead, no more: the last ones are shared out evenly)
        if (!room && !__all_sync(0xffffffffu, wait_for(bar(B_IE + (n & 1)), ((n >> 1) & 1) ^ 1))) {
          ok = false;
          break;
        }
        room = true;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(B_CLC), 16);
          clc_try_cancel(smem_u32(smem + OFF_ANSWER), bar(B_CLC));
        }
        __syncwarp();
        if (!__all_sync(0xffffffffu, wait_for(bar(B_CLC), asked & 1))) {
          ok = false;
          break;
        }
        ++asked;
        const bool more = clc_answer(smem_u32(smem + OFF_ANSWER), x, y, z);
        fence_proxy_async_smem();  // (the next answer is written behind this read)
        __syncwarp();
        if (!__any_sync(0xffffffffu, more)) break;
      }
      if (ok && lane == 0) {
        misc->item[n & 1].req = -2;
        mbar_arrive(bar(B_IF + (n & 1)));
      }
    } else if (warp == WARP_TMA) {
      // ---------------- TMA warp ----------------
      int slot = 0, phase = 0, vt = 0, qn0 = 0, qn1 = 0;  // of the next key chunk; value tiles and queries loaded so far
      for (int n = 0; next_item(n); ++n) {
        const Item it = misc->item[n & 1];
        const int cnt = max(it.cnt[0], it.cnt[1]);
        if (lane == 0) {
          auto query = [&](int g) {
            if (!ok || !wait_for(bar(B_QE + g), ((g ? qn1 : qn0) & 1) ^ 1)) {
              ok = false;
              return;
            }
            if (g) ++qn1;
            else ++qn0;
            mbar_arrive_expect_tx(bar(B_QF + g), nk * CHUNK);
            for (int c = 0; c < nk; ++c)
              tma_load_3d(smem_u32(smem + OFF_Q + (3 * g + c) * CHUNK), &maps.q, c < nn ? 64 * c : dn, it.h, it.q0 + TQ * g,
                          bar(B_QF + g));
          };
          for (int lt = 0; lt < cnt && ok; ++lt) {
            if (lt == 0 && it.cnt[0] > 0) query(0);
            const int n0 = it.k0 + (it.t_begin + lt) * TK;
            for (int c = 0; c < nk && ok; ++c) {
              if (!wait_for(bar(B_KE + slot), phase ^ 1)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(bar(B_KF + slot), CHUNK);
              const uint32_t dst = smem_u32(smem + OFF_K + slot * CHUNK);
              if (c < nn) tma_load_3d(dst, &maps.kv, 64 * c, it.h, n0, bar(B_KF + slot));
              else tma_load_3d(dst, &maps.rope, 0, 0, n0, bar(B_KF + slot));
              if (++slot == KSLOTS) slot = 0, phase ^= 1;
            }
            if (lt == 0 && it.cnt[1] > 0) query(1);
            const int s = vt % VST;
            if (!ok || !wait_for(bar(B_VE + s), ((vt / VST) & 1) ^ 1)) {
              ok = false;
              break;
            }
            if (lt >= it.fix0) mbar_arrive(bar(B_GO + s));
            mbar_arrive_expect_tx(bar(B_VF + s), nv * CHUNK);
            for (int c = 0; c < nv; ++c)
              tma_load_3d(smem_u32(smem + OFF_V + (2 * s + c) * CHUNK), &maps.kv, dn + 64 * c, it.h, n0, bar(B_VF + s));
            ++vt;
          }
        }
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        item_done(n);
      }
      if (!ok && lane == 0) {  // no copy may land after the CTA is gone
        if (qn0 > 0) wait_for(bar(B_QF), (qn0 - 1) & 1);
        if (qn1 > 0) wait_for(bar(B_QF + 1), (qn1 - 1) & 1);
        for (int s = 0; s < KSLOTS; ++s) wait_for(bar(B_KF + s), s < slot ? phase : phase ^ 1);
        for (int v = max(0, vt - VST); v < vt; ++v) wait_for(bar(B_VF + v % VST), (v / VST) & 1);
      }
      __syncwarp();
    } else if (warp == WARP_MMA) {
      // ---------------- MMA warp ----------------
      const uint32_t ID_QK = idesc_f16_f32(TQ, TK, 0, 0, 1);
      const uint32_t ID_PV = STD ? idesc_f16_f32(TQ, 128, 0, 1, 1) : idesc_f16_f32(TQ, dv, 0, 1, 1);
      // (reductions over the warp: their results are in uniform registers)
      auto wait_u = [&](int b, uint32_t parity) { return __reduce_min_sync(0xffffffffu, (uint32_t)wait_for(bar(b), parity)); };
      auto uniform = [&](int v) { return (int)__reduce_max_sync(0xffffffffu, (uint32_t)v); };
      const uint64_t q_desc = smem_desc(smem_u32(smem + OFF_Q), 16, 1024, SWIZZLE_128B);
      const uint64_t k_desc = smem_desc(smem_u32(smem + OFF_K), 16, 1024, SWIZZLE_128B);
      const uint64_t v_desc = smem_desc(smem_u32(smem + OFF_V), CHUNK, 1024, SWIZZLE_128B);
      uint32_t good = __reduce_min_sync(0xffffffffu, (uint32_t)(tmem == 0));
      int slot = 0, phase = 0;           // of the first key chunk of the tile to come
      int vs = 0, vphase = 0, vx = 0;    // value stage, its phase, and the phases of B_VX (a bit each)
      int pn0 = 0, pn1 = 0, qn0 = 0, qn1 = 0;  // phases of B_PF and B_QF
      // Waits inside an item only note that they gave up: one reduction a tile (30 cycles or more in
      // which no MMA is issued) instead of one a wait; what is issued until then stays in bounds.
      uint32_t fine = 1;
      auto wait = [&](int b, uint32_t parity) { fine &= (uint32_t)mbar_wait(bar(b), parity, good ? WAIT_NS : 0); };
      // S_g = Q_g K^T; the last of the tile's users frees its chunks
      auto issue_qk = [&](int g, bool first_user, bool last_user, bool last_tile) {
        int s = slot, ph = phase;
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (c < nk) {
            if (first_user) {
              wait(B_KF + s, ph);
              tc_fence_after_sync();
            }
            const uint64_t qa = q_desc + (uint32_t)((3 * g + c) * (CHUNK >> 4)), kb = k_desc + (uint32_t)(s * (CHUNK >> 4));
            const int steps = STD ? 4 : (c < nn ? min(4, (dn - 64 * c) / 16) : dr / 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (STD || kk < steps) mma_f16_ss_warp(TM_S + 128 * g, qa + 2 * kk, kb + 2 * kk, ID_QK, c | kk ? 1u : 0u);
            if (last_user) mma_commit_warp(bar(B_KE + s));
            if (++s == KSLOTS) s = 0, ph ^= 1;
          }
        }
        mma_commit_warp(bar(B_SF + g));
        if (last_tile) mma_commit_warp(bar(B_QE + g));
        if (last_user) slot = s, phase = ph;
      };
      auto issue_pv = [&](int g, uint32_t acc, uint32_t parity, bool last_user) {
        const uint64_t vb = v_desc + (uint32_t)(vs * (2 * CHUNK >> 4));
        wait(B_PF + g, parity);
        tc_fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < TK / 16; ++kk)
          mma_f16_ts_warp(TM_O + 128 * g, TM_S + 128 * g + 8 * kk, vb + 128 * kk, ID_PV, kk > 0 ? 1u : acc);
        mma_commit_warp(bar(B_PVD + g));
        if (last_user) mma_commit_warp(bar(B_VE + vs));
      };
      for (int n = 0; good; ++n) {
        // (every branch here hangs on a reduction's result: what a load or a vote decides would take the
        // loop's values out of the uniform registers, and an MMA's issue would cost twice as much)
        good = wait_u(B_IF + (n & 1), (n >> 1) & 1);
        const Item* it = &misc->item[n & 1];
        if (!good || uniform(it->req) == -2) break;
        const int c0 = uniform(it->cnt[0]), c1 = uniform(it->cnt[1]), fix = uniform(it->fix0), cnt = max(c0, c1);
        slot = uniform(slot), phase = uniform(phase), vs = uniform(vs), vphase = uniform(vphase), vx = uniform(vx);
        pn0 = uniform(pn0), pn1 = uniform(pn1);
        if (c0 > 0) {
          wait(B_QF, qn0);
          qn0 ^= 1;
          tc_fence_after_sync();
          issue_qk(0, true, c1 == 0, c0 == 1);
        }
        if (c1 > 0) {
          wait(B_QF + 1, qn1);
          qn1 ^= 1;
          tc_fence_after_sync();
          issue_qk(1, c0 == 0, true, c1 == 1);
        }
        for (int lt = 0; lt < cnt && good; ++lt) {
          wait(B_VF + vs, vphase);
          if (lt >= fix) {
            wait(B_VX + vs, (vx >> vs) & 1);
            vx ^= 1 << vs;
          }
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int mine = g ? c1 : c0, other = g ? c0 : c1;
            if (lt < mine) {
              issue_pv(g, lt > 0 ? 1u : 0u, g ? pn1 : pn0, g == 1 || lt >= other);
              if (g) pn1 ^= 1;
              else pn0 ^= 1;
              if (lt + 1 < mine) issue_qk(g, g == 0 || lt + 1 >= other, g == 1 || lt + 1 >= other, lt + 2 == mine);
            }
          }
          if (++vs == VST) vs = 0, vphase ^= 1;
          good = __reduce_min_sync(0xffffffffu, fine);
        }
        item_done(n);
      }
      if (!good) ok = false;
    } else if (warp == WARP_FIX) {
      // ---------------- values that are not finite ----------------
      int vt = 0, go = 0;  // value tiles so far, phases of B_GO (a bit each)
      for (int n = 0; ok && next_item(n); ++n) {
        const Item* it = &misc->item[n & 1];
        const int cnt = max(it->cnt[0], it->cnt[1]);
        for (int lt = min(it->fix0, cnt); lt < cnt; ++lt) {
          const int v = vt + lt, s = v % VST;
          // (B_VF alone would not do: a wait on a barrier whose phase before the one that is meant
          // has not ended returns at once)
          if (!__all_sync(0xffffffffu, wait_for(bar(B_GO + s), (go >> s) & 1) && wait_for(bar(B_VF + s), (v / VST) & 1))) {
            ok = false;
            break;
          }
          go ^= 1 << s;
          __nv_bfloat162 top = __floats2bfloat162_rn(0.f, 0.f);  // the largest magnitudes, NaN if there is one
          for (int r = lane; r < TK; r += 32) {
            const unsigned char* row = smem + OFF_V + 2 * s * CHUNK + r * 128;
            for (int c = 0; c < nv; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) {  // (every lane at another bank; the order does not matter)
                const uint4 w = *reinterpret_cast<const uint4*>(row + c * CHUNK + 16 * ((e + lane) & 7));
                auto look = [&](uint32_t u) { top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u))); };
                look(w.x), look(w.y), look(w.z), look(w.w);
              }
          }
          const bool odd = !isfinite(__low2float(top)) || !isfinite(__high2float(top));
          if (__any_sync(0xffffffffu, odd)) {
            // (what is kept from tile to tile is in shared memory: the search above needs the registers)
            volatile Item* const item = &misc->item[n & 1];
            int4* const kept = reinterpret_cast<int4*>(misc->first_bad) + lane;  // of columns 4 lane .. + 3
            int first[4] = {INT32_MAX, INT32_MAX, INT32_MAX, INT32_MAX};
            if (item->any_bad) {
              const int4 f = *kept;
              first[0] = f.x, first[1] = f.y, first[2] = f.z, first[3] = f.w;
            } else if (n > 0 && !__all_sync(0xffffffffu, wait_for(bar(B_IE + ((n - 1) & 1)), ((n - 1) >> 1) & 1))) {
              ok = false;  // (the places are the item's before until all are done with that)
              break;
            }
            __syncwarp();
            // Four columns a lane, four rows at a time: what is not finite becomes 0.
            const int at = (item->t_begin + lt) * TK;
            const __nv_bfloat162 inf = __floats2bfloat162_rn(INFINITY, INFINITY);
            uint32_t open[2] = {0, 0};  // columns without a first one
#pragma unroll
            for (int e = 0; e < 4; ++e) open[e / 2] |= first[e] == INT32_MAX ? 0xffffu << (16 * (e & 1)) : 0u;
            unsigned char* col = smem + OFF_V + (2 * s + (lane >> 4)) * CHUNK + 8 * (lane & 1);
            if (lane >> 4 < nv)
#pragma unroll 1
              for (int r0 = 0; r0 < TK; r0 += 4) {
                uint32_t w[4][2];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const uint2 v = *reinterpret_cast<const uint2*>(col + (r0 + r) * 128 + 16 * (((lane & 15) >> 1) ^ (r0 & 4) ^ r));
                  w[r][0] = v.x, w[r][1] = v.y;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const uint32_t fine = __hlt2_mask(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[r][e])), inf);
                    const uint32_t fresh = open[e] & ~fine;
                    if (fresh) {
                      if (fresh & 0xffffu) first[2 * e] = at + r0 + r;
                      if (fresh >> 16) first[2 * e + 1] = at + r0 + r;
                      open[e] &= fine;
                    }
                    w[r][e] &= fine;
                  }
                  *reinterpret_cast<uint2*>(col + (r0 + r) * 128 + 16 * (((lane & 15) >> 1) ^ (r0 & 4) ^ r)) = make_uint2(w[r][0], w[r][1]);
                }
              }
            *kept = make_int4(first[0], first[1], first[2], first[3]);
            // (a query tile that is done before this one is looked through may read both now)
            __threadfence_block();
            __syncwarp();
            if (lane == 0) item->any_bad = 1;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_VX + s));
        }
        vt += cnt;
        item_done(n);
      }
    }
  } else {
    // ---------------- softmax warps ----------------
    reg_more<REGS_SOFTMAX>();
    const int g = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
    const int qrow = TQ * g + 32 * quad + lane;  // this thread's query row of the CTA's QT
    const uint32_t lanes = (uint32_t)(32 * quad) << 16, ts = TM_S + 128 * g + lanes, to = TM_O + 128 * g + lanes;
    const uint32_t mine_p = smem_u32(&misc->pair[g][half][32 * quad + lane]), other_p = mine_p + (half ? -4 * TQ : 4 * TQ);
    const int pair_bar = 1 + 4 * g + quad;  // the two warps of these 32 rows
    const float c = fmaxf(a.softmax_scale * LOG2E, 0x1p-149f);  // (0 would make NaN of masked logits; of none it makes 2^-21)
    int sn = 0;  // tiles so far
    // The two warps of a pair share a barrier, which has no limit: they leave their loops only by what it
    // tells both, whether a wait of either gave up.
    for (int n = 0;; ++n) {
      const bool more = next_item(n);
      if (named_barrier_or(pair_bar, 64, !more || !ok)) break;
      const volatile Item& it = misc->item[n & 1];  // (read again where it is needed: the loop needs the registers)
      const int mine = it.cnt[g], whole = it.whole[g], tile0 = it.t_begin;
      if (max(it.cnt[0], it.cnt[1]) == 0) {
        for (int i = warp; i < it.rows; i += SM_WARPS)
          write_nothing(a, (int64_t)(it.q0 + i) * a.heads + it.h, it.split, lane, 32);
      }
      int last = -1;
      if (it.req >= 0 && qrow < it.rows) {
        last = __ldg(a.q_pos + it.q0 + qrow);
        if (last < -1 || last >= it.kv_len) {
          if (half == 0) report(a.dev_status, DSA_DEV_BAD_QPOS);
          last = -1;
        }
      }
      float m = -INFINITY, r = 0.f;  // the reference, and in units of x
      uint64_t l2 = 0;
      for (int lt = 0; lt < mine; ++lt, ++sn) {
        if (!__all_sync(0xffffffffu, wait_for(bar(B_SF + g), sn & 1))) ok = false;
        tc_fence_after_sync();
        float s[HALF];
#pragma unroll
        for (int b = 0; b < 2; ++b) tmem_ld32(ts + HALF * half + 32 * b, *reinterpret_cast<float(*)[32]>(s + 32 * b));
        tmem_wait_ld();
        if (lt >= whole) {
          const int seen = last - (tile0 + lt) * TK - HALF * half;
#pragma unroll
          for (int j = 0; j < HALF; ++j) s[j] = j <= seen ? s[j] : -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // (a NaN is no maximum)
#pragma unroll
        for (int j = 0; j < HALF; j += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[j + 2 * e], s[j + 2 * e + 1]);
        float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        // The other thread's; after the barrier S has been read by both, and P may take its place.  (The one
        // behind that keeps a value here until it is read: both pass B_SF's next phase only after P is whole.)
        st_shared(mine_p, top);
        tc_fence_before_sync();
        if (named_barrier_or(pair_bar, 64, !ok)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        top = fmaxf(top, ld_shared(other_p));
        const bool move = (top - m) * c > RISE;
        if (__any_sync(0xffffffffu, move)) {
          float f = 1.f;
          if (move) {
            const float to_r = top * c;
            f = fabsf(top) * c < HUGE_X ? ex2(r - to_r) : ex2((m - top) * c);  // (from -inf: 0)
            if (m == -INFINITY) f = 0.f;
            m = top, r = to_r;
          }
          l2 = mul2(l2, pk2(f, f));
          if (lt > 0) {  // each thread half of the columns (a multiple of 16)
            if (!__all_sync(0xffffffffu, wait_for(bar(B_PVD + g), (sn - 1) & 1))) ok = false;
            tc_fence_after_sync();
            for (int b = half; b < dv / 16; b += 2) {
              float o[16];
              tmem_ld16(to + 16 * b, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= f;
              tmem_st16(to + 16 * b, o);
            }
          }
        }
        // x = c s - r, r = c m rounded: the reference is any number, so r's rounding changes no weight's share.
        // Past 2^28 it would (r's steps reach 2^4 and more): x = c (s - m) there, where s - m is exact.
        const bool huge = !(fabsf(m) * c < HUGE_X) && m > -INFINITY;
        if (__any_sync(0xffffffffu, huge)) {
#pragma unroll
          for (int j = 0; j < HALF; ++j) s[j] = huge ? (s[j] - m) * c : fmaf(s[j], c, -r);
        } else {
          const uint64_t r2 = pk2(-r, -r), c2 = pk2(c, c);
#pragma unroll
          for (int j = 0; j < HALF; j += 2) upk2(fma2(pk2(s[j], s[j + 1]), c2, r2), s[j], s[j + 1]);
        }
        // (few weights at a time: with all of them in registers beside the logits, some of both spill)
        uint64_t sum = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t p[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x0 = ex2(s[16 * b + 2 * j]), x1 = ex2(s[16 * b + 2 * j + 1]);
            if (j & 1) sum = add2(sum, pk2(x0, x1));
            else l2 = add2(l2, pk2(x0, x1));
            // A weight enters the products as bf16, the type of the values (both factors of an MMA have the same),
            // 2^-8 of it off at most: out's error against 64 bits is 1.9 to 2.3e-3 with it, out's own rounding alone
            // 1.6 to 1.7e-3.  A second bf16 for the rest would be two fifths more products.  The sum takes it unrounded.
            const __nv_bfloat162 y = __floats2bfloat162_rn(x0, x1);
            p[j] = *reinterpret_cast<const uint32_t*>(&y);
          }
          tmem_st8(ts + 32 * half + 8 * b, p);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PF + g));
        l2 = add2(l2, sum);
      }
      if (mine > 0) {
        if (ok && !__all_sync(0xffffffffu, wait_for(bar(B_PVD + g), (sn - 1) & 1))) ok = false;
        if (named_barrier_or(pair_bar, 64, !ok)) {  // (and the maxima have been read)
          ok = false;
          break;
        }
      }
      tc_fence_after_sync();
      float l, lb;
      upk2(l2, l, lb);
      l += lb;
      const int64_t row = (int64_t)(it.q0 + qrow) * a.heads + it.h, part = (int64_t)it.split * a.num_tokens * a.heads + row;
      const bool live = qrow < it.rows;
      if (mine == 0) {
        if (live && it.cnt[g ^ 1] > 0) write_nothing(a, row, it.split, half, 2);
      } else {
        st_shared(mine_p, l);
        named_barrier_sync(pair_bar, 64);
        l = half ? ld_shared(other_p) + l : l + ld_shared(other_p);  // (the same sum in both)
        named_barrier_sync(pair_bar, 64);
        const bool any = !(l == 0.f);  // (NaN counts)
        const float inv = any ? 1.f / l : 0.f;
        const bool look = it.any_bad != 0;
        for (int b = half; b < dv / 32; b += 2) {
          float o[32];
          tmem_ld32(to + 32 * b, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = any ? o[e] * inv : 0.f;
          finish(a, misc->first_bad, o, 32 * b, 32, last, look, live, row, part, dv, S);
        }
        if (dv % 32 && half == 1) {
          float o[32];
          tmem_ld16(to + dv - 16, *reinterpret_cast<float(*)[16]>(o));
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = any ? o[e] * inv : 0.f;
          finish(a, misc->first_bad, o, dv - 16, 16, last, look, live, row, part, dv, S);
        }
        if (live && half == 0) {
          const float z = !any ? -INFINITY : fabsf(m) * c < HUGE_X ? r * LN2 + __logf(l) : m * a.softmax_scale + __logf(l);
          if (S > 1) a.lse_part[part] = z;
          else if (a.lse) a.lse[row] = z;
        }
      }
      tc_fence_before_sync();
      item_done(n);
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
