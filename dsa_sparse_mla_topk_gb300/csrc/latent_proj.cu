// Products of latent attention around the cache's latent space: queries into
// it (dsa_absorb_q), attention's outputs out of it (dsa_project_out), and
// cached rows to every head's keys and values (dsa_expand_kv).
//
//   absorb:   y[t, h, :] = x[t, h, :dn] W_k[h],        W_k[h] = w[h, :dn, :]   [dn, dl]
//   project:  y[t, h, :] = x[t, h, :dl] W_v[h]^T,      W_v[h] = w[h, dn:, :]   [dv, dl]
//   expand:   y[n, (h, j)] = s_n (code[n, :] . w[h, j, :])
//
// All three are C = s A B with bf16 factors and fp32 sums, 128 rows of A a CTA and tile
// (tcgen05 + TMEM + TMA), by persistent CTAs.  A unit is a head's columns (absorb: up to 512,
// project: up to 128) or 256 of expand's; its B, at most 128 KB a CTA, stays in shared
// memory while the CTA goes through tiles of rows, whose A comes in 64-column chunks.
// The (unit, tile) pairs are dealt in contiguous runs, one a CTA, equal to one tile; B of the
// next unit follows chunk by chunk behind the last tile of the one before.
// Results leave from one half of TMEM while the next tile's products run into the other:
// absorb's, whose heads' rows are 1,152 bytes apart from the rotated part, through shared memory
// and TMA stores of 32 rows x 64 columns; the others' straight from registers, 32 bytes a
// store, which leaves room for two more chunks of A (project, 8,192 tokens: 112 -> 108 us).
// absorb and project read and write more than they compute (85 and 102 flop a byte).  Measured, device time
// back to back, 64 heads of 128 + 64, latent 512: absorb 4,099 tokens 76 us (5.4 TB/s, most of it stores), 8
// tokens 4.7; project 8,192 tokens 107.6 us (6.3 TB/s, 93% of a copy), 128 tokens 6.3.
// expand is bound by the tensor cores (512): pairs of CTAs (cta_group::2) take 256 x 256
// outputs a tile, each holding half of the columns' weights, so that A is half
// as many bytes a product (with single CTAs of 128 columns 16,384 rows take 283 us, in pairs 211 at
// that step and 168 now: 1,637 TFLOP/s, with L2 between A's reads and the results).  Five
// requests of 167 to 333 rows: 27 us, two launches and 4 to 5 tiles a pair.
// Warps: 0-7 results, 8 TMA, 9 MMA, 10 the rotated part of the queries, which is copied.
// All waits are bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.cuh"
#include "mla_tc_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

using namespace sm100;

enum Mode { ABSORB, PROJECT, EXPAND };

constexpr int TM = 128, CHUNK = TM * 128;  // rows of a tile; a chunk of A: 128 rows x 64 columns
constexpr int SLOTS = 4;                   // chunks of A in flight (absorb: one less, the rotated part's place)
constexpr int N_MMA = 256;                 // columns of one accumulator; two of them
constexpr int OUT_WARPS = 8, WARP_TMA = 8, WARP_MMA = 9, WARP_ROPE = 10, THREADS = 352;
constexpr int B_BYTES = 128 * 1024, STAGE = 32 * 128;  // a warp's 32 rows x 64 columns of results
constexpr int OFF_B = 0;
constexpr int OFF_A = OFF_B + B_BYTES;
constexpr int OFF_OUT = OFF_A + SLOTS * CHUNK;  // [OUT_WARPS]
constexpr int OFF_BAR = OFF_OUT + OUT_WARPS * STAGE;
constexpr int B_AF = 0;             // [SLOTS + 2] a chunk of A has landed
constexpr int B_AE = B_AF + SLOTS + 2;  // [SLOTS + 2] its slot is free
constexpr int MAX_KC = 8;           // chunks of k
constexpr int B_BF = B_AE + SLOTS + 2;  // [MAX_KC] chunk of B of the unit has landed (absorb: [0], all of it)
constexpr int B_BE = B_BF + MAX_KC; // [MAX_KC] its products are done
constexpr int B_DF = B_BE + MAX_KC; // [2] an accumulator is complete
constexpr int B_DE = B_DF + 2;      // [2] it has been read
constexpr int B_RF = B_DE + 2;      // the rotated part has landed
constexpr int NBAR = B_RF + 1;
constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr int SMEM_BYTES = OFF_TMEM + 16 + 1024;  // with alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

struct ProductMaps {
  CUtensorMap a, b, c, c_rope;  // (results by TMA: absorb's)
};
struct Product {
  int m, n, k;             // rows; columns of a head (expand: of all); the sum's length
  int n_unit, per_group;   // columns of a unit, units of a head (expand: of all)
  int units;
  int b_row0, b_group;     // B's first row, and rows from head to head
  int rope_x;              // absorb: the rotated part's column in A, -1: none
  const int32_t* rows;     // expand: the rows there are, on the device
  const float* scale;      // expand: [m]
  __nv_bfloat16* out;      // not absorb: rows of ldc values, a head after the other
  int64_t ldc;
  bool wide;               // it is 32-byte aligned
  int32_t* dev_status;
};

template <Mode MODE>
__global__ void __launch_bounds__(THREADS, 1) product_kernel(const Product p, const __grid_constant__ ProductMaps maps) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
  auto bar = [&](int b) { return smem_u32(bars + b); };
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr bool PAIR = MODE == EXPAND;
  constexpr int NSLOT = MODE == ABSORB ? SLOTS - 1 : SLOTS + 2;
  constexpr int CTAS = PAIR ? 2 : 1, TROWS = CTAS * TM;  // rows of a tile
  const int rank = PAIR ? (int)cluster_rank() : 0;

  if (warp == WARP_MMA) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  if (tid == WARP_TMA * 32) {
    for (int b = 0; b < NBAR; ++b) mbar_init(bar(b), b >= B_DE && b < B_DE + 2 ? (uint32_t)(OUT_WARPS * CTAS) : 1u);
    fence_mbarrier_init();
    tma_prefetch_map(&maps.a);
    tma_prefetch_map(&maps.b);
    if (MODE == ABSORB) tma_prefetch_map(&maps.c);
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) {  // the other CTA's barriers and tensor memory are there, too
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int workers = gridDim.x / CTAS, worker = blockIdx.x / CTAS;
  const int nkc = (p.k + 63) / 64;
  const int b_rows = p.n_unit / CTAS;  // columns of a unit whose weights this CTA holds
  // unit u: head (expand: 0) and the first of its columns there
  auto group_of = [&](int u) { return MODE == EXPAND ? 0 : u / p.per_group; };
  auto col_of = [&](int u) { return (u % p.per_group) * p.n_unit; };
  auto cols_of = [&](int u) { return min(p.n_unit, p.n - col_of(u)); };
  // A barrier's bytes are those of both CTAs, counted on the first one's
  auto load = [&](int b, int off, const CUtensorMap* map, int x, int y, int z) {
    if constexpr (PAIR) tma_load_3d_pair(smem_u32(smem + off), map, x, y, z, cluster_addr(bar(b), 0));
    else tma_load_3d(smem_u32(smem + off), map, x, y, z, bar(b));
  };
  auto expect = [&](int b, uint32_t bytes) {
    if (rank == 0) mbar_arrive_expect_tx(bar(b), bytes * CTAS);
  };
  // chunk c of B of unit u: 64 columns of k, b_rows rows (not absorb)
  auto load_b = [&](int u, int c) {
    expect(B_BF + c, b_rows * 128);
    load(B_BF + c, OFF_B + c * b_rows * 128, &maps.b, 64 * c, 0, p.b_row0 + group_of(u) * p.b_group + col_of(u) + rank * b_rows);
  };
  int m_all = p.m;
  if constexpr (MODE == EXPAND) {
    // the first unit's weights do not depend on the rows (floor(floor(x mt) / mt) = floor(x))
    if (warp == WARP_TMA && lane == 0)
      for (int c = 0; c < nkc; ++c) load_b((int)((int64_t)p.units * worker / workers), c);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    m_all = min(max(*reinterpret_cast<const volatile int32_t*>(p.rows), 0), p.m);
  }
  const int mt = m_all / TROWS + (m_all % TROWS != 0);  // (up to 2^31 - 1 rows)
  const int64_t tiles = (int64_t)p.units * mt;
  const int t0 = (int)(tiles * worker / workers), t1 = (int)(tiles * (worker + 1) / workers);
  bool ok = true;
  // Results past half of L2 are marked as the first to go, or they push out what is read again (expand: 16,384 rows
  // 203 us, 188 so; absorb: 4,099 tokens 79.7 and 75.7); those that fit stay for the call that reads them.
  const uint64_t policy = l2_policy((int64_t)m_all * p.n * (MODE == EXPAND ? 1 : p.units / p.per_group) * 2 > (int64_t)64 << 20);

  if (warp == WARP_TMA) {
    if (lane == 0) {
      int slot = 0, phase = 0, unit = -1, loads = 0;
      for (int t = t0; t < t1 && ok; ++t) {
        const int u = t / mt, m0 = (t - u * mt) * TROWS + rank * TM, g = group_of(u), n0 = col_of(u);
        const bool fresh = u != unit;
        if (fresh) unit = u, ++loads;
        if (MODE == ABSORB && fresh) {  // slices of 64 columns, k rows each
          if (!mbar_wait(bar(B_BE), (loads & 1))) {
            ok = false;
            break;
          }
          const int slices = (cols_of(u) + 63) / 64;
          expect(B_BF, slices * p.k * 128);
          for (int s = 0; s < slices; ++s) load(B_BF, OFF_B + s * p.k * 128, &maps.b, n0 + 64 * s, 0, p.b_row0 + g * p.b_group);
        }
        for (int c = 0; c < nkc; ++c) {
          if (MODE != ABSORB && fresh && !(MODE == EXPAND && loads == 1)) {
            if (!mbar_wait(bar(B_BE + c), (loads & 1))) {
              ok = false;
              break;
            }
            load_b(u, c);
          }
          if (!mbar_wait(bar(B_AE + slot), phase ^ 1)) {
            ok = false;
            break;
          }
          expect(B_AF + slot, CHUNK);
          load(B_AF + slot, OFF_A + slot * CHUNK, &maps.a, 64 * c, g, m0);
          if (++slot == NSLOT) slot = 0, phase ^= 1;
        }
      }
      if (MODE == EXPAND && t0 >= t1) loads = 1;
      if ((!ok || t0 >= t1) && rank == 0) {  // no copy may land after the CTA is gone
        for (int c = 0; c < (MODE == ABSORB ? 1 : nkc) && loads; ++c) mbar_wait(bar(B_BF + c), (loads - 1) & 1);
        for (int s = 0; s < NSLOT && !ok; ++s) mbar_wait(bar(B_AF + s), s < slot ? phase : phase ^ 1);
      }
    }
    __syncwarp();
  } else if (warp == WARP_MMA) {
    if (rank == 0) {
      auto wait_u = [&](int b, uint32_t parity) {
        return __reduce_min_sync(0xffffffffu, (uint32_t)mbar_wait(bar(b), parity));
      };
      auto commit = [&](int b) {
        if constexpr (PAIR) mma_commit_pair_warp(bar(b));
        else mma_commit_warp(bar(b));
      };
      const uint64_t a_desc = smem_desc(smem_u32(smem + OFF_A), 16, 1024, SWIZZLE_128B);
      // absorb's B has its columns contiguous: from one 64-column slice to the next k rows of 128 bytes
      const uint64_t b_desc = smem_desc(smem_u32(smem + OFF_B), MODE == ABSORB ? p.k * 128 : 16, 1024, SWIZZLE_128B);
      uint32_t good = __reduce_min_sync(0xffffffffu, (uint32_t)(tmem == 0));
      const int ut0 = __reduce_min_sync(0xffffffffu, (uint32_t)t0), ut1 = __reduce_min_sync(0xffffffffu, (uint32_t)t1);
      int slot = 0, phase = 0, unit = -1, loads = 0, d = 0;  // d: accumulators filled so far
      for (int t = ut0; t < ut1 && good; ++t) {
        const int u = t / mt, nb = MODE == EXPAND ? p.n_unit : cols_of(u);
        const bool fresh = u != unit, last = t + 1 == ut1 || (t + 1) / mt != u;  // of the unit's tiles here
        if (fresh) unit = u, ++loads;
        if (MODE == ABSORB && fresh) good = wait_u(B_BF, (loads - 1) & 1);
        const int subs = MODE == ABSORB ? (nb + N_MMA - 1) / N_MMA : 1;
        int s = slot, ph = phase;
        for (int j = 0; j < subs && good; ++j, ++d) {
          good = wait_u(B_DE + (d & 1), ((d >> 1) & 1) ^ 1);
          tc_fence_after_sync();
          const uint32_t idesc = idesc_f16_f32(TROWS, min(N_MMA, nb - j * N_MMA), 0, MODE == ABSORB ? 1 : 0, 1);
          s = slot, ph = phase;
          for (int c = 0; c < nkc && good; ++c) {
            if (MODE != ABSORB && fresh) good = wait_u(B_BF + c, (loads - 1) & 1);
            if (j == 0 && good) good = wait_u(B_AF + s, ph);
            tc_fence_after_sync();
            const uint64_t ad = a_desc + (uint32_t)(s * (CHUNK >> 4));
            // 16 of k: 32 bytes along a row, or 16 rows of 128 bytes
            const uint64_t bd = MODE == ABSORB ? b_desc + (uint32_t)(j * (N_MMA / 64) * p.k * 8 + c * 64 * 8)
                                               : b_desc + (uint32_t)(c * b_rows * 8);
            const int steps = min(4, (p.k - 64 * c) / 16);
            if (good) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (kk < steps) {
                  if constexpr (PAIR)
                    mma_f16_ss_pair_warp(N_MMA * (d & 1), ad + 2 * kk, bd + 2 * kk, idesc, c | kk ? 1u : 0u);
                  else
                    mma_f16_ss_warp(N_MMA * (d & 1), ad + 2 * kk, bd + (MODE == ABSORB ? 128 : 2) * kk, idesc,
                                    c | kk ? 1u : 0u);
                }
              if (j == subs - 1) commit(B_AE + s);
              if (MODE != ABSORB && last) commit(B_BE + c);
            }
            if (++s == NSLOT) s = 0, ph ^= 1;
          }
          if (good) commit(B_DF + (d & 1));
        }
        if (MODE == ABSORB && last && good) commit(B_BE);
        slot = s, phase = ph;
      }
      if (!good) ok = false;
    }
  } else if (warp == WARP_ROPE) {
    if (MODE == ABSORB && p.rope_x >= 0 && lane == 0) {
      const uint32_t buf = smem_u32(smem + OFF_A + NSLOT * CHUNK);
      int done = 0;
      for (int t = t0; t < t1; ++t) {
        const int u = t / mt, m0 = (t - u * mt) * TM, g = group_of(u);
        if (col_of(u) != 0) continue;  // one of the head's units does it
        mbar_arrive_expect_tx(bar(B_RF), CHUNK);
        tma_load_3d(buf, &maps.a, p.rope_x, g, m0, bar(B_RF));
        if (!mbar_wait(bar(B_RF), done & 1)) {
          ok = false;
          break;
        }
        ++done;
        for (int i = 0; i < 4 && m0 + 32 * i < m_all; ++i) tma_store_3d(&maps.c_rope, buf + i * STAGE, 0, g, m0 + 32 * i, policy);
        tma_store_commit();
        tma_store_wait_read<0>();
      }
      tma_store_wait_all();
    }
    __syncwarp();
  } else {
    // ---- results: warp w has rows 32 (w % 4) .. + 31 of a tile, one a lane, and every other 64 columns ----
    const uint32_t buf = smem_u32(smem + OFF_OUT + warp * STAGE);
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    int d = 0;
    for (int t = t0; t < t1 && ok; ++t) {
      const int u = t / mt, m0 = (t - u * mt) * TROWS + rank * TM + 32 * quad, g = group_of(u), n0 = col_of(u);
      const int nb = MODE == EXPAND ? p.n_unit : cols_of(u);
      float scale = 1.f;
      if constexpr (MODE == EXPAND) scale = m0 + lane < m_all ? *const_cast<const volatile float*>(p.scale + m0 + lane) : 0.f;
      for (int j = 0; j < nb; j += N_MMA, ++d) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(B_DF + (d & 1)), (d >> 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const int width = min(N_MMA, nb - j);
        auto read = [&] {  // this warp's share of the accumulator
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR) mbar_arrive_cluster_relaxed(cluster_addr(bar(B_DE + (d & 1)), 0));
            else mbar_arrive(bar(B_DE + (d & 1)));
          }
        };
        if (64 * half >= width) read();
        for (int c = 64 * half; c < width; c += 128) {
          float x[64];
          tmem_ld32(N_MMA * (d & 1) + c + lanes, *reinterpret_cast<float(*)[32]>(x));
          if (c + 32 < width) tmem_ld32(N_MMA * (d & 1) + c + 32 + lanes, *reinterpret_cast<float(*)[32]>(x + 32));
          tmem_wait_ld();
          if (c + 128 >= width) read();
          if (m0 >= m_all || n0 + j + c >= p.n) continue;
          __align__(16) uint32_t y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const __nv_bfloat162 v = MODE == EXPAND ? __floats2bfloat162_rn(x[2 * e] * scale, x[2 * e + 1] * scale)
                                                    : __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            y[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
          if (MODE != ABSORB) {
            // straight to memory, a row's 128 bytes a lane
            if (m0 + lane < m_all) {
              __nv_bfloat16* dst = p.out + (int64_t)(m0 + lane) * p.ldc + (int64_t)g * p.n + n0 + j + c;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n0 + j + c + 16 * e < p.n) {
                  if (p.wide) {
                    store32(dst + 16 * e, y + 8 * e, policy);
                  } else {
                    *reinterpret_cast<uint4*>(dst + 16 * e) = make_uint4(y[8 * e], y[8 * e + 1], y[8 * e + 2], y[8 * e + 3]);
                    *reinterpret_cast<uint4*>(dst + 16 * e + 8) = make_uint4(y[8 * e + 4], y[8 * e + 5], y[8 * e + 6], y[8 * e + 7]);
                  }
                }
            }
            continue;
          }
          if (lane == 0) tma_store_wait_read<0>();  // the store before has left the buffer
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((e ^ (lane & 7)) << 4)),
                         "r"(y[4 * e]), "r"(y[4 * e + 1]), "r"(y[4 * e + 2]), "r"(y[4 * e + 3])
                         : "memory");
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&maps.c, buf, n0 + j + c, g, m0, policy);
            tma_store_commit();
          }
        }
      }
    }
    if (lane == 0) tma_store_wait_all();
    __syncwarp();
  }
  if (!ok && lane == 0) report(p.dev_status, DSA_DEV_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) {  // neither CTA leaves while the other's products read its shared memory
    cluster_arrive();
    cluster_wait();
  }
  if (warp == WARP_MMA) {
    tc_fence_after_sync();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

template <Mode MODE>
cudaError_t launch_product(const Product& p, const ProductMaps& maps, cudaStream_t stream) {
  auto kernel = product_kernel<MODE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  constexpr int CTAS = MODE == EXPAND ? 2 : 1;
  const int64_t tiles = (int64_t)p.units * (((int64_t)p.m + CTAS * TM - 1) / (CTAS * TM)), workers = device_sm_count() / CTAS;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CTAS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // after the rows' kernel
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(CTAS * (tiles < workers ? tiles : workers)));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = MODE == EXPAND ? 2 : 0;
  const cudaError_t r = cudaLaunchKernelEx(&cfg, kernel, p, maps);
  return r != cudaSuccess ? r : cudaGetLastError();
}

// Columns of a unit: the whole head's, halved while twice as many units still find SMs.
int columns_of_unit(int n, int most, int64_t groups_tiles) {
  int unit = (n + 63) / 64 * 64;
  unit = unit < most ? unit : most;
  while (unit > 64 && groups_tiles * ((n + unit - 1) / unit) * 2 <= device_sm_count()) unit = (unit / 2 + 63) / 64 * 64;
  return unit;
}

// ---- cached rows: codes as bf16 numbers (exact), scales and rotated parts ----

constexpr int EX_THREADS = 256, EX_WARPS = EX_THREADS / 32, EX_ROWS = 32;  // rows a CTA

// Every CTA takes the running sum of the lengths for itself.
__global__ void __launch_bounds__(EX_THREADS) expand_rows_kernel(const ExpandArgs a, __nv_bfloat16* x, float* scale) {
  extern __shared__ int32_t cu[];  // [num_req + 1]
  asm volatile("griddepcontrol.launch_dependents;");  // the products' CTAs may get ready meanwhile
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

  // ---- where the CTA's rows are, a thread a row; then 16 bytes a thread ----
  __shared__ int32_t s_slot[EX_ROWS];
  const int n0 = blockIdx.x * EX_ROWS;
  if (tid < EX_ROWS && n0 + tid < total) {
    const int n = n0 + tid;
    int lo = 0, hi = R - 1;  // the request with cu[r] <= n < cu[r + 1]
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (cu[mid + 1] > n) hi = mid;
      else lo = mid + 1;
    }
    const int pos = n - cu[lo], page = a.block_table[(int64_t)lo * a.bt_stride + pos / a.page_size];
    const bool good = page >= 0 && page < a.num_pages;
    if (!good) report(a.dev_status, DSA_DEV_BAD_PAGE);
    const int slot = good ? page * a.page_size + pos % a.page_size : -1;  // (num_pages page_size < 2^31)
    s_slot[tid] = slot;
  }
  __syncthreads();
  const int dl = a.d_latent, row_bytes = dl + a.d_rope, chunks = row_bytes / 16;
  const int rows = min(EX_ROWS, total - n0);
  for (int e = tid; e < rows * chunks; e += EX_THREADS) {
    const int i = e / chunks, c = e - i * chunks, slot = s_slot[i], n = n0 + i;
    // (the row's scale beside its bytes, where it is needed)
    const float sc = slot >= 0 && 16 * (c + 1) >= dl ? __ldg(a.kv_scale + slot) : 0.f;
    if (16 * (c + 1) == dl) scale[n] = sc;
    const uint4 v = slot >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.kv + (int64_t)slot * row_bytes) + c) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const bool rope = 16 * c >= dl;
    __align__(16) __nv_bfloat162 y[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[q / 2] >> (16 * (q & 1))), __NV_E4M3));
      float2 f = __half22float2(h);
      if (rope) f.x *= sc, f.y *= sc;
      y[q] = __floats2bfloat162_rn(f.x, f.y);  // (a code is exact in bf16)
    }
    __nv_bfloat16* dst = rope ? static_cast<__nv_bfloat16*>(a.k_rope) + (int64_t)n * a.d_rope + (16 * c - dl)
                              : x + (int64_t)n * dl + 16 * c;
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<uint4*>(y);
    *reinterpret_cast<uint4*>(dst + 8) = *reinterpret_cast<uint4*>(y + 4);
  }
}

}  // namespace

cudaError_t launch_absorb_q(const LatentProjArgs& a, cudaStream_t stream) {
  const int d_w = a.d_nope + a.d_v, d_out = a.d_latent + a.d_rope;
  const int64_t mt = ((int64_t)a.num_tokens + TM - 1) / TM;
  Product p = {};
  p.m = a.num_tokens, p.n = a.d_latent, p.k = a.d_nope;
  p.n_unit = columns_of_unit(p.n, 512, a.heads * mt);
  p.per_group = (p.n + p.n_unit - 1) / p.n_unit;
  p.units = a.heads * p.per_group;
  p.b_row0 = 0, p.b_group = d_w;
  p.rope_x = a.d_rope > 0 ? a.d_nope : -1;
  p.dev_status = a.dev_status;
  ProductMaps maps = {};
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y);
  if (!make_rows_map(&maps.a, a.x, a.num_tokens, a.heads, a.d_nope + a.d_rope, a.tok_stride, a.head_stride, TM) ||
      !make_rows_map(&maps.b, a.w, (int64_t)a.heads * d_w, 1, a.d_latent, a.d_latent, 0, (uint32_t)a.d_nope) ||
      !make_rows_map(&maps.c, y, a.num_tokens, a.heads, a.d_latent, (int64_t)a.heads * d_out, d_out, 32) ||
      !make_rows_map(&maps.c_rope, y + (a.d_rope > 0 ? a.d_latent : 0), a.num_tokens, a.heads,
                     a.d_rope > 0 ? a.d_rope : a.d_latent, (int64_t)a.heads * d_out, d_out, 32))
    return cudaErrorInvalidValue;
  return launch_product<ABSORB>(p, maps, stream);
}

cudaError_t launch_project_out(const LatentProjArgs& a, cudaStream_t stream) {
  const int d_w = a.d_nope + a.d_v;
  const int64_t mt = ((int64_t)a.num_tokens + TM - 1) / TM;
  Product p = {};
  p.m = a.num_tokens, p.n = a.d_v, p.k = a.d_latent;
  p.n_unit = columns_of_unit(p.n, 128, a.heads * mt);
  p.per_group = (p.n + p.n_unit - 1) / p.n_unit;
  p.units = a.heads * p.per_group;
  p.b_row0 = a.d_nope, p.b_group = d_w;
  p.dev_status = a.dev_status;
  p.out = static_cast<__nv_bfloat16*>(a.y), p.ldc = (int64_t)a.heads * a.d_v;
  p.wide = reinterpret_cast<uintptr_t>(a.y) % 32 == 0;
  p.rope_x = -1;
  ProductMaps maps = {};
  if (!make_rows_map(&maps.a, a.x, a.num_tokens, a.heads, a.d_latent, a.tok_stride, a.head_stride, TM) ||
      !make_rows_map(&maps.b, a.w, (int64_t)a.heads * d_w, 1, a.d_latent, a.d_latent, 0, (uint32_t)p.n_unit))
    return cudaErrorInvalidValue;
  return launch_product<PROJECT>(p, maps, stream);
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
  Product p = {};
  p.m = a.capacity, p.n = a.heads * a.d_kv, p.k = a.d_latent;
  p.n_unit = 256;
  p.per_group = p.units = (p.n + p.n_unit - 1) / p.n_unit;
  p.rope_x = -1;
  p.rows = a.cu_k + a.num_req;
  p.scale = scale;
  p.out = static_cast<__nv_bfloat16*>(a.kv_out), p.ldc = p.n;
  p.wide = reinterpret_cast<uintptr_t>(a.kv_out) % 32 == 0;
  p.dev_status = a.dev_status;
  ProductMaps maps = {};
  if (!make_rows_map(&maps.a, x, a.capacity, 1, a.d_latent, a.d_latent, 0, TM) ||
      !make_rows_map(&maps.b, a.w, p.n, 1, a.d_latent, a.d_latent, 0, (uint32_t)p.n_unit / 2))
    return cudaErrorInvalidValue;
  return launch_product<EXPAND>(p, maps, stream);
}

}  // namespace dsa
