// Attention of a chunk of new tokens over every visible position of the paged
// FP8 cache, on the Blackwell tensor cores (tcgen05 + TMEM + TMA).
//
// "Accelerating GLM-5.3-Flash on H200", section 3: QK^T, online softmax and
// the weighted value sum one KV tile at a time, splits merged by a Combine
// step; "GLM-5.3 Optimizations, Part 2" ("Interpretation"): a latent KV row is
// shared by all 64 heads.  For token i with request r and position p:
//   z_j = softmax_scale q . x_j,  x_j = e4m3(kv[slot_j]) s_j,  j = 0 .. p
//   out = sum_j softmax(z)_j x_j[:512],  lse = ln sum_j exp z_j
//
// One CTA = one token x one KV split (the 64 heads are the work that shares a
// row; the tokens of a request run side by side and share its rows in L2).
// A 64-row tile is 64 x 64 x (576 + 512) products twice (below), 1,376 cycles of
// MMAs, and takes about 1,900: the P V of a tile needs its weights, and those its
// QK^T, so the softmax's latency is hidden by two tiles only, and a long call
// runs at the power limit.  Measured, pages of 64: 1,024 tokens at the end of 16,384
// positions in 1.48 ms (1,525 TFLOP/s of the formula's bf16 products, the
// weights' second half not counted); 128 tokens of 16 requests, 4,096 positions
// each, 62 us in one split and 77 in the two that the rule takes where it does not
// know that all are live; 32 requests of 4,096 to 8,192 positions 40.4 us in four
// (118 MB of rows, 2.9 TB/s).  Warps:
//  * 3 (or 7) TMA warps bring KV tiles of 64 rows, FP8 as they are in the cache, five
//    tiles in flight.  A tile whose positions are all visible comes in boxes
//    of 64, 32, 16 or 8 rows, the largest that divides the page size (5 to
//    40 copies; a bad page reads as zeros); the last tile, and page sizes that
//    are not a multiple of 8, four rows a copy (tile::gather4, 80 copies), rows past the
//    last position reading as zeros, so that nothing behind it reaches an MMA.
//  * 1 MMA warp issues kind::f8f6f4 MMAs:
//        S    = [Q_hi ; Q_lo] K^T          M = 128, N = 64 rows, K = 576
//        O^T += V^T P_hi^T + V^T P_lo^T    M = 4 x 128 latent dims, N = 64 heads, K = 64 rows
//    Q's latent part is the A operand in tensor memory, its rope part and K
//    are in shared memory; V^T is the same tile read MN-major.
//  * 16 softmax warps turn S into P: lane quadrant q holds heads 16 q .. + 15,
//    Q_hi rows in lanes 0-15 and Q_lo rows in lanes 16-31.  A thread owns one
//    head and 8 rows of the tile; two 16-lane loads, whose half-warps take
//    different columns, bring it both halves of its logits.
// Q = Q_hi + Q_lo: two E4M3 numbers of a head scaled by a power of two, exact for
// bf16 values down to 2^-9 of the head's largest, below that to 2^-17 of it (E4M3's
// steps end: 0.4% of a Gaussian head).
// A weight P' = p s_j F is E4M3 + E5M2.  p = 2^(z - m) with a reference m for each
// head, and F, also the head's, puts the largest p s_j at 16: what counts is how much
// a row adds, not its scale alone, so one row of a huge scale and no weight takes no
// bits from the others (with one F for the largest scale, 2^14 times the others': 5%
// off, 2^22: nothing left).  16 is an exact value: a head that looks at one row
// gives that row.  Weights down to 2^-10 of the largest have a relative error of at
// most 2^-8 (0.13% root mean square, a bf16 weight's is 0.08%); smaller ones an
// absolute one of 2^-14 (of 16), and only below 2^-21 of the largest nothing is left
// of them.  A second E4M3 number would end at 2^-14: over a long context the many
// small weights of a flat tail are a share of the result that must not be rounded away.
// Lazy rescaling: m and F move when a weight nears 448, the largest E4M3 value; l is
// summed in fp32 from unrounded p.  (Of 64 heads some weight passes a bound in few
// tiles; with a bound 2^2 above 16, 152 tokens of 4,096 take 82 instead of 62 us.)
// All waits are bounded.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.cuh"
#include "mla_tc_common.cuh"
#include "sm100_ptx.cuh"

namespace cg = cooperative_groups;

namespace dsa {
namespace {

using namespace sm100;

constexpr int H = 64, DL = 512, DR = 64, DQK = DL + DR;
constexpr int T = 64;                           // KV rows per tile
constexpr int NST = 5;                          // KV tiles in flight
constexpr int NLAT = DL / 128;                  // 128-column latent slices per row
constexpr int LAT_BYTES = T * 128;              // one latent slice of a tile (128-byte swizzle)
constexpr int ROPE_OFF = NLAT * LAT_BYTES;      // the rope slice (64-byte swizzle)
constexpr int STAGE_BYTES = ROPE_OFF + T * DR;  // 36 KB
constexpr int QM = 2 * H;
constexpr int QROPE_BYTES = QM * DR;
constexpr int P_BYTES = H * T;  // P_hi (or P_lo) of a tile: [head][row], K-major, 64-byte swizzle
constexpr int NPB = 2;
constexpr int MAX_MERGED = chunk_max_merged();
constexpr int SM_WARPS = 16, SM_THREADS = SM_WARPS * 32;
constexpr float P_REF_LOG2 = 4.0f;    // F puts the largest weight at 2^4,
constexpr float P_TOP_LOG2 = 8.5f;    // and moves before one reaches 448 = 2^8.8, the largest E4M3 value
constexpr float S_MIN_LOG2 = -60.0f;  // in both a scale counts as 2^-60 at least: neither F nor p grows past all bounds
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// TMEM columns: two S buffers, Q's latent operand, O^T (4 chunks of 64 heads).
// Q row (= lane) of head h: 32 (h / 16) + h % 16 for Q_hi, 16 more for Q_lo.
constexpr uint32_t TM_S = 0, TM_Q = 2 * T, TM_O = 256, TM_COLS = 512;
static_assert(TM_Q + DL / 4 == TM_O, "S, Q and O fill the 512 TMEM columns");
__device__ constexpr int q_row(int h, int lo) { return 32 * (h >> 4) + (h & 15) + 16 * lo; }

// shared memory (offsets from a 1024-byte aligned base)
constexpr int OFF_KV = 0;
constexpr int OFF_QR = OFF_KV + NST * STAGE_BYTES;
constexpr int OFF_P = OFF_QR + QROPE_BYTES;           // [buffer][hi, lo]
constexpr int OFF_RED = OFF_P + NPB * 2 * P_BYTES;    // [2][4 row parts][64 heads] floats
constexpr int OFF_ALPHA = OFF_RED + 8 * H * 4;        // per-head factor of O
constexpr int OFF_SROW = OFF_ALPHA + H * 4;           // [NST][64] the tiles' row scales
constexpr int OFF_SLOG = OFF_SROW + NST * T * 4;      // [NST][64] their logarithms
constexpr int OFF_INFO = OFF_SLOG + NST * T * 4;      // [NST][2] valid rows of each 32 (bits)
constexpr int OFF_ML = OFF_INFO + NST * 2 * 4;         // [2][64] for the cluster's merge
constexpr int OFF_QS = OFF_ML + 2 * H * 4;             // [64] the heads' 2^e of Q, and logits' factor
constexpr int OFF_FLAG = OFF_QS + H * 8;               // O flags [4]
constexpr int OFF_BAR = OFF_FLAG + 128;
constexpr int B_KVF = 0;               // [NST] the tile in stage s has landed
constexpr int B_KVE = B_KVF + NST;     // [NST] stage s is free
constexpr int B_SF = B_KVE + NST;      // [2] S buffer b is complete
constexpr int B_PF = B_SF + 2;         // [2] P buffer b is written (and O rescaled)
constexpr int B_PVD = B_PF + NPB;      // [2] P V of the tile in P buffer b is done
constexpr int B_FIN = B_PVD + NPB;     // every MMA is done
constexpr int B_QREADY = B_FIN + 1;    // Q is converted (and its staging stages are free)
constexpr int B_QLOAD = B_QREADY + 1;  // raw bf16 Q has landed in the staging stages
constexpr int NBAR = B_QLOAD + 1;
constexpr int QSTAGE = NST - 2;
static_assert(2 * STAGE_BYTES == H * DQK * 2, "bf16 Q fills two KV stages");
constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr int SMEM_BYTES = OFF_TMEM + 16 + 1024;  // with alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
static_assert(H * DL * 4 <= NST * STAGE_BYTES && MAX_MERGED * H * 4 <= NPB * 2 * P_BYTES, "the merge's O and factors");
static_assert(OFF_QR % 1024 == 0 && OFF_P % 1024 == 0 && STAGE_BYTES % 1024 == 0, "swizzle atoms stay aligned");

struct ChunkMaps {
  CUtensorMap lat_box, rope_box;  // box_rows rows
  CUtensorMap lat_row, rope_row;  // one row, for tile::gather4
};

// NTMA TMA warps (0 .. NTMA - 1), then the MMA warp, then the softmax warps.
// MERGE: a token's splits are the CTAs of a thread-block cluster and merge
// their results over distributed shared memory (no partials, no Combine kernel).
template <int NTMA, bool MERGE>
__global__ void __launch_bounds__((NTMA + 1 + SM_WARPS) * 32, 1)
    mla_chunk_kernel(const MlaArgs a, const int32_t* __restrict__ q_pos, const __grid_constant__ ChunkMaps maps,
                     const int box_rows, const FastDiv page_div) {
  constexpr int WARP_MMA = NTMA, SM_WARP0 = NTMA + 1, NTHREADS = (SM_WARP0 + SM_WARPS) * 32;
  static_assert(SM_WARP0 % 4 == 0, "a softmax warp's TMEM lanes are those of its warp number modulo 4");
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red_s = reinterpret_cast<float*>(smem + OFF_RED);
  float* alpha_s = reinterpret_cast<float*>(smem + OFF_ALPHA);
  int* resc_s = reinterpret_cast<int*>(smem + OFF_FLAG);
  float2* qs_s = reinterpret_cast<float2*>(smem + OFF_QS);
  float* srow = reinterpret_cast<float*>(smem + OFF_SROW);
  float* slog = reinterpret_cast<float*>(smem + OFF_SLOG);
  uint32_t* info = reinterpret_cast<uint32_t*>(smem + OFF_INFO);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
  auto bar = [&](int b) { return smem_u32(bars + b); };
  auto wait_warp = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity)); };

  // (the shuffles tell the compiler that a value is the same for the whole
  // warp: the MMA warp's loop and descriptors then need no vector registers)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // the last tokens first: in a causal chunk they see the most
  const int i = (int)gridDim.x - 1 - (int)blockIdx.x;
  const int split = blockIdx.y, S = gridDim.y;
  const int P = a.page_size;
  const int32_t r = __shfl_sync(0xffffffffu, a.q_req[i], 0), last = __shfl_sync(0xffffffffu, q_pos[i], 0);
  const bool req_ok = r >= 0 && r < a.num_req;
  const bool pos_ok = last >= -1 && last <= INT32_MAX - T && page_div(max(last, 0)) < a.bt_stride;
  if (tid == 0) {
    if (!req_ok && r != -1) report(a.dev_status, DSA_DEV_BAD_PAGE);
    if (req_ok && !pos_ok) report(a.dev_status, DSA_DEV_BAD_QPOS);
  }
  const int n = req_ok && pos_ok ? last + 1 : 0;  // visible positions
  const int ntiles = (n + T - 1) / T;
  const int t_begin = (int)((int64_t)ntiles * split / S), t_end = (int)((int64_t)ntiles * (split + 1) / S);
  const int ntl = t_end - t_begin;

  float* ml_s = reinterpret_cast<float*>(smem + OFF_ML);  // MERGE: [64] references, [64] l
  // A split without tiles goes the whole way (no tile, l = 0) where the
  // cluster's other CTAs need its answer.
  if (MERGE ? n == 0 : ntl == 0) {  // nothing to see: O = 0, lse = -inf
    if (MERGE && split > 0) return;
    for (int e = tid; e < H * DL; e += NTHREADS) {
      if (MERGE || S == 1) static_cast<__nv_bfloat16*>(a.out)[(int64_t)i * H * DL + e] = __float2bfloat16_rn(0.f);
      else a.o_part[((int64_t)split * a.num_q + i) * H * DL + e] = 0.f;
    }
    for (int h = tid; h < H; h += NTHREADS) {
      if (!MERGE && S > 1) a.lse_part[((int64_t)split * a.num_q + i) * H + h] = -INFINITY;
      else if (a.lse) a.lse[(int64_t)i * H + h] = -INFINITY;
    }
    return;
  }

  // ---------------- setup ----------------
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), TM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar(B_KVF + s), NTMA);
      mbar_init(bar(B_KVE + s), 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(bar(B_SF + b), 1);
    for (int b = 0; b < NPB; ++b) {
      mbar_init(bar(B_PF + b), SM_WARPS);
      mbar_init(bar(B_PVD + b), 1);
    }
    mbar_init(bar(B_FIN), 1);
    mbar_init(bar(B_QREADY), SM_WARPS);
    mbar_init(bar(B_QLOAD), 1);
    fence_mbarrier_init();
    tma_prefetch_map(&maps.lat_box);
    tma_prefetch_map(&maps.rope_box);
    tma_prefetch_map(&maps.lat_row);
    tma_prefetch_map(&maps.rope_row);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint32_t kv_base = smem_u32(smem + OFF_KV), qr_base = smem_u32(smem + OFF_QR), p_base = smem_u32(smem + OFF_P);
  bool ok = true;
  const int32_t* bt = a.block_table + (int64_t)r * a.bt_stride;
  // the page id of a visible position, and the position's cache row (-1: no such page)
  auto page_of = [&](int pos) -> int { return __ldg(bt + page_div(pos)); };
  auto slot_in = [&](int page, int pos) -> int {
    return page >= 0 && page < a.num_pages ? page * P + (pos - page_div(pos) * P) : -1;
  };

  if (warp < NTMA) {
    // ---------------- TMA warps ----------------
    if (tid == 0) {  // raw Q into the staging stages
      mbar_arrive_expect_tx(bar(B_QLOAD), 2 * STAGE_BYTES);
      tma_bulk_load(kv_base + QSTAGE * STAGE_BYTES, static_cast<const __nv_bfloat16*>(a.q) + (int64_t)i * H * DQK,
                    2 * STAGE_BYTES, bar(B_QLOAD));
    }
    // A tile's copies are numbered group-major, c = 5 g + slice (four latent
    // slices, then rope), and dealt to the warps in runs, one copy a lane.
    // Boxes: groups of box_rows rows, y the row of the first; else groups of 4.
    struct Deal {
      int g, part;
      bool has;
      uint32_t bytes;  // this warp's bytes per tile
    };
    auto deal = [&](int rows) {
      const int nc = (NLAT + 1) * (T / rows);
      // Warps 0 and 1 look up the scales too: of seven, they take a fifth of many copies (152
      // tokens of 4,096 positions at page size 4: 104 us, 111 with even shares).  At most
      // 32 each: 80 copies are 27 of three warps, 13 of seven.
      auto first = [&](int w) {
        if (NTMA < 7 || nc < 40) return nc * w / NTMA;
        return w < 2 ? nc * w / 10 : nc / 5 + (nc - nc / 5) * (w - 2) / (NTMA - 2);
      };
      const int c0 = first(warp), c = c0 + lane;
      Deal d;
      d.g = c / (NLAT + 1), d.part = c % (NLAT + 1);
      d.has = lane < first(warp + 1) - c0;
      d.bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, d.has && d.part < NLAT)) * 128u * rows +
                (uint32_t)__popc(__ballot_sync(0xffffffffu, d.has && d.part == NLAT)) * (uint32_t)DR * rows;
      return d;
    };
    const Deal db = deal(box_rows > 0 ? box_rows : 4), dg = deal(4);
    const int past = (int)(a.num_pages * P);  // a row past the pool: reads as zeros
    auto boxed = [&](int lt) { return box_rows > 0 && (t_begin + lt + 1) * T <= n; };
    // The loop looks ahead: the page ids of tile lt + 3 are loaded, and the scales
    // behind those of lt + 2, while tile lt's copies are issued; one round trip to
    // L2 an iteration, in the shadow of the tiles in flight.
    // Page ids of this lane's copy of tile lt (a box: the first row's, in x).
    auto pages_of = [&](int lt) -> int4 {
      int4 v = make_int4(-1, -1, -1, -1);
      if (lt >= ntl) return v;
      const int base = (t_begin + lt) * T;
      if (boxed(lt)) {
        if (db.has) v.x = page_of(base + db.g * box_rows);
      } else if (dg.has) {
        const int pos = base + 4 * dg.g;
        if (pos < n) v.x = page_of(pos);
        if (pos + 1 < n) v.y = page_of(pos + 1);
        if (pos + 2 < n) v.z = page_of(pos + 2);
        if (pos + 3 < n) v.w = page_of(pos + 3);
      }
      return v;
    };
    // Warps 0 and 1 also look up the scales of a tile's rows 32 warp + lane.
    auto row_pos = [&](int lt) { return (t_begin + lt) * T + 32 * warp + lane; };
    auto row_page = [&](int lt) { return warp < 2 && lt < ntl && row_pos(lt) < n ? page_of(row_pos(lt)) : -1; };
    auto row_slot = [&](int lt, int page) -> int {
      if (warp > 1 || lt >= ntl || row_pos(lt) >= n) return -1;
      const int s = slot_in(page, row_pos(lt));
      if (s < 0) report(a.dev_status, DSA_DEV_BAD_PAGE);
      return s;
    };
    auto row_scale = [&](int slot) -> float { return slot >= 0 ? __ldg(a.kv_scale + slot) : 0.f; };
    int issued = 0;
    int4 pg0 = pages_of(0), pg1 = pages_of(1), pg2 = pages_of(2);
    int rp2 = row_page(2);
    int slot0 = row_slot(0, row_page(0)), slot1 = row_slot(1, row_page(1));
    float sc0 = row_scale(slot0), sc1 = row_scale(slot1);
    auto scale_log = [](float sc) { return fmaxf(__log2f(fabsf(sc)), S_MIN_LOG2); };
    float lg0 = scale_log(sc0);
    for (int lt = 0; lt < ntl; ++lt) {
      const int s = lt % NST;
      const int4 pg3 = pages_of(lt + 3);
      const int rp3 = row_page(lt + 3);
      const int slot2 = row_slot(lt + 2, rp2);
      const float sc2 = row_scale(slot2);
      if (lt >= NST && !wait_warp(B_KVE + s, ((lt - NST) / NST) & 1)) {
        ok = false;
        break;
      }
      if (lt == QSTAGE && !wait_warp(B_QREADY, 0)) {  // the staging stages hold raw Q until then
        ok = false;
        break;
      }
      if (warp < 2) {
        const unsigned valid = __ballot_sync(0xffffffffu, slot0 >= 0);
        srow[s * T + 32 * warp + lane] = sc0;
        slog[s * T + 32 * warp + lane] = lg0;
        if (lane == 0) info[s * 2 + warp] = valid;
        __syncwarp();
      }
      const uint32_t dst = kv_base + s * STAGE_BYTES;
      const bool bx = boxed(lt);
      if (lane == 0) mbar_arrive_expect_tx(bar(B_KVF + s), bx ? db.bytes : dg.bytes);
      __syncwarp();
      const int base = (t_begin + lt) * T;
      if (bx) {
        if (db.has) {
          const int row0 = slot_in(pg0.x, base + db.g * box_rows), y = row0 >= 0 ? row0 : past;
          if (db.part < NLAT)
            tma_load_2d(dst + db.part * LAT_BYTES + db.g * box_rows * 128, &maps.lat_box, db.part * 128, y, bar(B_KVF + s));
          else
            tma_load_2d(dst + ROPE_OFF + db.g * box_rows * DR, &maps.rope_box, DL, y, bar(B_KVF + s));
        }
      } else if (dg.has) {  // (page -1 past the last position: row -1)
        const int pos = base + 4 * dg.g;
        const int4 rows = make_int4(slot_in(pg0.x, pos), slot_in(pg0.y, pos + 1), slot_in(pg0.z, pos + 2),
                                    slot_in(pg0.w, pos + 3));
        if (dg.part < NLAT)
          tma_gather4(dst + dg.part * LAT_BYTES + dg.g * 512, &maps.lat_row, dg.part * 128, rows, bar(B_KVF + s));
        else
          tma_gather4(dst + ROPE_OFF + dg.g * 256, &maps.rope_row, DL, rows, bar(B_KVF + s));
      }
      pg0 = pg1, pg1 = pg2, pg2 = pg3;
      rp2 = rp3;
      slot0 = slot1, slot1 = slot2;
      sc0 = sc1, sc1 = sc2;
      lg0 = scale_log(sc0);  // (after the copies are out)
      issued = lt + 1;
    }
    // no copy may land after the CTA is gone
    for (int lt = issued > NST ? issued - NST : 0; lt < issued; ++lt)
      if (!wait_warp(B_KVF + lt % NST, (lt / NST) & 1)) ok = false;
    if (warp == 0 && !wait_warp(B_QLOAD, 0)) ok = false;
    if (!ok && lane == 0) report(a.dev_status, DSA_DEV_TIMEOUT);
  } else if (warp == WARP_MMA) {
    // ---------------- MMA warp ----------------
    constexpr uint32_t ID_QK = idesc_f16_f32(QM, T, 0, 0, 0);      // kind::f8f6f4: E4M3 x E4M3 -> f32
    constexpr uint32_t ID_PV_HI = idesc_f16_f32(128, H, 1, 0, 0);
    constexpr uint32_t ID_PV_LO = ID_PV_HI | (1u << 10);           // B is E5M2
    // the tensor memory of a CTA that holds all 512 columns starts at 0: the
    // addresses below are then constants and the descriptors warp-uniform
    const uint64_t a_rope = smem_desc(qr_base, 16, 512, SWIZZLE_64B);
    const uint64_t lat0 = smem_desc(kv_base, 16, 1024, SWIZZLE_128B);
    const uint64_t rope0 = smem_desc(kv_base + ROPE_OFF, 16, 512, SWIZZLE_64B);
    const uint64_t v0 = smem_desc(kv_base, LAT_BYTES, 1024, SWIZZLE_128B);
    const uint64_t p0 = smem_desc(p_base, 16, 512, SWIZZLE_64B);
    auto issue_qk = [&](int stage, int sb) {
      const uint64_t b_lat = lat0 + (uint32_t)(stage * (STAGE_BYTES >> 4));
      const uint64_t b_rope = rope0 + (uint32_t)(stage * (STAGE_BYTES >> 4));
      const uint32_t d = TM_S + T * sb;
#pragma unroll
      for (int ka = 0; ka < NLAT; ++ka) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f8_ts_warp(d, TM_Q + 8 * (4 * ka + kk), b_lat + ((ka * LAT_BYTES + kk * 32) >> 4), ID_QK,
                         (ka | kk) ? 1u : 0u);
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) mma_f8_ss_warp(d, a_rope + ((kk * 32) >> 4), b_rope + ((kk * 32) >> 4), ID_QK, 1u);
      mma_commit_warp(bar(B_SF + sb));
    };
    auto issue_pv = [&](int stage, int pb, uint32_t acc) {
      const uint64_t a0 = v0 + (uint32_t)(stage * (STAGE_BYTES >> 4));
      const uint64_t b0 = p0 + (uint32_t)(pb * ((2 * P_BYTES) >> 4));
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int kk = 0; kk < T / 32; ++kk) {
#pragma unroll
          for (int c = 0; c < NLAT; ++c)  // consecutive MMAs never share an accumulator
            mma_f8_ss_warp(TM_O + 64 * c, a0 + ((c * LAT_BYTES + kk * 32 * 128) >> 4),
                           b0 + ((w * P_BYTES + kk * 32) >> 4), w ? ID_PV_LO : ID_PV_HI, w > 0 || kk > 0 ? 1u : acc);
        }
      }
      mma_commit_warp(bar(B_KVE + stage));
      mma_commit_warp(bar(B_PVD + pb));
    };
    // Reductions over the warp leave their result in a uniform register: the
    // loop's counters and descriptors then need no per-MMA moves.
    auto wait_u = [&](int b, uint32_t parity) { return __reduce_min_sync(0xffffffffu, (uint32_t)mbar_wait(bar(b), parity)); };
    const int nt = __reduce_max_sync(0xffffffffu, ntl);
    uint32_t good = __reduce_min_sync(0xffffffffu, (uint32_t)(tmem == 0)) & wait_u(B_QREADY, 0);
    for (int lt = 0; lt < 2 && lt < nt && good; ++lt) {
      good = wait_u(B_KVF + lt, 0);
      tc_fence_after_sync();
      if (good) issue_qk(lt, lt);
    }
    int stage = 0, far = 2, far_phase = 0;  // the stages of tiles lt and lt + 2
    for (int lt = 0; lt < nt && good; ++lt) {
      // the tile after next has usually landed long ago: looked at first, so
      // that nothing but the two MMA groups sits between two waits for P
      if (lt + 2 < nt) good = wait_u(B_KVF + far, far_phase);
      good &= wait_u(B_PF + (lt & 1), (lt >> 1) & 1);
      if (!good) break;
      tc_fence_after_sync();
      issue_pv(stage, lt & 1, lt > 0 ? 1u : 0u);
      if (lt + 2 < nt) issue_qk(far, lt & 1);  // S buffer lt % 2 has been read
      stage = stage == NST - 1 ? 0 : stage + 1;
      if (far == NST - 1) far = 0, far_phase ^= 1;
      else ++far;
    }
    ok = good != 0;
    __syncwarp();
    mma_commit_warp(bar(B_FIN));
    if (!wait_warp(B_FIN, 0)) ok = false;  // every MMA is done before TMEM is released
    if (!ok && lane == 0) report(a.dev_status, DSA_DEV_TIMEOUT);
  } else {
    // ---------------- softmax warps ----------------
    const int sw = warp - SM_WARP0, st = tid - SM_WARP0 * 32;
    const int q4 = warp & 3;              // TMEM lane quadrant: heads 16 q4 .. + 15
    const int part = sw >> 2;             // tile rows 16 part .. + 15; O heads 16 part .. + 15
    const int hh = 16 * q4 + (lane & 15);  // this thread's head
    const int up = lane >> 4;             // 0: this lane holds Q_hi logits, 1: Q_lo; rows 16 part + 8 up .. + 7
    const uint32_t t_lane = tmem + ((uint32_t)(32 * q4) << 16);
    auto group_sync = [] { named_barrier_sync(2, SM_THREADS); };

    // ---- Q: bf16 -> x 2^qexp -> E4M3 hi and lo, latent part to TMEM, rope part to shared memory ----
    {
      constexpr int CH = DQK / 8;  // 16-byte chunks (8 bf16) per head
      const uint4* qraw = reinterpret_cast<const uint4*>(smem + OFF_KV + QSTAGE * STAGE_BYTES);
      auto bf_lo = [](uint32_t w) { return __uint_as_float(w << 16); };
      auto bf_hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
      if (!wait_warp(B_QLOAD, 0)) ok = false;
      // Eight threads a head: its largest |q| < 2^e puts Q at 2^8 below (2^(8 - e) stays finite:
      // a query below 2^-120 is as good as zero).
      {
        const int h = st >> 3;
        float mx = 0.f;  // (a NaN loses to a number; it stays one in E4M3)
#pragma unroll
        for (int u = 0; u < CH / 8; ++u) {
          const uint4 v = qraw[h * CH + (st & 7) + 8 * u];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int t = 0; t < 4; ++t) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(w[t])), fabsf(bf_hi(w[t]))));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if ((st & 7) == 0) {
          int e = 0;
          frexpf(mx, &e);
          const int x = mx > 0.f && mx < INFINITY ? min(8 - e, 100) : 0;
          // A negative softmax scale is Q's sign.  E4M3 has no infinity: the factor makes its head NaN.
          const float qk = fabsf(a.softmax_scale) * LOG2E * ldexpf(1.f, -x);
          qs_s[h] = make_float2(copysignf(ldexpf(1.f, x), a.softmax_scale), mx < INFINITY ? qk : NAN);
        }
      }
      group_sync();
      auto split8 = [&](const uint4 v, float qs, uint2& hv, uint2& lv) {  // 8 elements as byte quadruples
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float y0, y1;
          upk2(mul2(pk2(bf_lo(w[t]), bf_hi(w[t])), pk2(qs, qs)), y0, y1);
          split_e4m3x2(f32x2_to_f16x2(y0, y1), hi[t], lo[t]);
        }
        hv = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
        lv = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
      };
      const float qs_own = qs_s[hh].x;
      // Lane u writes row 32 q4 + u: Q_hi (u < 16) or Q_lo of head hh.  The two
      // lanes of a head split each 32-element block's chunks and swap halves
      // (loads staggered over the banks).
      for (int j = part; j < DL / 32; j += 4) {
        const uint4* src = qraw + hh * CH + 4 * j + 2 * up;
        const uint4 ra = src[lane & 1], rb = src[(lane & 1) ^ 1];
        uint2 keep[2], recv[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint2 hv, lv;
          split8((t ^ (lane & 1)) ? rb : ra, qs_own, hv, lv);
          keep[t] = up ? lv : hv;
          const uint2 send = up ? hv : lv;
          recv[t] = make_uint2(__shfl_xor_sync(0xffffffffu, send.x, 16), __shfl_xor_sync(0xffffffffu, send.y, 16));
        }
        const uint2 c0 = up ? recv[0] : keep[0], c1 = up ? recv[1] : keep[1];
        const uint2 c2 = up ? keep[0] : recv[0], c3 = up ? keep[1] : recv[1];
        const uint32_t col[8] = {c0.x, c0.y, c1.x, c1.y, c2.x, c2.y, c3.x, c3.y};
        tmem_st8(t_lane + TM_Q + 8 * j, col);
      }
      tmem_wait_st();
      unsigned char* qr = smem + OFF_QR;
      for (int e = st; e < H * (DR / 8); e += SM_THREADS) {
        const int h = e >> 3, c = e & 7;
        uint2 hv, lv;
        split8(qraw[h * CH + DL / 8 + c], qs_s[h].x, hv, lv);
        const int cc = c >> 1, hf = c & 1, rh = q_row(h, 0), rl = q_row(h, 1);
        *reinterpret_cast<uint2*>(qr + rh * DR + ((cc ^ ((rh >> 1) & 3)) << 4) + hf * 8) = hv;
        *reinterpret_cast<uint2*>(qr + rl * DR + ((cc ^ ((rl >> 1) & 3)) << 4) + hf * 8) = lv;
      }
      // before the TMA warps' copies into the staging stages, and the MMAs
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_QREADY));
    }
    // logit (log2 domain) = (S_hi + S_lo) (s_j qk_scale), rounded as a number of its own: a
    // reference is one of the logits, and the difference to it is then exact however
    // large they are (in one fused step a logit of 2^31 was off by 2^7: weights of infinity)
    const float qk_scale = qs_s[hh].y;

    // ---- the tiles ----
    float m_ref = -INFINITY;      // head hh's reference m (log2 domain), the same in its 8 threads
    float f_log = 0.f, f_scale = 1.f;  // its log2 F and F
    uint64_t l2 = pk2(0.f, 0.f);  // its share of l = sum 2^(z - m), two running sums
    const uint64_t qk2 = pk2(qk_scale, qk_scale);
    int stage = 0, kv_phase = 0;
    for (int lt = 0; lt < ntl; ++lt) {  // no early exit: every warp reaches every barrier
      const int sb = lt & 1;
      if (ok && !wait_warp(B_KVF + stage, kv_phase)) ok = false;  // the tile's row scales
      // s_j qk_scale, s_j F, and log2(s_j F) - 8.5 - m: above 0 with the logit added, the
      // row's weight is too large (m = -inf: any)
      uint64_t sq[4], sf[4], su[4];
      const int row0 = stage * T + 16 * part + 8 * up;
      auto rows8 = [&](const float* of, uint64_t (&v)[4]) {
        const float4 lo = reinterpret_cast<const float4*>(of + row0)[0], hi = reinterpret_cast<const float4*>(of + row0)[1];
        v[0] = pk2(lo.x, lo.y), v[1] = pk2(lo.z, lo.w), v[2] = pk2(hi.x, hi.y), v[3] = pk2(hi.z, hi.w);
      };
      auto scaled = [&](const uint64_t (&v)[4], uint64_t f2, uint64_t (&to)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) to[c] = mul2(v[c], f2);
      };
      {
        uint64_t sj[4];
        rows8(srow, sj);
        scaled(sj, qk2, sq);
        scaled(sj, pk2(f_scale, f_scale), sf);
        rows8(slog, su);
        const float above = f_log - P_TOP_LOG2 - m_ref;
#pragma unroll
        for (int c = 0; c < 4; ++c) su[c] = add2(su[c], pk2(above, above));
      }
      if (ok && !wait_warp(B_SF + sb, (lt >> 1) & 1)) ok = false;
      const uint32_t rows = info[stage * 2 + (part >> 1)];
      tc_fence_after_sync();
      float z[8];  // the logits of head hh, rows 16 part + 8 up + c (invalid: -inf)
      {
        // lanes 0-15 of the quadrant hold the heads' S_hi, lanes 16-31 their S_lo
        float vh[8], vl[8];
        tmem_ld8x2(t_lane + TM_S + T * sb + 16 * part, vh);
        tmem_ld8x2(t_lane + (16u << 16) + TM_S + T * sb + 16 * part, vl);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; c += 2)
          upk2(mul2(add2(pk2(vh[c], vh[c + 1]), pk2(vl[c], vl[c + 1])), sq[c >> 1]), z[c], z[c + 1]);
        if (rows != 0xffffffffu) {  // a tile with rows past the last position, or bad pages
          const unsigned my_valid = rows >> (16 * (part & 1) + 8 * up);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (!((my_valid >> c) & 1u)) z[c] = -INFINITY;
        }
      }
      // Is a weight too large?  Every thread goes on as if none was; the vote comes
      // after the weights, which are computed again in the rare tile where some
      // thread's answer was yes.  (The answer from the weights themselves, which needs
      // no logarithms, comes so late that 1,024 tokens of 16,384 take 2.3 ms.)
      bool want;
      {
        float t[8];
#pragma unroll
        for (int c = 0; c < 8; c += 2) upk2(add2(pk2(z[c], z[c + 1]), su[c >> 1]), t[c], t[c + 1]);
        float tm = t[0];
#pragma unroll
        for (int c = 1; c < 8; ++c) tm = fmaxf(tm, t[c]);
        want = tm > 0.f;
      }
      uint32_t phi[4], plo[4];
      uint64_t ln;
      for (bool again = false;; again = true) {
        // p = 2^(z - m), summed into l; folded with s_j F, as E4M3 + E5M2
        const float shift = m_ref == -INFINITY ? 0.f : -m_ref;
        const uint64_t shift2 = pk2(shift, shift);
        ln = l2;
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          float d0, d1, w0, w1;
          upk2(add2(pk2(z[c], z[c + 1]), shift2), d0, d1);
          const uint64_t p = pk2(ex2(d0), ex2(d1));
          ln = add2(ln, p);
          upk2(mul2(p, sf[c >> 1]), w0, w1);
          split_e4m3_e5m2x2(f32x2_to_f16x2(w0, w1), phi[c >> 1], plo[c >> 1]);
        }
        if (again) break;
        if (!named_barrier_or(3, SM_THREADS, want)) break;  // one vote of the 16 warps: uniform
        // ---- move m to the largest logit, and F where the largest weight passed it; rescale O and l ----
        float zt = z[0], wt = -INFINITY;  // largest logit, and log2 of the largest p s_j with it as the reference
        uint64_t sj[4], sl[4];
        rows8(srow, sj);
        rows8(slog, sl);
#pragma unroll
        for (int c = 1; c < 8; ++c) zt = fmaxf(zt, z[c]);
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          float l0, l1;
          upk2(sl[c >> 1], l0, l1);
          wt = fmaxf(wt, fmaxf((z[c] - zt) + l0, (z[c + 1] - zt) + l1));
        }
        {
          const float zo = __shfl_xor_sync(0xffffffffu, zt, 16), wo = __shfl_xor_sync(0xffffffffu, wt, 16);
          const float zm = fmaxf(zt, zo);
          wt = fmaxf(wt + (zt - zm), wo + (zo - zm));
          zt = zm;
        }
        if (up == 0) red_s[part * H + hh] = zt, red_s[(4 + part) * H + hh] = wt;
        group_sync();
        float mn = m_ref;
#pragma unroll
        for (int c = 0; c < 4; ++c) mn = fmaxf(mn, red_s[c * H + hh]);
        wt = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) wt = fmaxf(wt, red_s[(4 + c) * H + hh] + (red_s[c * H + hh] - mn));
        float alpha = 1.f;
        if (mn != -INFINITY) {
          const float f_new = P_REF_LOG2 - wt;
          const float f_old = f_log + (mn - m_ref);  // F's exponent with m moved alone (m_ref = -inf: infinite)
          const bool move = f_old - f_new > P_TOP_LOG2 - P_REF_LOG2 - 0.5f;
          const float al = ex2(m_ref - mn);
          l2 = mul2(l2, pk2(al, al));
          if (move) alpha = ex2(f_new - f_old);
          f_log = move ? f_new : f_old;
          f_scale = ex2(f_log);
          m_ref = mn;
        }
        scaled(sj, pk2(f_scale, f_scale), sf);
        if (part == 0 && up == 0) alpha_s[hh] = alpha;
        const unsigned need = __ballot_sync(0xffffffffu, lt > 0 && alpha != 1.f);
        if (part == 0 && lane == 0) resc_s[q4] = need != 0u;
        group_sync();
        if (resc_s[0] | resc_s[1] | resc_s[2] | resc_s[3]) {
          // O must hold every P V issued so far: the previous tile's
          if (ok && !wait_warp(B_PVD + (lt - 1) % NPB, ((lt - 1) / NPB) & 1)) ok = false;
          tc_fence_after_sync();
          const float* al = alpha_s + 16 * part;
#pragma unroll 1
          for (int c = 0; c < NLAT; ++c) {
            float o[16];
            const uint32_t addr = t_lane + TM_O + 64 * c + 16 * part;
            tmem_ld16(addr, o);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 16; ++h) o[h] *= al[h];
            tmem_st16(addr, o);
          }
          tmem_wait_st();
        }
      }
      l2 = ln;
      // P buffer lt % 2 was last read by P V(lt - 2), issued before QK^T(lt): the
      // commit that completed S(lt) tracks it, so the buffer is free
      {
        unsigned char* pr = smem + OFF_P + (lt % NPB) * 2 * P_BYTES + hh * T + ((part ^ ((hh >> 1) & 3)) << 4) + 8 * up;
        *reinterpret_cast<uint2*>(pr) = make_uint2(phi[0] | (phi[1] << 16), phi[2] | (phi[3] << 16));
        *reinterpret_cast<uint2*>(pr + P_BYTES) = make_uint2(plo[0] | (plo[1] << 16), plo[2] | (plo[3] << 16));
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PF + lt % NPB));
      if (stage == NST - 1) stage = 0, kv_phase ^= 1;
      else ++stage;
    }
    // ---------------- epilogue ----------------
    if (ok && !wait_warp(B_FIN, 0)) ok = false;
    tc_fence_after_sync();
    {
      float la, lb;
      upk2(l2, la, lb);
      const float lp = la + lb, lw = lp + __shfl_xor_sync(0xffffffffu, lp, 16);
      if (up == 0) red_s[part * H + hh] = lw;
    }
    group_sync();
    if (part == 0 && up == 0) {
      const float l = (red_s[hh] + red_s[H + hh]) + (red_s[2 * H + hh] + red_s[3 * H + hh]);
      // (O carries F; a NaN is not an empty row)
      alpha_s[hh] = l != 0.f ? ex2(-f_log) * (MERGE ? 1.f : 1.f / l) : 0.f;
      const float lse = l != 0.f ? (m_ref + log2f(l)) * LN2 : -INFINITY;
      if (MERGE) ml_s[hh] = ok && l != 0.f ? m_ref : -INFINITY, ml_s[H + hh] = ok ? l : 0.f;
      else if (S > 1) a.lse_part[((int64_t)split * a.num_q + i) * H + hh] = lse;
      else if (a.lse) a.lse[(int64_t)i * H + hh] = lse;
    }
    group_sync();
    if (ok) {
      // thread (q4, lane) holds latent dim d = 128 c + 32 q4 + lane of heads
      // 16 part .. + 15: a warp's store covers 32 consecutive d of one head
      float inv[16];
#pragma unroll
      for (int h = 0; h < 16; ++h) inv[h] = alpha_s[16 * part + h];
#pragma unroll 1
      for (int c = 0; c < NLAT; ++c) {
        const int d = 128 * c + 32 * q4 + lane;
        float o[16];
        tmem_ld16(t_lane + TM_O + 64 * c + 16 * part, o);
        tmem_wait_ld();
        if (MERGE) {  // O into the idle KV stages, [head][dim]
          float* os = reinterpret_cast<float*>(smem + OFF_KV) + 16 * part * DL + d;
#pragma unroll
          for (int h = 0; h < 16; ++h) os[h * DL] = o[h] * inv[h];
        } else if (S == 1) {
          __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)i * H + 16 * part) * DL + d;
#pragma unroll
          for (int h = 0; h < 16; ++h) ob[h * DL] = __float2bfloat16_rn(o[h] * inv[h]);
        } else {
          float* op = a.o_part + (((int64_t)split * a.num_q + i) * H + 16 * part) * DL + d;
#pragma unroll
          for (int h = 0; h < 16; ++h) op[h * DL] = o[h] * inv[h];
        }
      }
    } else if (lane == 0) {
      report(a.dev_status, DSA_DEV_TIMEOUT);
    }
  }

  // ---------------- teardown ----------------
  tc_fence_before_sync();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, TM_COLS);
  }

  if constexpr (MERGE) {
    // ---------------- the cluster's splits together ----------------
    //   out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    float* fac = reinterpret_cast<float*>(smem + OFF_P);  // [S][64] factors of the splits' O (the P buffers are idle)
    if (tid < H) {
      float ms[MAX_MERGED], ls[MAX_MERGED];  // (all the remote loads together)
#pragma unroll
      for (int s = 0; s < MAX_MERGED; ++s) {
        ms[s] = s < S ? *cluster.map_shared_rank(ml_s + tid, s) : -INFINITY;
        ls[s] = s < S ? *cluster.map_shared_rank(ml_s + H + tid, s) : 0.f;
      }
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int s = 0; s < MAX_MERGED; ++s) m = fmaxf(m, ms[s]);
#pragma unroll
      for (int s = 0; s < MAX_MERGED; ++s) {
        ms[s] = ms[s] == -INFINITY ? 0.f : ex2(ms[s] - m);
        l = fmaf(ms[s], ls[s], l);
      }
      const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int s = 0; s < MAX_MERGED; ++s)
        if (s < S) fac[s * H + tid] = ms[s] * inv;
      if (split == 0 && a.lse) a.lse[(int64_t)i * H + tid] = l != 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
    }
    __syncthreads();
    // each CTA a share of the token's values, four at a time
    const float* os = reinterpret_cast<const float*>(smem + OFF_KV);
    for (int e = split * NTHREADS + tid; e < H * DL / 4; e += S * NTHREADS) {
      const int h = e / (DL / 4);
      float4 v[MAX_MERGED];
#pragma unroll
      for (int s = 0; s < MAX_MERGED; ++s) {
        // (an empty split's O was never written)
        if (s < S && fac[s * H + h] != 0.f) v[s] = reinterpret_cast<const float4*>(cluster.map_shared_rank(os, s))[e];
        else v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < MAX_MERGED; ++s) {
        const float f = s < S ? fac[s * H + h] : 0.f;
        o.x = fmaf(f, v[s].x, o.x), o.y = fmaf(f, v[s].y, o.y), o.z = fmaf(f, v[s].z, o.z), o.w = fmaf(f, v[s].w, o.w);
      }
      __nv_bfloat162* ob = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t)i * H * DL) + 2 * e;
      ob[0] = __floats2bfloat162_rn(o.x, o.y);
      ob[1] = __floats2bfloat162_rn(o.z, o.w);
    }
    cluster.sync();  // no CTA leaves while another reads its shared memory
  }
}

}  // namespace

cudaError_t launch_chunk_tc(const MlaArgs& a, const int32_t* q_pos, bool merge, cudaStream_t stream) {
  if (a.num_q == 0) return cudaSuccess;
  // the largest box of rows that never leaves a page (gather4 takes pages that no multiple of 8 fits)
  int box = T;
  while (box >= 8 && a.page_size % box != 0) box /= 2;
  if (box < 8) box = 0;
  ChunkMaps maps;
  const uint32_t rows = box > 0 ? box : 1;
  if (!make_kv_map(&maps.lat_box, a, DQK, 128, rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_kv_map(&maps.rope_box, a, DQK, DR, rows, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !make_kv_map(&maps.lat_row, a, DQK, 128, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_kv_map(&maps.rope_row, a, DQK, DR, 1, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  // Three TMA warps keep up with boxes of 16 rows or more, 5 to 20 copies a tile
  // (1,024 tokens of 16,384: 1.48 ms at page size 64, 1.64 at 16; with seven 1.75 and
  // 1.75: more warps that look tiles up, and the power limit); smaller boxes and
  // gathers need seven (page size 24: 1.78 against 1.97 ms; 152 tokens of 16,384
  // at page size 4: 343 against 454 us).
  auto launch = [&](auto kern, int ntma) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = merge ? (unsigned)a.num_splits : 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.num_q, a.num_splits);
    cfg.blockDim = dim3((ntma + 1 + SM_WARPS) * 32);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = merge ? 1 : 0;
    const cudaError_t st = cudaLaunchKernelEx(&cfg, kern, a, q_pos, maps, box, make_fast_div(a.page_size));
    return st != cudaSuccess ? st : cudaGetLastError();
  };
  if (merge) return box >= 16 ? launch(mla_chunk_kernel<3, true>, 3) : launch(mla_chunk_kernel<7, true>, 7);
  return box >= 16 ? launch(mla_chunk_kernel<3, false>, 3) : launch(mla_chunk_kernel<7, false>, 7);
}

}  // namespace dsa
