// Drafted tokens verified against the target's probabilities.
//
// "Accelerating GLM-5.3-Flash on H200", section 3: a speculative verify step
// runs the target over a block of drafted tokens.  With the target's
// probabilities p_i after i drafted tokens, the draft's q_i and uniform
// numbers u_i, draft x_i is taken while
//     u_i q_i(x_i) < p_i(x_i)                              (u < p / q)
// and the first one that is not, at a, is replaced by a token drawn from the
// rest of the distribution,
//     w = max(p_a - q_a, 0),   token = min { j : sum_{i <= j} w_i > u sum_i w_i };
// after the last draft the token comes from p itself (speculative sampling:
// every output token is then distributed as the target's).  A draft that
// comes without probabilities is certain: q = 1 at x_i, 0 elsewhere.
//
// The token hangs on comparisons of sums of up to a million terms, so the
// sums are whole numbers: a probability becomes the integer part of p 2^60
// (exact for p >= 2^-37), p - q and every sum are then exact, whatever the
// order and the number of CTAs, and u sum w is a 64 x 64 bit product.  An fp32
// sum would move a border by ~1e-7 at each of V places, which shows in the
// token about once in a hundred draws at V = 131,072.  The long sums take the
// 60 bits in three parts of 20 by fp32 additions (Parts); the one run that is
// read again takes them by shifts (fixed60).
//
// A thread-block cluster per request.  Every CTA finds a for itself (one lane
// a draft); the CTAs then sum their parts of the row (each warp one
// contiguous run, 16-byte loads where the rows allow), exchange the sums over
// distributed shared memory, and only the warp whose run holds the token
// reads it again (from L2), 128 values a turn.  Only rows a of p and q are
// read.  128 requests, V = 131,072, with draft probabilities: 34 us for 101 MB
// (2.9 TB/s; the sums' arithmetic and the cluster-wide waits are what is
// not hidden).  Few requests are one round trip after another: 4 take 5.7 us.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.cuh"

namespace cg = cooperative_groups;

namespace dsa {
namespace {

constexpr int VD_MAX_CLUSTER = 8;

// Shifts whose amounts past 31 give 0 (negative ones count as large).
__device__ __forceinline__ uint32_t shl(uint32_t x, int n) {
  uint32_t r;
  asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(n));
  return r;
}
__device__ __forceinline__ uint32_t shr(uint32_t x, int n) {
  uint32_t r;
  asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(n));
  return r;
}

// p in [0, 1] as a multiple of 2^-60 (NaN and negative values: 0; above 1: 1).
// The significand m < 2^24 of p = m 2^(e - 150) is put at 2^37 (its value for e =
// 127) and shifted right by 127 - e: eight integer operations, where the
// conversion of an fp32 number to 64 bits runs at a fraction of their rate.
__device__ __forceinline__ int64_t fixed60(float p) {
  const uint32_t x = __float_as_uint(fminf(fmaxf(p, 0.f), 1.f));
  const uint32_t top = ((x << 5) & 0x0fffffe0u) | 0x10000000u;  // m 2^5: the upper word of m 2^37
  const int r = 127 - (int)(x >> 23);
  const uint32_t hi = shr(top, r), lo = shl(top, 32 - r) | shr(top, r - 32);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

struct Row {
  const float* p;
  const float* q;   // null: nothing is taken off but `skip`
  int64_t skip;     // a column of weight 0, or -1
  int32_t vocab;
  __device__ __forceinline__ int64_t weight(float pv, float qv, int32_t j) const {
    const int64_t w = fixed60(pv) - (q ? fixed60(qv) : 0);
    return j == skip || w < 0 ? 0 : w;
  }
};

// Four columns j .. j + 3 (zero past the row's end); vec: 16-byte loads.
template <bool VEC>
__device__ __forceinline__ float4 load4(const float* row, int32_t j, int32_t vocab) {
  if (VEC && j + 4 <= vocab) return *reinterpret_cast<const float4*>(row + j);
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = j + e < vocab ? row[j + e] : 0.f;
  return make_float4(v[0], v[1], v[2], v[3]);
}

// The sum of fixed60 over many values, 20 bits at a time: adding 2^3 to p in [0, 1]
// with rounding towards 0 leaves floor(p 2^20) in the low bits of the sum, the
// remainder is exact, and the same with 2^-17 and 2^-37 gives the next two 20
// bits.  Seven fp32 additions at the full rate, and the three parts add up in
// 32-bit words (2^20 a value: up to 1,024 of them before they are put together).
struct Parts {
  uint32_t h = 0, m = 0, l = 0;
  __device__ __forceinline__ static void split(float p, uint32_t& h, uint32_t& m, uint32_t& l) {
    p = __saturatef(p);  // to [0, 1], NaN to 0
    const float a = __fadd_rz(p, 8.f), r1 = p - (a - 8.f);
    const float b = __fadd_rz(r1, 0x1p-17f), r2 = r1 - (b - 0x1p-17f);
    h = __float_as_uint(a), m = __float_as_uint(b), l = __float_as_uint(__fadd_rz(r2, 0x1p-37f));
  }
  __device__ __forceinline__ void add(float p) {
    uint32_t x, y, z;
    split(p, x, y, z);
    h += x - __float_as_uint(8.f), m += y - __float_as_uint(0x1p-17f), l += z - __float_as_uint(0x1p-37f);
  }
  // max(p - q, 0): the parts' differences (as two's complement; the sum is what counts)
  __device__ __forceinline__ void add_rest(float p, float q) {
    uint32_t x, y, z, u, v, w;
    split(p, x, y, z);
    split(q, u, v, w);
    if (__saturatef(p) > __saturatef(q)) h += x - u, m += y - v, l += z - w;
  }
  __device__ __forceinline__ int64_t total() const {
    return ((int64_t)(int32_t)h << 40) + ((int64_t)(int32_t)m << 20) + (int64_t)(int32_t)l;
  }
};

// A lane's part of the sum over columns [lo, hi) (without `skip`), lo a multiple
// of 128.  The full blocks' loads are unconditional, eight turns of them in flight.
template <bool VEC, bool Q>
__device__ __forceinline__ int64_t run_sum(const Row& r, int32_t lo, int32_t hi) {
  constexpr int TURNS = Q ? 4 : 8;
  auto add4 = [](Parts& acc, const float4 p, const float4 q) {
    if constexpr (Q) {
      acc.add_rest(p.x, q.x);
      acc.add_rest(p.y, q.y);
      acc.add_rest(p.z, q.z);
      acc.add_rest(p.w, q.w);
    } else {
      acc.add(p.x);
      acc.add(p.y);
      acc.add(p.z);
      acc.add(p.w);
    }
  };
  auto full4 = [](const float* row, int32_t j) {
    if constexpr (VEC) return __ldg(reinterpret_cast<const float4*>(row + j));
    else return make_float4(__ldg(row + j), __ldg(row + j + 1), __ldg(row + j + 2), __ldg(row + j + 3));
  };
  int64_t s = 0;
  int32_t j0 = lo;
  const int lane4 = 4 * (threadIdx.x & 31);
  while (hi - j0 >= 128 * TURNS) {
    Parts acc;
    for (int n = 0; n < 256 / TURNS && hi - j0 >= 128 * TURNS; ++n, j0 += 128 * TURNS) {  // 1,024 values at most
      float4 p[TURNS], q[TURNS];
#pragma unroll
      for (int k = 0; k < TURNS; ++k) {
        p[k] = full4(r.p, j0 + 128 * k + lane4);
        if constexpr (Q) q[k] = full4(r.q, j0 + 128 * k + lane4);
      }
#pragma unroll
      for (int k = 0; k < TURNS; ++k) add4(acc, p[k], q[k]);
    }
    s += acc.total();
  }
  Parts acc;
  for (int32_t j = j0 + lane4; j < hi; j += 128)
    add4(acc, load4<VEC>(r.p, j, r.vocab), Q ? load4<VEC>(r.q, j, r.vocab) : make_float4(0.f, 0.f, 0.f, 0.f));
  return s + acc.total();
}

template <bool VEC>
__device__ __forceinline__ void weights4(const Row& r, int32_t j, int64_t (&w)[4]) {
  const float4 p = load4<VEC>(r.p, j, r.vocab);
  const float4 q = r.q ? load4<VEC>(r.q, j, r.vocab) : make_float4(0.f, 0.f, 0.f, 0.f);
  w[0] = r.weight(p.x, q.x, j);
  w[1] = r.weight(p.y, q.y, j + 1);
  w[2] = r.weight(p.z, q.z, j + 2);
  w[3] = r.weight(p.w, q.w, j + 3);
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int VD_THREADS, bool VEC>
__global__ void __launch_bounds__(VD_THREADS) verify_draft_kernel(const VerifyArgs a) {
  constexpr int VD_WARPS = VD_THREADS / 32;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int req = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ int64_t wsum[VD_WARPS];
  __shared__ int64_t csum[VD_MAX_CLUSTER];  // the CTAs' sums, written by each of them
  __shared__ int32_t s_take;

  const int32_t row0 = a.cu_rows[req], row1 = a.cu_rows[req + 1];
  int32_t* out = a.tokens + (int64_t)req * a.max_out;
  bool bad = row0 < 0 || row1 < row0 || row1 > a.num_rows;
  bool none = bad || row1 == row0;
  if (a.q_req && !none) {  // a request that the layout refused has rows, but no positions for them
    const int32_t owner = a.q_req[row0];
    none = owner != req;
    bad = none && owner != -1;
  }
  if (none) {  // no rows (the same for the whole cluster)
    if (rank == 0) {
      if (tid == 0) {
        if (bad) report(a.dev_status, DSA_DEV_BAD_INDEX);
        a.num_out[req] = 0;
        if (a.ctx_out) a.ctx_out[req] = a.ctx_len[req];
      }
      for (int e = tid; e < a.max_out; e += VD_THREADS) out[e] = -1;
    }
    return;
  }
  // Waited for before the first write to another CTA's shared memory.  Nothing was
  // written yet that it would have to order: relaxed (a releasing arrive: 4 requests
  // 6.0 instead of 5.7 us).
  asm volatile("barrier.cluster.arrive.relaxed;");
  const int32_t* xs = a.draft_tokens + row0;
  int32_t n = row1 - row0 - 1;
  if (n > a.max_out - 1) {  // drafts past the output's width are not looked at
    n = a.max_out - 1;
    if (rank == 0 && tid == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);
  }

  // ---- how many drafts are taken: one lane a draft, 32 at a time ----
  if (warp == 0) {
    int32_t take = n;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      bool ok = true;
      if (i < n) {
        const int32_t x = xs[i];
        ok = x >= 0 && x < a.vocab;
        if (!ok && rank == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);
        if (ok) {
          const float p = a.target[(int64_t)(row0 + i) * a.ld_target + x];
          const float q = a.draft ? a.draft[(int64_t)(row0 + i) * a.ld_draft + x] : 1.f;
          // two 24-bit factors: the product is exact in 64 bits (a NaN rejects)
          ok = (double)a.u_accept[row0 + i] * (double)q < (double)p;
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !ok);
      if (no) {
        take = i0 + __ffs(no) - 1;
        break;
      }
    }
    if (lane == 0) s_take = take;
  }
  __syncthreads();
  const int32_t take = s_take;
  Row row = {a.target + (int64_t)(row0 + take) * a.ld_target, nullptr, -1, a.vocab};
  if (take < n) {
    if (a.draft) row.q = a.draft + (int64_t)(row0 + take) * a.ld_draft;
    else row.skip = xs[take];
  }

  // a row without any probability; the warp that finds the token writes it
  // after the cluster's barrier
  if (rank == 0 && tid == 0) out[take] = a.vocab - 1;

  // ---- this warp's run of the row: a multiple of 128 columns ----
  const int nw = C * VD_WARPS;
  const int32_t run = (int32_t)((((int64_t)a.vocab + nw - 1) / nw + 127) / 128) * 128;
  const int64_t lo64 = (int64_t)(rank * VD_WARPS + warp) * run;
  const int32_t lo = (int32_t)min(lo64, (int64_t)a.vocab), hi = (int32_t)min(lo64 + run, (int64_t)a.vocab);
  int64_t total = 0, before = 0, mine = 0;
  for (int turn = 0; turn < 2; ++turn) {
    int64_t s = 0;
    if (row.q) {
      s = run_sum<VEC, true>(row, lo, hi);
    } else {
      s = run_sum<VEC, false>(row, lo, hi);
      if (lane == 0 && row.skip >= lo && row.skip < hi) s -= fixed60(row.p[row.skip]);
    }
    s = warp_sum(s);
    mine = s;
    if (lane == 0) wsum[warp] = s;
    if (turn == 0) asm volatile("barrier.cluster.wait;" ::: "memory");  // every CTA of the cluster runs
    __syncthreads();
    if (tid < C) {
      int64_t cta = 0;
      for (int w = 0; w < VD_WARPS; ++w) cta += wsum[w];
      *cluster.map_shared_rank(&csum[rank], tid) = cta;
    }
    cluster.sync();
    total = 0, before = 0;
    for (int c = 0; c < C; ++c) {
      if (c < rank) before += csum[c];
      total += csum[c];
    }
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (total != 0 || (!row.q && row.skip < 0)) break;
    // nothing is left of the row (p <= q everywhere): the token comes from p
    row.q = nullptr;
    row.skip = -1;
    cluster.sync();  // every CTA has read the sums
  }

  // ---- the warp whose run holds the token reads it again ----
  const float u = a.u_sample[req];
  // u 2^64, u clamped to [0, 1) (NaN: 0); exact for u >= 2^-40
  const uint64_t u64 = __float2ull_rz(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f) * 0x1p64f);
  const int64_t t = (int64_t)__umul64hi(u64, (uint64_t)total);  // floor(u sum w): sum_{i <= j} w > t
  if (before <= t && t < before + mine) {
    // (four turns' loads together: a run is a few round trips to L2)
    constexpr int TURNS = 4;
    int64_t base = before;
    bool found = false;
    for (int32_t j0 = lo; j0 < hi && !found; j0 += 128 * TURNS) {
      int64_t w[TURNS][4];
#pragma unroll
      for (int k = 0; k < TURNS; ++k) {
        const int32_t j = j0 + 128 * k + 4 * lane;
        w[k][0] = w[k][1] = w[k][2] = w[k][3] = 0;
        if (j < hi) weights4<VEC>(row, j, w[k]);
      }
#pragma unroll
      for (int k = 0; k < TURNS; ++k) {
        if (found) break;
        const int64_t s = (w[k][0] + w[k][1]) + (w[k][2] + w[k][3]);
        int64_t inc = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const unsigned over = __ballot_sync(0xffffffffu, base + inc > t);
        if (over) {
          found = true;
          if (lane == __ffs(over) - 1) {
            int64_t c = base + inc - s;
            int e = 0;
            for (; e < 3; ++e) {
              if (c + w[k][e] > t) break;
              c += w[k][e];
            }
            out[take] = j0 + 128 * k + 4 * lane + e;
          }
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  if (rank == 0) {
    for (int e = tid; e < a.max_out; e += VD_THREADS)
      if (e != take) out[e] = e < take ? xs[e] : -1;
    if (tid == 0) {
      a.num_out[req] = take + 1;
      if (a.ctx_out) a.ctx_out[req] = a.ctx_len[req] + take + 1;
    }
  }
  // no CTA leaves while another may still write its sum here: all have passed the last cluster.sync
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t stream) {
  const bool vec = (reinterpret_cast<uintptr_t>(a.target) & 15u) == 0 && a.ld_target % 4 == 0 &&
                   (!a.draft || ((reinterpret_cast<uintptr_t>(a.draft) & 15u) == 0 && a.ld_draft % 4 == 0));
  // Eight CTAs a request, of 512 threads while two of them fit an SM at once
  // (one request: 8.7 us, 256 threads 9.7 us), of 256 beyond that (128 requests, V =
  // 131,072: 34 us; 512 threads 39 us, and with fewer CTAs a request 36 to 45 us);
  // fewer where a request's chain of loads would repeat in too many waves.
  const int sms = device_sm_count();
  int c = VD_MAX_CLUSTER;
  while (c > 1 && (int64_t)a.num_req * c > 8 * sms) c /= 2;
  const bool wide = (int64_t)a.num_req * c <= 2 * sms;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.num_req * c);
  cfg.blockDim = dim3(wide ? 512 : 256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = wide ? (vec ? cudaLaunchKernelEx(&cfg, verify_draft_kernel<512, true>, a)
                                    : cudaLaunchKernelEx(&cfg, verify_draft_kernel<512, false>, a))
                             : (vec ? cudaLaunchKernelEx(&cfg, verify_draft_kernel<256, true>, a)
                                    : cudaLaunchKernelEx(&cfg, verify_draft_kernel<256, false>, a));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dsa
