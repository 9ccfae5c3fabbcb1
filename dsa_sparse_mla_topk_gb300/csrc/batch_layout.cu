// Block tables and slot maps of a batch from its requests' lengths.
//
// "Accelerating GLM-5.3-Flash on H200", section 2 "KV-only decode
// RadixCache": KV rows live in a paged pool that a block table maps per
// request.  A serving step with requests r of ctx[r] cached positions and
// new[r] new tokens needs, before it can write or read a row,
//   cu[r]    = sum_{s < r} new[s]                     (the batch's token ranges)
//   total[r] = ceil((ctx[r] + new[r]) / P), need[r] = max(0, total[r] - held[r])
//   table[r, held[r] + x] = free[used + sum_{s < r} need[s] + x],  x < need[r]
//   req, pos, slot of every token t: pos = ctx[r] + t - cu[r],
//   slot = table[r, pos / P] P + pos % P
// with need[r] = 0 where new[r] = 0.
//
// One launch.  Both prefix sums are of at most 8,192 requests, so every CTA
// takes them for itself in shared memory (12 bytes a request from L2, one
// block scan) instead of waiting for another CTA; then the CTAs share out the
// tokens (four a thread: one binary search over cu and 16-byte stores) and
// the new pages.  No CTA reads a table entry that this call writes: a token on
// a new page takes the page from the free list.  Bound by launch and the
// chain of loads (lengths, scan, table): 8 requests of one token 5.5 us, 128 of
// 8 tokens 6.0 us; 512 of 2,001 tokens 9.2 us, of which the 12.3 MB written (12
// bytes a token) take 1.8 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.cuh"

namespace dsa {
namespace {

constexpr int BL_THREADS = 512;
constexpr int BL_WARPS = BL_THREADS / 32;
constexpr int BL_TOK = 4;  // consecutive tokens per thread and turn

struct Pair {
  int64_t tok, page;
};

// Sums over the threads before this one, and over the whole block.
__device__ __forceinline__ Pair block_scan(Pair v, Pair* warp_sum, Pair* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pair inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, inc.tok, o), b = __shfl_up_sync(0xffffffffu, inc.page, o);
    if (lane >= o) inc.tok += a, inc.page += b;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  Pair before = {0, 0}, all = {0, 0};
#pragma unroll
  for (int w = 0; w < BL_WARPS; ++w) {
    const Pair s = warp_sum[w];
    if (w < warp) before.tok += s.tok, before.page += s.page;
    all.tok += s.tok, all.page += s.page;
  }
  *total = all;
  return {before.tok + inc.tok - v.tok, before.page + inc.page - v.page};
}

// The last r in [0, n) with key[r] <= x, for nondecreasing key with key[0] <= x.
__device__ __forceinline__ int last_not_above(const int32_t* key, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (key[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(BL_THREADS) batch_layout_kernel(const BatchLayoutArgs a) {
  extern __shared__ int32_t bl_smem[];
  const int R = a.num_req;
  int32_t* cu = bl_smem;         // [R + 1] first token of each request
  int32_t* first = cu + R + 1;   // [R + 1] new pages of the requests before
  int32_t* ctx_s = first + R + 1;  // [R] cached positions; -1: the request gets no tokens
  int32_t* held_s = ctx_s + R;   // [R] pages the request already has
  __shared__ Pair warp_sum[BL_WARPS];
  __shared__ int32_t fit_tok;  // tokens of the requests that fit the capacity
  const int tid = threadIdx.x;
  const bool reporter = blockIdx.x == 0;
  const int32_t P = a.page_size;

  const int64_t used = *a.free_used;
  const bool pool_ok = used >= 0 && used <= a.num_free;
  if (!pool_ok && reporter && tid == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);
  const int64_t left = pool_ok ? a.num_free - used : 0;

  // ---- requests: each thread takes a run of them ----
  const int per = (R + BL_THREADS - 1) / BL_THREADS;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  // a request's new tokens and needed pages; false: it is left as it is
  auto lengths = [&](int r, int32_t& ctx, int32_t& held, int64_t& tok, int64_t& need, bool tell) -> bool {
    ctx = a.ctx_len[r];
    held = a.pages_held[r];
    const int32_t nw = a.new_len[r];
    tok = 0, need = 0;
    if (ctx < 0 || nw < 0 || held < 0) {  // no such lengths: no tokens
      if (tell) report(a.dev_status, DSA_DEV_BAD_QPOS);
      return false;
    }
    tok = nw;
    if (nw == 0) return true;
    const int64_t total = ((int64_t)ctx + nw + P - 1) / P;
    if (total > a.bt_stride || (int64_t)ctx + nw > INT32_MAX) {  // its block table row is too short
      if (tell) report(a.dev_status, DSA_DEV_BAD_INDEX);
      return false;
    }
    need = total > held ? total - held : 0;
    return true;
  };
  Pair mine = {0, 0};
  for (int r = r0; r < r1; ++r) {
    int32_t c, h;
    int64_t tok, need;
    lengths(r, c, h, tok, need, reporter);
    mine.tok += tok, mine.page += need;
  }
  if (tid == 0) fit_tok = 0;
  Pair all;
  Pair at = block_scan(mine, warp_sum, &all);  // (has the barrier that orders fit_tok)
  int32_t fits_to = 0;
  for (int r = r0; r < r1; ++r) {
    int32_t c, h;
    int64_t tok, need;
    bool ok = lengths(r, c, h, tok, need, false);
    const int64_t t0 = at.tok;
    at.tok += tok, at.page += need;
    if (at.tok <= a.capacity) {
      fits_to = (int32_t)at.tok;
    } else if (tok > 0) {
      ok = false;
      if (reporter) report(a.dev_status, DSA_DEV_BAD_INDEX);
    }
    if (ok && need > 0 && at.page > left) {
      ok = false;
      if (reporter) report(a.dev_status, DSA_DEV_NO_PAGES);
    }
    cu[r] = (int32_t)min(t0, (int64_t)a.capacity + 1);  // past the capacity: replaced below
    first[r] = (int32_t)min(at.page - need, (int64_t)INT32_MAX);
    ctx_s[r] = ok ? c : -1;
    held_s[r] = h;
  }
  if (fits_to > 0) atomicMax(&fit_tok, fits_to);
  if (tid == 0) {
    cu[R] = (int32_t)min(all.tok, (int64_t)a.capacity + 1);
    first[R] = (int32_t)min(all.page, (int64_t)INT32_MAX);
  }
  __syncthreads();
  // a request past the capacity ends the batch: cu stays at the last one that fits
  const int32_t tokens = fit_tok;
  for (int r = tid; r <= R; r += BL_THREADS) cu[r] = min(cu[r], tokens);
  __syncthreads();

  // ---- per request: the new lengths, by one CTA ----
  if (reporter) {
    int64_t taken = 0;
    for (int r = tid; r <= R; r += BL_THREADS) {
      a.cu_q[r] = cu[r];
      if (r == R) break;
      const int32_t nw = a.new_len[r];
      const bool ok = ctx_s[r] >= 0;
      const int32_t h = held_s[r], need = first[r + 1] - first[r];
      a.ctx_out[r] = ok ? ctx_s[r] + nw : a.ctx_len[r];
      a.held_out[r] = ok ? h + need : h;
      if (ok && need > 0) taken = first[r + 1];
    }
    // the requests that take pages are those whose running sum fits: the largest is the count taken
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    __syncthreads();
    if ((tid & 31) == 0) warp_sum[tid >> 5].page = taken;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < BL_WARPS; ++w) taken = max(taken, warp_sum[w].page);
      *a.free_used_out = (int32_t)(used + taken);
    }
  }

  // ---- tokens ----
  const int64_t step = (int64_t)gridDim.x * BL_THREADS;
  for (int64_t g = (int64_t)blockIdx.x * BL_THREADS + tid; g * BL_TOK < a.capacity; g += step) {
    const int32_t t0 = (int32_t)(g * BL_TOK);
    int32_t req[BL_TOK], pos[BL_TOK], slot[BL_TOK];
    int r = t0 < tokens ? last_not_above(cu, R, t0) : R;
#pragma unroll
    for (int e = 0; e < BL_TOK; ++e) {
      const int32_t t = t0 + e;
      req[e] = pos[e] = slot[e] = -1;
      if (t >= tokens) continue;
      while (t >= cu[r + 1]) ++r;
      const int32_t c = ctx_s[r];
      if (c < 0) continue;
      const int32_t p = c + (t - cu[r]), pg = p / P, h = held_s[r];
      const int32_t page = pg < h ? a.block_table[(int64_t)r * a.bt_stride + pg] : a.free_pages[used + first[r] + pg - h];
      req[e] = r;
      pos[e] = p;
      if (page < 0 || page >= a.num_pages) report(a.dev_status, DSA_DEV_BAD_PAGE);
      else slot[e] = page * P + p % P;
    }
    if (a.vec && t0 + BL_TOK <= a.capacity) {
      reinterpret_cast<int4*>(a.q_req)[g] = make_int4(req[0], req[1], req[2], req[3]);
      reinterpret_cast<int4*>(a.q_pos)[g] = make_int4(pos[0], pos[1], pos[2], pos[3]);
      reinterpret_cast<int4*>(a.slot)[g] = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int e = 0; e < BL_TOK; ++e) {
        if (t0 + e >= a.capacity) break;
        a.q_req[t0 + e] = req[e];
        a.q_pos[t0 + e] = pos[e];
        a.slot[t0 + e] = slot[e];
      }
    }
  }

  // ---- new pages (one per needed page; the requests that got theirs) ----
  const int64_t wanted = min((int64_t)first[R], left);
  for (int64_t x = (int64_t)blockIdx.x * BL_THREADS + tid; x < wanted; x += step) {
    const int r = last_not_above(first, R, (int32_t)x);  // the last request that starts at or before x: it needs x
    if (ctx_s[r] < 0) continue;
    a.block_table[(int64_t)r * a.bt_stride + held_s[r] + (x - first[r])] = a.free_pages[used + x];
  }
}

// four words a request (cu and first have one more)
size_t smem_bytes(int num_req) { return sizeof(int32_t) * (4 * (size_t)num_req + 2); }

}  // namespace

int batch_layout_max_requests() { return 8192; }

cudaError_t launch_batch_layout(const BatchLayoutArgs& a, cudaStream_t stream) {
  const size_t smem = smem_bytes(a.num_req);
  if (smem > 48 * 1024) {  // more than a launch may take unasked
    // The limit is the kernel's, for every thread of the process: always the largest
    // batch's, so that no call lowers it between another one's two steps.
    const cudaError_t e = cudaFuncSetAttribute(batch_layout_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem_bytes(batch_layout_max_requests()));
    if (e != cudaSuccess) return e;
  }
  const int64_t groups = ((int64_t)a.capacity + BL_TOK - 1) / BL_TOK;
  const int64_t ctas = (groups + BL_THREADS - 1) / BL_THREADS;
  // one CTA per SM at most: each takes the requests' scan once
  const int sms = device_sm_count();
  const unsigned grid = (unsigned)(ctas < 1 ? 1 : ctas < sms ? ctas : sms);
  batch_layout_kernel<<<grid, BL_THREADS, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa
