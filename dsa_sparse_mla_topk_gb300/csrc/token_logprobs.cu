// Log probabilities of given tokens, the rows' entropy, the tokens' ranks and the
// most probable alternatives, in one pass over the rows.
//
// With m the row's largest logit, at column a, and x_j = (z_j - m) log2 e <= 0:
//   rest    = sum_{j != a} 2^x_j,  lse = m + log1p(rest)
//   logprob = z_t - m - log1p(rest)
//   entropy = log1p(rest) - ln 2 sum_j 2^x_j x_j / (1 + rest)     (two terms >= 0: nothing cancels)
// The largest term, 1, stays out of the sum: the logarithm of a sure token is next
// to rest, which 1 + rest in fp32 would round to 2^-24.
//
// A row is read once, 16 bytes a load, by one CTA or a cluster of up to 8 (few rows).  A
// thread keeps its own largest value m_t and the sums of 2^x and 2^x x relative to it, and
// counts the columns before the token.  Then
//  * the sums are put together relative to the largest m_t.  Only the thread that holds it
//    has the term 1 among its terms: one warp reads that thread's columns again and sums
//    them without it.
//  * of the k-th largest m_t, tau, it is known that k columns at least reach it: all
//    alternatives are among the columns >= tau, which only the few threads with m_t >= tau
//    hold.  Their columns are read again (from L2) by a warp each; the columns
//    found, usually little more than k, are put in order by counting.  tau comes from
//    a bisection on the values' bits that ends as soon as not many more than k threads
//    reach it.  Too many columns >= tau (equal logits all over): k rounds of a search
//    for the next one.
// A row of 16-bit values costs 6.5 instructions a value (of 10.9 that the SMs have in the time
// that HBM takes): two-wide fp32 arithmetic, maxima and counts two-wide in the type.
// Measured: 1,024 rows of 131,072 bf16, 20 alternatives, 66 us (4.1 TB/s; the loads alone 47, with the sums
// 54), 128 such rows fp32 19 us, 4 rows of 32,003 fp32 9.4 us (launch and the chain of steps).
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

constexpr int THREADS = 512, WARPS = THREADS / 32, MAX_CLUSTER = 8, MAX_TOP = token_logprobs_max_top();
constexpr int TURNS = 4;    // loads of a thread in flight
constexpr int CAND = 1024;  // columns >= tau that are put in order
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float X_MIN = -200.f;  // 2^x is 0 from -150 on; x of a masked column (-inf) times 0 would be NaN

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Bits in the order of the values (NaN aside; -0 as +0).
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Whether (x, i) comes before (y, j): larger, or equal and of a lower column.
__device__ __forceinline__ bool before(float x, int i, float y, int j) { return x > y || (x == y && i < j); }

// Values two by two in a 16-byte load: their fp32 values, running maxima and counts.
template <class T>
struct Pack;
template <>
struct Pack<float> {
  static constexpr int N = 4;  // values of a load
  struct Most {
    float v = -INFINITY;
    __device__ __forceinline__ void take(const uint4& w) {
      v = fmaxf(fmaxf(v, fmaxf(__uint_as_float(w.x), __uint_as_float(w.y))), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
    __device__ __forceinline__ float value() const { return v; }
  };
  typedef float Bound;  // a value to compare with
  __device__ __forceinline__ static Bound bound(float x) { return x; }
  struct Count {
    int n = 0;
    __device__ __forceinline__ void take(const uint4& w, Bound thr) {
      n += __uint_as_float(w.x) > thr;
      n += __uint_as_float(w.y) > thr;
      n += __uint_as_float(w.z) > thr;
      n += __uint_as_float(w.w) > thr;
    }
    __device__ __forceinline__ int value() const { return n; }
  };
  __device__ __forceinline__ static uint64_t pair(const uint4& w, int i) {
    return i == 0 ? pk2(__uint_as_float(w.x), __uint_as_float(w.y)) : pk2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  __device__ __forceinline__ static float get(const uint4& w, int e) {
    return __uint_as_float(e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w);
  }
  __device__ __forceinline__ static uint32_t minus_inf() { return 0xff800000u; }
  // the largest value below x (finite)
  __device__ __forceinline__ static float below(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u << 1) == 0 ? __uint_as_float(0x80000001u) : __uint_as_float(u & 0x80000000u ? u + 1 : u - 1);
  }
};
template <class T2>
__device__ __forceinline__ T2 as_pair(uint32_t w) {
  return *reinterpret_cast<const T2*>(&w);
}
// T2: the type two-wide
template <class T, class T2>
struct Pack16 {
  static constexpr int N = 8;
  struct Most {
    T2 v = as_pair<T2>(Pack<T>::minus_inf());
    __device__ __forceinline__ void take(const uint4& w) {
      v = __hmax2(v, __hmax2(__hmax2(as_pair<T2>(w.x), as_pair<T2>(w.y)), __hmax2(as_pair<T2>(w.z), as_pair<T2>(w.w))));
    }
    __device__ __forceinline__ float value() const { return fmaxf((float)v.x, (float)v.y); }
  };
  typedef uint32_t Bound;  // a value to compare with, twice
  __device__ __forceinline__ static Bound bound(float x) {
    const T t = (T)x;
    return 0x10001u * *reinterpret_cast<const uint16_t*>(&t);
  }
  struct Count {  // as numbers of the type: exact up to 256 a half, 32 loads
    T2 v = as_pair<T2>(0u);
    __device__ __forceinline__ void take(const uint4& w, Bound thr) {
      const T2 t2 = as_pair<T2>(thr);
      v = __hadd2(v, __hadd2(__hadd2(__hgt2(as_pair<T2>(w.x), t2), __hgt2(as_pair<T2>(w.y), t2)),
                             __hadd2(__hgt2(as_pair<T2>(w.z), t2), __hgt2(as_pair<T2>(w.w), t2))));
    }
    __device__ __forceinline__ int value() const { return (int)(float)v.x + (int)(float)v.y; }
  };
  __device__ __forceinline__ static float get(const uint4& w, int e) {
    const uint32_t u = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
    const T2 p = as_pair<T2>(u);
    return e & 1 ? (float)p.y : (float)p.x;
  }
  __device__ __forceinline__ static float below(float x) {
    const T t = (T)x;
    const uint16_t u = *reinterpret_cast<const uint16_t*>(&t);
    const uint16_t b = (uint16_t)(u << 1) == 0 ? 0x8001u : (uint16_t)(u & 0x8000u ? u + 1 : u - 1);
    return (float)*reinterpret_cast<const T*>(&b);
  }
};
template <>
struct Pack<__nv_bfloat16> : Pack16<__nv_bfloat16, __nv_bfloat162> {
  __device__ __forceinline__ static uint64_t pair(const uint4& w, int i) {
    const uint32_t u = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return pk2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  __device__ __forceinline__ static uint32_t minus_inf() { return 0xff80ff80u; }
};
template <>
struct Pack<__half> : Pack16<__half, __half2> {
  __device__ __forceinline__ static uint64_t pair(const uint4& w, int i) {
    const float2 f = __half22float2(as_pair<__half2>(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w));
    return pk2(f.x, f.y);
  }
  __device__ __forceinline__ static uint32_t minus_inf() { return 0xfc00fc00u; }
};

// A row as 16-byte loads: load v holds columns N v - shift .. + N - 1; what lies beside the row
// reads as masked.
template <class T>
struct Row {
  static constexpr int N = Pack<T>::N;
  const T* p;
  int vocab, shift, loads;
  __device__ __forceinline__ Row(const T* row, int V) : p(row), vocab(V) {
    shift = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    loads = (V + shift + N - 1) / N;
  }
  __device__ __forceinline__ bool inside(int v) const { return v * N >= shift && v * N - shift + N <= vocab; }
  __device__ __forceinline__ uint4 full(int v) const { return __ldg(reinterpret_cast<const uint4*>(p - shift) + v); }
  __device__ __forceinline__ uint4 load(int v) const {
    if (inside(v)) return full(v);
    __align__(16) T e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = v * N - shift + i;
      e[i] = j >= 0 && j < vocab ? p[j] : (T)-INFINITY;
    }
    return *reinterpret_cast<const uint4*>(e);
  }
};

// What a CTA found in its share of a row.
struct Part {
  float top, rest, ent;  // the largest value, the sums without (one of) it
  int count, n;          // columns before the token; alternatives listed
};
struct Shared {
  float wf[2][WARPS];
  int wi[WARPS];
  uint32_t wk[2][WARPS];
  float m_t[THREADS];
  Part part[MAX_CLUSTER];
  float lz[MAX_CLUSTER][MAX_TOP];
  int lc[MAX_CLUSTER][MAX_TOP];
  float cz[CAND];
  int cc[CAND];
  int list[THREADS];
  int owner, flagged, cands;
  float own_rest, own_ent;
};

// Sums and order over the share [v0, v1) of a row's loads by this CTA.
template <class T>
__device__ __forceinline__ void share_of_row(const Row<T>& row, int v0, int v1, const int32_t* token, int& t, float& zt,
                                             bool& bad, int top, Shared* sh, Part* part, float* lz, int* lc) {
  constexpr int N = Pack<T>::N;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // a turn's loads are on their way while the one before is worked on, the first while the token is looked up
  auto fetch = [&](int vb, uint4 (&w)[TURNS]) {
    const bool whole = vb + THREADS * TURNS <= v1 && row.inside(vb) && row.inside(vb + THREADS * TURNS - 1);
#pragma unroll
    for (int k = 0; k < TURNS; ++k) {
      const int v = vb + THREADS * k + tid;
      if (whole) w[k] = row.full(v);
      else if (v < v1) w[k] = row.load(v);
      else w[k] = make_uint4(Pack<T>::minus_inf(), Pack<T>::minus_inf(), Pack<T>::minus_inf(), Pack<T>::minus_inf());
    }
  };
  uint4 next[TURNS];
  fetch(v0, next);
  t = __ldg(token);
  bad = t < -1 || t >= row.vocab;
  if (bad) t = -1;
  zt = t >= 0 ? (float)row.p[t] : 0.f;
  const int vt = t >= 0 ? (t + row.shift) / N : 0;  // the token's load
  // before it equal values count, from it on they do not
  const typename Pack<T>::Bound thr_hi = Pack<T>::bound(t >= 0 ? zt : INFINITY);
  const typename Pack<T>::Bound thr_lo = Pack<T>::bound(t >= 0 ? Pack<T>::below(zt) : INFINITY);
  float m = -INFINITY;
  uint64_t s2 = 0, e2 = 0;
  int count = 0;
  for (int vb = v0; vb < v1; vb += THREADS * TURNS) {
    uint4 w[TURNS];
#pragma unroll
    for (int k = 0; k < TURNS; ++k) w[k] = next[k];
    if (vb + THREADS * TURNS < v1) fetch(vb + THREADS * TURNS, next);
    typename Pack<T>::Most most;
    typename Pack<T>::Count n;
#pragma unroll
    for (int k = 0; k < TURNS; ++k) {
      most.take(w[k]);
      n.take(w[k], vb + THREADS * k + tid < vt ? thr_lo : thr_hi);
    }
    count += n.value();
    const float up = fmaxf(m, most.value());
    if (up > m) {  // the sums relative to the new largest value: 2^(x + d) (x + d)
      const float d = fmaxf((m - up) * LOG2E, X_MIN), f = ex2(d);
      const uint64_t d2 = pk2(d, d), f2 = pk2(f, f);
      e2 = mul2(fma2(s2, d2, e2), f2);
      s2 = mul2(s2, f2);
      m = up;
    }
    const float ref = m == -INFINITY ? 0.f : -m;
    const uint64_t ref2 = pk2(ref, ref), l2 = pk2(LOG2E, LOG2E);
#pragma unroll
    for (int k = 0; k < TURNS; ++k)
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        float x0, x1;
        upk2(mul2(add2(Pack<T>::pair(w[k], i), ref2), l2), x0, x1);
        x0 = max_nan(x0, X_MIN), x1 = max_nan(x1, X_MIN);
        const uint64_t p = pk2(ex2(x0), ex2(x1));
        s2 = add2(s2, p);
        e2 = fma2(p, pk2(x0, x1), e2);
      }
  }
  float s, e, hi;
  upk2(s2, s, hi);
  s += hi;
  upk2(e2, e, hi);
  e += hi;

  // ---- the largest value, and one thread that holds it ----
  if (tid == 0) sh->owner = THREADS, sh->flagged = 0, sh->cands = 0;
  sh->m_t[tid] = m;
  const uint32_t key = order_of(m), wmost = __reduce_max_sync(0xffffffffu, key), wleast = __reduce_min_sync(0xffffffffu, key);
  if (lane == 0) sh->wk[0][warp] = wmost, sh->wk[1][warp] = wleast;
  __syncthreads();
  uint32_t most = 0, least = UINT32_MAX;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) most = max(most, sh->wk[0][w]), least = min(least, sh->wk[1][w]);
  if (key == most) atomicMin(&sh->owner, tid);
  __syncthreads();
  const int owner = sh->owner;
  const float M = sh->m_t[owner];
  const float d = fmaxf((m - M) * LOG2E, X_MIN), f = m == -INFINITY ? 0.f : ex2(d);
  // (a thread without values: s is 0, or NaN where there was one)
  e = fmaf(s, m == -INFINITY ? 0.f : d, e) * f;
  s = m == -INFINITY ? s : s * f;
  if (tid == owner && M > -INFINITY) s = 0.f, e = 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    e += __shfl_xor_sync(0xffffffffu, e, o);
  }
  count = (int)__reduce_add_sync(0xffffffffu, (uint32_t)count);
  if (lane == 0) sh->wf[0][warp] = s, sh->wf[1][warp] = e, sh->wi[warp] = count;

  // ---- tau: at least `top` threads reach it, few more if the values allow ----
  // (by the whole block: one warp over all 512 values takes 0.5 us longer)
  uint32_t tau = 0;
  if (top > 0) {
    const uint32_t none = order_of(-INFINITY);
    // reached by at least `top` threads (or all that hold values); by none
    uint32_t lo = max(least, none + 1), up = most + 1;
    if (most > none && (least > none || __syncthreads_count(key >= lo) > top)) {
      while (up - lo > 1) {
        const uint32_t mid = lo + (up - lo) / 2;
        const int c = __syncthreads_count(key >= mid);
        if (c >= top) {
          lo = mid;
          if (c <= top + top / 4 + 4) break;
        } else {
          up = mid;
        }
      }
    }
    tau = lo;
    if (key >= tau) sh->list[atomicAdd(&sh->flagged, 1)] = tid;
  }
  __syncthreads();
  // ---- columns read again, a warp a thread's: the owner's for the sum, the others' for tau ----
  const int flagged = sh->flagged;
  auto turn = [&](int who, int i) { return v0 + who + THREADS * i; };
  if (warp == 0 && M > -INFINITY) {
    float rs = 0.f, re = 0.f;
    int same = 0;
    for (int i = lane; turn(owner, i) < v1; i += 32) {
      const uint4 w = row.load(turn(owner, i));
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const float z = Pack<T>::get(w, q);
        if (z == M) {
          ++same;
        } else {
          const float x = max_nan((z - M) * LOG2E, X_MIN), p = ex2(x);
          rs += p;
          re = fmaf(p, x, re);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      rs += __shfl_xor_sync(0xffffffffu, rs, o);
      re += __shfl_xor_sync(0xffffffffu, re, o);
    }
    same = (int)__reduce_add_sync(0xffffffffu, (uint32_t)same);
    if (lane == 0) sh->own_rest = rs + (float)(same - 1), sh->own_ent = re;
  }
  for (int q = WARPS - 1 - warp; q < flagged; q += WARPS) {
    const int who = sh->list[q];
    for (int i = lane; turn(who, i) < v1; i += 32) {
      const int v = turn(who, i);
      const uint4 w = row.load(v);
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const float z = Pack<T>::get(w, c);
        if (z > -INFINITY && order_of(z) >= tau) {
          const int at = atomicAdd(&sh->cands, 1);
          if (at < CAND) sh->cz[at] = z, sh->cc[at] = v * N - row.shift + c;
        }
      }
    }
  }
  __syncthreads();
  const int cands = sh->cands;
  if (tid == 0) {
    float rs = M > -INFINITY ? sh->own_rest : 0.f, re = M > -INFINITY ? sh->own_ent : 0.f;
    int c = 0;
    for (int w = 0; w < WARPS; ++w) rs += sh->wf[0][w], re += sh->wf[1][w], c += sh->wi[w];
    part->top = M, part->rest = rs, part->ent = re, part->count = c;
    part->n = cands <= CAND ? min(top, cands) : top;
  }
  if (cands <= CAND) {
    for (int i = tid; i < cands; i += THREADS) {
      const float z = sh->cz[i];
      const int c = sh->cc[i];
      int r = 0;
      for (int j = 0; j < cands; ++j) r += before(sh->cz[j], sh->cc[j], z, c);
      if (r < top) lz[r] = z, lc[r] = c;
    }
  } else {
    // more than CAND columns reach tau (and so at least `top`): the next one, `top` times
    float pz = INFINITY;
    int pc = -1;
    for (int k = 0; k < top; ++k) {
      float x = -INFINITY;
      int xi = INT32_MAX;
      for (int v = v0 + tid; v < v1; v += THREADS) {
        const uint4 w = row.load(v);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const float z = Pack<T>::get(w, q);
          const int c = v * N - row.shift + q;
          if (z > -INFINITY && before(pz, pc, z, c) && before(z, c, x, xi)) x = z, xi = c;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        const int yi = __shfl_xor_sync(0xffffffffu, xi, o);
        if (before(y, yi, x, xi)) x = y, xi = yi;
      }
      __syncthreads();
      if (lane == 0) sh->cz[warp] = x, sh->cc[warp] = xi;
      __syncthreads();
      x = sh->cz[0], xi = sh->cc[0];
      for (int w = 1; w < WARPS; ++w)
        if (before(sh->cz[w], sh->cc[w], x, xi)) x = sh->cz[w], xi = sh->cc[w];
      if (tid == 0) lz[k] = x, lc[k] = xi;
      pz = x, pc = xi;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(THREADS, 2) logprobs_kernel(const LogprobArgs a, const int C) {
  __shared__ Shared sh;
  const int tid = threadIdx.x;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = C > 1 ? (int)cluster.block_rank() : 0;
  const int64_t i = blockIdx.x / C;
  const T* p = static_cast<const T*>(a.logits) + i * a.ld;
  const Row<T> row(p, a.vocab);
  // waited for before the first write to another CTA's shared memory
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed;");
  const int each = (row.loads + C - 1) / C, v0 = min(rank * each, row.loads), v1 = min(v0 + each, row.loads);
  int t;
  float zt;
  bool bad;
  share_of_row(row, v0, v1, a.tokens + i, t, zt, bad, a.top, &sh, &sh.part[rank], sh.lz[rank], sh.lc[rank]);
  if (bad && tid == 0 && rank == 0) report(a.dev_status, DSA_DEV_BAD_INDEX);
  __syncthreads();
  if (C > 1) {
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (rank > 0) {
      Shared* to = cluster.map_shared_rank(&sh, 0);
      if (tid == 0) to->part[rank] = sh.part[rank];
      for (int k = tid; k < sh.part[rank].n; k += THREADS) to->lz[rank][k] = sh.lz[rank][k], to->lc[rank][k] = sh.lc[rank][k];
    }
    cluster.sync();
    if (rank > 0) return;
  }
  // ---- the shares together ----
  float M = -INFINITY;
  int first = 0;
  for (int c = 0; c < C; ++c)
    if (sh.part[c].top > M) M = sh.part[c].top, first = c;
  float rest = 0.f, ent = 0.f;
  int count = 0;
  for (int c = 0; c < C; ++c) {
    const Part& q = sh.part[c];
    count += q.count;
    if (q.top == -INFINITY || c == first) {
      rest += q.rest;
      ent += q.ent;
    } else {
      const float d = fmaxf((q.top - M) * LOG2E, X_MIN), f = ex2(d), s = 1.f + q.rest;
      rest = fmaf(s, f, rest);
      ent = fmaf(fmaf(s, d, q.ent), f, ent);
    }
  }
  const bool odd = isnan(rest) || M == INFINITY, none = M == -INFINITY;
  const float log_total = log1pf(rest);
  if (tid == 0) {
    a.logprob[i] = odd ? NAN : t < 0 || none ? -INFINITY : (zt - M) - log_total;
    a.entropy[i] = odd ? NAN : none ? 0.f : log_total - LN2 * ent / (1.f + rest);
    // equal values of lower columns in the token's own load
    if (t >= 0 && zt > -INFINITY)
      for (int j = max(0, t - (t + row.shift) % Row<T>::N); j < t; ++j) count += (float)p[j] == zt;
    if (!(t >= 0 && zt == -INFINITY)) a.rank[i] = t < 0 ? -1 : min(count, a.vocab - 1);
  }
  if (t >= 0 && zt == -INFINITY) {  // a masked token: counted on its own
    int n = 0;
    for (int j = tid; j < a.vocab; j += THREADS) {
      const float z = (float)p[j];
      n += z > -INFINITY || (z == -INFINITY && j < t);
    }
    n = (int)__reduce_add_sync(0xffffffffu, (uint32_t)n);
    __syncthreads();
    if ((tid & 31) == 0) sh.wi[tid >> 5] = n;
    __syncthreads();
    if (tid == 0) {
      n = 0;
      for (int w = 0; w < WARPS; ++w) n += sh.wi[w];
      a.rank[i] = min(n, a.vocab - 1);
    }
  }
  if (a.top == 0) return;
  int have = 0;
  for (int c = 0; c < C; ++c) have += sh.part[c].n;
  for (int e = tid; e < C * MAX_TOP; e += THREADS) {
    const int c = e / MAX_TOP, k = e % MAX_TOP;
    if (k >= sh.part[c].n) continue;
    const float z = sh.lz[c][k];
    const int col = sh.lc[c][k];
    int r = k;
    for (int o = 0; o < C; ++o)
      if (o != c)
        for (int j = 0; j < sh.part[o].n && before(sh.lz[o][j], sh.lc[o][j], z, col); ++j) ++r;
    if (r < a.top) {
      a.top_ids[i * a.top + r] = col;
      a.top_logprobs[i * a.top + r] = odd ? NAN : (z - M) - log_total;
    }
  }
  for (int k = have + tid; k < a.top; k += THREADS) {
    a.top_ids[i * a.top + k] = -1;
    a.top_logprobs[i * a.top + k] = odd ? NAN : -INFINITY;
  }
}

template <class T>
cudaError_t launch(const LogprobArgs& a, cudaStream_t stream) {
  // CTAs a row: few rows share the GPU, as long as a thread has a load and all CTAs run at once, two an
  // SM (64 x 50,000 values 10 us in 256 CTAs, 20 in 512; 128 x 131,072 fp32 19 us in 256, 31 in 512).  Rows
  // past that go a CTA each (sharing out the last wave's among clusters: 1,024 rows 66 -> 72 us).
  const int64_t loads = ((int64_t)a.vocab + Pack<T>::N - 1) / Pack<T>::N;
  int c = 1;
  while (c < MAX_CLUSTER && (int64_t)a.num_rows * c * 2 <= 2 * device_sm_count() && loads > (int64_t)THREADS * c) c *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.num_rows * c);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a, c);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  if (a.dtype == DSA_BF16) return launch<__nv_bfloat16>(a, stream);
  if (a.dtype == DSA_FP16) return launch<__half>(a, stream);
  return launch<float>(a, stream);
}

}  // namespace dsa
