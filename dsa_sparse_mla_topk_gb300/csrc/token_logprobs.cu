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
//    has the term 1 among its terms: its columns are read again and summed without it.
//  * of the k-th largest of 128 groups of threads' maxima, tau, it is known that k columns
//    at least reach it: all alternatives are among the columns >= tau, which only a few threads
//    hold (about as many as k).  Their columns are read again (from L2) too; those that reach
//    tau, usually little more than k, are put in order by counting.  Too many of them (equal
//    logits all over): k rounds of a search for the next one.
// A row of 16-bit values costs 10 instructions a value, as many as the SMs have in the time that HBM takes:
// 6.6 are arithmetic (fp32 two-wide, maxima and counts two-wide in the type), the rest a turn's; nothing is
// checked in turns that lie in the row as a whole (with checks at each load 11.2).
// What follows a row is a chain of ten thousand cycles that mostly waits; a row a CTA of 256 threads,
// four an SM, lets other rows' loads run under it.
// Measured: 1,024 rows of 131,072 bf16, 20 alternatives, 59 us (4.6 TB/s), fp32 103 us (5.2 TB/s), 4,096 rows bf16 203 us (5.3 TB/s),
// 4,096 of 32,000 83 us, 128 of 131,072 fp32 19 us, 4 of 32,003 fp32 9.1 us (launch and the chain of steps).
// Rows that do not start at 16 bytes pay for their ends, two waits and a turn more: 1,024 x 131,071 75 us.
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

constexpr int MAX_CLUSTER = 8, MAX_TOP = token_logprobs_max_top();
constexpr int SLOTS = 512;  // parts of a share, each with its largest value: a thread's, cut in time where there are fewer threads
constexpr int TURNS = 4;    // loads of a thread in flight
constexpr int CAND = 1024;  // columns >= tau that are put in order
constexpr int GROUPS = 128;  // of slots, slot mod GROUPS: as many hold values as loads do, at most all
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

__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o); }

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
  struct Count {
    // of masks of ones (at most 2^15 a half): a lower and b upper halves sum to 2^16 (a - b) - a mod 2^32
    uint32_t v = 0;
    __device__ __forceinline__ void take(const uint4& w, Bound thr) {
      const T2 t2 = as_pair<T2>(thr);
      v += __hgt2_mask(as_pair<T2>(w.x), t2) + __hgt2_mask(as_pair<T2>(w.y), t2);
      v += __hgt2_mask(as_pair<T2>(w.z), t2) + __hgt2_mask(as_pair<T2>(w.w), t2);
    }
    __device__ __forceinline__ int value() const {
      const int a = (int)(0u - v & 0xffffu);
      return 2 * a - ((int)(v + (uint32_t)a) >> 16);
    }
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
  __device__ __forceinline__ uint4 load(int v) const {
    if (inside(v)) return __ldg(reinterpret_cast<const uint4*>(p - shift) + v);
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
  float wf[2][16];
  int wi[2][16], wt[16];
  uint32_t wk[2][16];
  float m_s[SLOTS];
  __align__(16) float gm[GROUPS];
  Part part[MAX_CLUSTER];
  float lz[MAX_CLUSTER][MAX_TOP];
  int lc[MAX_CLUSTER][MAX_TOP];
  float cz[CAND];
  int cc[CAND];
  int list[SLOTS + 4];
  int listed, cands;
};

// Sums and order over the share [v0, v1) of a row's loads by this CTA.
template <class T, int THREADS>
__device__ __forceinline__ void share_of_row(const Row<T>& row, int v0, int v1, const int32_t* token, int& t, float& zt,
                                             bool& bad, int top, Shared* sh, Part* part, float* lz, int* lc) {
  constexpr int N = Pack<T>::N, WARPS = THREADS / 32, SEG = SLOTS / THREADS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // A turn's loads are on their way while the one before is worked on, the first while the token is looked up.
  // Loads that lie in the row as a whole, in0 .. in1 - 1 of the share, wait for nothing; the row's ends are patched in.
  constexpr int TURN = THREADS * TURNS;
  const int in0 = max(v0, row.inside(0) ? 0 : 1), in1 = min(v1, row.inside(row.loads - 1) ? row.loads : row.loads - 1);
  const uint4* from = reinterpret_cast<const uint4*>(row.p - row.shift) + v0 + tid;
  auto fetch = [&](int vb, uint4 (&w)[TURNS]) {
    if (vb >= in0 && vb + TURN <= in1) {
#pragma unroll
      for (int k = 0; k < TURNS; ++k) w[k] = __ldg(from + THREADS * k);
    } else {
#pragma unroll
      for (int k = 0; k < TURNS; ++k) {
        const int v = vb + THREADS * k + tid;
        w[k] = make_uint4(Pack<T>::minus_inf(), Pack<T>::minus_inf(), Pack<T>::minus_inf(), Pack<T>::minus_inf());
        if (v >= in0 && v < in1) w[k] = __ldg(from + THREADS * k);
      }
      if ((vb < in0 && v0 < v1) || (in1 < v1 && vb + TURN > in1)) {
#pragma unroll
        for (int k = 0; k < TURNS; ++k) {
          const int v = vb + THREADS * k + tid;
          if (v < v1 && (v < in0 || v >= in1)) w[k] = row.load(v);
        }
      }
    }
    from += TURN;
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
  // a thread's slots: `per` turns each
  const int per = ((v1 - v0 + TURN - 1) / TURN + SEG - 1) / SEG;
  float m_seg = -INFINITY;
  int seg = 0, left = per;
  if (tid == 0 && v0 == 0 && t >= 0) {  // equal values of lower columns in the token's own load
    const uint4 w = row.load(vt);
#pragma unroll
    for (int c = 0; c < N; ++c) count += Pack<T>::get(w, c) == zt && vt * N - row.shift + c < t;
  }
  int room = 512;
  typename Pack<T>::Count n;
#pragma unroll 1
  for (int vb = v0; vb < v1; vb += TURN) {
    uint4 w[TURNS];
#pragma unroll
    for (int k = 0; k < TURNS; ++k) w[k] = next[k];
    if (vb + TURN < v1) fetch(vb + TURN, next);
    typename Pack<T>::Most most;
    const int before_t = vt - tid - vb;
#pragma unroll
    for (int k = 0; k < TURNS; ++k) {
      most.take(w[k]);
      n.take(w[k], THREADS * k < before_t ? thr_lo : thr_hi);
    }
    if (--room == 0) count += n.value(), n = {}, room = 512;
    const float now = most.value(), up = fmaxf(m, now);
    if (SEG > 1) {
      m_seg = fmaxf(m_seg, now);
      if (--left == 0) sh->m_s[seg * THREADS + tid] = m_seg, m_seg = -INFINITY, ++seg, left = per;
    }
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
  count += n.value();
  float s, e, hi;
  upk2(s2, s, hi);
  s += hi;
  upk2(e2, e, hi);
  e += hi;

  // ---- the largest value, and one thread that holds it ----
  if (tid == 0) sh->listed = SEG, sh->cands = 0;  // the owner's first
  if (SEG == 1) sh->m_s[tid] = m;
  else
    for (; seg < SEG; ++seg) sh->m_s[seg * THREADS + tid] = m_seg, m_seg = -INFINITY;
  const uint32_t key = order_of(m), wmost = __reduce_max_sync(0xffffffffu, key);
  const int wfirst = __ffs(__ballot_sync(0xffffffffu, key == wmost)) - 1;
  if (lane == 0) sh->wk[0][warp] = wmost, sh->wt[warp] = warp * 32 + wfirst;
  __syncthreads();
  const uint32_t kw = sh->wk[0][lane % WARPS], most = __reduce_max_sync(0xffffffffu, kw);
  const int owner = sh->wt[__ffs(__ballot_sync(0xffffffffu, kw == most)) - 1];
  const float M = value_of(most);

  // ---- tau: the top-th largest of the groups' maxima ----
  uint32_t tau = UINT32_MAX;
  if (top > 0) {
    if (tid < GROUPS) {
      float g = sh->m_s[tid];
#pragma unroll
      for (int k = GROUPS; k < SLOTS; k += GROUPS) g = fmaxf(g, sh->m_s[tid + k]);
      sh->gm[tid] = g;
    }
    __syncthreads();
    // a group's threads count the groups that reach it
    constexpr int EACH = THREADS / GROUPS;
    const float x = sh->gm[tid / EACH];
    int c = 0;
#pragma unroll
    for (int j = tid % EACH; j < GROUPS / 4; j += EACH) {
      const float4 y = reinterpret_cast<const float4*>(sh->gm)[j];
      c += y.x >= x;
      c += y.y >= x;
      c += y.z >= x;
      c += y.w >= x;
    }
#pragma unroll
    for (int o = EACH / 2; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    const uint32_t reached = __reduce_max_sync(0xffffffffu, c >= top ? order_of(x) : 0u);
    if (lane == 0) sh->wk[1][warp] = reached;
    __syncthreads();
    // (fewer groups that hold values: every value)
    tau = max(__reduce_max_sync(0xffffffffu, sh->wk[1][lane % WARPS]), order_of(-INFINITY) + 1);
#pragma unroll
    for (int g = 0; g < SEG; ++g) {
      const uint32_t flags = __ballot_sync(0xffffffffu, order_of(sh->m_s[g * THREADS + tid]) >= tau && tid != owner);
      if (flags) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&sh->listed, __popc(flags));
        at = __shfl_sync(0xffffffffu, at, 0);
        if (flags >> lane & 1) sh->list[at + __popc(flags & ((1u << lane) - 1))] = g * THREADS + tid;
      }
    }
    __syncthreads();
  }

  // ---- columns read again: the owner's for the sum, the listed threads' for tau ----
  const float d = fmaxf((m - M) * LOG2E, X_MIN), f = m == -INFINITY ? 0.f : ex2(d);
  // (a thread without values: s is 0, or NaN where there was one)
  e = fmaf(s, m == -INFINITY ? 0.f : d, e) * f;
  s = m == -INFINITY ? s : s * f;
  if (tid == owner && M > -INFINITY) s = 0.f, e = 0.f;
  int same = 0;
  const int listed = sh->listed, loads = SEG > 1 ? per * TURNS : (v1 - v0 + THREADS - 1) / THREADS;  // of a slot
  const int lg = loads > 1 ? 32 - __clz(loads - 1) : 0;
  constexpr int AT_ONCE = 1024 / THREADS;  // the listed slots' loads in a round or two
  for (int q0 = tid; q0 < listed << lg; q0 += THREADS * AT_ONCE) {
    uint4 w[AT_ONCE];
    int who[AT_ONCE], v[AT_ONCE];
#pragma unroll
    for (int h = 0; h < AT_ONCE; ++h) {
      const int q = q0 + THREADS * h, k = q >> lg, j = q & ((1 << lg) - 1);
      const int slot = k < SEG ? k * THREADS + owner : k < listed ? sh->list[k] : 0;
      who[h] = slot % THREADS;
      v[h] = v0 + who[h] + THREADS * (slot / THREADS * loads + j);
      if (k >= listed || j >= loads || v[h] >= v1) who[h] = -1;
      else w[h] = row.load(v[h]);
    }
#pragma unroll
    for (int h = 0; h < AT_ONCE; ++h) {
      if (who[h] < 0) continue;
      int hits = 0;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const float z = Pack<T>::get(w[h], c);
        hits += z > -INFINITY && order_of(z) >= tau;
      }
      if (hits > 0) {
        int at = atomicAdd(&sh->cands, hits);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float z = Pack<T>::get(w[h], c);
          if (z > -INFINITY && order_of(z) >= tau) {
            if (at < CAND) sh->cz[at] = z, sh->cc[at] = v[h] * N - row.shift + c;
            ++at;
          }
        }
      }
      if (who[h] == owner && M > -INFINITY) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float z = Pack<T>::get(w[h], c);
          if (z == M) {
            ++same;
          } else {
            const float x = max_nan((z - M) * LOG2E, X_MIN), p = ex2(x);
            s += p;
            e = fmaf(p, x, e);
          }
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    e += __shfl_xor_sync(0xffffffffu, e, o);
  }
  count = (int)__reduce_add_sync(0xffffffffu, (uint32_t)count);
  same = (int)__reduce_add_sync(0xffffffffu, (uint32_t)same);
  if (lane == 0) sh->wf[0][warp] = s, sh->wf[1][warp] = e, sh->wi[0][warp] = count, sh->wi[1][warp] = same;
  __syncthreads();
  const int cands = sh->cands;
  if (warp == 0) {
    s = lane < WARPS ? sh->wf[0][lane] : 0.f, e = lane < WARPS ? sh->wf[1][lane] : 0.f;
#pragma unroll
    for (int o = WARPS / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    count = (int)__reduce_add_sync(0xffffffffu, lane < WARPS ? sh->wi[0][lane] : 0);
    same = (int)__reduce_add_sync(0xffffffffu, lane < WARPS ? sh->wi[1][lane] : 0);
    if (lane == 0) {
      part->top = M, part->rest = M > -INFINITY ? s + (float)(same - 1) : s, part->ent = e, part->count = count;
      part->n = cands <= CAND ? min(top, cands) : top;
    }
  }
  if (cands <= CAND) {
    // eight threads a column
    for (int q0 = 0; q0 < cands; q0 += THREADS / 8) {
      const int q = q0 + tid / 8;
      const float z = q < cands ? sh->cz[q] : 0.f;
      const int c = q < cands ? sh->cc[q] : 0;
      int r = 0;
      if (q < cands)
        for (int j = tid % 8; j < cands; j += 8) r += before(sh->cz[j], sh->cc[j], z, c);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
      if (q < cands && tid % 8 == 0 && r < top) lz[r] = z, lc[r] = c;
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

template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logprobs_kernel(const LogprobArgs a, const int C) {
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
  share_of_row<T, THREADS>(row, v0, v1, a.tokens + i, t, zt, bad, a.top, &sh, &sh.part[rank], sh.lz[rank], sh.lc[rank]);
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
    if ((tid & 31) == 0) sh.wi[0][tid >> 5] = n;
    __syncthreads();
    if (tid == 0) {
      n = 0;
      for (int w = 0; w < THREADS / 32; ++w) n += sh.wi[0][w];
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

template <class T, int THREADS>
cudaError_t launch(const LogprobArgs& a, cudaStream_t stream) {
  // CTAs a row: few rows share the GPU, as long as a thread has a load and all CTAs run at once, two an
  // SM (64 x 50,000 values 10 us in 256 CTAs, 20 in 512; 128 x 131,072 fp32 19 us in 256, 31 in 512).  Rows
  // past that go a CTA each (sharing out the last wave's among clusters costs 1,024 rows 6 us more).
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, logprobs_kernel<T, THREADS>, a, c);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  // Many rows: CTAs of half the threads, whose chains behind a row overlap.  512, 256, 128 threads, us: 400 x 8,000
  // bf16 13.0, 8.7, 9.8; 4,096 x 8,000 93, 54, 55; 4,096 x 32,000 114, 83, 94; 1,024 x 131,072 63, 59, 77; fp32
  // 4,096 x 8,000 84, 56, 54; 4,096 x 32,000 128, 110, 123; 1,024 x 131,072 107, 103, 112; fp16 as bf16.
  const bool many = a.num_rows > 2 * device_sm_count();
  if (a.dtype == DSA_BF16) return many ? launch<__nv_bfloat16, 256>(a, stream) : launch<__nv_bfloat16, 512>(a, stream);
  if (a.dtype == DSA_FP16) return many ? launch<__half, 256>(a, stream) : launch<__half, 512>(a, stream);
  return many ? launch<float, 256>(a, stream) : launch<float, 512>(a, stream);
}

}  // namespace dsa
