// Log probabilities of given tokens, log-sum-exp, entropy and the top
// alternatives of rows of logits.
#include <cfloat>
#include <cmath>

#include "float2.cuh"
#include "float_io.cuh"
#include "launch.h"
#include "step_launch.h"

namespace qmv {

constexpr int LP_UNROLL = 4;        // 16-byte loads of a thread on their way
constexpr int LP_MAX_CLUSTER = 8;
constexpr int LP_SEGS = 16;         // stretches of a thread's loads whose largest logit is kept
constexpr int LP_CAND = 1024;       // candidates for the top list that shared memory holds
constexpr int LP_CHAIN = 512;       // terms that a thread adds up in 32 bits before they join its sums in 64
// The smallest exponent (of 2) that matters; also what exp2 of a masked logit takes,
// so that 0 * -inf never enters a sum.
constexpr float LP_LOWEST = -1.0e4f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float at_least(float a, float b) {  // NaN stays NaN
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
// 16 bytes of logits.
template <int DT>
struct LogitVec {
  using T = typename Elem<DT>::type;
  static constexpr int N = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ float2 pair(int i) const {  // values 2i, 2i + 1
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (DT == QMV_DT_F32) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    if constexpr (DT == QMV_DT_BF16) return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    if constexpr (DT == QMV_DT_F16) return __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
  }
  // The first of the values that equals m, if any, becomes -inf; true if there was one.
  __device__ __forceinline__ bool leave_out(float m) {
    uint32_t* const w[4] = {&raw.x, &raw.y, &raw.z, &raw.w};
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (DT == QMV_DT_F32) {
        const bool here = !found && __uint_as_float(*w[i]) == m;
        if (here) *w[i] = 0xff800000u;
        found |= here;
      } else {
        const float2 v = pair(i);
        const uint32_t low = DT == QMV_DT_BF16 ? 0xff80u : 0xfc00u;
        const bool a = !found && v.x == m, b = !found && !a && v.y == m;
        if (a) *w[i] = (*w[i] & 0xffff0000u) | low;
        if (b) *w[i] = (*w[i] & 0xffffu) | low << 16;
        found |= a || b;
      }
    }
    return found;
  }
  __device__ __forceinline__ void mask() {  // all -inf
    const uint32_t w = DT == QMV_DT_F32 ? 0xff800000u : DT == QMV_DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;
    raw = make_uint4(w, w, w, w);
  }
};

// The largest of some vectors' logits (NaN left out).
template <int DT, int U>
__device__ __forceinline__ float largest(const LogitVec<DT> (&x)[U]) {
  if constexpr (DT == QMV_DT_F32) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const float2 v = x[u].pair(i);
        m = fmaxf(m, fmaxf(v.x, v.y));
      }
    return m;
  } else {
    using Two = typename std::conditional<DT == QMV_DT_BF16, __nv_bfloat162, __half2>::type;
    Two m;
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t w[4] = {x[u].raw.x, x[u].raw.y, x[u].raw.z, x[u].raw.w};
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const Two v = *reinterpret_cast<const Two*>(&w[i]);
        m = u + i ? __hmax2(m, v) : v;
      }
    }
    return fmaxf(fmaxf(to_float(m.x), to_float(m.y)), -INFINITY);  // (both NaN: -inf)
  }
}

__device__ __forceinline__ unsigned long long candidate(float v, int at) {  // larger first, then the lower index
  v += 0.0f;  // (-0 as 0)
  const uint32_t b = __float_as_uint(v), o = (int)b < 0 ? ~b : b | 0x80000000u;
  return (unsigned long long)o << 32 | (0xffffffffu - (uint32_t)at);
}
__device__ __forceinline__ float value_of(unsigned long long c) {
  const uint32_t o = (uint32_t)(c >> 32);
  return __uint_as_float((int)o < 0 ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int index_of(unsigned long long c) { return (int)(0xffffffffu - (uint32_t)c); }

// What a warp knows of its part of a row: its largest logit m, and over its other
// logits s = sum 2^d and t = sum 2^d d with d = (l - m) k, k = scale / ln 2.  The
// largest one itself (2^0) is left out, so that a row that is nearly certain keeps
// the digits of what is left: log-sum-exp = scale m + log1p(s).
struct LpPart {
  float m, s, t;  // m -inf: no logit above -inf (s and t are 0, or NaN)
};

__device__ __forceinline__ uint32_t peer(const void* here, int rank) {  // the same place in another CTA of the cluster
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(here)), "r"(rank));
  return at;
}

// A cluster a row, each CTA a run of its 16-byte vectors; a thread takes every NT-th.
//
// One pass over the logits: sums of 2^d and 2^d d relative to the warp's largest
// logit so far, that one left out (when it grows, both are rescaled and the former
// one joins them), and the largest of each stretch of each thread's loads.  For the
// top list a little of the row is then read again from L2: the stretches whose
// largest reaches a floor that at least n_top threads reach, the q-th largest among all
// warps' r-th largest thread maxima, q r >= n_top.  Every logit of the list is at least
// that floor and lies in such a stretch.  These candidates are ordered by (value,
// index), so no order of arrival shows; where they overflow shared memory (many equal
// logits) the list is found entry by entry, each by a pass of its own of one CTA over the
// row: 20 of a row of 151936 equal fp32 logits 485 us (7.5 where they differ), of 2^20 3.2 ms.
//
// Bound by HBM for many rows, with about 8 instructions a logit: 2048 x 151936 bfloat16
// (622 MB) 119 us, 5.2 TB/s (three CTAs of 256 threads an SM with the next loads on
// their way; four without 121, two 139).  One row of 151936 fp32 6.6 us: three rounds of
// loads, two barriers of the cluster and the loads of the candidates in turn.
//
// LONG: more than FOLD vectors a CTA.  There a thread's sums join sums in 64 bits every
// LP_CHAIN terms: in 32 bits alone rows of 2^24 logits were off by 5e-5 where all were
// equal, and by 1.1e-4 where they rose slowly (a rescaling a step).  Shorter rows, which
// never fold, keep a loop without it (16 rows of 151936 fp32 7.3 us, with it 7.7; 2048 of
// bfloat16 119 and 123).
template <int DT, int NT>
constexpr int lp_fold() {  // vectors from one fold to the next
  return NT * LP_CHAIN / (LogitVec<DT>::N / 2);
}
template <int DT, int NT, bool LONG>
__global__ void __launch_bounds__(NT, NT == 512 ? 1 : 3) logprobs_kernel(const LogprobsParams p, int ranks) {
  using Vec = LogitVec<DT>;
  using T = typename Vec::T;
  constexpr int N = Vec::N, WARPS = NT / 32, MAX_PARTS = (NT == 512 ? LP_MAX_CLUSTER : 2) * WARPS;
  static_assert(sizeof(double2) * NT <= sizeof(unsigned long long) * LP_CAND, "the threads' long sums lie in cand");
  __shared__ __align__(16) unsigned long long cand[LP_CAND];  // the first CTA's: the row's
  __shared__ float seg_max[LP_SEGS][NT];
  __shared__ LpPart parts[MAX_PARTS];              // the first CTA's: all warps'
  __shared__ float reach[MAX_PARTS];               // all warps' r-th largest thread maxima
  __shared__ int n_cand, n_again, again[NT];
  __shared__ float s_floor, s_top, s_log;
  __shared__ unsigned long long w_best[WARPS];
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = ranks > 1 ? blockIdx.x % ranks : 0;
  const long long r = ranks > 1 ? blockIdx.x / ranks : blockIdx.x;
  const int n_parts = ranks * WARPS;
  if (tid == 0) n_cand = n_again = 0;
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  const T* row = static_cast<const T*>(p.logits) + r * p.ld;
  // vectors of 16 aligned bytes; the first may begin before the row, the last end after it
  const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
  const int n_vec = (int)((p.V + shift + N - 1) / N);
  const int v0 = (int)((long long)n_vec * rank / ranks), v1 = (int)((long long)n_vec * (rank + 1) / ranks);
  const int whole0 = max(v0, shift > 0), whole1 = min(v1, (p.V + shift) / N);  // whole ones of the CTA
  // vector v of the row if it lies before `end`
  auto load = [&](int v, int end) {
    Vec x;
    x.mask();
    if (v < end) {
      const int e = v * N - shift;
      if (e >= 0 && e + N <= p.V) {
        if (QMV_CHECK(in_range(r * p.ld + e, N, p.logits_len, p.err))) x.raw = __ldg(reinterpret_cast<const uint4*>(row + e));
      } else {
        alignas(16) T t[N];
        *reinterpret_cast<uint4*>(t) = x.raw;
#pragma unroll
        for (int j = 0; j < N; j++)
          if (e + j >= 0 && e + j < p.V && QMV_CHECK(in_range(r * p.ld + e + j, 1, p.logits_len, p.err))) t[j] = row[e + j];
        x.raw = *reinterpret_cast<const uint4*>(t);
      }
    }
    return x;
  };
  // the given tokens' logits
  float given = 0.f;
  int token = -1;
  if (rank == 0 && tid < p.n_given) {
    token = p.tokens[r * p.n_given + tid];
    if (token >= p.V) set_error(p.err, QMV_DEVERR_TOKEN);
    if (token >= 0 && token < p.V) given = to_float(row[token]);
  }

  const float k = p.scale * 1.4426950408889634f;
  const F2 k2 = F2::of(k, k);
  float m = -FLT_MAX, mine = -INFINITY, stretch = -INFINITY;
  bool out = false;  // the warp's largest is left out of the sums
  F2 S = F2::of(0.f, 0.f), D = S;
  constexpr int STEP = NT * LP_UNROLL, FOLD = lp_fold<DT, NT>();
  static_assert(FOLD % STEP == 0, "whole steps");
  // s and t of the vectors folded before (until the candidates come), relative to fold_m
  double2& folded = reinterpret_cast<double2*>(cand)[tid];
  float fold_m = -FLT_MAX;
  auto fold = [&](bool some) {
    double2 sum = some ? folded : make_double2(0., 0.);
    if (some && fold_m != m) {  // (seldom: exp2 in 64 bits takes as long as some steps)
      const double d = fmax(((double)fold_m - m) * k, (double)LP_LOWEST), f = exp2(d);
      sum = make_double2(f * sum.x, f * (sum.y + d * sum.x));
    }
    sum.x += (double)S.x() + (double)S.y();
    sum.y += (double)D.x() + (double)D.y();
    return sum;
  };
  const int steps = (v1 - v0 + STEP - 1) / STEP, per_seg = (steps + LP_SEGS - 1) / LP_SEGS;
  int seg = 0, in_seg = 0;
  auto fetch = [&](int v, Vec(&x)[LP_UNROLL]) {
    const int w = v - lane;  // the warp's first
    if (w >= whole0 && w + NT * (LP_UNROLL - 1) + 32 <= whole1 &&
        QMV_CHECK(in_range(r * p.ld + (long long)v * N - shift, (long long)NT * (LP_UNROLL - 1) * N + N, p.logits_len, p.err))) {
      const uint4* at = reinterpret_cast<const uint4*>(row + (v * N - shift));
#pragma unroll
      for (int u = 0; u < LP_UNROLL; u++) x[u].raw = __ldg(at + u * NT);
    } else {
#pragma unroll
      for (int u = 0; u < LP_UNROLL; u++) x[u] = load(v + u * NT, v1);
    }
  };
  Vec next[LP_UNROLL];
  fetch(v0 + tid, next);
  for (int v = v0 + tid;;) {
    const int end = LONG ? min(v1, v - tid + FOLD) : v1;
#pragma unroll 2
    for (; v - tid < end; v += STEP) {
      Vec x[LP_UNROLL];
#pragma unroll
      for (int u = 0; u < LP_UNROLL; u++) x[u] = next[u];
      fetch(v + STEP, next);  // (the next step's are on their way)
      const float bm = largest(x);
      mine = fmaxf(mine, bm);
      stretch = fmaxf(stretch, bm);
      if (++in_seg == per_seg) {
        seg_max[seg][tid] = stretch;
        seg++;
        in_seg = 0;
        stretch = -INFINITY;
      }
      const unsigned above = __ballot_sync(0xffffffffu, bm > m || (!out && bm == m));
      if (above) {
        const float now = warp_max(bm), d = fmaxf((m - now) * k, LP_LOWEST), f = ex2(d);
        const F2 f2 = F2::of(f, f), was = F2::of(out && lane == 0 ? 1.f : 0.f, 0.f);
        // the former largest joins the sums (d is 0 for it)
        S = S + was;
        D = f2 * fma2(F2::of(d, d), S, D);
        S = f2 * S;
        m = now;
        out = true;
        if (lane == __ffs(__ballot_sync(0xffffffffu, bm == now)) - 1) {
          bool left = false;
#pragma unroll
          for (int u = 0; u < LP_UNROLL; u++)
            if (!left) left = x[u].leave_out(now);
        }
      }
      const F2 m2 = F2::of(-m, -m);
#pragma unroll
      for (int u = 0; u < LP_UNROLL; u++)
#pragma unroll
        for (int i = 0; i < N / 2; i++) {
          const float2 l = x[u].pair(i);
          F2 d = (F2::of(l.x, l.y) + m2) * k2;
          d = F2::of(at_least(d.x(), LP_LOWEST), at_least(d.y(), LP_LOWEST));
          const F2 e = F2::of(ex2(d.x()), ex2(d.y()));
          S = S + e;
          D = fma2(e, d, D);
        }
    }
    if (!LONG || v - tid >= v1) break;
    folded = fold(v - tid - v0 > FOLD);
    fold_m = m;
    S = D = F2::of(0.f, 0.f);
  }
  if (in_seg) seg_max[seg][tid] = stretch;

  const int n_top = p.n_top;
  const int nr = (2 * n_top + n_parts - 1) / n_parts, nq = nr ? (n_top + nr - 1) / nr : 0;  // (n_parts is at least 8)
  float s = S.x() + S.y(), t = D.x() + D.y();
  if (LONG && v1 - v0 > FOLD) {
    const double2 sum = fold(true);
    s = (float)sum.x;
    t = (float)sum.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  float rth = -INFINITY;
  {
    float left = mine;
    for (int i = 0; i < nr; i++) {
      rth = warp_max(left);
      if (i + 1 < nr && lane == __ffs(__ballot_sync(0xffffffffu, left == rth)) - 1) left = -INFINITY;
    }
  }
  const LpPart part{out ? m : -INFINITY, s, t};
  const int me = rank * WARPS + warp;
  if (ranks > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all CTAs are there
    if (lane < ranks && n_top)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer(&reach[me], lane)), "f"(rth) : "memory");
    if (lane == 0) {
      const uint32_t to = peer(&parts[me], 0);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(part.m) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(part.s) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(part.t) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank > 0 && !n_top) return;
  } else {
    if (lane == 0) {
      reach[me] = rth;
      parts[me] = part;
    }
    __syncthreads();
  }
  if (n_top) {
    // The floor: the nq-th largest of all warps' values (one of equal ones before the
    // next).  Four threads count for each.
    if (tid < 4 * n_parts) {
      const int of = tid >> 2, quarter = n_parts >> 2;  // (n_parts is a multiple of 8)
      const float v = reach[of];
      int before = 0;
#pragma unroll 8
      for (int j = 0; j < quarter; j++) {
        const int i = 4 * j + (tid & 3);
        before += reach[i] > v || (reach[i] == v && i < of);
      }
      before += __shfl_xor_sync(0xffffffffu, before, 1);
      before += __shfl_xor_sync(0xffffffffu, before, 2);
      if (before == nq - 1) s_floor = v;
    }
    __syncthreads();
    const float floor = s_floor;
    // the stretches that reach it
    if (mine >= floor && mine > -INFINITY)
      for (int i = 0; i * per_seg < steps; i++)
        if (seg_max[i][tid] >= floor) {
          const int at = atomicAdd(&n_again, 1);
          if (at < NT) again[at] = i * NT + tid;
        }
    __syncthreads();
    const bool all = n_again > NT;  // too many to list: everything again
    const int loads = per_seg * LP_UNROLL, items = all ? v1 - v0 : n_again * loads;
    const uint32_t counter = peer(&n_cand, 0);
    for (int i = tid; i < items; i += NT) {
      int v = v0 + i;
      if (!all) {
        const int which = i / loads, of = again[which], first = of / NT * per_seg * STEP;
        v = v0 + first + of % NT + (i - which * loads) * NT;
      }
      const Vec x = load(v, v1);
#pragma unroll
      for (int j = 0; j < N; j++) {
        const float2 two = x.pair(j / 2);
        const float l = j & 1 ? two.y : two.x;
        if (l >= floor && l > -INFINITY) {
          const unsigned long long c = candidate(l, v * N - shift + j);
          int at;
          if (ranks > 1) {
            asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(at) : "r"(counter) : "memory");
            if (at < LP_CAND) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer(&cand[at], 0)), "l"(c) : "memory");
          } else {
            at = atomicAdd(&n_cand, 1);
            if (at < LP_CAND) cand[at] = c;
          }
        }
      }
    }
    if (ranks > 1) {
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      if (rank > 0) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        return;
      }
    }
  }

  // The row's largest, s and t: the warps' in a fixed order, by the first warp.
  if (warp == 0) {
    LpPart q[MAX_PARTS / 32 + (MAX_PARTS < 32)];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < MAX_PARTS; j += 32) {
      q[j / 32] = LpPart{-INFINITY, 0.f, 0.f};
      if (j + lane < n_parts) q[j / 32] = parts[j + lane];
      top = fmaxf(top, q[j / 32].m);
    }
    top = warp_max(top);
    int owner = n_parts;  // the warp whose largest stays out of s
#pragma unroll
    for (int j = 0; j < MAX_PARTS; j += 32)
      if (q[j / 32].m == top) owner = min(owner, j + lane);
    owner = __reduce_min_sync(0xffffffffu, owner);
    float rs = 0.f, rt = 0.f;
#pragma unroll
    for (int j = 0; j < MAX_PARTS; j += 32) {
      const LpPart& of = q[j / 32];
      if (j + lane == owner || !(of.m > -INFINITY)) {
        rs += of.s;  // (0 or NaN where there is no logit)
        rt += of.t;
      } else {
        const float d = at_least((of.m - top) * k, LP_LOWEST), f = ex2(d);
        rs += f * (1.0f + of.s);
        rt += f * (of.t + d * (1.0f + of.s));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      rs += __shfl_xor_sync(0xffffffffu, rs, o);
      rt += __shfl_xor_sync(0xffffffffu, rt, o);
    }
    if (top == INFINITY) rs = NAN;
    const bool none = !(top > -INFINITY) && rs == rs;  // every logit is -inf
    const float log_s = log1pf(rs);
    if (lane == 0) {
      s_top = none ? 0.f : top;
      s_log = none ? INFINITY : log_s;
      if (QMV_CHECK(in_range(r, 1, p.rows_len, p.err))) {
        if (p.lse) p.lse[r] = none ? -INFINITY : fmaf(top, p.scale, log_s);
        if (p.entropy) p.entropy[r] = none ? 0.f : log_s - 0.6931471805599453f * rt / (1.0f + rs);
      }
    }
  }
  if (ranks > 1 && n_top) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  const float top = s_top, log_s = s_log;  // (0 and inf where every logit is -inf: log probabilities are -inf)
  // (halves: the difference of finite logits stays finite)
  auto logp = [&](float l) { return (0.5f * l - 0.5f * top) * (2.0f * p.scale) - log_s; };
  if (tid < p.n_given && QMV_CHECK(in_range(r * p.n_given + tid, 1, p.given_len, p.err)))
    p.logp[r * p.n_given + tid] = token < 0 ? 0.f : token >= p.V ? NAN : logp(given);
  if (!n_top) return;
  auto list = [&](int at, unsigned long long c) {
    if (QMV_CHECK(in_range(r * n_top + at, 1, p.top_len, p.err))) {
      p.top_ids[r * n_top + at] = c ? index_of(c) : -1;
      p.top_logp[r * n_top + at] = c ? logp(value_of(c)) : -INFINITY;
    }
  };
  const int n = n_cand;
  if (n <= LP_CAND) {
    for (int i = warp; i < n; i += WARPS) {
      const unsigned long long c = cand[i];
      int before = 0;
      for (int j = 0; j < n; j += 32) before += __popc(__ballot_sync(0xffffffffu, j + lane < n && cand[j + lane] > c));
      if (lane == 0 && before < n_top) list(before, c);
    }
    for (int i = n + tid; i < n_top; i += NT) list(i, 0);
    return;
  }
  unsigned long long last = ~0ull;
  for (int i = 0; i < n_top; i++) {
    unsigned long long best = 0;
    for (int v = tid; v < n_vec; v += NT) {
      const Vec x = load(v, n_vec);
#pragma unroll
      for (int j = 0; j < N; j++) {
        const float2 two = x.pair(j / 2);
        const float l = j & 1 ? two.y : two.x;
        const unsigned long long c = l > -INFINITY ? candidate(l, v * N - shift + j) : 0;
        if (c < last && c > best) best = c;
      }
    }
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    __syncthreads();  // (the last entry's values are read)
    if (lane == 0) w_best[warp] = best;
    __syncthreads();
    for (int j = 0; j < WARPS; j++) best = max(best, w_best[j]);
    if (tid == 0) list(i, best);
    last = best;
  }
}

template <int DT, int NT, bool LONG>
static cudaError_t launch_long(const LogprobsParams& p, int ranks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  make_config(cfg, attr, dim3((unsigned)(p.rows * ranks)), dim3(NT), 0, stream, true);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, NT, LONG>, p, ranks);
}
template <int DT, int NT>
static cudaError_t launch_as(const LogprobsParams& p, int ranks, cudaStream_t stream) {
  // (a CTA's vectors, with the two that a row may begin and end in)
  const int vecs = (p.V / LogitVec<DT>::N + 2) / ranks + 1;
  return vecs > lp_fold<DT, NT>() ? launch_long<DT, NT, true>(p, ranks, stream) : launch_long<DT, NT, false>(p, ranks, stream);
}

template <int DT>
static cudaError_t launch_dt(const LogprobsParams& p, cudaStream_t stream) {
  // Few rows: a cluster each, while CTAs have a round of loads each and all clusters
  // find room at once (an SM a CTA, and clusters do not fill their part of the GPU:
  // 16 rows in clusters of 4 9 us, of 8 12 us); up to a row an SM two smaller CTAs.
  const int round = 512 * LP_UNROLL * LogitVec<DT>::N / 2;
  int ranks = 1;
  while (ranks < LP_MAX_CLUSTER && 4 * p.rows * ranks <= device_sm_count() && p.V > (long long)ranks * round) ranks *= 2;
  if (ranks > 1) return launch_as<DT, 512>(p, ranks, stream);
  return launch_as<DT, 256>(p, p.rows <= device_sm_count() && p.V > round ? 2 : 1, stream);
}

cudaError_t launch_logprobs(int dtype, const LogprobsParams& p, cudaStream_t stream) {
  switch (dtype) {
    case QMV_DT_F16: return launch_dt<QMV_DT_F16>(p, stream);
    case QMV_DT_BF16: return launch_dt<QMV_DT_BF16>(p, stream);
    default: return launch_dt<QMV_DT_F32>(p, stream);
  }
}

}  // namespace qmv
