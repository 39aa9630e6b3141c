// Log probabilities of given tokens, log-sum-exp, entropy and the top
// alternatives of rows of logits.
#include <cfloat>
#include <cmath>

#include "float_io.cuh"
#include "launch.h"
#include "step_launch.h"

namespace qmv {

constexpr int LP_THREADS = 512, LP_WARPS = LP_THREADS / 32;
constexpr int LP_UNROLL = 4;        // 16-byte loads of a thread on their way
constexpr int LP_MAX_CLUSTER = 8;
constexpr int LP_CAND = 2048;       // candidates for the top list that shared memory holds
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
// Two floats at once (packed fp32 arithmetic).
struct F2 {
  unsigned long long u;
  __device__ __forceinline__ static F2 of(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.u) : "f"(x), "f"(y));
    return r;
  }
  __device__ __forceinline__ float x() const { return __uint_as_float((uint32_t)u); }
  __device__ __forceinline__ float y() const { return __uint_as_float((uint32_t)(u >> 32)); }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return r;
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
  __device__ __forceinline__ void mask() {  // all -inf
    const uint32_t w = DT == QMV_DT_F32 ? 0xff800000u : DT == QMV_DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;
    raw = make_uint4(w, w, w, w);
  }
  __device__ __forceinline__ float largest() const {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N / 2; i++) {
      const float2 v = pair(i);
      m = fmaxf(m, fmaxf(v.x, v.y));
    }
    return m;
  }
};

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

// What a CTA knows of its part of a row: its largest logit M, and over its other
// logits s = sum 2^d and t = sum 2^d d with d = (l - M) k, k = scale / ln 2.  The
// largest one itself (2^0) is left out, so that a row that is nearly certain keeps
// the digits of what is left: log-sum-exp = scale M + log1p(s).
struct LpPart {
  float M, s, t;
  int n;  // entries of its list
};

// A cluster a row, each CTA a run of its 16-byte vectors; a thread takes every 512th.
//
// One pass over the logits: sums of 2^d and 2^d d relative to the warp's largest
// logit so far (when that grows, both are rescaled), and each thread's largest.
// Then a little of the row is read again from L2: the thread that met the CTA's
// largest has its sums formed anew without that one (above), and the top list's
// candidates are taken from the threads whose largest reaches a floor that at least
// n_top threads reach: the q-th largest among the warps' r-th largest thread maxima,
// q r >= n_top.  Every logit of the list is at least that floor and is met by such a
// thread.  Candidates are ordered by (value, index), so no order of arrival shows;
// where they overflow shared memory (many equal logits) the list is found entry
// by entry, each by a pass of its own.
//
// Bound by HBM for many rows: about 6 instructions a logit.
template <int DT>
__global__ void __launch_bounds__(LP_THREADS, 2) logprobs_kernel(const LogprobsParams p, int ranks) {
  using Vec = LogitVec<DT>;
  using T = typename Vec::T;
  constexpr int N = Vec::N;
  __shared__ unsigned long long cand[LP_CAND];
  __shared__ unsigned long long lists[LP_MAX_CLUSTER][QMV_MAX_TOP];
  __shared__ LpPart parts[LP_MAX_CLUSTER];
  __shared__ float w_max[LP_WARPS], w_floor[LP_WARPS], w_s[LP_WARPS], w_t[LP_WARPS];
  __shared__ int w_owner[LP_WARPS];
  __shared__ int n_cand;
  __shared__ unsigned long long w_best[LP_WARPS];
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = ranks > 1 ? blockIdx.x % ranks : 0;
  const long long r = blockIdx.x / ranks;
  if (tid == 0) n_cand = 0;
  pdl_wait();
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const T* row = static_cast<const T*>(p.logits) + r * p.ld;
  // vectors of 16 aligned bytes; the first may begin before the row
  const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
  const int n_vec = (int)((p.V + shift + N - 1) / N);
  const int v0 = (int)((long long)n_vec * rank / ranks), v1 = (int)((long long)n_vec * (rank + 1) / ranks);
  auto load = [&](int v) {
    Vec x;
    x.mask();
    if (v < v1) {
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
  float m = -FLT_MAX, mine = -INFINITY;
  F2 S = F2::of(0.f, 0.f), D = S;
  for (int v = v0 + tid; v - lane < v1; v += LP_THREADS * LP_UNROLL) {
    Vec x[LP_UNROLL];
#pragma unroll
    for (int u = 0; u < LP_UNROLL; u++) x[u] = load(v + u * LP_THREADS);
    float bm = x[0].largest();
#pragma unroll
    for (int u = 1; u < LP_UNROLL; u++) bm = fmaxf(bm, x[u].largest());
    mine = fmaxf(mine, bm);
    if (__any_sync(0xffffffffu, bm > m)) {
      const float now = fmaxf(m, warp_max(bm)), d = fmaxf((m - now) * k, LP_LOWEST), f = ex2(d);
      const F2 f2 = F2::of(f, f);
      D = f2 * fma2(F2::of(d, d), S, D);
      S = f2 * S;
      m = now;
    }
    const F2 m2 = F2::of(-m, -m), k2 = F2::of(k, k);
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

  // the warp's largest thread maximum and its r-th
  const int n_top = p.n_top, nr = (n_top + 7) / 8, nq = nr ? (n_top + nr - 1) / nr : 0;
  {
    float left = mine;
    for (int i = 0; i < max(nr, 1); i++) {
      const float w = warp_max(left);
      const int from = __ffs(__ballot_sync(0xffffffffu, left == w)) - 1;
      if (lane == 0) {
        if (i == 0) w_max[warp] = w, w_owner[warp] = from;
        w_floor[warp] = w;
      }
      if (lane == from) left = -INFINITY;
    }
  }
  __syncthreads();
  float M = lane < LP_WARPS ? w_max[lane] : -INFINITY;
  const float all = warp_max(M);
  const int owner_warp = __ffs(__ballot_sync(0xffffffffu, M == all)) - 1;
  M = all;
  const bool owner = warp == owner_warp && lane == w_owner[warp];
  float floor = INFINITY;
  if (n_top) {
    float left = lane < LP_WARPS ? w_floor[lane] : -INFINITY;
    for (int i = 0; i < nq; i++) {
      floor = warp_max(left);
      const int from = __ffs(__ballot_sync(0xffffffffu, left == floor)) - 1;
      if (lane == from) left = -INFINITY;
    }
  }
  // the sums relative to M, without the owner's
  float s = 0.f, t = 0.f;
  if (!owner || !(mine > -INFINITY)) {
    const float d = fmaxf((m - fmaxf(M, -FLT_MAX)) * k, LP_LOWEST), f = ex2(d);
    s = f * (S.x() + S.y());
    t = f * (D.x() + D.y()) + d * s;
  }
  // some threads' logits again
  unsigned again = __ballot_sync(0xffffffffu, (owner || mine >= floor) && mine > -INFINITY);
  while (again) {
    const int from = __ffs(again) - 1;
    again &= again - 1;
    const bool sums = warp == owner_warp && from == w_owner[warp];
    int equal = 0;
    for (int v = v0 + warp * 32 + from + lane * LP_THREADS; v < v1; v += 32 * LP_THREADS) {
      const Vec x = load(v);
#pragma unroll
      for (int i = 0; i < N; i++) {
        const float2 two = x.pair(i / 2);
        const float l = i & 1 ? two.y : two.x;
        if (l >= floor && l > -INFINITY) {
          const int at = atomicAdd(&n_cand, 1);
          if (at < LP_CAND) cand[at] = candidate(l, v * N - shift + i);
        }
        if (sums) {
          if (l == M) equal++;
          else {
            const float d = at_least((l - M) * k, LP_LOWEST), e = ex2(d);
            s += e;
            t = fmaf(e, d, t);
          }
        }
      }
    }
    if (sums) {  // all but one of those that equal it
      equal = __reduce_add_sync(0xffffffffu, equal) - 1;
      if (lane == 0) s += (float)equal;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  if (lane == 0) {
    w_s[warp] = s;
    w_t[warp] = t;
  }
  __syncthreads();
  // the CTA's list, largest first
  int have = min(n_cand, n_top);
  if (n_cand <= LP_CAND) {
    for (int i = tid; i < n_cand; i += LP_THREADS) {
      const unsigned long long c = cand[i];
      int before = 0;
      for (int j = 0; j < n_cand; j++) before += cand[j] > c;
      if (before < n_top) lists[0][before] = c;
    }
  } else {
    unsigned long long last = ~0ull;
    have = 0;
    for (int i = 0; i < n_top; i++) {
      unsigned long long best = 0;
      for (int v = v0 + tid; v < v1; v += LP_THREADS) {
        const Vec x = load(v);
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
      for (int j = 0; j < LP_WARPS; j++) best = max(best, w_best[j]);
      if (!best) break;
      if (tid == 0) lists[0][i] = best;
      last = best;
      have = i + 1;
    }
  }
  LpPart part;
  if (warp == 0) {
    s = lane < LP_WARPS ? w_s[lane] : 0.f;
    t = lane < LP_WARPS ? w_t[lane] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    part = LpPart{M, s, t, have};
  }
  __syncthreads();
  if (ranks > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (rank > 0) {
      uint32_t to;
      if (tid < have) {
        asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_u32(&lists[rank][tid])));
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(lists[0][tid]) : "memory");
      }
      if (tid == 0) {
        asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_u32(&parts[rank])));
        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(__float_as_uint(part.M)),
                     "r"(__float_as_uint(part.s)), "r"(__float_as_uint(part.t)), "r"(part.n)
                     : "memory");
      }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank > 0) return;
  }
  if (tid == 0) parts[0] = part;
  __syncthreads();
  // the row's M, s and t, in the CTAs' order, by every thread
  float top = parts[0].M;
  for (int i = 1; i < ranks; i++) top = fmaxf(top, parts[i].M);
  float rs = 0.f, rt = 0.f;
  bool left_out = false;  // the one that is left out of s
  for (int i = 0; i < ranks; i++) {
    const LpPart q = parts[i];
    if (!(q.M > -INFINITY)) {
      rs += q.s, rt += q.t;  // 0, or NaN
      continue;
    }
    if (q.M == top && !left_out) {
      left_out = true;
      rs += q.s;
      rt += q.t;
    } else {
      const float d = at_least((q.M - top) * k, LP_LOWEST), f = ex2(d);
      rs += f * (1.0f + q.s);
      rt += f * (q.t + d * (1.0f + q.s));
    }
  }
  if (top == INFINITY) rs = NAN;
  const bool none = !(top > -INFINITY) && rs == rs;  // every logit is -inf
  const float log_s = log1pf(rs);
  auto logp = [&](float l) { return none ? -INFINITY : (l - top) * p.scale - log_s; };
  if (tid == 0) {
    if (QMV_CHECK(in_range(r, 1, p.rows_len, p.err))) {
      if (p.lse) p.lse[r] = none ? -INFINITY : fmaf(top, p.scale, log_s);
      if (p.entropy) p.entropy[r] = none ? 0.f : log_s - 0.6931471805599453f * rt / (1.0f + rs);
    }
  }
  if (tid < p.n_given && QMV_CHECK(in_range(r * p.n_given + tid, 1, p.given_len, p.err)))
    p.logp[r * p.n_given + tid] = token < 0 ? 0.f : token >= p.V ? NAN : logp(given);
  if (n_top) {
    // entry i of list j: as many before it as in its own list and, by a search, in the others
    for (int e = tid; e < ranks * n_top; e += LP_THREADS) {
      const int j = e / n_top, i = e - j * n_top;
      if (i >= parts[j].n) continue;
      const unsigned long long c = lists[j][i];
      int before = i;
      for (int o = 0; o < ranks; o++) {
        if (o == j) continue;
        int lo = 0, hi = parts[o].n;
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (lists[o][mid] > c) lo = mid + 1;
          else hi = mid;
        }
        before += lo;
      }
      if (before < n_top && QMV_CHECK(in_range(r * n_top + before, 1, p.top_len, p.err))) {
        p.top_ids[r * n_top + before] = index_of(c);
        p.top_logp[r * n_top + before] = logp(value_of(c));
      }
    }
    int total = 0;
    for (int i = 0; i < ranks; i++) total += parts[i].n;
    for (int e = total + tid; e < n_top; e += LP_THREADS)
      if (QMV_CHECK(in_range(r * n_top + e, 1, p.top_len, p.err))) {
        p.top_ids[r * n_top + e] = -1;
        p.top_logp[r * n_top + e] = -INFINITY;
      }
  }
}

template <int DT>
static cudaError_t launch_dt(const LogprobsParams& p, cudaStream_t stream) {
  // Few rows: a cluster each, while all of them still fit the GPU twice over and a
  // CTA keeps a round of loads of its own.
  const int round = LP_THREADS * LP_UNROLL * LogitVec<DT>::N / 2;
  int ranks = 1;
  while (ranks < LP_MAX_CLUSTER && p.rows * ranks <= device_sm_count() && p.V > (long long)ranks * round) ranks *= 2;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  make_config(cfg, attr, dim3((unsigned)(p.rows * ranks)), dim3(LP_THREADS), 0, stream, true);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<DT>, p, ranks);
}

cudaError_t launch_logprobs(int dtype, const LogprobsParams& p, cudaStream_t stream) {
  switch (dtype) {
    case QMV_DT_F16: return launch_dt<QMV_DT_F16>(p, stream);
    case QMV_DT_BF16: return launch_dt<QMV_DT_BF16>(p, stream);
    default: return launch_dt<QMV_DT_F32>(p, stream);
  }
}

}  // namespace qmv
