// Experts of each token from its router logits: scores, balance bias, groups,
// top-k and gates.
#include <cfloat>
#include <cmath>

#include "float_io.cuh"
#include "launch.h"
#include "step_launch.h"

namespace qmv {

constexpr int ROUTE_WARPS = 4;  // tokens of a CTA

// Where a lane's experts lie: each group of gs experts is given to 2^log lanes,
// `per` consecutive experts to each, so that lane order is expert order.
struct RoutePlace {
  int log, per;
};

// A value's place in the order of real numbers, above 0; NaN as -inf.
__device__ __forceinline__ uint32_t order_of(float v) {
  v = v == v ? v + 0.0f : -INFINITY;  // (-0 + 0 = 0: equal numbers are equal)
  const uint32_t b = __float_as_uint(v);
  return (int)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((int)o < 0 ? o & 0x7fffffffu : ~o);
}

// A logit as the scores take it: NaN as -inf, at most FLT_MAX.
__device__ __forceinline__ float tame(float l) { return l == l ? fminf(l, FLT_MAX) : -INFINITY; }

// The whole selection of a token in 64 bits, by one warp, for tokens whose
// 32-bit scores come too close to a decision: the same steps as in the kernel
// below, whose result it replaces.  Called for about one token in 300, so the
// logits are read again and nothing is tuned.
template <int PER, class T>
__device__ __noinline__ void select_exactly(const RouteParams& p, RoutePlace pl, const T* row, int (&pick)[QMV_MAX_TOPK],
                                            float (&gate)[QMV_MAX_TOPK]) {
  const int lane = threadIdx.x & 31;
  const int lpg = 1 << pl.log, gs = p.E / p.groups, g = lane >> pl.log;
  const int first = (lane & (lpg - 1)) * pl.per;
  const int have = g < p.groups ? max(0, min(pl.per, gs - first)) : 0;
  const int e0 = g * gs + first;
  double top = -INFINITY, total = 0;
  for (int i = 0; i < have; i++) top = fmax(top, (double)tame(to_float(row[e0 + i])));
  for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool soft = p.gating == QMV_GATING_SOFTMAX;
  auto raw = [&](int i) -> double {  // the score, not yet over the softmax's sum
    const double l = tame(to_float(row[e0 + i]));
    if (l == -INFINITY) return 0.0;
    return soft ? exp(l - top) : 1.0 / (1.0 + exp(-l));
  };
  if (soft) {
    for (int i = 0; i < have; i++) total += raw(i);
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  double s[PER], c[PER];
  double one = -INFINITY, two = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    s[i] = 0, c[i] = -INFINITY;
    if (i < have) {
      s[i] = raw(i);
      if (soft) s[i] = total > 0 ? s[i] / total : 0.0;
      c[i] = s[i];
      if (p.bias) c[i] += (double)p.bias[e0 + i];
      if (!(c[i] == c[i])) c[i] = -INFINITY;
      if (c[i] > one) two = one, one = c[i];
      else if (c[i] > two) two = c[i];
      // without a bias larger logits are larger scores, whatever 64 bits leave of them
      if (!p.bias) c[i] = tame(to_float(row[e0 + i]));
    }
  }
  if (p.keep < p.groups) {
    for (int o = 1; o < lpg; o <<= 1) {
      const double a = __shfl_xor_sync(0xffffffffu, one, o), b = __shfl_xor_sync(0xffffffffu, two, o);
      two = fmax(fmin(one, a), one >= a ? two : b);
      one = fmax(one, a);
    }
    const double mine = p.group_top == 2 ? one + two : one;
    int before = 0;
    for (int j = 0; j < p.groups; j++) {
      const double other = __shfl_sync(0xffffffffu, mine, j << pl.log);
      before += other > mine || (other == mine && j < g);
    }
    if (before >= p.keep) {
#pragma unroll
      for (int i = 0; i < PER; i++) s[i] = -1;  // left out
    }
  }
  double picked[QMV_MAX_TOPK], sum = 0;
  for (int k = 0; k < p.top_k; k++) {
    double best = -INFINITY, score = 0;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (i < have && s[i] >= 0 && (at == 0x7fffffff || c[i] > best)) best = c[i], score = s[i], at = e0 + i;
    for (int o = 16; o > 0; o >>= 1) {
      const double b = __shfl_xor_sync(0xffffffffu, best, o), sc = __shfl_xor_sync(0xffffffffu, score, o);
      const int a = __shfl_xor_sync(0xffffffffu, at, o);
      if (a != 0x7fffffff && (at == 0x7fffffff || b > best || (b == best && a < at))) best = b, score = sc, at = a;
    }
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (i < have && e0 + i == at) s[i] = -1;
    pick[k] = at;
    picked[k] = score;
    sum += score;
  }
  for (int k = 0; k < p.top_k; k++)
    gate[k] = (float)((p.renorm ? (sum > 0 ? picked[k] / sum : 0.0) : picked[k]) * (double)p.scale);
}

// One warp a token: s = softmax(l) or sigmoid(l), c = s + bias; a group's score
// is the sum of its one or two largest c; of the kept groups' experts the top_k
// largest c are picked, larger first, ties to the lower index; gates are their s,
// over their sum if renorm, times scale.
//
// Without a bias an expert's c orders as its logit does, and the logits are
// compared.  With one, and for sums of two, what is compared carries the errors of
// fp32: score and sum are within about 2^-21 of s + |bias|.  Where two compared
// values at a border (kept and next group; consecutive picks and the first left
// out) lie closer than 2^-20 of their size plus 2^-24, the token is decided again
// in 64 bits, so the picks are those of 64 bits everywhere.
//
// Bound by the picks: 2 steps across the warp and one over a lane's experts each.
template <int PER, int DT>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_select_kernel(const RouteParams p, const RoutePlace pl) {
  using T = typename Elem<DT>::type;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * ROUTE_WARPS + (threadIdx.x >> 5);
  if (t >= p.n_tok) return;
  const T* row = static_cast<const T*>(p.logits) + (long long)t * p.ld;
  const int lpg = 1 << pl.log, gs = p.E / p.groups, g = lane >> pl.log;
  const int first = (lane & (lpg - 1)) * pl.per;
  const int have = g < p.groups ? max(0, min(pl.per, gs - first)) : 0;
  const int e0 = g * gs + first;
  float s[PER];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    s[i] = i < have && QMV_CHECK(in_range((long long)t * p.ld + e0 + i, 1, p.logits_len, p.err))
               ? tame(to_float(row[e0 + i]))
               : -INFINITY;
    top = fmaxf(top, s[i]);
  }
  uint32_t key[PER];  // the place of what picks compare; 0: none
#pragma unroll
  for (int i = 0; i < PER; i++) key[i] = !p.bias && i < have ? order_of(s[i]) : 0;
  float inv = 1.f;  // scores are inv * s
  if (p.gating == QMV_GATING_SOFTMAX) {
    top = value_of(__reduce_max_sync(0xffffffffu, order_of(top)));
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      s[i] = s[i] > -INFINITY ? expf(s[i] - top) : 0.f;
      total += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    inv = total > 0.f ? 1.0f / total : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < PER; i++) s[i] = s[i] > -INFINITY ? __frcp_rn(1.0f + expf(-s[i])) : 0.f;
  }
  float one = -INFINITY, two = -INFINITY, widest = 0.f;
#pragma unroll
  for (int i = 0; i < PER; i++)
    if (i < have) {
      float c = s[i] * inv;
      if (p.bias) {
        const float b = p.bias[e0 + i];
        c += b;
        key[i] = order_of(c);
        c = value_of(key[i]);
        if (fabsf(b) < INFINITY) widest = fmaxf(widest, fabsf(b));
      }
      two = fmaxf(two, fminf(one, c));
      one = fmaxf(one, c);
    }
  widest = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(widest)));
  // two values that this close may stand the other way round
  auto close = [&](float a, float b) {
    return a == b || fabsf(a - b) <= 0x1p-20f * (fabsf(a) + fabsf(b) + 2.0f * widest) + 0x1p-24f;
  };
  bool doubt = false;
  if (p.keep < p.groups) {
    for (int o = 1; o < lpg; o <<= 1) {
      const float a = __shfl_xor_sync(0xffffffffu, one, o), b = __shfl_xor_sync(0xffffffffu, two, o);
      two = fmaxf(fminf(one, a), one >= a ? two : b);
      one = fmaxf(one, a);
    }
    const float mine = p.group_top == 2 ? one + two : one;
    int before = 0;
    bool near = false;
    for (int j = 0; j < p.groups; j++) {
      const float other = __shfl_sync(0xffffffffu, mine, j << pl.log);
      const bool first_of = other > mine || (other == mine && j < g);
      before += first_of;
      near |= j != g && close(mine, other);
    }
    // only a group next to the border between kept and left matters
    doubt = near && g < p.groups && before + 1 >= p.keep && before <= p.keep;
    if (before >= p.keep || g >= p.groups) {
#pragma unroll
      for (int i = 0; i < PER; i++) key[i] = 0;
    }
  }
  doubt = __any_sync(0xffffffffu, doubt);

  int pick[QMV_MAX_TOPK];
  float gate[QMV_MAX_TOPK];
  float sum = 0.f, last = 0.f;
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < PER; i++) mine = max(mine, key[i]);
#pragma unroll
  for (int k = 0; k <= QMV_MAX_TOPK; k++) {
    if (k > p.top_k) break;
    const uint32_t best = __reduce_max_sync(0xffffffffu, mine);
    if (p.bias && best) {
      const float now = value_of(best);
      if (k > 0) doubt |= close(last, now);
      last = now;
    }
    if (k >= p.top_k || k >= QMV_MAX_TOPK) break;
    const int from = __ffs(__ballot_sync(0xffffffffu, mine == best)) - 1;
    int at = 0;
    float sc = 0.f;
    if (lane == from) {
      bool found = false;
      mine = 0;
#pragma unroll
      for (int i = 0; i < PER; i++) {
        if (!found && key[i] == best) {
          found = true;
          at = e0 + i;
          sc = s[i];
          key[i] = 0;
        }
        mine = max(mine, key[i]);
      }
    }
    pick[k] = __shfl_sync(0xffffffffu, at, from);
    gate[k] = __shfl_sync(0xffffffffu, sc, from);
    sum += gate[k];
  }
  if (doubt) {
    select_exactly<PER, T>(p, pl, row, pick, gate);
  } else {
#pragma unroll
    for (int k = 0; k < QMV_MAX_TOPK; k++)
      if (k < p.top_k) gate[k] = (!p.renorm ? gate[k] * inv : sum > 0.f ? gate[k] / sum : 0.f) * p.scale;
  }
#pragma unroll
  for (int k = 0; k < QMV_MAX_TOPK; k++)
    if (k < p.top_k && lane == k && QMV_CHECK(in_range((long long)t * p.top_k + k, 1, p.ids_len, p.err))) {
      p.ids[(long long)t * p.top_k + k] = pick[k];
      p.gates[(long long)t * p.top_k + k] = gate[k];
    }
}

template <int DT>
static cudaError_t launch_dt(const RouteParams& p, cudaStream_t stream) {
  const int gs = p.E / p.groups;
  RoutePlace pl{0, 0};
  while ((2 << pl.log) * p.groups <= 32) pl.log++;
  pl.per = (gs + (1 << pl.log) - 1) >> pl.log;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3((unsigned)((p.n_tok + ROUTE_WARPS - 1) / ROUTE_WARPS)), dim3(32 * ROUTE_WARPS), 0, stream,
              true);
  if (pl.per <= 4) return cudaLaunchKernelEx(&cfg, route_select_kernel<4, DT>, p, pl);
  if (pl.per <= 8) return cudaLaunchKernelEx(&cfg, route_select_kernel<8, DT>, p, pl);
  if (pl.per <= 16) return cudaLaunchKernelEx(&cfg, route_select_kernel<16, DT>, p, pl);
  return cudaLaunchKernelEx(&cfg, route_select_kernel<32, DT>, p, pl);
}

cudaError_t launch_route_select(int dtype, const RouteParams& p, cudaStream_t stream) {
  switch (dtype) {
    case QMV_DT_F16: return launch_dt<QMV_DT_F16>(p, stream);
    case QMV_DT_BF16: return launch_dt<QMV_DT_BF16>(p, stream);
    default: return launch_dt<QMV_DT_F32>(p, stream);
  }
}

}  // namespace qmv
