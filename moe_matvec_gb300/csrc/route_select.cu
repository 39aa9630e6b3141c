// Experts of each token from its router logits: scores, balance bias, groups,
// top-k and gates.
#include <cfloat>
#include <cmath>

#include "float_io.cuh"
#include "launch.h"
#include "step_launch.h"

namespace qmv {

constexpr int ROUTE_WARPS = 4;  // tokens of a CTA

__device__ __forceinline__ float rcp(float x) {  // 1 ulp
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float ex2(float x) {  // 2 ulp
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float LOG2E = 1.4426950408889634f;

// Where a lane's experts lie: each group of gs experts is given to 2^log lanes,
// `per` consecutive experts to each, so that lane order is expert order.
struct RoutePlace {
  int log, per;
};

// A number's place in the order of real numbers, above 0 (-0 is not for it).
__device__ __forceinline__ uint32_t order_of(float v) {
  const int b = __float_as_int(v);
  return (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ ((uint32_t)~((int)o >> 31) | 0x80000000u));
}

// A logit or bias as it is taken: NaN as -inf, at most FLT_MAX, -0 as 0.
__device__ __forceinline__ float tame(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX) + 0.0f; }

__device__ __forceinline__ void put(const RouteParams& p, int t, int k, int expert, double gate) {
  const long long at = (long long)t * p.top_k + k;
  if (QMV_CHECK(in_range(at, 1, p.ids_len, p.err))) {
    p.ids[at] = expert;
    p.gates[at] = (float)gate;
  }
}
__device__ __forceinline__ void put(const RouteParams& p, int t, int k, int expert, float gate) {
  const long long at = (long long)t * p.top_k + k;
  if (QMV_CHECK(in_range(at, 1, p.ids_len, p.err))) {
    p.ids[at] = expert;
    p.gates[at] = gate;
  }
}

// The whole selection of token t in 64 bits, by one warp, where more experts are in
// doubt than it has lanes: the same steps as in the kernel below.  Rare, so the
// logits are read again and nothing is tuned.
template <int PER, class T>
__device__ __noinline__ void select_exactly(const RouteParams& p, RoutePlace pl, int t) {
  const T* row = static_cast<const T*>(p.logits) + (long long)t * p.ld;
  const int lane = threadIdx.x & 31;
  const int lpg = 1 << pl.log, gs = p.size, g = lane >> pl.log;
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
      if (p.bias) c[i] += (double)tame(p.bias[e0 + i]);
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
  double mine = 0, sum = 0;  // lane k: pick k's score
  int pick = 0;
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
    if (lane == k) pick = at, mine = score;
    sum += score;
  }
  if (lane < p.top_k) put(p, t, lane, pick, (p.renorm ? (sum > 0 ? mine / sum : 0.0) : mine) * (double)p.scale);
}

// Exact values of token t's experts, where some are in doubt.  Scores of a softmax
// without a bias are compared without their common divisor.
template <class T>
struct Exact {
  const RouteParams& p;
  const T* row;
  double top, total = 1;
  __device__ __forceinline__ Exact(const RouteParams& p, int t, float top)
      : p(p), row(static_cast<const T*>(p.logits) + (long long)t * p.ld), top(top) {
    if (p.gating != QMV_GATING_SOFTMAX || !p.bias) return;
    total = 0;
    for (int e = threadIdx.x & 31; e < p.E; e += 32) {
      const float l = tame(to_float(row[e]));
      total += l > -INFINITY ? exp((double)l - this->top) : 0.0;
    }
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  __device__ __forceinline__ double score(float l) const {
    if (!(l > -INFINITY)) return 0.0;
    return p.gating == QMV_GATING_SOFTMAX ? exp((double)l - top) / total : 1.0 / (1.0 + exp(-(double)l));
  }
  __device__ __forceinline__ double choice(int e, double s) const { return p.bias ? s + (double)tame(p.bias[e]) : s; }
};

// Groups about the border: whether the lane's group, if it is `open`, is among the
// `want` largest of the open ones.
template <class T>
__device__ __noinline__ bool settle_groups(const RouteParams& p, int log, int t, float top, bool open, int want) {
  const int lane = threadIdx.x & 31, g = lane >> log;
  const unsigned opened = __ballot_sync(0xffffffffu, open && (lane & ((1 << log) - 1)) == 0);
  const Exact<T> exact(p, t, top);
  double value = 0;  // of the lane's group
  for (unsigned todo = opened; todo; todo &= todo - 1) {
    const int group = (__ffs(todo) - 1) >> log;
    double a = -INFINITY, b = -INFINITY;
    for (int i = lane; i < p.size; i += 32) {
      const int e = group * p.size + i;
      const double v = exact.choice(e, exact.score(tame(to_float(exact.row[e]))));
      if (v > a) b = a, a = v;
      else if (v > b) b = v;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const double x = __shfl_xor_sync(0xffffffffu, a, o), y = __shfl_xor_sync(0xffffffffu, b, o);
      b = fmax(fmin(a, x), a >= x ? b : y);
      a = fmax(a, x);
    }
    if (g == group) value = p.group_top == 2 ? a + b : a;
  }
  int ahead = 0;
  for (unsigned todo = opened; todo; todo &= todo - 1) {
    const int of = __ffs(todo) - 1;
    const double other = __shfl_sync(0xffffffffu, value, of);
    ahead += other > value || (other == value && (of >> log) < g);
  }
  return ahead < want;
}

// The token's picks and gates from n candidates, expert e of each of the first n lanes.
template <class T>
__device__ __noinline__ void settle_picks(const RouteParams& p, int t, float top, float inv, int n, int e) {
  const int lane = threadIdx.x & 31;
  const Exact<T> exact(p, t, top);
  double v = -INFINITY, score = 0;
  if (lane < n) {
    const float l = tame(to_float(exact.row[e]));
    score = exact.score(l);
    v = p.bias ? exact.choice(e, score) : (double)l;
    if (!p.bias) score *= (double)inv;
  }
  int before = 0;
  for (int j = 0; j < n; j++) {
    const double other = __shfl_sync(0xffffffffu, v, j);
    const int i = __shfl_sync(0xffffffffu, e, j);
    before += other > v || (other == v && i < e);
  }
  const bool in = lane < n && before < p.top_k;
  double sum = in ? score : 0.0;
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (in) put(p, t, before, e, (p.renorm ? (sum > 0 ? score / sum : 0.0) : score) * (double)p.scale);
}

// Largest first, by a bitonic network.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {
#pragma unroll
  for (int k = 2; k <= N; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2)
#pragma unroll
      for (int i = 0; i < N; i++)
        if ((i ^ j) > i) {
          const uint32_t lo = min(v[i], v[i ^ j]), hi = max(v[i], v[i ^ j]);
          v[i] = i & k ? lo : hi;
          v[i ^ j] = i & k ? hi : lo;
        }
}

// A warp a token, by turns: s = softmax(l) or sigmoid(l), c = s + bias; a group's
// score is the sum of its one or two largest c; of the kept groups' experts the
// top_k largest c are picked, larger first, ties to the lower index; gates are their
// s, over their sum if renorm, times scale.
//
// Each lane has consecutive experts (lane order is expert order) and sorts their
// keys: the places of c, or without a bias of the logits, in the order of real
// numbers, whose lowest bits (8 for 8 experts a lane) give way to the expert's lane
// and slot, the first ones largest.  A pick is then the largest of the lanes' first
// keys and a shift of the keys of the lane that has it; lane k keeps pick k.
//
// What is compared carries errors: those of fp32 (a score's exponent is rounded twice,
// s |l| 2^-24 at most 2^-25 s + 2^-24, and the rest is within 2^-20 of two scores with
// up to 8 experts a lane, and c's own rounding; a logit is exact) and the bits given
// way (0 in logits of 16).  Where two compared values at a border (kept and next group; consecutive picks and the first left out)
// lie closer than that, what is in doubt is decided in 64 bits: the groups about the
// border by their exact scores, the picks by the exact values of the picks and of
// all experts that are as close after them, one a lane.  So the picks are those of 64
// bits everywhere, at the cost of 64-bit arithmetic for a few tokens in a hundred.
//
// Bound by a token's dependent steps (eight picks one after another, each a maximum over
// the warp) and about 700 instructions, the ALU pipe half full: 16384 tokens of 256
// experts in 8 groups with a bias 19 us, without groups 16, softmax without both 14; one
// token 2.6 us.  More or fewer CTAs an SM (8, 5), the next token's logits on their way and
// cheaper scores changed that by less than a tenth.
template <int PER, int DT, bool VEC, bool FULL>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, PER <= 8 ? 6 : PER <= 16 ? 4 : 2) route_select_kernel(const __grid_constant__ RouteParams p, const RoutePlace pl) {
  using T = typename Elem<DT>::type;
  constexpr uint32_t PLACE = 32 * PER - 1;  // the bits of a lane and slot
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lpg = 1 << pl.log, gs = p.size, g = lane >> pl.log;
  const int per = FULL ? PER : pl.per, first = (lane & (lpg - 1)) * per;
  const int have = FULL ? PER : g < p.groups ? max(0, min(per, gs - first)) : 0;
  const int e0 = FULL ? lane * PER : g * gs + first;
  const bool soft = p.gating == QMV_GATING_SOFTMAX, biased = p.bias != nullptr;
  float bias[PER], widest = 0.f;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    bias[i] = 0.f;
    if (biased && i < have) {
      bias[i] = tame(p.bias[e0 + i]);
      if (fabsf(bias[i]) < INFINITY) widest = fmaxf(widest, fabsf(bias[i]));
    }
  }
  widest = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(widest)));
  // How far c of up to two scores whose values add up to `of` may be off: s (at most 1,
  // and at most |c| + |bias|) by the roundings of the softmax's sum, exp2, quotient and
  // exponent, c by its own.  Infinite ones (of a bias) are not off.
  constexpr float REL = PER <= 8 ? 0x1p-20f : PER <= 16 ? 0x1p-19f : 0x1p-18f;
  auto off = [&](float of) { return fminf(REL * fminf(of + 2.0f * widest, 2.0f) + 0x1p-22f * of + 0x1p-22f, FLT_MAX); };
  auto expert = [&](int f) {  // of lane f / PER, slot f % PER
    const int of = f / PER;
    return FULL ? f : (of >> pl.log) * gs + (of & (lpg - 1)) * per + f % PER;
  };
  auto placed = [&](float v, int i) { return i < have ? (order_of(v) & ~PLACE) | (PLACE - lane * PER - i) : 0u; };
  for (int t = blockIdx.x * ROUTE_WARPS + warp; t < p.n_tok; t += gridDim.x * ROUTE_WARPS) {
    const T* row = static_cast<const T*>(p.logits) + (long long)t * p.ld;
    float s[PER];
    if constexpr (VEC) {  // lanes have whole fours
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        Packed<T, 4> x;
        float l[4];
        const bool in = i < have && QMV_CHECK(in_range((long long)t * p.ld + e0 + i, 4, p.logits_len, p.err));
        x.clear();
        if (in) x.load(row + e0 + i);
        x.to(l);
#pragma unroll
        for (int j = 0; j < 4; j++) s[i + j] = in ? l[j] : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; i++)
        s[i] = i < have && QMV_CHECK(in_range((long long)t * p.ld + e0 + i, 1, p.logits_len, p.err)) ? to_float(row[e0 + i]) : -INFINITY;
    }
    float top = -INFINITY;
    uint32_t key[PER];  // 0: none
#pragma unroll
    for (int i = 0; i < PER; i++) {
      s[i] = tame(s[i]);
      if (!biased) key[i] = placed(s[i], i);
    }
    float inv = 1.f;  // scores are inv * s
    if (soft) {
#pragma unroll
      for (int i = 0; i < PER; i++) top = fmaxf(top, s[i]);
      top = value_of(__reduce_max_sync(0xffffffffu, order_of(top)));
      float total = 0.f;
#pragma unroll
      for (int i = 0; i < PER; i++) {
        s[i] = s[i] > -INFINITY ? ex2((s[i] - top) * LOG2E) : 0.f;
        total += s[i];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      inv = total > 0.f ? 1.0f / total : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < PER; i++) s[i] = rcp(1.0f + ex2(-LOG2E * s[i]));  // (-inf: 1 / inf = 0)
    }
    float c[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) {
      c[i] = fmaf(s[i], inv, bias[i]);
      if (biased) key[i] = placed(c[i], i);
    }

    if (p.keep < p.groups) {
      float one = -INFINITY, two = -INFINITY;
#pragma unroll
      for (int i = 0; i < PER; i++)
        if (i < have) {
          two = fmaxf(two, fminf(one, c[i]));
          one = fmaxf(one, c[i]);
        }
      for (int o = 1; o < lpg; o <<= 1) {
        const float a = __shfl_xor_sync(0xffffffffu, one, o), b = __shfl_xor_sync(0xffffffffu, two, o);
        two = fmaxf(fminf(one, a), one >= a ? two : b);
        one = fmaxf(one, a);
      }
      const float score = p.group_top == 2 ? one + two : one;
      const uint32_t mine = order_of(score + 0.0f);
      int before = 0;
#pragma unroll 8
      for (int j = 0; j < p.groups; j++) {
        const uint32_t other = __shfl_sync(0xffffffffu, mine, j << pl.log);
        before += other > mine || (other == mine && j < g);
      }
      bool in = g < p.groups && before < p.keep;
      const float err = off(fabsf(one) + (p.group_top == 2 ? fabsf(two) : 0.f));
      const uint32_t lo = order_of(score - err + 0.0f), hi = order_of(score + err + 0.0f);
      // the least that a group that is in may have, and the most of one that is not
      const uint32_t last = __reduce_min_sync(0xffffffffu, in ? lo : 0xffffffffu);
      const uint32_t next = __reduce_max_sync(0xffffffffu, in || g >= p.groups ? 0u : hi);
      if (next >= last) {
        const bool open = g < p.groups && (in ? lo <= next : hi >= last);
        // what is left to be kept of these groups
        const int sure = __popc(__ballot_sync(0xffffffffu, in && !open && (lane & (lpg - 1)) == 0));
        const bool among = settle_groups<T>(p, pl.log, t, top, open, p.keep - sure);
        if (open) in = among;
      }
      if (!in) {
#pragma unroll
        for (int i = 0; i < PER; i++) key[i] = 0;
      }
    }
    sort_down(key);

    uint32_t picked = 0;  // lane k: pick k's key
    auto pick = [&](int k) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
      if (lane == k) picked = best;
      if (key[0] == best) {
#pragma unroll
        for (int i = 0; i < PER; i++) key[i] = i + 1 < PER ? key[i + 1] : 0;
      }
    };
#pragma unroll
    for (int k = 0; k < QMV_MAX_TOPK; k++)
      if (k < p.top_k) pick(k);
    // consecutive picks, and the last one and what comes after it
    const uint32_t after = __reduce_max_sync(0xffffffffu, key[0]);
    auto near = [&](uint32_t a, uint32_t b) {  // b is not above a
      a &= ~PLACE, b &= ~PLACE;
      if (!biased) return DT == QMV_DT_F32 && a == b;  // (logits of 16 bits are whole in their keys)
      const float x = value_of(a), y = value_of(b);
      return x - y <= off(fabsf(x) + fabsf(y)) + (float)(32 * PER) * 0x1p-23f * fmaxf(fabsf(x), fabsf(y));
    };
    uint32_t follower = __shfl_down_sync(0xffffffffu, picked, 1);
    if (lane == p.top_k - 1) follower = after;
    const bool doubt = __any_sync(0xffffffffu, lane < p.top_k && follower && near(picked, follower));
    int from = PLACE - (picked & PLACE);  // lane k: pick k's lane and slot
    // The picks' scores, as they enter the gates: lane k's (rather than those above, whose
    // exponents are rounded once too often for small scores).
    float held = 0.f;
    if (lane < p.top_k) {
      const float l = tame(to_float(row[expert(from)]));
      held = l > -INFINITY ? (soft ? expf(l - top) : __frcp_rn(1.0f + expf(-l))) : 0.f;
    }
    float of_all = held;
#pragma unroll
    for (int o = QMV_MAX_TOPK / 2; o > 0; o >>= 1) of_all += __shfl_xor_sync(0xffffffffu, of_all, o);
    of_all = __shfl_sync(0xffffffffu, of_all, 0);
    // (scores down to 2^-126 are whole: smaller sums are formed anew)
    if (!doubt && (!p.renorm || of_all >= 0x1p-60f)) {
      if (lane < p.top_k) put(p, t, lane, expert(from), (p.renorm ? held / of_all : held * inv) * p.scale);
      continue;
    }
    int n = p.top_k;
    while (n < 32) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
      if (!best || !near(__shfl_sync(0xffffffffu, picked, n - 1), best)) break;
      pick(n++);
    }
    from = PLACE - (picked & PLACE);
    if (n == 32) {  // more than a warp can hold
      select_exactly<PER, T>(p, pl, t);
      continue;
    }
    settle_picks<T>(p, t, top, inv, n, expert(from));
  }
}

template <int DT, bool VEC>
static cudaError_t launch_as(const RouteParams& p, RoutePlace pl, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  // as many CTAs as the SMs hold at once (80 registers a thread with up to 8 experts a lane,
  // of which 64 to 68 bytes spill, 128 with 16, where 80 to 84 do, 246 with 32); warps take
  // tokens by turns
  const int ctas = (p.n_tok + ROUTE_WARPS - 1) / ROUTE_WARPS;
  const int cap = (pl.per <= 8 ? 6 : pl.per <= 16 ? 4 : 2) * device_sm_count();
  make_config(cfg, attr, dim3((unsigned)(ctas < cap ? ctas : cap)), dim3(32 * ROUTE_WARPS), 0, stream, true);
  if constexpr (VEC) {
    // every lane full (128, 256, 512 experts in 1, 2, 4 .. groups): nothing to ask for
    if (p.groups << pl.log == 32 && p.size == pl.per << pl.log) {
      if (pl.per == 4) return cudaLaunchKernelEx(&cfg, route_select_kernel<4, DT, true, true>, p, pl);
      if (pl.per == 8) return cudaLaunchKernelEx(&cfg, route_select_kernel<8, DT, true, true>, p, pl);
      if (pl.per == 16) return cudaLaunchKernelEx(&cfg, route_select_kernel<16, DT, true, true>, p, pl);
    }
  }
  if (pl.per <= 4) return cudaLaunchKernelEx(&cfg, route_select_kernel<4, DT, VEC, false>, p, pl);
  if (pl.per <= 8) return cudaLaunchKernelEx(&cfg, route_select_kernel<8, DT, VEC, false>, p, pl);
  if (pl.per <= 16) return cudaLaunchKernelEx(&cfg, route_select_kernel<16, DT, VEC, false>, p, pl);
  return cudaLaunchKernelEx(&cfg, route_select_kernel<32, DT, VEC, false>, p, pl);
}

template <int DT>
static cudaError_t launch_dt(RouteParams p, cudaStream_t stream) {
  p.size = p.E / p.groups;
  RoutePlace pl{0, 0};
  while ((2 << pl.log) * p.groups <= 32) pl.log++;
  pl.per = (p.size + (1 << pl.log) - 1) >> pl.log;
  // four experts a load where no lane's run of them is cut and all are aligned
  const bool vec = pl.per % 4 == 0 && p.size % 4 == 0 && p.ld % 4 == 0;
  return vec ? launch_as<DT, true>(p, pl, stream) : launch_as<DT, false>(p, pl, stream);
}

cudaError_t launch_route_select(int dtype, const RouteParams& p, cudaStream_t stream) {
  switch (dtype) {
    case QMV_DT_F16: return launch_dt<QMV_DT_F16>(p, stream);
    case QMV_DT_BF16: return launch_dt<QMV_DT_BF16>(p, stream);
    default: return launch_dt<QMV_DT_F32>(p, stream);
  }
}

}  // namespace qmv
