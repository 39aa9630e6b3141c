// Norm of each query and key head and the position rotation, in one pass.
#include "float2.cuh"
#include "float_io.cuh"
#include "kv_cache.cuh"
#include "launch.h"
#include "step_launch.h"

namespace qmv {

constexpr int ROPE_WARPS = 4;         // warps of a CTA, each on its own
constexpr int ROPE_MAX_PAIRS = 128;   // of a head of 256 values
constexpr int ROPE_AHEAD = 3;         // head groups of a warp on their way
constexpr int ROPE_CTAS = 4;          // CTAs an SM (5: 20.0 us, 6 with 2 ahead 22.4, for 17.8)

// A frequency (radians a position) in turns a position, as a fraction of 2^64: a
// position times it, modulo 2^64, is the turn's fraction, whatever the position (in
// fp32 a position of 131072 would leave 2^-7 of the angle).  Formed in 64-bit floats,
// once per warp and pair.
__device__ __forceinline__ unsigned long long turns_a_position(float freq) {
  double f = (double)freq * 0.15915494309189535;  // 1 / (2 pi)
  f -= rint(f);                                   // [-1/2, 1/2]
  // (half a turn either way is 2^63; a frequency that is no number turns by 0)
  return (unsigned long long)__double2ll_rn(f * 0x1p63) << 1;
}
// cos and sin of what is left of a turn: at most half a turn, to 2^-25 of it in fp32.
__device__ __forceinline__ float2 turn_of(int pos, unsigned long long freq, float scale) {
  const int left = (int)((unsigned long long)(long long)pos * freq >> 32);
  float s, c;
  sincospif((float)left * 0x1p-31f, &s, &c);
  return make_float2(c * scale, s * scale);
}

// One float or two at once.
template <int W>
struct Wide {
  using type = float;
  __device__ __forceinline__ static float of(const float* x) { return *x; }
  __device__ __forceinline__ static float both(float x) { return x; }
  __device__ __forceinline__ static float fma(float a, float b, float c) { return fmaf(a, b, c); }
  __device__ __forceinline__ static float sum(float a) { return a; }
  __device__ __forceinline__ static void to(float a, float* x) { *x = a; }
};
template <>
struct Wide<2> {
  using type = F2;
  __device__ __forceinline__ static F2 of(const float* x) { return F2::of(x[0], x[1]); }
  __device__ __forceinline__ static F2 both(float x) { return F2::of(x, x); }
  __device__ __forceinline__ static F2 fma(F2 a, F2 b, F2 c) { return fma2(a, b, c); }
  __device__ __forceinline__ static float sum(F2 a) { return a.x() + a.y(); }
  __device__ __forceinline__ static void to(F2 a, float* x) { x[0] = a.x(), x[1] = a.y(); }
};

// The first of x, the second of y.
__device__ __forceinline__ float first(float x, float) { return x; }
__device__ __forceinline__ F2 first(F2 x, F2 y) { return F2::of(x.x(), y.y()); }

// The 2 CH consecutive values (a, b) of a unit whose pairs are neighbours: the
// pairs' first values and their second ones, and back.
template <int CH>
__device__ __forceinline__ void to_pairs(float (&a)[CH], float (&b)[CH]) {
  float x[2 * CH];
#pragma unroll
  for (int j = 0; j < CH; j++) x[j] = a[j], x[CH + j] = b[j];
#pragma unroll
  for (int j = 0; j < CH; j++) a[j] = x[2 * j], b[j] = x[2 * j + 1];
}
template <int CH>
__device__ __forceinline__ void from_pairs(float (&a)[CH], float (&b)[CH]) {
  float x[2 * CH];
#pragma unroll
  for (int j = 0; j < CH; j++) x[2 * j] = a[j], x[2 * j + 1] = b[j];
#pragma unroll
  for (int j = 0; j < CH; j++) a[j] = x[j], b[j] = x[CH + j];
}

// y = x * w / sqrt(mean(x^2) + eps) (w given, else y = x), then each pair (a, b) of
// the first R values becomes (a cos - b sin, b cos + a sin).
//
// A head is D / (2 CH) units of two chunks of CH consecutive values, one unit a
// lane (up to UL units for short chunks): the two halves of CH pairs (pair i: values i and
// i + R / 2), or 2 CH consecutive values (pair i: 2i, 2i + 1), or two chunks
// that do not turn.  So a lane holds whole pairs, the norm is a sum over the
// head's lanes, and the same lane has the same pairs in every head: the products
// of its cosines and sines with the weights stay in registers while the warp goes
// through the token's heads, 32 / (lanes of a head) at a time, the next ones on
// their way.  The warp's lanes share out the token's angles (64 bits, the only
// costly arithmetic) through shared memory; meanwhile the first heads travel.
//
// Bound for many tokens by latency with few warps: 4096 x 40 heads of 128 bfloat16 (84
// MB) 17.7 us, 4.7 TB/s, with 47% of the issue slots taken by 23% of the warps, which wait
// for their own chains, for the turns in shared memory and for loads, in this order.  The
// loads run dry at each token's end: the next one's first heads and angles (with the
// products with the weights a third of the instructions) begin there.  One token of 40
// heads 2.8 us: a load, the angle, the sum and the store in turn.
// ALL: every pair turns (R = D).
template <int DT, int CH, int UL, bool INTER, bool ALL>
__global__ void __launch_bounds__(32 * ROPE_WARPS, UL <= 2 ? ROPE_CTAS : 3)
    norm_rope_kernel(const RopeParams p, int lph_log, unsigned per, unsigned rest) {
  using T = typename Elem<DT>::type;
  using Chunk = Packed<T, CH>;
  constexpr int PF = UL == 1 ? ROPE_AHEAD : UL == 2 ? 2 : 1;  // head groups on their way
  __shared__ float2 turns[ROPE_WARPS][ROPE_MAX_PAIRS];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int hpw = 32 >> lph_log, li = lane & ((1 << lph_log) - 1), sub = lane >> lph_log;
  const int units = p.D / (2 * CH), turning = p.R / (2 * CH);
  const int q_steps = (p.q.n + hpw - 1) >> (5 - lph_log), steps = q_steps + ((p.k.n + hpw - 1) >> (5 - lph_log));
  // `per` groups for this warp, one more for the first `rest` warps
  const unsigned w = blockIdx.x * ROPE_WARPS + wid, g0 = w * per + min(w, rest);
  int todo = (int)(per + (w < rest));
  unsigned t = g0 / (unsigned)steps;
  int s0 = (int)(g0 - t * steps);
  // the lane's pairs of the token's angles
  unsigned long long freq[ROPE_MAX_PAIRS / 32];
  int axis[ROPE_MAX_PAIRS / 32];
#pragma unroll
  for (int i = 0; i < ROPE_MAX_PAIRS / 32; i++) {
    freq[i] = 0;
    axis[i] = 0;
    if (32 * i < p.R / 2) {
      const int pair = lane + 32 * i;
      freq[i] = turns_a_position(pair < p.R / 2 ? p.freq[pair] : 0.f);
      if (p.axis && pair < p.R / 2) axis[i] = p.axis[pair];
      if (axis[i] >= p.n_axes) {
        set_error(p.err, QMV_DEVERR_BATCH);
        axis[i] = 0;
      }
    }
  }
  // the lane's unit i, and the places of its two chunks in a head
  auto unit = [&](int i) { return li + (i << lph_log); };
  int pa[UL], pb[UL];
#pragma unroll
  for (int i = 0; i < UL; i++) {
    const int u = unit(i);
    if (INTER || u >= turning) {
      pa[i] = u * 2 * CH;
      pb[i] = pa[i] + CH;
    } else {
      pa[i] = u * CH;
      pb[i] = p.R / 2 + pa[i];
    }
  }
  // The token's head groups in order, queries first: the lane's head of a group
  // (x) and how many heads there are from the group's first on.
  struct Cursor {
    T* x;
    int left;
  };
  auto group = [&](int s, bool out) {
    const bool keys = s >= q_steps;
    const RopeHeads& h = keys ? p.k : p.q;
    const int head = (keys ? s - q_steps : s) * hpw;
    T* x = out ? static_cast<T*>(h.y) + t * h.ys : const_cast<T*>(static_cast<const T*>(h.x)) + t * h.xs;
    return Cursor{x + (head + sub) * p.D, h.n - head};
  };
  auto advance = [&](Cursor& c, int s, bool out) {  // from group s - 1 to s
    if (s == q_steps) {
      c = group(s, out);
    } else {
      c.x += hpw * p.D;
      c.left -= hpw;
    }
  };
  const float inv_d = 1.0f / (float)p.D;
  // (cleared once: lanes without a unit keep zeros, lanes without a head what they had,
  // which goes nowhere)
  Chunk ra[PF][UL], rb[PF][UL];
#pragma unroll
  for (int k = 0; k < PF; k++)
#pragma unroll
    for (int i = 0; i < UL; i++) ra[k][i].clear(), rb[k][i].clear();
  for (; todo > 0; t++, s0 = 0) {
    const int s1 = min(s0 + todo, steps);
    todo -= s1 - s0;
    Cursor in = group(s0, false), out = group(s0, true);
    int ahead = s0;
    auto fetch = [&](Chunk(&xa)[UL], Chunk(&xb)[UL]) {
#pragma unroll
      for (int i = 0; i < UL; i++) {
        QMV_DEBUG_ONLY(const RopeHeads& h = ahead < q_steps ? p.q : p.k; const long long at = in.x - static_cast<const T*>(h.x);)
        if (ahead < s1 && sub < in.left && unit(i) < units) {
          if (QMV_CHECK(in_range(at + pa[i], CH, h.x_len, p.err))) xa[i].load(in.x + pa[i]);
          if (QMV_CHECK(in_range(at + pb[i], CH, h.x_len, p.err))) xb[i].load(in.x + pb[i]);
        }
      }
      advance(in, ++ahead, false);
    };
#pragma unroll
    for (int k = 0; k < PF; k++) fetch(ra[k], rb[k]);

    int pos = 0;
    if (!p.pos) {
      int seq = (int)t, a = seq, b = seq + 1;
      if (p.starts) {
        seq = last_seq_at_most(p.n_seq, (int)t, [&](int s) { return p.starts[s]; });
        a = p.starts[seq];
        b = p.starts[seq + 1];
      }
      int len = p.lens[seq];
      if (a < 0 || b < a || b > p.n_tok || len < 0) {  // clamped as by the cache calls (kv_seq)
        set_error(p.err, QMV_DEVERR_BATCH);
        a = min(max(a, 0), p.n_tok);
        b = min(max(b, a), p.n_tok);
        len = max(len, 0);
      }
      if ((int)t < a || (int)t >= b) continue;  // no sequence's token (the whole warp)
      if (len > 0 && len < b - a) set_error(p.err, QMV_DEVERR_BATCH);  // tokens before the first
      pos = len - b + (int)t;
    }
    __syncwarp();  // (the last token's turns are read)
#pragma unroll
    for (int i = 0; i < ROPE_MAX_PAIRS / 32; i++) {
      const int pair = lane + 32 * i;
      if (pair >= p.R / 2) break;
      const int at = p.pos ? p.pos[(long long)t * p.n_axes + axis[i]] : pos;
      turns[wid][pair] = turn_of(at, freq[i], p.scale);
    }
    __syncwarp();
    // Pair (a, b) becomes rstd (a ca - b sb, b cb + a sa): cosines and sines times the
    // weights of a and b (sb holds -sb).  Two pairs at once where a lane has more than one.
    constexpr int NP = UL * CH, W = CH > 1 ? 2 : 1;
    using V = typename Wide<W>::type;
    V ca[NP / W], sa[NP / W], cb[NP / W], sb[NP / W];
    auto factors = [&](const float* w) {
#pragma unroll
      for (int i = 0; i < UL; i++) {
        const int pair0 = unit(i) * CH;  // pairs below R / 2 turn (whole units but where pairs are neighbours)
        float wa[CH], wb[CH];
#pragma unroll
        for (int j = 0; j < CH; j++) wa[j] = wb[j] = 1.f;
        if (w && unit(i) < units) {
          if constexpr (CH > 1) {
            load_vec<CH>(w + pa[i], wa);
            load_vec<CH>(w + pb[i], wb);
          } else {
            wa[0] = w[pa[i]];
            wb[0] = w[pb[i]];
          }
          if (INTER) to_pairs(wa, wb);
        }
        float c[CH], n[CH];
#pragma unroll
        for (int j = 0; j < CH; j++) {
          const float2 cs = pair0 + j < p.R / 2 ? turns[wid][pair0 + j] : make_float2(1.f, 0.f);
          c[j] = cs.x, n[j] = cs.y;
        }
#pragma unroll
        for (int j = 0; j < CH; j += W) {
          const int e = (i * CH + j) / W;
          const V a = Wide<W>::of(&wa[j]), b = Wide<W>::of(&wb[j]), co = Wide<W>::of(&c[j]), si = Wide<W>::of(&n[j]);
          ca[e] = co * a, sa[e] = si * a;
          cb[e] = co * b, sb[e] = Wide<W>::both(-1.f) * (si * b);
        }
      }
    };
    factors(s0 < q_steps ? p.q.w : p.k.w);
    for (int s = s0; s < s1; s += PF) {
#pragma unroll
      for (int k = 0; k < PF; k++) {
        if (s + k >= s1) break;
        if (s + k == q_steps && s + k > s0) factors(p.k.w);  // from queries to keys
        const bool norm = (s + k < q_steps ? p.q.w : p.k.w) != nullptr;
        V va[NP / W], vb[NP / W];
#pragma unroll
        for (int i = 0; i < UL; i++) {
          float xa[CH], xb[CH];
          ra[k][i].to(xa);
          rb[k][i].to(xb);
          if (INTER) to_pairs(xa, xb);
#pragma unroll
          for (int j = 0; j < CH; j += W) va[(i * CH + j) / W] = Wide<W>::of(&xa[j]), vb[(i * CH + j) / W] = Wide<W>::of(&xb[j]);
        }
        fetch(ra[k], rb[k]);
        V rstd = Wide<W>::both(1.f);
        if (norm) {
          V one = Wide<W>::both(0.f), two = one;
#pragma unroll
          for (int i = 0; i < NP / W; i++) {
            one = Wide<W>::fma(va[i], va[i], one);
            two = Wide<W>::fma(vb[i], vb[i], two);
          }
          float sum = Wide<W>::sum(one + two);
          for (int o = 1; o < 1 << lph_log; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          rstd = Wide<W>::both(rsqrtf(fmaf(sum, inv_d, p.eps)));  // at most 2 units in the last place off
        }
#pragma unroll
        for (int i = 0; i < UL; i++) {
          Chunk oa, ob;
          float ya[CH], yb[CH];
          // (what does not turn has nothing of its partner, which may be infinite)
          const int turn = p.R / 2 - unit(i) * CH;  // pairs of the unit that turn: all or none but where they are neighbours
#pragma unroll
          for (int j = 0; j < CH; j += W) {
            const int e = (i * CH + j) / W;
            V a = va[e] * ca[e], b = vb[e] * cb[e];
            if (ALL || turn > j) {
              const V a1 = Wide<W>::fma(vb[e], sb[e], a), b1 = Wide<W>::fma(va[e], sa[e], b);
              if (!ALL && INTER && W == 2 && turn == j + 1) a = first(a1, a), b = first(b1, b);
              else a = a1, b = b1;
            }
            Wide<W>::to(rstd * a, &ya[j]);
            Wide<W>::to(rstd * b, &yb[j]);
          }
          if (INTER) from_pairs(ya, yb);
          oa.from(ya);
          ob.from(yb);
          QMV_DEBUG_ONLY(const RopeHeads& h = s + k < q_steps ? p.q : p.k; const long long at = out.x - static_cast<const T*>(h.y);)
          if (sub < out.left && unit(i) < units) {
            if (QMV_CHECK(in_range(at + pa[i], CH, h.y_len, p.err))) oa.store(out.x + pa[i]);
            if (QMV_CHECK(in_range(at + pb[i], CH, h.y_len, p.err))) ob.store(out.x + pb[i]);
          }
        }
        advance(out, s + k + 1, true);
      }
    }
  }
}

template <int DT, int CH, int UL>
static cudaError_t launch_as(bool interleaved, const RopeParams& p, cudaStream_t stream) {
  const int units = p.D / (2 * CH);
  int log = 0;
  while ((1 << log) < units && log < 5) log++;
  const int hpw = 32 >> log;
  const int steps = (p.q.n + hpw - 1) / hpw + (p.k.n + hpw - 1) / hpw;
  // As many warps as the GPU holds at once, or a group of heads each.
  const long long total = (long long)p.n_tok * steps, ctas = (total + ROPE_WARPS - 1) / ROPE_WARPS;
  const long long cap = (long long)(UL <= 2 ? ROPE_CTAS : 3) * device_sm_count();
  const unsigned grid = (unsigned)(ctas < cap ? ctas : cap);
  const unsigned per = (unsigned)(total / (grid * ROPE_WARPS)), rest = (unsigned)(total % (grid * ROPE_WARPS));
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3(grid), dim3(32 * ROPE_WARPS), 0, stream, true);
  // (knowing that every pair turns saves 0.7 us of 17 with 4096 x 40 heads of 128
  // bfloat16; with short chunks it does not show)
  if constexpr (CH >= 4)
    if (p.R == p.D) {
      if (interleaved) return cudaLaunchKernelEx(&cfg, norm_rope_kernel<DT, CH, UL, true, true>, p, log, per, rest);
      return cudaLaunchKernelEx(&cfg, norm_rope_kernel<DT, CH, UL, false, true>, p, log, per, rest);
    }
  if (interleaved) return cudaLaunchKernelEx(&cfg, norm_rope_kernel<DT, CH, UL, true, false>, p, log, per, rest);
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<DT, CH, UL, false, false>, p, log, per, rest);
}

// Chunks of 16 bytes where whole ones pair up, else shorter ones, down to single
// values (4096 x 40 heads of 128 bfloat16, the halves of R values as pairs: R 64 and 128
// 18 us, 120 24, 124 and 126 43).  Where pairs are neighbours only the head's size counts
// (19 us).  The lanes of a head are a power of two: with heads of 72 values (21.6 us), 80
// (17.3) and 192 (31.4) 44, 38 and 25% of them have no unit.
template <int DT>
static cudaError_t launch_dt(bool interleaved, const RopeParams& p, cudaStream_t stream) {
  const int R = interleaved ? 0 : p.R;
  if constexpr (DT != QMV_DT_F32)
    if (p.D % 16 == 0 && R % 16 == 0) return launch_as<DT, 8, 1>(interleaved, p, stream);
  if (p.D % 8 == 0 && R % 8 == 0) return launch_as<DT, 4, 1>(interleaved, p, stream);
  if (p.D % 4 == 0 && R % 4 == 0)
    return p.D <= 128 ? launch_as<DT, 2, 1>(interleaved, p, stream) : launch_as<DT, 2, 2>(interleaved, p, stream);
  return p.D <= 128 ? launch_as<DT, 1, 2>(interleaved, p, stream) : launch_as<DT, 1, 4>(interleaved, p, stream);
}

cudaError_t launch_norm_rope(int dtype, bool interleaved, const RopeParams& p, cudaStream_t stream) {
  switch (dtype) {
    case QMV_DT_F16: return launch_dt<QMV_DT_F16>(interleaved, p, stream);
    case QMV_DT_BF16: return launch_dt<QMV_DT_BF16>(interleaved, p, stream);
    default: return launch_dt<QMV_DT_F32>(interleaved, p, stream);
  }
}

}  // namespace qmv
