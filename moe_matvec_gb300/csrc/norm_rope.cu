// Norm of each query and key head and the position rotation, in one pass.
#include "float_io.cuh"
#include "kv_cache.cuh"
#include "launch.h"
#include "step_launch.h"

namespace qmv {

constexpr int ROPE_WARPS = 4;         // warps of a CTA, each on its own
constexpr int ROPE_MAX_PAIRS = 128;   // head_dim 256

// cos and sin of pair i at position pos.  The turn pos * freq / (2 pi) is formed
// and reduced to its fraction in 64 bits: in 32 a position of 131072 leaves 2^-7
// of the angle.  What remains is at most half a turn, to 2^-25 of a turn in fp32.
__device__ __forceinline__ float2 turn_of(int pos, float freq, float scale) {
  const double turn = (double)pos * ((double)freq * 0.15915494309189535);
  float s, c;
  sincospif(2.0f * (float)(turn - rint(turn)), &s, &c);
  return make_float2(c * scale, s * scale);
}

// y = x * w / sqrt(mean(x^2) + eps) (w given, else y = x), then each pair (a, b) of
// the first R values becomes (a cos - b sin, a sin + b cos).
//
// A head is D / (2 CH) units of two chunks of CH consecutive values, one unit a
// lane (UL units for CH = 1): the two halves of CH pairs (pair i: values i and
// i + R / 2), or 2 CH consecutive values (pair i: 2i, 2i + 1), or two chunks
// that do not turn.  So a lane holds whole pairs, the norm is a sum over the
// head's lanes, and the same lane has the same pairs in every head: its cosines
// and sines stay in registers while the warp goes through the token's heads,
// 32 / (lanes of a head) at a time.  The warp's lanes share out the token's angles
// (64 bits, the only costly arithmetic) through shared memory; meanwhile the first
// heads are on their way.
//
// Bound by HBM for many tokens.
template <int DT, int CH, int UL, bool INTER>
__global__ void __launch_bounds__(32 * ROPE_WARPS) norm_rope_kernel(const RopeParams p, int lph_log, int split) {
  using T = typename Elem<DT>::type;
  struct alignas(CH * sizeof(T) < 16 ? CH * sizeof(T) : 16) Chunk {
    T v[CH];
  };
  constexpr int PF = UL == 1 ? 4 : 1;  // head groups on their way at once
  __shared__ float2 turns[ROPE_WARPS][ROPE_MAX_PAIRS];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const long long item = (long long)blockIdx.x * ROPE_WARPS + wid;
  const long long t = item / split;
  const int part = (int)(item - t * split);
  if (t >= p.n_tok) return;
  const int hpw = 32 >> lph_log, li = lane & ((1 << lph_log) - 1), sub = lane >> lph_log;
  const int units = p.D / (2 * CH), turning = p.R / (2 * CH);
  const int q_steps = (p.q.n + hpw - 1) / hpw, steps = q_steps + (p.k.n + hpw - 1) / hpw;
  const int s0 = (int)((long long)steps * part / split), s1 = (int)((long long)steps * (part + 1) / split);
  // the two chunks of the lane's unit i
  auto unit = [&](int i) { return li + (i << lph_log); };
  auto places = [&](int u, int& a, int& b) {
    if (INTER || u >= turning) {
      a = u * 2 * CH;
      b = a + CH;
    } else {
      a = u * CH;
      b = p.R / 2 + a;
    }
  };
  Chunk ra[PF][UL], rb[PF][UL];
  auto fetch = [&](int s, Chunk(&xa)[UL], Chunk(&xb)[UL]) {
    const RopeHeads& h = s < q_steps ? p.q : p.k;
    const int head = (s < q_steps ? s : s - q_steps) * hpw + sub;
#pragma unroll
    for (int i = 0; i < UL; i++) {
#pragma unroll
      for (int j = 0; j < CH; j++) from_float(0.f, xa[i].v[j]), from_float(0.f, xb[i].v[j]);
      int a, b;
      places(unit(i), a, b);
      const long long at = t * h.xs + (long long)head * p.D;
      if (s < s1 && head < h.n && unit(i) < units && QMV_CHECK(in_range(at + a, CH, h.x_len, p.err)) &&
          QMV_CHECK(in_range(at + b, CH, h.x_len, p.err))) {
        xa[i] = *reinterpret_cast<const Chunk*>(static_cast<const T*>(h.x) + at + a);
        xb[i] = *reinterpret_cast<const Chunk*>(static_cast<const T*>(h.x) + at + b);
      }
    }
  };
#pragma unroll
  for (int k = 0; k < PF; k++) fetch(s0 + k, ra[k], rb[k]);

  int pos = 0;
  if (!p.pos) {
    int seq = (int)t, a = seq, b = seq + 1;
    if (p.starts) {
      seq = last_seq_at_most(p.n_seq, (int)t, [&](int s) { return p.starts[s]; });
      a = p.starts[seq];
      b = p.starts[seq + 1];
    }
    const int len = p.lens[seq];
    if (a < 0 || b < a || b > p.n_tok || len < 0) set_error(p.err, QMV_DEVERR_BATCH);
    if (t < a || t >= b) return;  // no sequence's token (the whole warp)
    pos = (int)((long long)max(len, 0) - b + t);
  }
  for (int i = lane; i < p.R / 2; i += 32) {
    int at = pos;
    if (p.pos) {
      int ax = p.axis ? p.axis[i] : 0;
      if (ax >= p.n_axes) {
        set_error(p.err, QMV_DEVERR_BATCH);
        ax = 0;
      }
      at = p.pos[t * p.n_axes + ax];
    }
    turns[wid][i] = turn_of(at, p.freq[i], p.scale);
  }
  __syncwarp();
  float co[UL][CH], si[UL][CH];
#pragma unroll
  for (int i = 0; i < UL; i++)
#pragma unroll
    for (int j = 0; j < CH; j++) {
      const bool turns_here = unit(i) < turning;
      const float2 cs = turns[wid][turns_here ? unit(i) * CH + j : 0];
      co[i][j] = turns_here ? cs.x : 1.f;
      si[i][j] = turns_here ? cs.y : 0.f;
    }
  float wa[UL][CH], wb[UL][CH];
  const float* w_held = nullptr;
  const float inv_d = 1.0f / (float)p.D;
  for (int s = s0; s < s1; s += PF) {
    if (s > s0) {
#pragma unroll
      for (int k = 0; k < PF; k++) fetch(s + k, ra[k], rb[k]);
    }
#pragma unroll
    for (int k = 0; k < PF; k++) {
      if (s + k >= s1) break;
      const RopeHeads& h = s + k < q_steps ? p.q : p.k;
      const int head = (s + k < q_steps ? s + k : s + k - q_steps) * hpw + sub;
      float va[UL][CH], vb[UL][CH];
#pragma unroll
      for (int i = 0; i < UL; i++)
#pragma unroll
        for (int j = 0; j < CH; j++) {
          va[i][j] = to_float(ra[k][i].v[j]);
          vb[i][j] = to_float(rb[k][i].v[j]);
        }
      if (h.w) {
        if (h.w != w_held) {  // queries' weights, then keys'
          w_held = h.w;
#pragma unroll
          for (int i = 0; i < UL; i++) {
            int a, b;
            places(unit(i), a, b);
#pragma unroll
            for (int j = 0; j < CH; j++) {
              wa[i][j] = unit(i) < units ? h.w[a + j] : 0.f;
              wb[i][j] = unit(i) < units ? h.w[b + j] : 0.f;
            }
          }
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < UL; i++)
#pragma unroll
          for (int j = 0; j < CH; j++) sum = fmaf(va[i][j], va[i][j], fmaf(vb[i][j], vb[i][j], sum));
        for (int o = 1; o < 1 << lph_log; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float rstd = rsqrtf(fmaf(sum, inv_d, p.eps));  // at most 2 units in the last place off
#pragma unroll
        for (int i = 0; i < UL; i++)
#pragma unroll
          for (int j = 0; j < CH; j++) {
            va[i][j] = (va[i][j] * rstd) * wa[i][j];
            vb[i][j] = (vb[i][j] * rstd) * wb[i][j];
          }
      }
#pragma unroll
      for (int i = 0; i < UL; i++) {
        Chunk oa, ob;
#pragma unroll
        for (int j = 0; j < CH; j++) {
          if (INTER && CH > 1) {  // pairs 0 .. CH / 2 of the unit lie in the first chunk
            if (j % 2 == 0) {
              const float c = co[i][j / 2], n = si[i][j / 2], c2 = co[i][(CH + j) / 2], n2 = si[i][(CH + j) / 2];
              from_float(va[i][j] * c - va[i][j + 1] * n, oa.v[j]);
              from_float(va[i][j + 1] * c + va[i][j] * n, oa.v[j + 1]);
              from_float(vb[i][j] * c2 - vb[i][j + 1] * n2, ob.v[j]);
              from_float(vb[i][j + 1] * c2 + vb[i][j] * n2, ob.v[j + 1]);
            }
          } else {
            from_float(va[i][j] * co[i][j] - vb[i][j] * si[i][j], oa.v[j]);
            from_float(vb[i][j] * co[i][j] + va[i][j] * si[i][j], ob.v[j]);
          }
        }
        int a, b;
        places(unit(i), a, b);
        const long long at = t * h.ys + (long long)head * p.D;
        if (head < h.n && unit(i) < units && QMV_CHECK(in_range(at + a, CH, h.y_len, p.err)) &&
            QMV_CHECK(in_range(at + b, CH, h.y_len, p.err))) {
          *reinterpret_cast<Chunk*>(static_cast<T*>(h.y) + at + a) = oa;
          *reinterpret_cast<Chunk*>(static_cast<T*>(h.y) + at + b) = ob;
        }
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
  // Few tokens: their heads are shared out to more warps, as many as 8 warps an SM.
  const long long warps = 8ll * device_sm_count();
  int split = (int)(warps / p.n_tok);
  if (split > steps) split = steps;
  if (split < 1) split = 1;
  const long long items = (long long)p.n_tok * split;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3((unsigned)((items + ROPE_WARPS - 1) / ROPE_WARPS)), dim3(32 * ROPE_WARPS), 0, stream, true);
  if (interleaved) return cudaLaunchKernelEx(&cfg, norm_rope_kernel<DT, CH, UL, true>, p, log, split);
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<DT, CH, UL, false>, p, log, split);
}

// Chunks of 16 bytes where whole ones pair up (of 8 for 16-bit types whose sizes
// leave that), else single values.
template <int DT>
static cudaError_t launch_dt(bool interleaved, const RopeParams& p, cudaStream_t stream) {
  if constexpr (DT != QMV_DT_F32)
    if (p.D % 16 == 0 && p.R % 16 == 0) return launch_as<DT, 8, 1>(interleaved, p, stream);
  if (p.D % 8 == 0 && p.R % 8 == 0) return launch_as<DT, 4, 1>(interleaved, p, stream);
  return launch_as<DT, 1, 4>(interleaved, p, stream);
}

cudaError_t launch_norm_rope(int dtype, bool interleaved, const RopeParams& p, cudaStream_t stream) {
  switch (dtype) {
    case QMV_DT_F16: return launch_dt<QMV_DT_F16>(interleaved, p, stream);
    case QMV_DT_BF16: return launch_dt<QMV_DT_BF16>(interleaved, p, stream);
    default: return launch_dt<QMV_DT_F32>(interleaved, p, stream);
  }
}

}  // namespace qmv
