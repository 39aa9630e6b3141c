// Page selection: an upper bound of each page's quantized logits from the
// smallest and largest key codes of its dimensions, then the n_sel largest.
#include <limits.h>

#include "float_io.cuh"
#include "kv_cache.cuh"
#include "kv_launch.h"
#include "launch.h"

namespace qmv {

constexpr int SC_THREADS = 128;
constexpr int SC_PAGES = 128;  // pages of one block
constexpr int SC_UNROLL = 4;   // pages a lane works on at once
constexpr int PICK_THREADS = 512;

// The sequence that holds token t, or -1.
__device__ __forceinline__ int seq_of_token(const KvParams& p, int t) {
  if (!p.starts) return t;
  int lo = 0, hi = p.n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.starts[mid] <= t) lo = mid; else hi = mid;
  }
  const KvSeq q = kv_seq(p, lo);
  return t >= q.t0 && t < q.t0 + q.n ? lo : -1;
}

__device__ __forceinline__ float load_any(const void* x, long long at, int dt) {
  return dt == QMV_DT_F32 ? static_cast<const float*>(x)[at]
                          : dt == QMV_DT_F16 ? to_float(static_cast<const __half*>(x)[at])
                                             : to_float(static_cast<const __nv_bfloat16*>(x)[at]);
}

struct SelectParams {
  KvParams kv;
  const void* q;
  long long q_stride;
  int dtype, G, n_sel;
  float* scores;  // [n_tok][H][max_pages]
  int32_t* ids;
#ifdef QMV_DEBUG
  long long q_len, scores_len, ids_len;
#endif
};

// scores of SC_PAGES pages of one (token, kv head).  The group's query heads
// are quantized into shared memory, split by sign: with q = q+ + q-,
//   sum_i max(q_i lo_i, q_i hi_i) = q+ . hi + q- . lo,
// two chains of dp4a, exact in int32.  D / 16 lanes share a page (16 bytes of
// each extreme per lane), SC_UNROLL pages a lane at once.  Reads 2 D + 4 bytes
// per page; bound by that read up to about 8 query heads per kv head, by dp4a
// beyond.
template <int D>
__global__ void __launch_bounds__(SC_THREADS) kv_score_kernel(const SelectParams p) {
  constexpr int LP = D == 64 ? 4 : D == 128 ? 8 : 16, LIVE = D / 16, PPW = 32 / LP, W4 = D / 4;
  extern __shared__ __align__(16) uint32_t sq[];  // [G][2][D / 4] codes, then [G] scales
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.z, head = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = seq_of_token(p.kv, t);
  if (s < 0) return;
  const KvSeq q = kv_seq(p.kv, s);
  const int pos = q.len - q.n + (t - q.t0);
  if (pos < 0) return;
  const int last = pos / p.kv.P;  // the token's own page: picked whatever its score
  const int pg0 = blockIdx.x * SC_PAGES;
  if (last < p.n_sel || pg0 >= last) return;  // every page is picked / nothing here
  float* dq = reinterpret_cast<float*>(sq + p.G * 2 * W4);
  for (int g = warp; g < p.G; g += SC_THREADS / 32) {
    const long long at = t * p.q_stride + (long long)(head * p.G + g) * D;
    float x[D / 32], amax = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; i++) {
      const int dd = i * 32 + lane;
      x[i] = QMV_CHECK(in_range(at + dd, 1, p.q_len, p.kv.err)) ? load_any(p.q, at + dd, p.dtype) : 0.f;
      amax = fmaxf(amax, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float d = __fdiv_rn(amax, 127.f), inv = d > 0.f ? __frcp_rn(d) : 0.f;
    int8_t* pos8 = reinterpret_cast<int8_t*>(sq + g * 2 * W4);
#pragma unroll
    for (int i = 0; i < D / 32; i++) {
      const int c = min(max(__float2int_rn(__fmul_rn(x[i], inv)), -127), 127);
      pos8[i * 32 + lane] = (int8_t)max(c, 0);
      pos8[D + i * 32 + lane] = (int8_t)min(c, 0);
    }
    if (lane == 0) dq[g] = d;
  }
  __syncthreads();
  const int sub = lane / LP, li = lane % LP;
  constexpr int STEP = SC_THREADS / 32 * PPW;  // pages between a lane's pages
  const int bb = kv_bounds_bytes(D);
  for (int pb = pg0 + warp * PPW + sub; pb - sub < min(pg0 + SC_PAGES, last); pb += STEP * SC_UNROLL) {
    uint4 lo[SC_UNROLL], hi[SC_UNROLL];
    float dk[SC_UNROLL];
    bool ok[SC_UNROLL];
#pragma unroll
    for (int i = 0; i < SC_UNROLL; i++) {
      const int pg = pb + i * STEP;
      lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
      dk[i] = 0.f;
      ok[i] = pg < min(pg0 + SC_PAGES, last);
      const int id = ok[i] ? kv_page(p.kv, s, pg) : -1;
      if (id >= 0) {
        const long long at = ((long long)id * p.kv.H + head) * bb;
        if (QMV_CHECK(in_range(at, bb, p.kv.bounds_len, p.kv.err))) {
          const uint8_t* b = p.kv.bounds + at;
          dk[i] = *reinterpret_cast<const float*>(b);
          if (li < LIVE) {
            lo[i] = *reinterpret_cast<const uint4*>(b + KV_HEADER + 16 * li);
            hi[i] = *reinterpret_cast<const uint4*>(b + KV_HEADER + D + 16 * li);
          }
        }
      }
    }
    float best[SC_UNROLL];
#pragma unroll
    for (int i = 0; i < SC_UNROLL; i++) best[i] = -INFINITY;
    for (int g = 0; g < p.G; g++) {
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (li < LIVE) {
        a = *reinterpret_cast<const uint4*>(sq + g * 2 * W4 + 4 * li);
        b = *reinterpret_cast<const uint4*>(sq + g * 2 * W4 + W4 + 4 * li);
      }
      const float d = dq[g];
#pragma unroll
      for (int i = 0; i < SC_UNROLL; i++) {
        int u = __dp4a((int)a.x, (int)hi[i].x, 0);
        u = __dp4a((int)a.y, (int)hi[i].y, u);
        u = __dp4a((int)a.z, (int)hi[i].z, u);
        u = __dp4a((int)a.w, (int)hi[i].w, u);
        u = __dp4a((int)b.x, (int)lo[i].x, u);
        u = __dp4a((int)b.y, (int)lo[i].y, u);
        u = __dp4a((int)b.z, (int)lo[i].z, u);
        u = __dp4a((int)b.w, (int)lo[i].w, u);
#pragma unroll
        for (int o = LP / 2; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
        best[i] = fmaxf(best[i], __fmul_rn((float)u, d));
      }
    }
    if (li == 0) {
#pragma unroll
      for (int i = 0; i < SC_UNROLL; i++) {
        const long long at = ((long long)t * p.kv.H + head) * p.kv.max_pages + pb + i * STEP;
        if (ok[i] && QMV_CHECK(in_range(at, 1, p.scores_len, p.kv.err))) p.scores[at] = __fmul_rn(best[i], dk[i]);
      }
    }
  }
}

// Order-preserving unsigned key of a score (-0 as +0).
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum over the block; every thread gets it, and the exclusive prefix of its
// own value.
__device__ __forceinline__ int block_scan(int v, int& total, int* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = inc;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < PICK_THREADS / 32; i++) {
    if (i < warp) before += buf[i];
    total += buf[i];
  }
  return before + inc - v;
}

// The picks of one (token, kv head): the n_sel - 1 largest scores of pages [0,
// last), ties to the lower index, and page `last`, ascending.  A radix
// selection finds the key of the last pick in four passes over the scores
// (8 bits a pass, most significant first); a pass in index order then writes
// the pages above it and the first of those equal to it.
__global__ void __launch_bounds__(PICK_THREADS) kv_pick_kernel(const SelectParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int hist[256], buf[PICK_THREADS / 32], s_bin, s_left;
  const int t = blockIdx.y, head = blockIdx.x, tid = threadIdx.x;
  const int s = seq_of_token(p.kv, t);
  if (s < 0) return;
  const KvSeq q = kv_seq(p.kv, s);
  const int pos = q.len - q.n + (t - q.t0);
  const long long row = (long long)t * p.kv.H + head;
  if (!QMV_CHECK(in_range(row * p.n_sel, p.n_sel, p.ids_len, p.kv.err))) return;
  int32_t* ids = p.ids + row * p.n_sel;
  const int last = pos < 0 ? -1 : pos / p.kv.P;
  if (last < p.n_sel) {  // all of them
    for (int i = tid; i < p.n_sel; i += PICK_THREADS) ids[i] = i <= last ? i : -1;
    return;
  }
  const float* sc = p.scores + row * p.kv.max_pages;
  if (!QMV_CHECK(in_range(row * p.kv.max_pages, last, p.scores_len, p.kv.err))) return;
  const int want = p.n_sel - 1;
  uint32_t prefix = 0;
  int left = want;  // picks still to find among the keys that match the prefix
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += PICK_THREADS) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < last; i += PICK_THREADS) {
        const uint32_t k = score_key(sc[i]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid < 32) {
        // lane: 8 bins from the top; the bin where the running count reaches `left`
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          c[i] = hist[255 - (tid * 8 + i)];
          sum += c[i];
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int n = __shfl_up_sync(0xffffffffu, inc, o);
          if (tid >= o) inc += n;
        }
        int run = inc - sum;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          if (run < left && run + c[i] >= left) {
            s_bin = 255 - (tid * 8 + i);
            s_left = left - run;
          }
          run += c[i];
        }
      }
      __syncthreads();
      prefix |= (uint32_t)s_bin << shift;
      left = s_left;
      __syncthreads();
    }
  }
  int out = 0, equal = 0;  // written; seen equal to the threshold
  for (int b = 0; b < last; b += PICK_THREADS) {
    const int i = b + tid;
    const uint32_t k = i < last ? score_key(sc[i]) : 0;
    const bool gt = want > 0 && i < last && k > prefix, eq = want > 0 && i < last && k == prefix;
    int n_eq, n_out;
    const int rank = equal + block_scan(eq, n_eq, buf);
    const bool take = gt || (eq && rank < left);
    const int at = out + block_scan(take, n_out, buf);
    if (take) ids[at] = i;
    equal += n_eq;
    out += n_out;
  }
  if (tid == 0) ids[want] = last;
}

size_t kv_select_ws_bytes(int H, int n_tok, int max_pages) { return (size_t)n_tok * H * max_pages * sizeof(float); }

template <int D>
static cudaError_t launch_score(const SelectParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)p.G * (2 * D + sizeof(float));
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kv_score_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3((p.kv.max_pages + SC_PAGES - 1) / SC_PAGES, p.kv.H, p.kv.n_tok), dim3(SC_THREADS), smem,
              stream, true);
  return cudaLaunchKernelEx(&cfg, kv_score_kernel<D>, p);
}

cudaError_t launch_kv_select(const KvParams& kv, int D, const SelectArgs& a, cudaStream_t stream) {
  SelectParams p{};
  p.kv = kv;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.dtype = a.dtype;
  p.G = a.n_heads / kv.H;
  p.n_sel = a.n_sel;
  p.scores = static_cast<float*>(a.ws);
  p.ids = a.ids;
  QMV_DEBUG_ONLY(p.q_len = (long long)(kv.n_tok - 1) * a.q_stride + (long long)a.n_heads * D;
                 p.scores_len = (long long)kv.n_tok * kv.H * kv.max_pages;
                 p.ids_len = output_extent((long long)kv.n_tok * kv.H * a.n_sel);)
  cudaError_t e = cudaSuccess;
  if (kv.max_pages > a.n_sel) {  // else every page of every token is picked
    switch (D) {
      case 64: e = launch_score<64>(p, stream); break;
      case 128: e = launch_score<128>(p, stream); break;
      case 192: e = launch_score<192>(p, stream); break;
      default: e = launch_score<256>(p, stream); break;
    }
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3(kv.H, kv.n_tok), dim3(PICK_THREADS), 0, stream, true);
  return cudaLaunchKernelEx(&cfg, kv_pick_kernel, p);
}

}  // namespace qmv
