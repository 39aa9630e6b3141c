// Page selection: an upper bound of each page's quantized logits from the
// smallest and largest key codes of its dimensions, then the n_sel largest.
#include <limits.h>

#include <atomic>

#include "float_io.cuh"
#include "kv_cache.cuh"
#include "kv_launch.h"
#include "launch.h"

namespace qmv {

constexpr int SEL_THREADS = 512;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_UNROLL = 2;     // pages a lane works on at once
constexpr int SEL_TABLE = 2048;   // page indices brought into shared memory at a time
constexpr int SEL_MAX_CLUSTER = 8;
constexpr int SEL_MAX_GROUP = 256;  // query heads per kv head
constexpr int SEL_CACHED = 8192;  // keys kept in shared memory while picking

// The sequence that holds token t, or -1.
__device__ __forceinline__ int seq_of_token(const KvParams& p, int t) {
  if (!p.starts) return t;
  const int lo = last_seq_at_most(p.n_seq, t, [&](int s) { return p.starts[s]; });
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

// Order-preserving unsigned key of a score (-0 as +0).
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive prefix of v over the block's threads, and the sum.
__device__ __forceinline__ int block_scan(int v, int& total, int (&buf)[SEL_WARPS]) {
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
  for (int i = 0; i < SEL_WARPS; i++) {
    if (i < warp) before += buf[i];
    total += buf[i];
  }
  return before + inc - v;
}

// One cluster per (token, kv head): its CTAs score a share of the pages each,
// and the first, in whose shared memory the scores' keys meet, then picks.
// 16 sequences of up to 65536 tokens, 8 heads of 128, pages of 64 (26 MB of
// bounds): 14 us, of them 6-8 the scores of the longest sequence and 5 its picks;
// 2 sequences of 16384: 6 us, steps that wait for one another throughout.
//
// Scores: the group's query heads are quantized into shared memory, split by
// sign: with q = q+ + q-,
//   sum_i max(q_i lo_i, q_i hi_i) = q+ . hi + q- . lo,
// two chains of dp4a, exact in int32.  D / 16 lanes share a page (16 bytes of
// each extreme per lane), SEL_UNROLL pages a lane at once.  2 D + 4 bytes are
// read per page; bound by that read (or, for few pages, by the chain of
// dependent loads: lens, table, bounds) up to about 8 query heads per kv head,
// by dp4a beyond.
//
// Picks: the n_sel - 1 largest of the pages before the token's own, ties to the
// lower index, and the own page, ascending.  A radix selection finds the
// smallest key that is picked, 8 bits a pass from the highest bit in which the
// keys differ, done as soon as a whole bin is picked; then every thread counts
// in a contiguous run of pages and writes at its place.
template <int D>
__global__ void __launch_bounds__(SEL_THREADS, 2) kv_select_kernel(const SelectParams p) {
  constexpr int LP = D == 64 ? 4 : D == 128 ? 8 : 16, LIVE = D / 16, PPW = 32 / LP, W4 = D / 4, E = D / 32;
  extern __shared__ __align__(16) uint32_t sq[];  // [G][2][D / 4] codes, then [G] scales
  __shared__ uint32_t keys[SEL_CACHED];
  __shared__ int table[SEL_TABLE];
  __shared__ int hist[256], buf[SEL_WARPS], s_bin, s_left, s_done;
  __shared__ uint32_t s_lo[SEL_WARPS], s_hi[SEL_WARPS];
  pdl_launch_dependents();
  pdl_wait();
  const int rank = blockIdx.x, ranks = gridDim.x;  // of the cluster
  const int t = blockIdx.z, head = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (everything up to the cluster barrier's condition is the same in the whole cluster)
  const int s = seq_of_token(p.kv, t);
  if (s < 0) return;
  const KvSeq q = kv_seq(p.kv, s);
  const int pos = q.len - q.n + (t - q.t0);
  const long long row = (long long)t * p.kv.H + head;
  int32_t* ids = p.ids + row * p.n_sel;
  auto put = [&](int i, int page) {
    if (QMV_CHECK(in_range(row * p.n_sel + i, 1, p.ids_len, p.kv.err))) ids[i] = page;
  };
  const int last = pos < 0 ? -1 : pos / p.kv.P;  // the token's own page: picked whatever its score
  if (last < p.n_sel) {                          // all of them
    if (rank == 0)
      for (int i = tid; i < p.n_sel; i += SEL_THREADS) put(i, i <= last ? i : -1);
    return;
  }
  if (!QMV_CHECK(in_range(row * p.kv.max_pages, last, p.scores_len, p.kv.err))) return;
  float* const sc = p.scores + row * p.kv.max_pages;
  const int want = p.n_sel - 1;
  if (want == 0) {
    if (rank == 0 && tid == 0) put(0, last);
    return;
  }

  // Up to SEL_CACHED keys go straight into the first CTA's shared memory (once it
  // is known to run), more of them by the workspace.
  const bool cached = last <= SEL_CACHED;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  uint32_t first_keys;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(first_keys) : "r"(smem_u32(keys)));

  // ---- scores of pages [pg0, pg1)
  const int per = (last + ranks - 1) / ranks, pg0 = min(rank * per, last), pg1 = min(pg0 + per, last);
  const int sub = lane / LP, li = lane % LP;
  constexpr int STEP = SEL_WARPS * PPW;  // pages between a lane's pages
  const int bb = kv_bounds_bytes(D);
  // The cache's indices of up to SEL_TABLE pages from `from` on: one load for
  // the block, and the bounds' addresses then hang on shared memory alone.
  auto load_table = [&](int from) {
    for (int i = tid; i < min(SEL_TABLE, pg1 - from); i += SEL_THREADS) table[i] = kv_page(p.kv, s, from + i);
  };
  load_table(pg0);
  float* dq = reinterpret_cast<float*>(sq + p.G * 2 * W4);
  for (int g = warp; g < p.G; g += SEL_WARPS) {
    const long long at = t * p.q_stride + (long long)(head * p.G + g) * D;
    float x[E], amax = 0.f;
#pragma unroll
    for (int i = 0; i < E; i++) {
      const int dd = i * 32 + lane;
      x[i] = QMV_CHECK(in_range(at + dd, 1, p.q_len, p.kv.err)) ? load_any(p.q, at + dd, p.dtype) : 0.f;
      amax = fmaxf(amax, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float d = __fdiv_rn(amax, 127.f), inv = d > 0.f ? __frcp_rn(d) : 0.f;
    int8_t* pos8 = reinterpret_cast<int8_t*>(sq + g * 2 * W4);
#pragma unroll
    for (int i = 0; i < E; i++) {
      const int c = min(max(__float2int_rn(__fmul_rn(x[i], inv)), -127), 127);
      pos8[i * 32 + lane] = (int8_t)max(c, 0);
      pos8[D + i * 32 + lane] = (int8_t)min(c, 0);
    }
    if (lane == 0) dq[g] = d;
  }
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  __syncthreads();
  for (int from = pg0; from < pg1; from += SEL_TABLE) {
    if (from > pg0) {
      __syncthreads();
      load_table(from);
      __syncthreads();
    }
    const int upto = min(from + SEL_TABLE, pg1);
    // warps go their own ways: their loads and products overlap
    for (int pb = from + warp * PPW + sub; pb - sub < upto; pb += STEP * SEL_UNROLL) {
      uint4 lo[SEL_UNROLL], hi[SEL_UNROLL];
      float dk[SEL_UNROLL];
#pragma unroll
      for (int i = 0; i < SEL_UNROLL; i++) {
        const int pg = pb + i * STEP, id = pg < upto ? table[pg - from] : -1;
        lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
        dk[i] = 0.f;
        const long long at = ((long long)max(id, 0) * p.kv.H + head) * bb;
        if (id >= 0 && QMV_CHECK(in_range(at, bb, p.kv.bounds_len, p.kv.err))) {
          const uint8_t* b = p.kv.bounds + at;
          dk[i] = *reinterpret_cast<const float*>(b);
          if (li < LIVE) {
            lo[i] = *reinterpret_cast<const uint4*>(b + KV_HEADER + 16 * li);
            hi[i] = *reinterpret_cast<const uint4*>(b + KV_HEADER + D + 16 * li);
          }
        }
      }
      float best[SEL_UNROLL];
#pragma unroll
      for (int i = 0; i < SEL_UNROLL; i++) best[i] = -INFINITY;
      for (int g = 0; g < p.G; g++) {
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (li < LIVE) {
          a = *reinterpret_cast<const uint4*>(sq + g * 2 * W4 + 4 * li);
          b = *reinterpret_cast<const uint4*>(sq + g * 2 * W4 + W4 + 4 * li);
        }
        const float d = dq[g];
#pragma unroll
        for (int i = 0; i < SEL_UNROLL; i++) {
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
        for (int i = 0; i < SEL_UNROLL; i++)
          if (pb + i * STEP < upto) {
            const float score = __fmul_rn(best[i], dk[i]);
            if (cached && QMV_CHECK(in_range(pb + i * STEP, 1, SEL_CACHED, p.kv.err)))
              asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(first_keys + 4 * (pb + i * STEP)), "r"(score_key(score)) : "memory");
            if (!cached) sc[pb + i * STEP] = score;
          }
      }
    }
  }
  // the cluster's scores are written; the first CTA goes on
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank != 0) return;

  // ---- picks
  uint32_t kmin = 0xffffffffu, kmax = 0;
  auto key = [&](int i) { return cached ? keys[i] : score_key(__ldcg(sc + i)); };
  for (int i = tid; i < last; i += SEL_THREADS) {
    const uint32_t k = key(i);
    kmin = min(kmin, k);
    kmax = max(kmax, k);
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0) {
    s_lo[warp] = kmin;
    s_hi[warp] = kmax;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SEL_WARPS; i++) {
    kmin = min(kmin, s_lo[i]);
    kmax = max(kmax, s_hi[i]);
  }
  // keys less kmin have `bits` bits; picked are those >= floor, and of those
  // equal to floor the first `left`
  int bits = 32 - __clz((int)(kmax - kmin)), left = want;
  uint32_t floor = 0;
  bool whole = false;  // every key >= floor is picked
  while (bits > 0 && !whole) {
    const int shift = max(bits - 8, 0);
    for (int i = tid; i < 256; i += SEL_THREADS) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < last; i += SEL_THREADS) {
      const uint32_t k = key(i) - kmin;
      if (bits == 32 || (k >> bits) == (floor >> bits)) atomicAdd(&hist[(k >> shift) & 255u & ((1u << (bits - shift)) - 1)], 1);
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
          s_done = run + c[i] == left;
        }
        run += c[i];
      }
    }
    __syncthreads();
    floor |= (uint32_t)s_bin << shift;
    left = s_left;
    whole = s_done != 0;
    bits = shift;
    __syncthreads();
  }
  // a thread's run of pages
  const int run = (last + SEL_THREADS - 1) / SEL_THREADS, b0 = min(tid * run, last), b1 = min(b0 + run, last);
  int n_eq = 0, n_gt = 0, total;
  for (int i = b0; i < b1; i++) {
    const uint32_t k = key(i) - kmin;
    n_gt += k > floor || (whole && k == floor);
    n_eq += !whole && k == floor;
  }
  int rank_eq = whole ? 0 : block_scan(n_eq, total, buf);
  const int take = n_gt + min(max(left - rank_eq, 0), n_eq);
  int at = block_scan(take, total, buf);
  for (int i = b0; i < b1; i++) {
    const uint32_t k = key(i) - kmin;
    if (k > floor || (k == floor && (whole || rank_eq++ < left))) put(at++, i);
  }
  if (tid == 0) put(want, last);
}

size_t kv_select_ws_bytes(int H, int n_tok, int max_pages) { return (size_t)n_tok * H * max_pages * sizeof(float); }

template <int D>
static cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)p.G * (2 * D + sizeof(float));
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(configured.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kv_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SEL_MAX_GROUP * (2 * D + (int)sizeof(float)));
    if (e != cudaSuccess) return e;
    configured.fetch_or(1ull << dev);
  }
  // CTAs of a cluster: a round of the lanes' pages each or more, while all
  // clusters still fit the GPU at once (two CTAs an SM), up to the portable size
  const int round = SEL_WARPS * (32 / (D == 64 ? 4 : D == 128 ? 8 : 16)) * SEL_UNROLL;
  int ranks = 1;
  const long long heads = (long long)p.kv.H * p.kv.n_tok;
  while (ranks < SEL_MAX_CLUSTER && p.kv.max_pages > ranks * round && heads * ranks <= device_sm_count()) ranks *= 2;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  make_config(cfg, attr, dim3(ranks, p.kv.H, p.kv.n_tok), dim3(SEL_THREADS), smem, stream, true);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kv_select_kernel<D>, p);
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
  switch (D) {
    case 64: return launch_select<64>(p, stream);
    case 128: return launch_select<128>(p, stream);
    case 192: return launch_select<192>(p, stream);
    default: return launch_select<256>(p, stream);
  }
}

}  // namespace qmv
