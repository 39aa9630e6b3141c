// Low-rank adapters of many requests beside a shared projection:
// y = res + scale_a B_a (A_a x), each token with its own adapter a.
#include "float_io.cuh"
#include "launch.h"
#include "step_launch.h"

namespace qmv {

constexpr int LORA_WARPS = 8, LORA_THREADS = 32 * LORA_WARPS;
constexpr int LORA_TOK = 4;      // tokens of one adapter that a CTA takes
constexpr int LORA_COLS = 8;     // consecutive columns a lane
constexpr int LORA_WIN = 32 * LORA_COLS;
constexpr int LORA_ROWS = 8;     // rows of A a warp holds sums for

// The tokens of one CTA: up to LORA_TOK of those with token t's adapter, from t
// on; n = 0 where another CTA (an earlier token's) has t among its own.
struct LoraTokens {
  int a;  // the adapter, -1: none
  int n;
  int tok[LORA_TOK];
};
// (two loads a lane: ids, as every warp of a CTA comes by them)
__device__ __forceinline__ LoraTokens lora_tokens(const LoraParams& p, int t) {
  const int lane = threadIdx.x & 31;
  int id[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int k = lane + 32 * i;
    id[i] = k < p.n_tok ? __ldcg(p.ids + k) : -2;
    if (k < p.n_tok && (id[i] < 0 || id[i] >= p.n)) {
      if (id[i] >= p.n && k == t) set_error(p.err, QMV_DEVERR_ADAPTER);
      id[i] = -1;
    }
  }
  LoraTokens q;
  q.a = __shfl_sync(0xffffffffu, t < 32 ? id[0] : id[1], t & 31);
  unsigned long long same = (unsigned long long)__ballot_sync(0xffffffffu, id[1] == q.a) << 32 |
                            __ballot_sync(0xffffffffu, id[0] == q.a);
  q.n = 0;
  if (__popcll(same & ((1ull << t) - 1)) % LORA_TOK) return q;
  same &= ~0ull << t;
#pragma unroll
  for (int i = 0; i < LORA_TOK; i++) {
    q.tok[i] = same ? __ffsll(same) - 1 : t;
    if (same) q.n = i + 1;
    same &= same - 1;
  }
  return q;
}
__device__ __forceinline__ int rank_of(const LoraParams& p, int a) {
  return p.ranks ? min(max(__ldcg(p.ranks + a), 0), p.r) : p.r;
}

// Raw values of 16-byte (or 8-byte) loads.
template <class T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Raw {
  T v[N];
};

// v = A x over one split of the columns: part[split][token][row].  A warp takes
// every 8th row, eight at a time; a lane has 8 columns of each window of 256, and
// the eight rows' sums for up to four tokens are added over the lanes together
// (31 shuffles for 32 sums).  Adapter rows are read once per four of its tokens.
template <int DT>
__global__ void __launch_bounds__(LORA_THREADS) lora_down_kernel(const LoraParams p) {
  using T = typename Elem<DT>::type;
  using Row = Raw<T, LORA_COLS>;
  // The second kernel may start (and read the adapters' other half) once what came
  // before this call is done.
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const LoraTokens q = lora_tokens(p, blockIdx.y);
  if (q.n == 0 || q.a < 0) return;
  const int rank = rank_of(p, q.a);
  const int c0 = blockIdx.x * p.window, c1 = min(c0 + p.window, p.K);
  const T* A = static_cast<const T*>(p.A) + (long long)q.a * p.r * p.K;
  for (int j0 = warp; j0 < rank; j0 += LORA_WARPS * LORA_ROWS) {
    float acc[LORA_ROWS][LORA_TOK];
#pragma unroll
    for (int i = 0; i < LORA_ROWS; i++)
#pragma unroll
      for (int k = 0; k < LORA_TOK; k++) acc[i][k] = 0.f;
    for (int c = c0 + lane * LORA_COLS; c - lane * LORA_COLS < c1; c += LORA_WIN) {
      Row w[LORA_ROWS];
#pragma unroll
      for (int i = 0; i < LORA_ROWS; i++) {
        const int j = j0 + i * LORA_WARPS;
#pragma unroll
        for (int e = 0; e < LORA_COLS; e++) from_float(0.f, w[i].v[e]);
        if (j < rank && c < c1 && QMV_CHECK(in_range((long long)(q.a * p.r + j) * p.K + c, LORA_COLS, p.a_len, p.err)))
          w[i] = *reinterpret_cast<const Row*>(A + (long long)j * p.K + c);
      }
#pragma unroll
      for (int k = 0; k < LORA_TOK; k++) {
        if (k < q.n) {
          float x[LORA_COLS];
#pragma unroll
          for (int e = 0; e < LORA_COLS; e++) x[e] = 0.f;
          if (c < c1) load_vec<LORA_COLS>(p.x + (long long)q.tok[k] * p.K + c, x);
#pragma unroll
          for (int i = 0; i < LORA_ROWS; i++)
#pragma unroll
            for (int e = 0; e < LORA_COLS; e++) acc[i][k] = fmaf(to_float(w[i].v[e]), x[e], acc[i][k]);
        }
      }
    }
    // sum `lane` of the 32 over the lanes: halves the sums a lane holds at each step
    float* s = &acc[0][0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < o; i++) {
        const float give = up ? s[i] : s[i + o], keep = up ? s[i + o] : s[i];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    const int j = j0 + (lane / LORA_TOK) * LORA_WARPS, k = lane % LORA_TOK;
    int tok = q.tok[0];
#pragma unroll
    for (int i = 1; i < LORA_TOK; i++)
      if (i == k) tok = q.tok[i];
    if (j < rank && k < q.n) p.part[((long long)blockIdx.x * p.n_tok + tok) * p.r + j] = s[0];
  }
}

// y = res + scale B v for a tile of rows: v's parts are added in order, then each
// row of B lies with LPR lanes, VW values each, and the tile's results go through
// shared memory so that y and res are read and written in whole lines.  The tile's
// rows of B are on their way before the first kernel has finished.
template <int DT, int VW, int STEPS>
__global__ void __launch_bounds__(LORA_THREADS) lora_up_kernel(const LoraParams p, int lpr_log) {
  using T = typename Elem<DT>::type;
  using Row = Raw<T, VW>;
  extern __shared__ float lora_smem[];
  __shared__ float v[LORA_TOK][QMV_MAX_RANK];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rpw = 32 >> lpr_log, rows = STEPS * LORA_WARPS * rpw;  // rows of a tile
  const long long m0 = (long long)blockIdx.x * rows;
  pdl_launch_dependents();
  const LoraTokens q = lora_tokens(p, blockIdx.y);
  if (q.n == 0) return;  // (res of its tokens is another CTA's)
  if (q.a < 0) {         // no adapter
    pdl_wait();
    if (p.y != p.res)
      for (int k = 0; k < q.n; k++)
        for (long long m = m0 + tid; m < min(m0 + rows, p.M); m += LORA_THREADS)
          if (QMV_CHECK(in_range(q.tok[k] * p.M + m, 1, p.y_len, p.err))) p.y[q.tok[k] * p.M + m] = p.res[q.tok[k] * p.M + m];
    return;
  }
  const int rank = rank_of(p, q.a);
  const int j0 = (lane & ((1 << lpr_log) - 1)) * VW, sub = lane >> lpr_log;
  const T* B = static_cast<const T*>(p.B) + (long long)q.a * p.M * p.r;
  Row w[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; i++) {
    const long long m = m0 + (i * LORA_WARPS + warp) * rpw + sub;
#pragma unroll
    for (int e = 0; e < VW; e++) from_float(0.f, w[i].v[e]);
    if (m < p.M && j0 < rank && QMV_CHECK(in_range(((long long)q.a * p.M + m) * p.r + j0, VW, p.b_len, p.err)))
      w[i] = *reinterpret_cast<const Row*>(B + m * p.r + j0);
  }
  const float scale = p.scales ? __ldcg(p.scales + q.a) : 1.0f;
  pdl_wait();
  for (int i = tid; i < LORA_TOK * p.r; i += LORA_THREADS) {
    const int k = i / p.r, j = i - k * p.r;
    float sum = 0.f;
    if (k < q.n && j < rank) {
      int tok = q.tok[0];
#pragma unroll
      for (int o = 1; o < LORA_TOK; o++)
        if (o == k) tok = q.tok[o];
      for (int s = 0; s < p.splits; s++) sum += __ldcg(p.part + ((long long)s * p.n_tok + tok) * p.r + j);
    }
    v[k][j] = sum * scale;
  }
  __syncthreads();
  float x[LORA_TOK][VW];
#pragma unroll
  for (int k = 0; k < LORA_TOK; k++)
#pragma unroll
    for (int e = 0; e < VW; e++) x[k][e] = j0 + e < rank && k < q.n ? v[k][j0 + e] : 0.f;
#pragma unroll
  for (int i = 0; i < STEPS; i++) {
    float b[VW];
#pragma unroll
    for (int e = 0; e < VW; e++) b[e] = j0 + e < rank ? to_float(w[i].v[e]) : 0.f;
#pragma unroll
    for (int k = 0; k < LORA_TOK; k++) {
      if (k < q.n) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < VW; e++) sum = fmaf(b[e], x[k][e], sum);
        for (int o = 1; o < 1 << lpr_log; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (j0 == 0) lora_smem[k * rows + (i * LORA_WARPS + warp) * rpw + sub] = sum;
      }
    }
  }
  __syncthreads();
  const int live = (int)min((long long)rows, p.M - m0);
  for (int i = tid; i < live; i += LORA_THREADS)
#pragma unroll
    for (int k = 0; k < LORA_TOK; k++)
      if (k < q.n) {
        const long long at = q.tok[k] * p.M + m0 + i;
        if (QMV_CHECK(in_range(at, 1, p.y_len, p.err))) p.y[at] = p.res[at] + lora_smem[k * rows + i];
      }
}

// Splits of the columns: windows of 256 a split as long as there are at most 16
// (each tile of the second kernel adds all splits' parts).
int lora_splits(long long K, int n_tok) {
  (void)n_tok;
  const long long wins = (K + LORA_WIN - 1) / LORA_WIN, per = (wins + 15) / 16;
  return (int)((wins + per - 1) / per);
}

template <int DT, int VW, int STEPS>
static cudaError_t launch_up(const LoraParams& p, int log, cudaStream_t stream) {
  const int rows = STEPS * LORA_WARPS * (32 >> log);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3((unsigned)((p.M + rows - 1) / rows), p.n_tok), dim3(LORA_THREADS),
              (size_t)LORA_TOK * rows * sizeof(float), stream, true);
  return cudaLaunchKernelEx(&cfg, lora_up_kernel<DT, VW, STEPS>, p, log);
}

template <int DT, int VW>
static cudaError_t launch_vw(const LoraParams& p, cudaStream_t stream) {
  int log = 0;
  while ((VW << log) < p.r) log++;
  // Steps of a warp: as many as leave two CTAs an SM, each token taken to have an
  // adapter of its own.
  const long long rows = LORA_WARPS * (32 >> log), tiles = (p.M + rows - 1) / rows * p.n_tok;
  const long long want = 2ll * device_sm_count();
  if (tiles >= 8 * want) return launch_up<DT, VW, 8>(p, log, stream);
  if (tiles >= 4 * want) return launch_up<DT, VW, 4>(p, log, stream);
  if (tiles >= 2 * want) return launch_up<DT, VW, 2>(p, log, stream);
  return launch_up<DT, VW, 1>(p, log, stream);
}

template <int DT>
static cudaError_t launch_dt(const LoraParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3(p.splits, p.n_tok), dim3(LORA_THREADS), 0, stream, true);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, lora_down_kernel<DT>, p);
  if (e != cudaSuccess) return e;
  if constexpr (DT != QMV_DT_F32)
    if (p.r % 8 == 0) return launch_vw<DT, 8>(p, stream);
  return launch_vw<DT, 4>(p, stream);
}

cudaError_t launch_lora(int dtype, LoraParams p, cudaStream_t stream) {
  p.splits = lora_splits(p.K, p.n_tok);
  const int wins = (p.K + LORA_WIN - 1) / LORA_WIN;
  p.window = (wins + p.splits - 1) / p.splits * LORA_WIN;
  switch (dtype) {
    case QMV_DT_F16: return launch_dt<QMV_DT_F16>(p, stream);
    case QMV_DT_BF16: return launch_dt<QMV_DT_BF16>(p, stream);
    default: return launch_dt<QMV_DT_F32>(p, stream);
  }
}

}  // namespace qmv
