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
constexpr int LORA_ROWS = 4;     // rows of A a warp holds sums for
constexpr int LORA_SMS = 152;    // what the splits of the columns are made for (on any device: they decide the sums' order)

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

// v = A x over one split of the columns: part[split][token][row].  A warp takes
// four rows; a lane has 8 columns of each window of 256, the next window's rows on
// their way while one is worked on.  The four rows' sums for up to four tokens are
// added over the lanes together (16 shuffles for 16 sums).  x of the CTA's tokens
// lies in shared memory.  Adapter rows are read once per four of its tokens.
template <int DT>
__global__ void __launch_bounds__(LORA_THREADS, 2) lora_down_kernel(const LoraParams p) {
  using T = typename Elem<DT>::type;
  using Row = Packed<T, LORA_COLS>;
  extern __shared__ __align__(16) float lora_x[];  // [LORA_TOK][window]
  // The second kernel may start (and read the adapters' other half) once what came
  // before this call is done.
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const LoraTokens q = lora_tokens(p, blockIdx.y);
  if (q.n == 0 || q.a < 0) return;
  const int rank = rank_of(p, q.a);
  const int c0 = blockIdx.x * p.window, c1 = min(c0 + p.window, p.K);
  const T* A = static_cast<const T*>(p.A) + (long long)q.a * p.r * p.K;
  constexpr int AHEAD = DT == QMV_DT_F32 ? 1 : 2;  // windows on their way: 4 KB a warp
  Row w[AHEAD][LORA_ROWS];
  auto fetch = [&](Row& x, int j, int c) {
    x.clear();
    if (j < rank && c < c1 && QMV_CHECK(in_range(((long long)q.a * p.r + j) * p.K + c, LORA_COLS, p.a_len, p.err)))
      x.load(A + (long long)j * p.K + c);
  };
  auto begin = [&](int j0) {
#pragma unroll
    for (int u = 0; u < AHEAD; u++)
#pragma unroll
      for (int i = 0; i < LORA_ROWS; i++) fetch(w[u][i], j0 + i, c0 + lane * LORA_COLS + u * LORA_WIN);
  };
  begin(warp * LORA_ROWS);
  for (int i = 4 * tid; i < p.window; i += 4 * LORA_THREADS)
#pragma unroll
    for (int k = 0; k < LORA_TOK; k++)
      if (k < q.n)
        *reinterpret_cast<float4*>(lora_x + k * p.window + i) =
            c0 + i < p.K ? *reinterpret_cast<const float4*>(p.x + (long long)q.tok[k] * p.K + c0 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  for (int j0 = warp * LORA_ROWS; j0 < rank; j0 += LORA_WARPS * LORA_ROWS) {
    if (j0 != warp * LORA_ROWS) begin(j0);
    float acc[LORA_ROWS][LORA_TOK];
#pragma unroll
    for (int i = 0; i < LORA_ROWS; i++)
#pragma unroll
      for (int k = 0; k < LORA_TOK; k++) acc[i][k] = 0.f;
    for (int base = c0; base < c1; base += AHEAD * LORA_WIN) {
#pragma unroll
      for (int u = 0; u < AHEAD; u++) {
        const int c = base + u * LORA_WIN + lane * LORA_COLS;
        if (base + u * LORA_WIN >= c1) break;
        float x[LORA_TOK][LORA_COLS];
#pragma unroll
        for (int k = 0; k < LORA_TOK; k++)
          if (k < q.n) load_vec<LORA_COLS>(lora_x + k * p.window + c - c0, x[k]);
#pragma unroll
        for (int i = 0; i < LORA_ROWS; i++) {
          float v[LORA_COLS];
          w[u][i].to(v);
          fetch(w[u][i], j0 + i, c + AHEAD * LORA_WIN);
#pragma unroll
          for (int k = 0; k < LORA_TOK; k++)
            if (k < q.n)
#pragma unroll
              for (int e = 0; e < LORA_COLS; e++) acc[i][k] = fmaf(v[e], x[k][e], acc[i][k]);
        }
      }
    }
    // sum `lane` % 16 of the 16 over the lanes: halves the sums a lane holds at each step
    float* s = &acc[0][0];
#pragma unroll
    for (int o = LORA_ROWS * LORA_TOK / 2; o > 0; o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < o; i++) {
        const float give = up ? s[i] : s[i + o], keep = up ? s[i + o] : s[i];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    s[0] += __shfl_xor_sync(0xffffffffu, s[0], LORA_ROWS * LORA_TOK);
    const int j = j0 + lane / LORA_TOK, k = lane % LORA_TOK;
    int tok = q.tok[0];
#pragma unroll
    for (int i = 1; i < LORA_TOK; i++)
      if (i == k) tok = q.tok[i];
    if (lane < LORA_ROWS * LORA_TOK && j < rank && k < q.n) p.part[((long long)blockIdx.x * p.n_tok + tok) * p.r + j] = s[0];
  }
}

// y = res + scale B v: v's parts are added in order, then each warp goes through
// rows of its own, eight loads of 16 bytes a lane on their way (the first ones
// before the first kernel has finished).  A row of B lies with 2^lpr_log lanes, VW
// values each; the partial sums of `gather` loads are added over those lanes
// together, so that afterwards each lane has one row's sum and up to 32 consecutive
// rows of y and res are read and written at once.
template <int DT, int VW, int LPR_LOG>
__global__ void __launch_bounds__(LORA_THREADS, 2) lora_up_kernel(const LoraParams p, int rows_per_warp) {
  using T = typename Elem<DT>::type;
  using Row = Packed<T, VW>;
  constexpr int LPR = 1 << LPR_LOG, RPL = 32 >> LPR_LOG;               // lanes a row, rows a load
  constexpr int GATHER_LOG = LPR_LOG < 3 ? LPR_LOG : 3, GATHER = 1 << GATHER_LOG;
  constexpr int LOADS = 8, BLOCK = GATHER * RPL;                       // rows whose sums are gathered at once
  __shared__ float v[LORA_TOK][QMV_MAX_RANK];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long first = ((long long)blockIdx.x * LORA_WARPS + warp) * rows_per_warp;
  const long long m0 = min(first, p.M), m1 = min(first + rows_per_warp, p.M);
  pdl_launch_dependents();
  const LoraTokens q = lora_tokens(p, blockIdx.y);
  if (q.n == 0) return;  // (another CTA has these rows of the token)
  if (q.a < 0) {         // no adapter
    pdl_wait();
    if (p.y != p.res)
      for (int k = 0; k < q.n; k++)
        for (long long m = m0 + lane; m < m1; m += 32)
          if (QMV_CHECK(in_range(q.tok[k] * p.M + m, 1, p.y_len, p.err))) p.y[q.tok[k] * p.M + m] = p.res[q.tok[k] * p.M + m];
    return;
  }
  const int rank = rank_of(p, q.a);
  const int li = lane & (LPR - 1), j0 = li * VW, sub = lane >> LPR_LOG;
  const T* B = static_cast<const T*>(p.B) + (long long)q.a * p.M * p.r + j0;
  Row w[LOADS];
  auto fetch = [&](Row& x, long long m) {
    x.clear();
    if (m < m1 && j0 < rank && QMV_CHECK(in_range(((long long)q.a * p.M + m) * p.r + j0, VW, p.b_len, p.err)))
      x.load(B + m * p.r);
  };
#pragma unroll
  for (int i = 0; i < LOADS; i++) fetch(w[i], m0 + i * RPL + sub);
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
      const float* part = p.part + (long long)tok * p.r + j;
      const long long step = (long long)p.n_tok * p.r;
#pragma unroll 8
      for (int s = 0; s < p.splits; s++) sum += __ldcg(part + s * step);
    }
    v[k][j] = sum * scale;
  }
  __syncthreads();
  float x[LORA_TOK][VW];
#pragma unroll
  for (int k = 0; k < LORA_TOK; k++)
#pragma unroll
    for (int e = 0; e < VW; e++) x[k][e] = j0 + e < rank && k < q.n ? v[k][j0 + e] : 0.f;
  // the row of a block whose sum ends up here
  const int mine = GATHER == 1 ? sub : (li & (GATHER - 1)) * RPL + sub;
  const bool writer = LPR <= GATHER || li < GATHER;
  for (long long m = m0; m < m1; m += LOADS * RPL) {
#pragma unroll
    for (int g = 0; g < LOADS / GATHER; g++) {
      float acc[LORA_TOK][GATHER], res[LORA_TOK];
      const long long row = m + g * BLOCK + mine;
#pragma unroll
      for (int k = 0; k < LORA_TOK; k++) res[k] = k < q.n && writer && row < m1 ? p.res[q.tok[k] * p.M + row] : 0.f;
#pragma unroll
      for (int i = 0; i < GATHER; i++) {
        float b[VW];
        w[g * GATHER + i].to(b);
        fetch(w[g * GATHER + i], m + (LOADS + g * GATHER + i) * RPL + sub);
        if (j0 + VW > rank) {
#pragma unroll
          for (int e = 0; e < VW; e++)
            if (j0 + e >= rank) b[e] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < LORA_TOK; k++) {
          acc[k][i] = 0.f;
          if (k < q.n)
#pragma unroll
            for (int e = 0; e < VW; e++) acc[k][i] = fmaf(b[e], x[k][e], acc[k][i]);
        }
      }
#pragma unroll
      for (int k = 0; k < LORA_TOK; k++) {
        if (k < q.n) {
#pragma unroll
          for (int o = GATHER / 2; o > 0; o >>= 1) {
            const bool up = li & o;
#pragma unroll
            for (int i = 0; i < o; i++) {
              const float give = up ? acc[k][i] : acc[k][i + o], keep = up ? acc[k][i + o] : acc[k][i];
              acc[k][i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
          }
#pragma unroll
          for (int o = GATHER; o < LPR; o <<= 1) acc[k][0] += __shfl_xor_sync(0xffffffffu, acc[k][0], o);
          const long long at = q.tok[k] * p.M + row;
          if (writer && row < m1 && QMV_CHECK(in_range(at, 1, p.y_len, p.err))) p.y[at] = res[k] + acc[k][0];
        }
      }
    }
  }
}

// Splits of the columns: as many as give every SM two CTAs (each token taken to
// have an adapter of its own), at most 16, a window of 256 columns each or more, and
// at most 2048 columns (x of four tokens in shared memory).
static int lora_window(long long K, int n_tok) {
  const long long wins = (K + LORA_WIN - 1) / LORA_WIN;
  long long splits = (2ll * LORA_SMS + n_tok - 1) / n_tok;
  if (splits > 16) splits = 16;
  if (splits > wins) splits = wins;
  long long per = (wins + splits - 1) / splits;
  if (per > 8) per = 8;
  return (int)(per * LORA_WIN);
}
int lora_splits(long long K, int n_tok) {
  const int w = lora_window(K, n_tok);
  return (int)((K + w - 1) / w);
}

template <int DT, int VW, int LPR_LOG>
static cudaError_t launch_up(const LoraParams& p, cudaStream_t stream) {
  // Rows of a warp: so many that all warps fit the GPU at once (16 an SM), each
  // token taken to have an adapter of its own; whole blocks.
  constexpr int RPL = 32 >> LPR_LOG, BLOCK = (LPR_LOG < 3 ? 1 << LPR_LOG : 8) * RPL;
  const long long warps = 16ll * device_sm_count() / p.n_tok;
  long long rows = (p.M + warps - 1) / warps;
  rows = (rows + BLOCK - 1) / BLOCK * BLOCK;
  const long long per_cta = rows * LORA_WARPS;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3((unsigned)((p.M + per_cta - 1) / per_cta), p.n_tok), dim3(LORA_THREADS), 0, stream, true);
  return cudaLaunchKernelEx(&cfg, lora_up_kernel<DT, VW, LPR_LOG>, p, (int)rows);
}

template <int DT, int VW>
static cudaError_t launch_vw(const LoraParams& p, cudaStream_t stream) {
  if (p.r <= VW) return launch_up<DT, VW, 0>(p, stream);
  if (p.r <= 2 * VW) return launch_up<DT, VW, 1>(p, stream);
  if (p.r <= 4 * VW) return launch_up<DT, VW, 2>(p, stream);
  if (p.r <= 8 * VW) return launch_up<DT, VW, 3>(p, stream);
  if (p.r <= 16 * VW) return launch_up<DT, VW, 4>(p, stream);
  if constexpr (VW == 4) return launch_up<DT, VW, 5>(p, stream);
  return cudaErrorInvalidValue;  // (a rank above QMV_MAX_RANK)
}

template <int DT>
static cudaError_t launch_dt(const LoraParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3(p.splits, p.n_tok), dim3(LORA_THREADS), (size_t)LORA_TOK * p.window * sizeof(float), stream, true);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, lora_down_kernel<DT>, p);
  if (e != cudaSuccess) return e;
  if constexpr (DT != QMV_DT_F32)
    if (p.r % 8 == 0) return launch_vw<DT, 8>(p, stream);
  return launch_vw<DT, 4>(p, stream);
}

cudaError_t launch_lora(int dtype, LoraParams p, cudaStream_t stream) {
  p.window = lora_window(p.K, p.n_tok);
  p.splits = lora_splits(p.K, p.n_tok);
  switch (dtype) {
    case QMV_DT_F16: return launch_dt<QMV_DT_F16>(p, stream);
    case QMV_DT_BF16: return launch_dt<QMV_DT_BF16>(p, stream);
    default: return launch_dt<QMV_DT_F32>(p, stream);
  }
}

}  // namespace qmv
