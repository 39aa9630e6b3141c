// Low-rank adapters of many requests beside a shared projection:
// y = res + scale_a B_a (A_a x), each token with its own adapter a.
#include "float_io.cuh"
#include "launch.h"
#include "step_launch.h"

namespace qmv {

constexpr int LORA_WARPS = 4, LORA_THREADS = 32 * LORA_WARPS;
constexpr int LORA_CTAS = 4;     // CTAs an SM
constexpr int LORA_CLUSTER = 8;  // CTAs of a cluster, where one launch does both products
constexpr int LORA_TOK = 4;      // tokens of one adapter that a CTA takes
constexpr int LORA_COLS = 8;     // consecutive columns a lane
constexpr int LORA_WIN = 32 * LORA_COLS;
constexpr int LORA_ROWS = 4;     // rows of A a warp holds sums for
constexpr int LORA_SMS = 152;    // what the splits of the columns are made for (on any device: they decide the sums' order)

// The tokens of one CTA (or cluster): up to LORA_TOK with the same adapter, and what
// part of their work is its own.  The tokens of each adapter (and those without one)
// form groups of LORA_TOK in their order; the call's CTAs are dealt out to the groups,
// which only the device knows.
struct LoraTokens {
  int a;             // the adapter, -1: none
  int rank;          // how much of it counts
  int n;             // 0: nothing left for it
  int part, parts;   // its part of its group's work
  int tok[LORA_TOK];
};
// (every warp of a CTA comes by them alone: a lane has tokens `lane` and `lane` + 32)
__device__ __forceinline__ LoraTokens lora_tokens(const LoraParams& p, int unit, int units) {
  const int lane = threadIdx.x & 31;
  int id[2], before[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int k = lane + 32 * i;
    id[i] = k < p.n_tok ? __ldcg(p.ids + k) : -2;
    if (k < p.n_tok && (id[i] < 0 || id[i] >= p.n)) {
      if (id[i] >= p.n && unit == 0) set_error(p.err, QMV_DEVERR_ADAPTER);
      id[i] = -1;
    }
  }
  // (the ranks travel while the groups are formed)
  int rank[2];
#pragma unroll
  for (int i = 0; i < 2; i++) rank[i] = id[i] >= 0 && p.ranks ? __ldcg(p.ranks + id[i]) : p.r;
  // tokens of the same adapter before the lane's
  const unsigned below = (1u << lane) - 1;
  before[0] = __popc(__match_any_sync(0xffffffffu, id[0]) & below);
  if (p.n_tok > 32) {
    before[1] = __popc(__match_any_sync(0xffffffffu, id[1]) & below);
#pragma unroll
    for (int j = 0; j < 32; j++) before[1] += __shfl_sync(0xffffffffu, id[0], j) == id[1];
  }
  const unsigned lead0 = __ballot_sync(0xffffffffu, lane < p.n_tok && before[0] % LORA_TOK == 0);
  const unsigned lead1 = __ballot_sync(0xffffffffu, lane + 32 < p.n_tok && before[1] % LORA_TOK == 0);
  const int first = __popc(lead0), groups = first + __popc(lead1);
  const int g = unit % groups;
  // the group's first token: the g-th of those that lead one
  const unsigned at0 = __ballot_sync(0xffffffffu, (lead0 >> lane & 1) && __popc(lead0 & below) == g);
  const unsigned at1 = __ballot_sync(0xffffffffu, (lead1 >> lane & 1) && first + __popc(lead1 & below) == g);
  const int t = at0 ? __ffs(at0) - 1 : __ffs(at1) + 31;
  LoraTokens q;
  q.a = __shfl_sync(0xffffffffu, t < 32 ? id[0] : id[1], t & 31);
  q.part = unit / groups;
  q.parts = units / groups;
  unsigned long long same = (unsigned long long)__ballot_sync(0xffffffffu, id[1] == q.a) << 32 |
                            __ballot_sync(0xffffffffu, id[0] == q.a);
  same &= ~0ull << t;
  q.n = 0;
#pragma unroll
  for (int i = 0; i < LORA_TOK; i++) {
    q.tok[i] = same ? __ffsll(same) - 1 : t;
    if (same) q.n = i + 1;
    same &= same - 1;
  }
  if (q.part >= q.parts) q.n = 0;
  q.rank = min(max(__shfl_sync(0xffffffffu, t < 32 ? rank[0] : rank[1], t & 31), 0), p.r);
  return q;
}
// v = A x: part[split][token][row], each over one split of the columns.  The work
// of a group of tokens is (split, four rows) units; a CTA takes a run of rows of one
// split, a warp every fourth unit of it, and a lane has 8 columns of each window of
// 256.  The next windows' rows are on their way while one is worked on, across
// units.  The four rows' sums for up to four tokens are added over the lanes
// together (16 shuffles for 16 sums).  x of the CTA's tokens lies in shared memory.
// Adapter rows are read once per four of its tokens.
//
// Bound by latency and HBM: 64 adapters of rank 64, K 5120 (42 MB) 13.8 us by itself, 3.1 TB/s:
// ids, ranks and first loads in turn, then a warp has two units of five windows.
template <int DT, int NT, class Store>
__device__ __forceinline__ void lora_down(const LoraParams& p, const LoraTokens& q, float* lora_x, int split, int nth,
                                          int of, Store store) {
  using T = typename Elem<DT>::type;
  using Row = Packed<T, LORA_COLS>;
  constexpr int AHEAD = DT == QMV_DT_F32 ? 1 : 2;  // windows on their way: 4 KB a warp
  constexpr int SUMS = LORA_ROWS * NT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = q.rank;
  // the nth of `of` runs of units
  const int units = (rank + LORA_ROWS - 1) / LORA_ROWS;
  const int u0 = units * nth / of, u1 = units * (nth + 1) / of;
  if (nth >= of || u0 == u1) return;  // (the whole CTA)
  const int c0 = split * p.window, cols = min(p.window, p.K - c0), wins = (cols + LORA_WIN - 1) / LORA_WIN;
  const T* A = static_cast<const T*>(p.A) + (long long)q.a * p.r * p.K + c0 + lane * LORA_COLS;
  Row w[AHEAD][LORA_ROWS];
  // The loads go through (unit, window) in order, AHEAD of the sums.
  int next_unit = u0 + warp, next_win = 0;
  const T* next = A + (long long)next_unit * LORA_ROWS * p.K;
  auto fetch = [&](Row& x, int i) {  // row i of the next unit's next window
    x.clear();
    if (next_unit < u1 && next_unit * LORA_ROWS + i < rank && next_win * LORA_WIN + lane * LORA_COLS < cols &&
        QMV_CHECK(in_range(next + (long long)i * p.K - static_cast<const T*>(p.A), LORA_COLS, p.a_len, p.err)))
      x.load(next + (long long)i * p.K);
  };
  auto advance = [&]() {
    next += LORA_WIN;
    if (++next_win == wins) {
      next_win = 0;
      next_unit += LORA_WARPS;
      next = A + (long long)next_unit * LORA_ROWS * p.K;
    }
  };
#pragma unroll
  for (int u = 0; u < AHEAD; u++) {
#pragma unroll
    for (int i = 0; i < LORA_ROWS; i++) fetch(w[u][i], i);
    advance();
  }
  // (asynchronous copies: all on their way at once; past the columns they write zeros)
  for (int i = 4 * tid; i < p.window; i += 4 * LORA_THREADS)
#pragma unroll
    for (int k = 0; k < NT; k++)
      if (k < q.n) {
        const bool in = i < cols && QMV_CHECK(in_range((long long)q.tok[k] * p.K + c0 + i, 4, p.x_len, p.err));
        const float* from = p.x + (in ? (long long)q.tok[k] * p.K + c0 + i : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(lora_x + k * p.window + i)), "l"(from),
                     "r"(in ? 16 : 0)
                     : "memory");
      }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  int win = 0, unit = u0 + warp;
  float acc[LORA_ROWS][NT];
#pragma unroll
  for (int i = 0; i < LORA_ROWS; i++)
#pragma unroll
    for (int k = 0; k < NT; k++) acc[i][k] = 0.f;
  while (unit < u1) {
#pragma unroll
    for (int u = 0; u < AHEAD; u++) {
      if (unit >= u1) break;
      float x[NT][LORA_COLS];
#pragma unroll
      for (int k = 0; k < NT; k++)
        load_vec<LORA_COLS>(lora_x + (k < q.n ? k : 0) * p.window + win * LORA_WIN + lane * LORA_COLS, x[k]);
#pragma unroll
      for (int i = 0; i < LORA_ROWS; i++) {
        float v[LORA_COLS];
        w[u][i].to(v);
        fetch(w[u][i], i);
#pragma unroll
        for (int k = 0; k < NT; k++)
#pragma unroll
          for (int e = 0; e < LORA_COLS; e++) acc[i][k] = fmaf(v[e], x[k][e], acc[i][k]);
      }
      advance();
      if (++win < wins) continue;
      // The unit's sums over the lanes, by lane bits 3, 2, 1, 0, 4 (one order for any
      // number of sums): halves the sums that a lane holds at each step, down to one.
      float* s = &acc[0][0];
      int have = SUMS;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        if (have > 1) {
          have /= 2;
          const bool up = lane & o;
#pragma unroll
          for (int i = 0; i < SUMS / 2; i++)
            if (i < have) {
              const float give = up ? s[i] : s[i + have], keep = up ? s[i + have] : s[i];
              s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        } else {
          s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
        }
      }
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], 16);
      constexpr int SHARE = 16 / SUMS;  // lanes that end with the same sum
      const int at = (lane & 15) / SHARE, j = unit * LORA_ROWS + at / NT, k = at % NT;
      if (lane < 16 && lane % SHARE == 0 && j < rank && k < q.n) store(k, j, s[0]);
      win = 0;
      unit += LORA_WARPS;
#pragma unroll
      for (int i = 0; i < LORA_ROWS; i++)
#pragma unroll
        for (int k2 = 0; k2 < NT; k2++) acc[i][k2] = 0.f;
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(LORA_THREADS, LORA_CTAS) lora_down_kernel(const LoraParams p) {
  extern __shared__ __align__(16) float lora_x[];  // [LORA_TOK][window]
  // The second kernel may start (and read the adapters' other half) once what came
  // before this call is done.
  pdl_wait();
  pdl_launch_dependents();
  const LoraTokens q = lora_tokens(p, blockIdx.x, gridDim.x);
  if (q.n == 0 || q.a < 0) return;
  const int split = q.part % p.splits, nth = q.part / p.splits, of = q.parts / p.splits;
  auto store = [&](int k, int j, float sum) {
    int tok = q.tok[0];
#pragma unroll
    for (int i = 1; i < LORA_TOK; i++)
      if (i == k) tok = q.tok[i];
    const long long at = ((long long)split * p.n_tok + tok) * p.r + j;
    if (QMV_CHECK(in_range(at, 1, p.part_len, p.err))) p.part[at] = sum;
  };
  if (q.n == 1) lora_down<DT, 1>(p, q, lora_x, split, nth, of, store);
  else if (q.n == 2) lora_down<DT, 2>(p, q, lora_x, split, nth, of, store);
  else lora_down<DT, LORA_TOK>(p, q, lora_x, split, nth, of, store);
}

// y = res + scale B v: v's parts (part(k, j, s) once ready() returns) are added in
// order, then each warp goes through rows of its own, eight loads of 16 bytes a lane on
// their way (the first ones before ready()).  A row of B lies with 2^lpr_log lanes, VW
// values each; the partial sums of `gather` loads are added over those lanes
// together, so that afterwards each lane has one row's sum and up to 32 consecutive
// rows of y and res are read and written at once.
//
// A kernel holds the variants of one, two and four tokens, and the widest takes all 128
// registers: 76 bytes spill (132 are read back) for bfloat16 with 8 lanes a row, the rank
// 64 of the cases below, and 160 (220) in lora_both_kernel with 2 lanes, rank 16.
//
// Bound by HBM for many adapters: 64 of rank 64, M 17408 (152 MB) 32.8 us by itself, 4.6 TB/s,
// both products 37.6; a few groups of tokens by the chain of ids, v's parts, rows and res:
// 24 tokens on 10 adapters (21 MB in all) 16.7 us.  Tokens that share an adapter are far
// from their bytes: each group of four reads and converts it anew (64 tokens on one, 13 MB
// in all, 18.9 us; on eight 21.2).
template <int DT, int VW, int LPR_LOG, int NT, class Ready, class Part>
__device__ __forceinline__ void lora_up(const LoraParams& p, const LoraTokens& q, float (&v)[LORA_TOK][QMV_MAX_RANK],
                                        long long m0, int rows, Ready ready, Part part) {
  using T = typename Elem<DT>::type;
  using Row = Packed<T, VW>;
  constexpr int LPR = 1 << LPR_LOG, RPL = 32 >> LPR_LOG;               // lanes a row, rows a load
  constexpr int GATHER_LOG = LPR_LOG < 3 ? LPR_LOG : 3, GATHER = 1 << GATHER_LOG;
  constexpr int LOADS = 8, BLOCK = GATHER * RPL;                       // rows whose sums are gathered at once
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = q.rank;
  const int li = lane & (LPR - 1), j0 = li * VW, sub = lane >> LPR_LOG;
  const bool ragged = rank % VW != 0;  // a lane's values may end at the rank
  const T* B = static_cast<const T*>(p.B) + ((long long)q.a * p.M + m0 + sub) * p.r + j0;
  // rows that the lane may load: none past its adapter's rank
  const int live = j0 < rank ? rows - sub : 0, step = RPL * p.r;
  Row w[LOADS];
  auto fetch = [&](Row& x, const T* at, int m) {
    x.clear();
    if (m < live && QMV_CHECK(in_range(at - static_cast<const T*>(p.B), VW, p.b_len, p.err))) x.load(at);
  };
#pragma unroll
  for (int i = 0; i < LOADS; i++) fetch(w[i], B + i * step, i * RPL);
  // The row of a block whose sum ends up here; res of the next blocks' rows is on its way
  // too (asked for where it is used, 64 adapters of rank 16 took 20.4 us instead of 17.0).
  const int mine = (li & (GATHER - 1)) * RPL + sub;
  const bool writer = LPR <= GATHER || li < GATHER;
  constexpr int BLOCKS = LOADS / GATHER, RES = BLOCKS < 8 / NT ? BLOCKS : 8 / NT;
  const float* from[NT];
  float* y[NT];
  float res[RES][NT];
#pragma unroll
  for (int k = 0; k < NT; k++) {
    from[k] = p.res + q.tok[k] * p.M + m0 + mine;
    y[k] = p.y + q.tok[k] * p.M + m0 + mine;
  }
  auto fetch_res = [&](float(&x)[NT], int row) {
#pragma unroll
    for (int k = 0; k < NT; k++)
      if (writer && row + mine < rows && k < q.n && QMV_CHECK(in_range(from[k] + row - p.res, 1, p.n_tok * p.M, p.err)))
        x[k] = from[k][row];
  };
#pragma unroll
  for (int i = 0; i < RES; i++) {
#pragma unroll
    for (int k = 0; k < NT; k++) res[i][k] = 0.f;
    fetch_res(res[i], i * BLOCK);
  }
  const float scale = p.scales ? __ldcg(p.scales + q.a) : 1.0f;
  ready();
  for (int i = tid; i < NT * p.r; i += LORA_THREADS) {
    const int k = i / p.r, j = i - k * p.r;
    float sum = 0.f;
    if (k < q.n && j < rank) {
#pragma unroll 8
      for (int s = 0; s < p.splits; s++) sum += part(k, j, s);
    }
    v[k][j] = sum * scale;
  }
  __syncthreads();
  float x[NT][VW];
#pragma unroll
  for (int k = 0; k < NT; k++)
#pragma unroll
    for (int e = 0; e < VW; e++) x[k][e] = j0 + e < rank && k < q.n ? v[k][j0 + e] : 0.f;
  for (int m = 0; m < rows; m += LOADS * RPL) {
    B += LOADS * step;
#pragma unroll
    for (int g = 0; g < LOADS / GATHER; g++) {
      float acc[NT][GATHER], r[NT];
      const int row = m + g * BLOCK;
      const bool here = writer && row + mine < rows;
#pragma unroll
      for (int k = 0; k < NT; k++) r[k] = res[g % RES][k];
      fetch_res(res[g % RES], row + RES * BLOCK);
#pragma unroll
      for (int i = 0; i < GATHER; i++) {
        float b[VW];
        w[g * GATHER + i].to(b);
        fetch(w[g * GATHER + i], B + (g * GATHER + i) * step, m + (LOADS + g * GATHER + i) * RPL);
        if (ragged) {
#pragma unroll
          for (int e = 0; e < VW; e++)
            if (j0 + e >= rank) b[e] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < NT; k++) {
          acc[k][i] = 0.f;
#pragma unroll
          for (int e = 0; e < VW; e++) acc[k][i] = fmaf(b[e], x[k][e], acc[k][i]);
        }
      }
#pragma unroll
      for (int k = 0; k < NT; k++) {
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
        if (here && k < q.n && QMV_CHECK(in_range(y[k] + row - p.y, 1, p.y_len, p.err))) y[k][row] = r[k] + acc[k][0];
      }
    }
  }
}

// The rows of a warp, `nth` of `of`: equal runs, multiples of 32.
__device__ __forceinline__ int lora_rows(long long M, long long nth, long long of, long long& m0) {
  const int per = (int)(((M + of - 1) / of + 31) / 32 * 32);
  m0 = min(nth * per, M);
  return (int)min((long long)per, M - m0);
}
// Rows of tokens without an adapter.
__device__ __forceinline__ void lora_copy(const LoraParams& p, const LoraTokens& q, long long m0, int rows) {
  if (p.y == p.res) return;
#pragma unroll
  for (int k = 0; k < LORA_TOK; k++)
    if (k < q.n)
      for (int m = threadIdx.x & 31; m < rows; m += 32)
        if (QMV_CHECK(in_range(q.tok[k] * p.M + m0 + m, 1, p.y_len, p.err)))
          p.y[q.tok[k] * p.M + m0 + m] = p.res[q.tok[k] * p.M + m0 + m];
}

template <int DT, int VW, int LPR_LOG>
__global__ void __launch_bounds__(LORA_THREADS, LORA_CTAS) lora_up_kernel(const LoraParams p) {
  __shared__ float v[LORA_TOK][QMV_MAX_RANK];
  pdl_launch_dependents();
  const LoraTokens q = lora_tokens(p, blockIdx.x, gridDim.x);
  if (q.n == 0) return;  // (more CTAs than the groups' parts)
  long long m0;
  const int rows = lora_rows(p.M, (long long)q.part * LORA_WARPS + (threadIdx.x >> 5), (long long)q.parts * LORA_WARPS, m0);
  if (q.a < 0) {
    pdl_wait();
    lora_copy(p, q, m0, rows);
    return;
  }
  auto ready = [] { pdl_wait(); };
  auto part = [&](int k, int j, int s) {
    int tok = q.tok[0];
#pragma unroll
    for (int o = 1; o < LORA_TOK; o++)
      if (o == k) tok = q.tok[o];
    const long long at = ((long long)s * p.n_tok + tok) * p.r + j;
    return QMV_CHECK(in_range(at, 1, p.part_len, p.err)) ? __ldcg(p.part + at) : 0.f;
  };
  if (q.n == 1) lora_up<DT, VW, LPR_LOG, 1>(p, q, v, m0, rows, ready, part);
  else if (q.n == 2) lora_up<DT, VW, LPR_LOG, 2>(p, q, v, m0, rows, ready, part);
  else lora_up<DT, VW, LPR_LOG, LORA_TOK>(p, q, v, m0, rows, ready, part);
}

// Both products in one launch, for a few tokens: a cluster of eight CTAs forms a
// group's v, a split of the columns each, every CTA's parts going to all of them
// through shared memory, and then its part of the rows.  Several clusters of a group
// form the same v, from L2.
//
// One token, rank 16, 4096 -> 4096: 3.5 us, 4.7 a call from Python (two launches 4.3
// and 7 to 10).
template <int DT, int VW, int LPR_LOG, int NT>
__device__ __forceinline__ void lora_both(const LoraParams& p, const LoraTokens& q, float* lora_x,
                                          float (&v)[LORA_TOK][QMV_MAX_RANK],
                                          float (&parts)[LORA_CLUSTER][LORA_TOK][QMV_MAX_RANK], int rank) {
  auto store = [&](int k, int j, float sum) {
#pragma unroll
    for (int i = 0; i < LORA_CLUSTER; i++) {
      uint32_t to;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(&parts[rank][k][j])), "r"(i));
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(sum) : "memory");
    }
  };
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all CTAs are there
  if (rank < p.splits) lora_down<DT, NT>(p, q, lora_x, rank, 0, 1, store);
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  long long m0;
  const int rows = lora_rows(p.M, ((long long)q.part * LORA_CLUSTER + rank) * LORA_WARPS + (threadIdx.x >> 5),
                             (long long)q.parts * LORA_CLUSTER * LORA_WARPS, m0);
  auto ready = [] { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); };
  auto part = [&](int k, int j, int s) { return parts[s][k][j]; };
  lora_up<DT, VW, LPR_LOG, NT>(p, q, v, m0, rows, ready, part);
}

template <int DT, int VW, int LPR_LOG>
__global__ void __launch_bounds__(LORA_THREADS, LORA_CTAS) lora_both_kernel(const LoraParams p) {
  extern __shared__ __align__(16) float lora_x[];  // [LORA_TOK][window]
  __shared__ float v[LORA_TOK][QMV_MAX_RANK];
  __shared__ float parts[LORA_CLUSTER][LORA_TOK][QMV_MAX_RANK];
  pdl_launch_dependents();
  pdl_wait();
  const int rank = (int)blockIdx.x % LORA_CLUSTER;
  LoraTokens q = lora_tokens(p, blockIdx.x / LORA_CLUSTER, gridDim.x / LORA_CLUSTER);
  // no more clusters of a group than have rows
  const long long rows_each = 32 * LORA_WARPS * LORA_CLUSTER;
  q.parts = (int)min((long long)q.parts, (p.M + rows_each - 1) / rows_each);
  if (q.n == 0 || q.part >= q.parts) return;  // (all CTAs of a cluster alike)
  if (q.a < 0) {
    long long m0;
    const int rows = lora_rows(p.M, ((long long)q.part * LORA_CLUSTER + rank) * LORA_WARPS + (threadIdx.x >> 5),
                               (long long)q.parts * LORA_CLUSTER * LORA_WARPS, m0);
    lora_copy(p, q, m0, rows);
    return;
  }
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (q.n == 1) lora_both<DT, VW, LPR_LOG, 1>(p, q, lora_x, v, parts, rank);
  else if (q.n == 2) lora_both<DT, VW, LPR_LOG, 2>(p, q, lora_x, v, parts, rank);
  else lora_both<DT, VW, LPR_LOG, LORA_TOK>(p, q, lora_x, v, parts, rank);
}

// One launch for both products, in clusters of eight CTAs: where a CTA's share of A is
// at most 64 KB (one token of rank 64, K 5120, 82 KB: 7.7 us, in two launches 5.0) and
// up to 32 tokens (64 on one adapter: 25 us for 18), x of four tokens beside the
// parts in 48 KB of shared memory.
static bool lora_one_launch(long long K, int n_tok, int r, int dtype) {
  const long long window = ((K + LORA_WIN - 1) / LORA_WIN + LORA_CLUSTER - 1) / LORA_CLUSTER * LORA_WIN;
  return n_tok <= 32 && window <= 1536 && window * r * (dtype == QMV_DT_F32 ? 4 : 2) <= 65536;
}

// Columns of a split: windows of 256, at most 8 (x of four tokens in shared memory)
// and at most 16 splits (the second kernel adds them) where that leaves a choice (not
// above 32768 columns, or 18432 with 64 tokens: 8 windows a split, up to 512 splits).
// Taken are those for which a warp has the fewest windows to go through, each token
// taken to have an adapter of its own and its share of four CTAs an SM; fewer
// splits among equals.
static int lora_window(long long K, int n_tok, int r, int dtype) {
  if (lora_one_launch(K, n_tok, r, dtype))
    return (int)(((K + LORA_WIN - 1) / LORA_WIN + LORA_CLUSTER - 1) / LORA_CLUSTER * LORA_WIN);
  const int wins = (int)((K + LORA_WIN - 1) / LORA_WIN), units = (r + LORA_ROWS - 1) / LORA_ROWS;
  const int parts = LORA_CTAS * LORA_SMS / n_tok;
  int best = 8, least = 0;
  for (int want = 1; want <= 16 && want <= wins; want++) {
    const int per = (wins + want - 1) / want, splits = (wins + per - 1) / per;
    if (per > 8 || splits > parts) continue;
    const int of = parts / splits, cost = ((units + of - 1) / of + LORA_WARPS - 1) / LORA_WARPS * per;
    if (!least || cost < least) least = cost, best = per;
  }
  return best * LORA_WIN;
}
int lora_splits(long long K, int n_tok, int r, int dtype) {
  const int w = lora_window(K, n_tok, r, dtype);
  return (int)((K + w - 1) / w);
}

// CTAs of a launch: what the SMs hold at once, but not more than `units` for each
// token, and at least `least` for each.
static unsigned lora_grid(const LoraParams& p, long long units, long long least) {
  long long ctas = (long long)LORA_CTAS * device_sm_count();
  if (ctas > units * p.n_tok) ctas = units * p.n_tok;
  if (ctas < least * p.n_tok) ctas = least * p.n_tok;
  return (unsigned)ctas;
}

template <int DT, int VW, int LPR_LOG>
static cudaError_t launch_up(const LoraParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  if (lora_one_launch(p.K, p.n_tok, p.r, DT)) {
    // clusters: a warp for every 32 rows of each token, as many as the GPU holds at once
    long long clusters = (p.M + 32 * LORA_WARPS * LORA_CLUSTER - 1) / (32 * LORA_WARPS * LORA_CLUSTER) * p.n_tok;
    const long long cap = (long long)LORA_CTAS * device_sm_count() / LORA_CLUSTER;
    if (clusters > cap) clusters = cap;
    if (clusters < p.n_tok) clusters = p.n_tok;  // (one for each group at least)
    make_config(cfg, attr, dim3((unsigned)(clusters * LORA_CLUSTER)), dim3(LORA_THREADS),
                (size_t)LORA_TOK * p.window * sizeof(float), stream, true);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = LORA_CLUSTER;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, lora_both_kernel<DT, VW, LPR_LOG>, p);
  }
  make_config(cfg, attr, dim3(lora_grid(p, (p.M + 32 * LORA_WARPS - 1) / (32 * LORA_WARPS), 1)), dim3(LORA_THREADS), 0, stream,
              true);
  return cudaLaunchKernelEx(&cfg, lora_up_kernel<DT, VW, LPR_LOG>, p);
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
static cudaError_t launch_down(const LoraParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  const long long units = (p.r + LORA_WARPS * LORA_ROWS - 1) / (LORA_WARPS * LORA_ROWS);
  make_config(cfg, attr, dim3(lora_grid(p, p.splits * units, p.splits)), dim3(LORA_THREADS),
              (size_t)LORA_TOK * p.window * sizeof(float), stream, true);
  return cudaLaunchKernelEx(&cfg, lora_down_kernel<DT>, p);
}

template <int DT>
static cudaError_t launch_dt(const LoraParams& p, cudaStream_t stream) {
  if (!lora_one_launch(p.K, p.n_tok, p.r, DT)) {
    const cudaError_t e = launch_down<DT>(p, stream);
    if (e != cudaSuccess) return e;
  }
  if constexpr (DT != QMV_DT_F32)
    if (p.r % 8 == 0) return launch_vw<DT, 8>(p, stream);
  return launch_vw<DT, 4>(p, stream);
}

cudaError_t launch_lora(int dtype, LoraParams p, cudaStream_t stream) {
  p.window = lora_window(p.K, p.n_tok, p.r, dtype);
  p.splits = lora_splits(p.K, p.n_tok, p.r, dtype);
  switch (dtype) {
    case QMV_DT_F16: return launch_dt<QMV_DT_F16>(p, stream);
    case QMV_DT_BF16: return launch_dt<QMV_DT_BF16>(p, stream);
    default: return launch_dt<QMV_DT_F32>(p, stream);
  }
}

}  // namespace qmv
