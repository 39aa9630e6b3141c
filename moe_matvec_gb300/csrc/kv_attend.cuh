// Attention over the paged 8-bit cache.
//
// out = softmax(scale q K^T) V for the rows (token, query head) that share a
// kv head.  Every byte of K and V is read once per item = (sequence, kv head,
// up to 8 or 16 MT of its rows); up to about 16 rows the kernel is bound by that
// read.  The units of work are tiles of 64 tokens of an item; the workers (the
// warps of all SMs, or pairs of them for head_dim above 128) take equal
// contiguous shares of all units of the batch, so ragged lengths and single
// long sequences fill the GPU alike.  Warps never wait for one another: a share
// that ends inside an item leaves its running maximum, sum and accumulator in
// the workspace, and a second kernel joins an item's parts in their order.
// (Batches of few units take a cluster per item and no second kernel instead, see
// clusters_for in kv_attend.cu.)
// (Shares per CTA, merged in shared memory, ended unevenly: a segment's end
// waited for its slowest warp, 2.8 us a tile; 32 x 8192 tokens 77 us.)
//
// A worker feeds itself: the halves of its tiles, K (with the scales) and V, go
// through two stages of its own by bulk copies (one per page and half).
// Once a half is read, the copies of the one that comes into its stage next are
// started, so that K and V of the next tile are on their way while this one is
// computed and no thread waits for a stage to become free.  What the tiles are
// made of is worked out 32 tiles at a time, a lane each.
//
// Measured: 32 sequences of up to 8192 tokens, 40 query and 8 kv heads of 128
// (395 MB): 67 us, 5.9 TB/s, 87% of a copy's bandwidth; one sequence of 131072
// (269 MB): 50 us; one of 1000 (clusters): 8.2 us, of which the copies and products
// of its one tile a worker are 3 and the rest is the launch, dependent loads and
// the join.  16 rows in halves (16 x 8192, 176 MB): 42 us; head_dim 192 / 256 (fp32,
// 132 / 176 MB): 32 / 38 us, 4.0-4.5 TB/s with 34-38% of the issue slots and 27-38%
// of the tensor pipe in use: two warps a scheduler, each of which waits for
// its own chain of codes, products and softmax.
//
// The arithmetic (mma.sync m16n8k16, f16 operands, fp32 sums) has codes, exact
// in f16, in B.  With fp32 queries the rows of A are 8 query rows in two f16
// parts, q = hi + lo, rows 0-7 hi and 8-15 lo, and so are the softmax weights:
// one MMA gives both products, and the padding that 8 rows would leave in a
// 16-row operand does the work of fp32 precision.  Where a kv head has more than
// 8 rows of f16 or bfloat16 queries (HALF) A holds 16 of them: hi alone is q
// then, exactly but for what lies 2^-25 below the row's largest; the weights
// keep their two parts, in two MMAs.
//
// The order of the contraction is free, so each lane takes the 16-byte pieces
// that the record layout puts in its reach: for S = q K^T lane (r, c) = (lane /
// 4, lane % 4) reads dimensions 64 h + 16 c .. + 15 of token 16 (r / 2) + 2 j +
// r % 2 of the tile (MMA column r of group j), and S then leaves lane c with
// tokens 16 c .. 16 c + 15 of row r: exactly the slots whose V codes are 16
// contiguous bytes of dimension 8 n + r.  No shuffle or transposition lies
// between the two products.
#pragma once
#include <limits.h>

#include <atomic>

#include "float_io.cuh"
#include "kv_cache.cuh"
#include "kv_launch.h"
#include "launch.h"

namespace qmv {

constexpr int AT_TILE = 64;  // tokens of a unit
// Stages of a worker: K of one tile while V of the one before is read and the
// other way round.  More bytes in flight cost HBM bandwidth (a bare copy loop:
// 7.2 TB/s with 80 KB in flight per SM, 6.7 with 210); with three stages a
// worker 32 x 8192 tokens of head_dim 128 took 71 us, with two 68.
constexpr int AT_RING = 2;
constexpr int AT_MAX_CTAS = 160;
// What enters f16 for a token of a row is a dv / ref: its softmax weight a = 2^(s -
// m), its page's value scale dv, and the row's own reference ref.  A running
// maximum m is only followed when it is left behind by more than 2^8, so a is below
// 2^8; ref follows the largest a dv / 2^8 of the tokens that the row sees, again
// once that exceeds 2^8 ref.  Times 2^6 / 2^8 the largest product so far lies
// between 2^6 and 2^14, and two f16 parts hold 22 bits of those down to 2^-9 of it
// and leave an error of 2^-31 of it below that.  (One reference for all rows of a
// worker, the largest dv of its pages, would cost rows their bits for pages that
// they do not see or give no weight.)  ref is 2^-125 at least, for the divisions by
// it: an error of less than 2^-132 where the values are too small for that.
constexpr float AT_P_SCALE = 0.25f;  // 2^6 / 2^8
constexpr float AT_LAZY = 8.f;       // powers of two
constexpr float AT_REF_MIN = 0x1p-117f;

// Warps of a CTA: the quarters of an SM hold whole warps, 8 of up to 255
// registers a thread or 12 of up to 168, and q and the accumulators take them.
__host__ __device__ constexpr int at_warps(int D, int MT, bool HALF) { return D * MT <= 64 && !HALF ? 12 : 8; }
// Warps that share a tile: from head_dim 192 on two, each for half the
// dimensions of K and of V (q and the accumulators of all would not fit a
// thread's registers; two warps with half the tokens each spilled, 16 x 8192
// tokens of head_dim 256: 47 us, now 39).  They add their products of q and
// K through shared memory and do the softmax each.
__host__ __device__ constexpr int at_split(int D) { return D > 128 ? 2 : 1; }
__host__ __device__ constexpr int at_exchange_bytes(int NR) { return NR * AT_TILE * 8 * (int)sizeof(float); }
// First dimension of k-step k of a warp (less the lane's 16 c): 64 dimensions a
// four steps, of which two warps share the middle ones of 192.
template <int D>
__device__ __forceinline__ int at_kdim(int part, int k) {
  if (D == 192 && k >= 4) return 64 + 8 * part + 4 * (k - 4);
  return 64 * ((D > 128 ? 2 * part : 0) + (k >> 2)) + 4 * (k & 3);
}
// A stage holds half a tile, K with the scales or V.  For head_dim 64 and pages
// under a tile it holds a whole one: a bulk copy takes an SM about 46 ns however
// small, and two for every page would take longer than the 8 KB of a tile from
// HBM (8 draft tokens on 4000 of head_dim 64 in pages of 16: 22 us, now 20
// with one copy a page; 32 sequences of 8192: 86 us, now 70).
__host__ __device__ constexpr bool at_whole(int D, int P) { return D == 64 && P < AT_TILE; }
// Shared-memory bytes from one page to the next, of K (or the whole record) and
// of V: a lane's V piece of page c / (P / 16) must fall into another bank group
// than its neighbours'.
__host__ __device__ constexpr int at_k_stride(int D, int P) {
  return at_whole(D, P) ? kv_page_bytes(D, P) + (P == 16 ? 16 : 48) : KV_HEADER + P * D;
}
__host__ __device__ constexpr int at_v_stride(int D, int P) {
  return at_whole(D, P) ? at_k_stride(D, P) : P * D + (P == 16 ? 32 : P == 32 ? 64 : 0);
}
__host__ __device__ constexpr int at_stage_bytes(int D, int P) {
  return at_whole(D, P) ? AT_TILE / P * at_k_stride(D, P) : AT_TILE * D + 128;
}

// A part in the workspace: m and l of each of the R rows, then the rows.  Slot 0
// of a worker: the item that its share begins inside of; slot 1: the one that it
// ends inside of.
__host__ __device__ constexpr int at_slot_floats(int D, int R) { return R * (D + 2); }
// What the join needs of an item: the workers first .. last that hold its
// parts (last < first: there is nothing to join), and its rows.
struct AttendJoin {
  int first, last, tbase, row0, nrows, head, pad[2];
};

struct AttendParams {
  KvParams kv;
  const void* q;
  void* out;
  long long q_stride;
  float scale_log2;  // scale * log2(e)
  int dtype, G, n_heads, causal, window;
  const int32_t* sel;
  int n_sel;
  float* slots;       // [worker][2]
  int* n_items;       // items of the batch
  AttendJoin* joins;  // [item]
  int max_items;
  int cluster;  // CL: CTAs of an item
#ifdef QMV_DEBUG
  long long q_len, out_len, sel_len, slots_len;
#endif
};

struct AttendItem {
  int s, tbase, nrows, row0, head;  // rows row0 .. of the item's row space; row r: token tbase + r / G
  KvSeq seq;
  int tile0, tiles;                 // first tile, units
  int k;                            // the unit asked for
  int id;                           // of the batch's items
};

// Tiles of a sequence that any of its tokens may see.
__device__ __forceinline__ void seq_tiles(const AttendParams& p, const KvSeq& q, int& tile0, int& tiles) {
  tile0 = p.window > 0 ? max(q.len - q.n - p.window + 1, 0) / AT_TILE : 0;
  tiles = max((q.len + AT_TILE - 1) / AT_TILE - tile0, 1);
}

// a / b for a >= 0, b > 0: in 32 bits where they do (a 64-bit division is some
// 150 cycles, and a share's first copy waits for four of them).
__device__ __forceinline__ long long divide(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// Unit u of the batch (ids: the sequences' first items; base: prefix sums of the sequences' units or, when each
// token has its own pages, their first tokens).
template <int R>
__device__ __forceinline__ AttendItem locate(const AttendParams& p, const long long* base, const int* ids, long long u) {
  AttendItem it;
  const int H = p.kv.H;
  long long key = u;
  if (p.sel) {
    const int tiles = (p.n_sel * p.kv.P + AT_TILE - 1) / AT_TILE, n_rt = (p.G + R - 1) / R;
    const int item = (int)divide(u, tiles);
    it.k = (int)(u - (long long)item * tiles);
    it.id = item;
    it.tiles = tiles;
    it.tile0 = 0;
    const int th = item / n_rt;
    it.row0 = (item - th * n_rt) * R;
    it.tbase = th / H;
    it.head = th - it.tbase * H;
    it.nrows = p.G;
    key = it.tbase;
  }
  int lo = 0, hi = p.kv.n_seq;  // base[lo] <= key < base[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (base[mid] <= key) lo = mid; else hi = mid;
  }
  it.s = lo;
  it.seq = kv_seq(p.kv, lo);
  if (!p.sel) {
    seq_tiles(p, it.seq, it.tile0, it.tiles);
    it.nrows = it.seq.n * p.G;
    const int n_rt = (it.nrows + R - 1) / R;
    const long long local = u - base[lo];
    const int item = (int)divide(local, it.tiles);
    it.k = (int)(local - (long long)item * it.tiles);
    it.id = ids[lo] + item;
    it.head = item / n_rt;
    it.row0 = (item - it.head * n_rt) * R;
    it.tbase = it.seq.t0;
  }
  return it;
}

// The item after `it`, from its first unit.
template <int R>
__device__ __forceinline__ void next_item(const AttendParams& p, const long long* base, AttendItem& it) {
  it.k = 0;
  it.id++;
  it.row0 += R;
  if (it.row0 < it.nrows) return;
  it.row0 = 0;
  if (++it.head < p.kv.H) return;
  it.head = 0;
  const int n_seq = p.kv.n_seq;
  if (p.sel) {
    it.tbase++;
    while (it.s + 1 < n_seq && base[it.s + 1] <= it.tbase) it.s++;
    it.seq = kv_seq(p.kv, it.s);
  } else {
    do {
      if (++it.s >= n_seq) return;  // there is none: the caller is at its last unit
    } while (base[it.s] == base[it.s + 1]);
    it.seq = kv_seq(p.kv, it.s);
    seq_tiles(p, it.seq, it.tile0, it.tiles);
    it.nrows = it.seq.n * p.G;
    it.tbase = it.seq.t0;
  }
}

// Position of row r's token (the row space of `it`).
__device__ __forceinline__ int row_pos(const AttendParams& p, const AttendItem& it, int r) {
  return it.seq.len - it.seq.n + (it.tbase - it.seq.t0) + r / p.G;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four code bytes (code + 128) as two f16 pairs, exactly: 0x6400 | b is 1024 +
// b, less 1152 is the code.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& a, uint32_t& b) {
  const __half2 off = __half2half2(__ushort_as_half(0x6480u));
  const uint32_t x = __byte_perm(w, 0x64646464u, 0x4140), y = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 hx = __hsub2(*reinterpret_cast<const __half2*>(&x), off);
  const __half2 hy = __hsub2(*reinterpret_cast<const __half2*>(&y), off);
  a = *reinterpret_cast<const uint32_t*>(&hx);
  b = *reinterpret_cast<const uint32_t*>(&hy);
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// (x, y) as two f16 pairs, hi + lo
__device__ __forceinline__ void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the same with a zero sum to start from
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Four consecutive values of a float tensor of type dt.
__device__ __forceinline__ void load4(const void* base, long long at, int dt, float (&v)[4]) {
  if (dt == QMV_DT_F32) load_vec<4>(static_cast<const float*>(base) + at, v);
  else if (dt == QMV_DT_F16) load_vec<4>(static_cast<const __half*>(base) + at, v);
  else load_vec<4>(static_cast<const __nv_bfloat16*>(base) + at, v);
}
// Two consecutive values into one (at even).
__device__ __forceinline__ void store2(void* base, long long at, int dt, float x, float y) {
  if (dt == QMV_DT_F32)
    *reinterpret_cast<float2*>(static_cast<float*>(base) + at) = make_float2(x, y);
  else if (dt == QMV_DT_F16)
    *reinterpret_cast<__half2*>(static_cast<__half*>(base) + at) = __floats2half2_rn(x, y);
  else
    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(base) + at) = __floats2bfloat162_rn(x, y);
}

// Item `id` of a batch dealt out by items, from its first unit; id -1 in the
// answer: there is none.  By a whole warp.  Where sequences have several tokens,
// sequence s owns the row tiles floor(starts[s] G / R) + s .. of each head, at
// least as many as its rows need.
template <int R>
__device__ __forceinline__ AttendItem item_of(const AttendParams& p, int id) {
  AttendItem it;
  it.id = id;
  it.k = 0;
  if (p.kv.starts && !p.sel) {
    const int x = id / p.kv.H;
    it.head = id - x * p.kv.H;
    auto first_tile = [&](int t0, int s) { return (int)((long long)t0 * p.G / R) + s; };
    it.s = last_seq_at_most(p.kv.n_seq, x, [&](int s) { return first_tile(p.kv.starts[s], s); });
    it.seq = kv_seq(p.kv, it.s);
    it.tbase = it.seq.t0;
    it.nrows = it.seq.n * p.G;
    const long long row0 = (long long)(x - first_tile(it.seq.t0, it.s)) * R;
    if (row0 < 0 || row0 >= it.nrows) it.id = -1;
    it.row0 = (int)row0;
    seq_tiles(p, it.seq, it.tile0, it.tiles);
    return it;
  }
  const int n_rt = (p.G + R - 1) / R, th = id / n_rt;
  it.row0 = (id - th * n_rt) * R;
  it.tbase = th / p.kv.H;
  it.head = th - it.tbase * p.kv.H;
  it.s = p.kv.starts ? last_seq_at_most(p.kv.n_seq, it.tbase, [&](int s) { return p.kv.starts[s]; }) : it.tbase;
  it.seq = kv_seq(p.kv, it.s);
  it.nrows = p.sel ? p.G : it.seq.n * p.G;
  if (p.sel) {
    it.tile0 = 0;
    it.tiles = (p.n_sel * p.kv.P + AT_TILE - 1) / AT_TILE;
  } else {
    seq_tiles(p, it.seq, it.tile0, it.tiles);
  }
  return it;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// p of this CTA, in CTA `rank` of the cluster.
__device__ __forceinline__ float2 load_peer(const float* p, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

// Adds parts of a row: M, L and the lane's columns of acc over the parts given
// by load(i, stat, x), N at a time.
template <int E, int N, class Load>
__device__ __forceinline__ void join_row(int parts, Load load, float& M, float& L, float (&acc)[E]) {
  M = -INFINITY, L = 0.f;
#pragma unroll
  for (int e = 0; e < E; e++) acc[e] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += N) {
    float2 st[N];
    float x[N][E];
#pragma unroll
    for (int i = 0; i < N; i++) load(min(i0 + i, parts - 1), st[i], x[i]);
    float top = M;
#pragma unroll
    for (int i = 0; i < N; i++) top = fmaxf(top, st[i].x);
    const float back = M == -INFINITY && L == L ? 0.f : ex2(M - top);
    M = top;
    L *= back;
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] *= back;
#pragma unroll
    for (int i = 0; i < N; i++) {
      if (i0 + i >= parts) continue;
      // (a row that is no number keeps its sum as one)
      const float f = st[i].x == -INFINITY && st[i].y == st[i].y ? 0.f : ex2(st[i].x - M);
      L = fmaf(st[i].y, f, L);
#pragma unroll
      for (int e = 0; e < E; e++) acc[e] = fmaf(x[i][e], f, acc[e]);
    }
  }
}

// Rows of an item, and of a lane's A fragment (its rows r and, with HALF, r + 8).
__host__ __device__ constexpr int at_rows(int MT, bool HALF) { return (HALF ? 16 : 8) * MT; }

// CL: a cluster per item, for batches of few units (see clusters_for): its
// workers share the item's tiles, and its rows are joined through shared memory,
// so that there is no second kernel and no prefix sum of the batch.
template <int D, int P, int MT, bool HALF, bool CL>
__global__ void __launch_bounds__(at_warps(D, MT, HALF) * 32, 1) kv_attend_kernel(const AttendParams p) {
  constexpr int W = at_warps(D, MT, HALF), SP = at_split(D), NG = W / SP, NJ = 8;
  // independent products in flight: a chain of MMAs into one accumulator waits
  // for each of them
  constexpr int IL = MT == 1 ? 4 : 2;
  constexpr int R = at_rows(MT, HALF), NR = HALF ? 2 : 1, ppt = AT_TILE / P;
  constexpr int DW = D / SP, KS = DW / 16, NV = DW / 8;  // dimensions of a warp, of K and of V
  constexpr bool WHOLE = at_whole(D, P);
  constexpr int K_STRIDE = at_k_stride(D, P), V_STRIDE = at_v_stride(D, P), STAGE = at_stage_bytes(D, P);
  constexpr int K_BYTES = KV_HEADER + P * D, V_BYTES = P * D;
  static_assert(ppt * K_STRIDE <= STAGE && (ppt - 1) * V_STRIDE + V_BYTES <= STAGE, "a stage holds either half");
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int S = AT_RING;
  const int n_seq = p.kv.n_seq;
  // stages [group][S] | products [group][SP] (SP > 1) | barriers [group][S] | first units | first items
  constexpr int XCH = SP > 1 ? at_exchange_bytes(NR) : 0;
  uint8_t* cur = smem + (size_t)NG * S * STAGE + NG * SP * XCH;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(cur);
  cur += NG * S * sizeof(uint64_t);
  long long* const base = reinterpret_cast<long long*>(cur);
  int* const ids = reinterpret_cast<int*>(base + n_seq + 1);
  __shared__ long long wtot[W];
  __shared__ int wids[W];
  __shared__ int stop;  // a wait ran out: no copy is started any more

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid < NG * S) mbar_init(&bars[tid], 1);
  if (tid == 0) stop = 0;
  fence_mbar_init();
  pdl_wait();
  const int group = warp / SP, part = warp % SP;
  AttendItem it;
  long long u0 = 0, u1 = 0, share = 1;
  int worker = 0;
  const int ranks = CL ? p.cluster : 1, rank = CL ? blockIdx.x % ranks : 0;
  if constexpr (CL) {
    it = item_of<R>(p, blockIdx.x / ranks);
    if (it.id < 0) return;  // (the whole cluster)
    const int each = (it.tiles + ranks * NG - 1) / (ranks * NG), w = group * ranks + rank;
    u0 = min(w * each, it.tiles);
    u1 = min((w + 1) * each, it.tiles);
    it.k = (int)u0;
    __syncthreads();  // the barriers are there
  } else {
    // the sequences' first units (first tokens) and items
    long long total = 0;
    int items = 0;
    for (int c = 0; c < n_seq; c += W * 32) {
      const int s = c + tid;
      long long units = 0;
      int first = 0, mine = 0;
      if (s < n_seq) {
        const KvSeq q = kv_seq(p.kv, s);
        int t0, tiles;
        seq_tiles(p, q, t0, tiles);
        mine = (q.n * p.G + R - 1) / R * p.kv.H;
        units = (long long)mine * tiles;
        first = q.t0;
      }
      long long inc = units;
      int inc_ids = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        const int w = __shfl_up_sync(0xffffffffu, inc_ids, o);
        if (lane >= o) inc += v, inc_ids += w;
      }
      if (lane == 31) wtot[warp] = inc, wids[warp] = inc_ids;
      __syncthreads();
      long long before = total;
      int before_ids = items;
#pragma unroll
      for (int i = 0; i < W; i++) {
        if (i < warp) before += wtot[i], before_ids += wids[i];
        total += wtot[i], items += wids[i];
      }
      if (s < n_seq) {
        base[s] = p.sel ? first : before + inc - units;
        ids[s] = before_ids + inc_ids - mine;
      }
      __syncthreads();
    }
    if (p.sel) {
      const int tiles = (p.n_sel * P + AT_TILE - 1) / AT_TILE;
      items = p.kv.n_tok * p.kv.H * ((p.G + R - 1) / R);
      total = (long long)items * tiles;
    } else if (tid == 0) {
      base[n_seq] = total;
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) *p.n_items = items;

    // The workers: SP warps that work on one tile at a time; neighbours in number
    // sit on different SMs, so that a small batch spreads.
    share = divide(total + NG * gridDim.x - 1, NG * gridDim.x);
    worker = group * gridDim.x + blockIdx.x;
    u0 = min(worker * share, total);
    u1 = min(total, u0 + share);
  }
  const int units = (int)(u1 - u0);
  if (!CL && units == 0) return;
  const int r = lane >> 2, c = lane & 3;
  uint8_t* const stages = smem + (size_t)group * S * STAGE;
  uint64_t* const full = bars + group * S;
  const uint64_t policy = policy_evict_first();
  bool dead = false;

  // ---- what the units [planned, planned + 32) of the share are made of, a lane
  // each: for each page of the tile its index in the cache and in the sequence
  // (or -1), and the kv head
  int planned = 0, page[ppt], idx[ppt], head = 0;
  auto plan = [&](int from) {
    planned = from;
#pragma unroll
    for (int i = 0; i < ppt; i++) page[i] = idx[i] = -1;
    if (from + lane >= units) return;
    AttendItem x = it;
    if constexpr (CL) x.k = (int)u0 + from + lane;
    else x = locate<R>(p, base, ids, u0 + from + lane);
    head = x.head;
    const int rows = min(x.row0 + R, x.nrows) - 1;
    // positions that some row of the item may see: [vis0, vis1)
    const int vis1 = p.causal ? row_pos(p, x, rows) + 1 : x.seq.len;
    const int vis0 = p.window > 0 ? row_pos(p, x, x.row0) - p.window + 1 : 0;
#pragma unroll
    for (int i = 0; i < ppt; i++) {
      int pg;
      if (p.sel) {
        const int j = x.k * ppt + i;
        const long long at = ((long long)x.tbase * p.kv.H + x.head) * p.n_sel + j;
        // a token that no sequence covers has no pages (its list may hold anything)
        const bool listed = j < p.n_sel && x.tbase >= x.seq.t0 && x.tbase < x.seq.t0 + x.seq.n;
        pg = listed && QMV_CHECK(in_range(at, 1, p.sel_len, p.kv.err)) ? p.sel[at] : -1;
        if (pg >= p.kv.max_pages) {
          set_error(p.kv.err, QMV_DEVERR_PAGE);
          pg = -1;
        }
      } else {
        pg = (x.tile0 + x.k) * ppt + i;
      }
      const long long pos = (long long)pg * P;
      if (pg < 0 || pos >= vis1 || pos >= x.seq.len || pos + P <= vis0) continue;
      page[i] = kv_page(p.kv, x.s, pg);
      idx[i] = page[i] < 0 ? -1 : pg;
    }
  };
  // Starts the copies of half h (unit h / 2 of the share: K, then V; WHOLE: of
  // unit h) into stage st, which nothing reads any more; by whole warps, lane 0
  // of the first posts the bytes and copies.  `now`: the unit that is worked on.
  auto fill = [&](int h, int st, int now) {
    const int t = WHOLE ? h : h >> 1;
    if (t >= units || dead) return;
    if (t - planned >= 32) plan(now);
    const int src = t - planned;
    int pg[ppt];
#pragma unroll
    for (int i = 0; i < ppt; i++) pg[i] = __shfl_sync(0xffffffffu, page[i], src);
    const int hd = __shfl_sync(0xffffffffu, head, src);
    if (part != 0 || lane != 0 || *const_cast<volatile int*>(&stop)) return;
    const bool v = !WHOLE && (h & 1);
    const uint32_t bytes = WHOLE ? K_BYTES + V_BYTES : v ? V_BYTES : K_BYTES;
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < ppt; i++) sum += pg[i] < 0 ? 0u : bytes;
    mbar_arrive_expect_tx(&full[st], sum);
#pragma unroll
    for (int i = 0; i < ppt; i++) {
      if (pg[i] < 0) continue;
      const long long at = ((long long)pg[i] * p.kv.H + hd) * kv_page_bytes(D, P) + (v ? K_BYTES : 0);
      uint8_t* dst = stages + st * STAGE + i * (v ? V_STRIDE : K_STRIDE);
      if (QMV_CHECK(in_range(at, bytes, p.kv.pages_len, p.kv.err)) && QMV_CHECK(smem_in_range(dst, bytes, p.kv.err)))
        bulk_copy_g2s_hint(dst, p.kv.pages + at, bytes, &full[st], policy);
      else
        mbar_complete_tx(&full[st], bytes);
    }
  };
  // The worker has read stage st: half h + S may come into it.
  auto release = [&](int h, int st, int now) {
    if constexpr (SP > 1) named_sync(2 + group, SP * 32);
    else __syncwarp();
    fill(h + S, st, now);
  };
  // A wait that runs out ends the warp's arithmetic, not its steps: it goes on
  // meeting its partner at the barriers.
  auto landed = [&](int st, int phase) {
    if (dead) return;
    if (__all_sync(0xffffffffu, mbar_wait(&full[st], phase, p.kv.err))) return;
    dead = true;
    stop = 1;
  };
  plan(0);
  for (int h = 0; h < S; h++) fill(h, h, 0);
  int tile = 0, st = 0, phase = 0;  // the next unit of the share; stage and phase of its next half
  auto next_stage = [&] {
    if (++st == S) {
      st = 0;
      phase ^= 1;
    }
  };

  long long u = u0;
  if constexpr (!CL) it = locate<R>(p, base, ids, u);
  for (;; next_item<R>(p, base, it)) {
    const int seg = (int)min((long long)(it.tiles - it.k), u1 - u);  // units of this item in the share
    // q of the lane's rows as A fragments
    uint32_t qa[MT][KS][4];
    float qs[MT][NR];
    int lim[MT][NR], low[MT][NR];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
      for (int nr = 0; nr < NR; nr++) {
        const int row = it.row0 + (mt * NR + nr) * 8 + r;
        const bool live = row < it.nrows;
        const int pos = live ? row_pos(p, it, row) : -1;
        lim[mt][nr] = live ? (p.causal ? min(pos + 1, it.seq.len) : it.seq.len) : 0;
        low[mt][nr] = p.window > 0 ? pos - p.window + 1 : INT_MIN;
        const long long at = (long long)(it.tbase + row / p.G) * p.q_stride + (long long)(it.head * p.G + row % p.G) * D;
        float v[KS][4], amax = 0.f;
#pragma unroll
        for (int k = 0; k < KS; k++) {
          const int d0 = at_kdim<D>(part, k) + 16 * c;
          v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.f;
          if (live && QMV_CHECK(in_range(at + d0, 4, p.q_len, p.kv.err))) load4(p.q, at + d0, p.dtype, v[k]);
#pragma unroll
          for (int e = 0; e < 4; e++) amax = fmaxf(amax, fabsf(v[k][e]));
        }
        if constexpr (SP > 1) {  // one scale for the row: the partner's dimensions count too
#pragma unroll
          for (int k = 0; k < KS; k++) {
            const int d0 = at_kdim<D>(1 - part, k) + 16 * c;
            float x[4] = {};
            if (live && QMV_CHECK(in_range(at + d0, 4, p.q_len, p.kv.err))) load4(p.q, at + d0, p.dtype, x);
#pragma unroll
            for (int e = 0; e < 4; e++) amax = fmaxf(amax, fabsf(x[e]));
          }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // the row over a power of two near its largest magnitude (exact), so that
        // two f16 parts hold 22 bits of it
        const int e = min(max((int)(__float_as_uint(amax) >> 23), 1), 253);
        const float down = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e)
        // (the sign of the scale goes into q: a larger product is then a larger logit)
        const float down1 = p.scale_log2 < 0.f ? -down : down;
        qs[mt][nr] = __uint_as_float((uint32_t)e << 23) * fabsf(p.scale_log2);
#pragma unroll
        for (int k = 0; k < KS; k++) {
          if constexpr (HALF) {
            qa[mt][k][nr] = pack_f16(v[k][0] * down1, v[k][1] * down1);
            qa[mt][k][2 + nr] = pack_f16(v[k][2] * down1, v[k][3] * down1);
          } else {
            split_f16(v[k][0] * down1, v[k][1] * down1, qa[mt][k][0], qa[mt][k][1]);
            split_f16(v[k][2] * down1, v[k][3] * down1, qa[mt][k][2], qa[mt][k][3]);
          }
        }
      }
    }
    float o[MT][NV][4], m[MT][NR], l[MT][NR], ref[MT][NR];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
      for (int nr = 0; nr < NR; nr++) {
        m[mt][nr] = -INFINITY;
        l[mt][nr] = 0.f;
        ref[mt][nr] = AT_REF_MIN;
      }
#pragma unroll
      for (int n = 0; n < NV; n++) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    }

    for (const int end = tile + seg; tile < end; tile++) {
      // the lane's 16 tokens are a piece of one page
      const int sub = 16 * c / P;
      int pidx = -1;
#pragma unroll
      for (int i = 0; i < ppt; i++) {
        const int v = __shfl_sync(0xffffffffu, idx[i], tile - planned);
        if (sub == i) pidx = v;
      }
      const int pos0 = pidx < 0 ? INT_MAX - 64 : pidx * P + (16 * c) % P;
      float dk = 0.f, dv = 0.f;
      float s[MT][NR][NJ][2];
      landed(st, phase);
      if (!dead && QMV_CHECK(smem_in_range(stages + st * STAGE, STAGE, p.kv.err))) {
        const uint8_t* stage = stages + st * STAGE;
        if (pidx >= 0) {
          const float2 sc = *reinterpret_cast<const float2*>(stage + sub * K_STRIDE);
          dk = sc.x;
          dv = sc.y;
        }
        // S = q K^T, group j: tokens 2 j, 2 j + 1 of the lane's, row r
        const int ksub = 16 * (r >> 1) / P, kt = (16 * (r >> 1)) % P + (r & 1);
        const uint8_t* krow = stage + ksub * K_STRIDE + KV_HEADER + kt * 64 + 16 * c;
#pragma unroll
        for (int jg = 0; jg < NJ; jg += IL) {
          float acc[MT][IL][4];
#pragma unroll
          for (int h = 0; h < (KS + 3) / 4; h++) {
            constexpr int LAST = KS % 4 ? KS % 4 : 4;  // k-steps of the last 64 dimensions
            const int at = at_kdim<D>(part, 4 * h), here = at / 64 * P * 64 + at % 64;
            uint32_t w[IL][4];
#pragma unroll
            for (int i = 0; i < IL; i++) {
              const uint8_t* from = krow + here + (jg + i) * 128;
              if (h == (KS + 3) / 4 - 1) {
                uint32_t x[LAST];
                load_words<LAST>(from, x);
#pragma unroll
                for (int k = 0; k < LAST; k++) w[i][k] = x[k];
              } else {
                load_words<4>(from, w[i]);
              }
            }
#pragma unroll
            for (int k = 0; k < 4 && 4 * h + k < KS; k++) {
#pragma unroll
              for (int i = 0; i < IL; i++) {
                uint32_t b0, b1;
                codes_to_f16(w[i][k], b0, b1);
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
                  if (h == 0 && k == 0) mma16816_first(acc[mt][i], qa[mt][0], b0, b1);
                  else mma16816(acc[mt][i], qa[mt][4 * h + k], b0, b1);
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < IL; i++) {
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
#pragma unroll
              for (int e = 0; e < 2; e++) {
                if constexpr (HALF) s[mt][0][jg + i][e] = acc[mt][i][e], s[mt][NR - 1][jg + i][e] = acc[mt][i][2 + e];
                else s[mt][0][jg + i][e] = acc[mt][i][e] + acc[mt][i][2 + e];
              }
            }
          }
        }
      }
      float4* const xch = reinterpret_cast<float4*>(smem + (size_t)NG * S * STAGE + (group * SP + part) * XCH) + lane;
      if constexpr (SP > 1) {
#pragma unroll
        for (int nr = 0; nr < NR; nr++) {
#pragma unroll
          for (int j = 0; j < NJ; j += 2)
            xch[(nr * NJ + j) * 16] = make_float4(s[0][nr][j][0], s[0][nr][j][1], s[0][nr][j + 1][0], s[0][nr][j + 1][1]);
        }
      }
      if constexpr (!WHOLE) {
        release(2 * tile, st, tile);
        next_stage();
      }
      if constexpr (SP > 1) {  // (both warps add the same two: their softmax is the same bit for bit)
        const float4* const other = xch + (part ? -1 : 1) * (XCH / 16);
#pragma unroll
        for (int nr = 0; nr < NR; nr++) {
#pragma unroll
          for (int j = 0; j < NJ; j += 2) {
            const float4 x = other[(nr * NJ + j) * 16];
            s[0][nr][j][0] += x.x, s[0][nr][j][1] += x.y, s[0][nr][j + 1][0] += x.z, s[0][nr][j + 1][1] += x.w;
          }
        }
      }
      uint32_t pa[MT][NJ / 2][4], pb[HALF ? MT : 1][NJ / 2][4];
      if (!dead) {
        // tiles at an end of some row's range: products out of it become -inf
        bool inside = true;
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
#pragma unroll
          for (int nr = 0; nr < NR; nr++) inside = inside && pos0 >= low[mt][nr] && pos0 + 2 * NJ <= lim[mt][nr];
        }
        if (!__all_sync(0xffffffffu, inside)) {
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
#pragma unroll
            for (int nr = 0; nr < NR; nr++) {
#pragma unroll
              for (int j = 0; j < NJ; j++) {
#pragma unroll
                for (int e = 0; e < 2; e++)
                  if (pos0 + 2 * j + e >= lim[mt][nr] || pos0 + 2 * j + e < low[mt][nr]) s[mt][nr][j][e] = -INFINITY;
              }
            }
          }
        }
        const float dvm = fminf(dv, 0x1p126f);  // (finite times a weight of 0; no finite scale is as large)
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
          float fix[NR];
#pragma unroll
          for (int nr = 0; nr < NR; nr++) {
            // the lane's products share one factor to logits in powers of two
            // (not 0: a masked product is -inf)
            const float f = fmaxf(qs[mt][nr] * dk, 0x1p-120f);
            float mine = s[mt][nr][0][0];
#pragma unroll
            for (int j = 0; j < NJ; j++) mine = fmaxf(mine, fmaxf(s[mt][nr][j][0], s[mt][nr][j][1]));
            mine *= f;
            float mx = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (mx > m[mt][nr] + AT_LAZY || (m[mt][nr] == -INFINITY && mx > m[mt][nr])) {
              const float alpha = ex2(m[mt][nr] - mx);
              l[mt][nr] *= alpha;
              ref[mt][nr] *= alpha;  // (in place of the sums)
              m[mt][nr] = mx;
            }
            const float ms = m[mt][nr] == -INFINITY ? 0.f : m[mt][nr];
            // the largest of the lanes' pages that the row sees
            float top = fmaxf(ex2(mine - ms - AT_LAZY) * dvm, AT_REF_MIN);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            fix[nr] = 1.f;
            if (top > ref[mt][nr] * 256.f) {
              fix[nr] = __fdividef(ref[mt][nr], top);
              ref[mt][nr] = top;
            }
            // (finite for pages that the row does not see, whose weights are 0)
            const float vrel = fminf(__fdividef(dv, ref[mt][nr]) * AT_P_SCALE, 0x1p127f);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; j++) {
              const float a = ex2(fmaf(s[mt][nr][j][0], f, -ms)), b = ex2(fmaf(s[mt][nr][j][1], f, -ms));
              sum += a + b;
              // HALF: high parts in A's rows of pa, low parts in those of pb
              if constexpr (HALF)
                split_f16(a * vrel, b * vrel, pa[mt][j >> 1][2 * (j & 1) + nr], pb[mt][j >> 1][2 * (j & 1) + nr]);
              else
                split_f16(a * vrel, b * vrel, pa[mt][j >> 1][2 * (j & 1)], pa[mt][j >> 1][2 * (j & 1) + 1]);
            }
            l[mt][nr] += sum;
          }
          if (__any_sync(0xffffffffu, fix[0] != 1.f || fix[NR - 1] != 1.f)) {
#pragma unroll
            for (int n2 = 0; n2 < NV; n2++) {
              o[mt][n2][0] *= fix[0], o[mt][n2][1] *= fix[0];
              o[mt][n2][2] *= fix[NR - 1], o[mt][n2][3] *= fix[NR - 1];
            }
          }
        }
      }
      if constexpr (!WHOLE) landed(st, phase);
      if (!dead) {
        // O += P V: k-step kk holds the lane's tokens 4 kk .. + 3
        const uint8_t* vrow = stages + st * STAGE + (WHOLE ? K_BYTES : 0) + sub * V_STRIDE + (DW * part + r) * P + (16 * c) % P;
#pragma unroll
        for (int ng = 0; ng < NV; ng += IL) {
          uint32_t w[IL][NJ / 2];
#pragma unroll
          for (int i = 0; i < IL; i++) load_words<NJ / 2>(vrow + (ng + i) * 8 * P, w[i]);
#pragma unroll
          for (int kk = 0; kk < NJ / 2; kk++) {
#pragma unroll
            for (int i = 0; i < IL; i++) {
              uint32_t b0, b1;
              codes_to_f16(w[i][kk], b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; mt++) {
                mma16816(o[mt][ng + i], pa[mt][kk], b0, b1);
                if constexpr (HALF) mma16816(o[mt][ng + i], pb[mt][kk], b0, b1);
              }
            }
          }
        }
      }
      release(WHOLE ? tile : 2 * tile + 1, st, tile);
      next_stage();
    }

    // ---- the item's rows, or the share's part of them
    const bool begins = it.k == 0, ends = it.k + seg == it.tiles, whole = begins && ends;
    // (with page lists a token may lie in no sequence: its row is not written)
    const bool covered = it.tbase >= it.seq.t0 && it.tbase < it.seq.t0 + it.seq.n;
    // column pair n2 of the lane's row: o in fp32 times f (the reference put back)
    auto pair = [&](int mt, int nr, int n2, float f) {
      const float(&x)[4] = o[mt][n2];
      return HALF ? make_float2(x[2 * nr] * f, x[2 * nr + 1] * f) : make_float2((x[0] + x[2]) * f, (x[1] + x[3]) * f);
    };
    auto write_slot = [&](float* slot, int mt, int nr) {
      if (CL ? !QMV_CHECK(smem_in_range(slot, at_slot_floats(D, R) * sizeof(float), p.kv.err))
             : !QMV_CHECK(in_range(slot - p.slots, at_slot_floats(D, R), p.slots_len, p.kv.err)))
        return;
      const int row = (mt * NR + nr) * 8 + r;
      if (c == 0 && part == 0) {
        // (the maximum of a row that is no number ignores that)
        slot[2 * row] = l[mt][nr] != l[mt][nr] ? NAN : m[mt][nr];
        slot[2 * row + 1] = l[mt][nr];
      }
      float* dst = slot + 2 * R + row * D + DW * part + 2 * c;
#pragma unroll
      for (int n2 = 0; n2 < NV; n2++) *reinterpret_cast<float2*>(dst + 8 * n2) = pair(mt, nr, n2, ref[mt][nr] * (1.f / AT_P_SCALE));
    };
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
      for (int nr = 0; nr < NR; nr++) {
        l[mt][nr] += __shfl_xor_sync(0xffffffffu, l[mt][nr], 1);
        l[mt][nr] += __shfl_xor_sync(0xffffffffu, l[mt][nr], 2);
      }
    }
    if constexpr (CL) {
      // Parts in the workers' stages (which nothing comes into any more), a CTA's
      // joined by its warps, a row each at a time, into the first; the cluster's
      // parts of a row then by one of its CTAs.
      static_assert(at_slot_floats(D, R) * (int)sizeof(float) <= S * STAGE, "a worker's stages hold its part");
      float* const slot = reinterpret_cast<float*>(stages);
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
#pragma unroll
        for (int nr = 0; nr < NR; nr++) write_slot(slot, mt, nr);
      }
      __syncthreads();
      constexpr int E = D / 32;
      float* const first = reinterpret_cast<float*>(smem);
      float M, L, acc[E];
      auto store = [&](int row) {
        const int rr = it.row0 + row;
        if (!covered || rr >= it.nrows) return;
        const float inv = L > 0.f ? 1.f / L : L != L ? NAN : 0.f;
        const long long at = ((long long)(it.tbase + rr / p.G) * p.n_heads + it.head * p.G + rr % p.G) * D + 2 * lane;
#pragma unroll
        for (int i = 0; i < E / 2; i++)
          if (QMV_CHECK(in_range(at + 64 * i, 2, p.out_len, p.kv.err)))
            store2(p.out, at + 64 * i, p.dtype, acc[2 * i] * inv, acc[2 * i + 1] * inv);
      };
      for (int row = warp; row < R; row += W) {
        join_row<E, NG < 8 ? 4 : 8>(
            NG,
            [&](int g, float2& st, float (&x)[E]) {
              const float* from = first + (size_t)g * (S * STAGE / sizeof(float));
              st = *reinterpret_cast<const float2*>(from + 2 * row);
#pragma unroll
              for (int i = 0; i < E / 2; i++) {
                const float2 v = *reinterpret_cast<const float2*>(from + 2 * R + row * D + 64 * i + 2 * lane);
                x[2 * i] = v.x, x[2 * i + 1] = v.y;
              }
            },
            M, L, acc);
        if (ranks == 1) {
          store(row);
          continue;
        }
        __syncwarp();
        if (lane == 0) *reinterpret_cast<float2*>(first + 2 * row) = make_float2(M, L);
#pragma unroll
        for (int i = 0; i < E / 2; i++)
          *reinterpret_cast<float2*>(first + 2 * R + row * D + 64 * i + 2 * lane) = make_float2(acc[2 * i], acc[2 * i + 1]);
      }
      if (ranks > 1) {
        cluster_sync();
        for (int row = rank + warp * ranks; row < R; row += W * ranks) {
          join_row<E, 4>(
              ranks,
              [&](int from, float2& st, float (&x)[E]) {
                st = load_peer(first + 2 * row, from);
#pragma unroll
                for (int i = 0; i < E / 2; i++) {
                  const float2 v = load_peer(first + 2 * R + row * D + 64 * i + 2 * lane, from);
                  x[2 * i] = v.x, x[2 * i + 1] = v.y;
                }
              },
              M, L, acc);
          store(row);
        }
        cluster_sync();  // nobody leaves while its parts are read
      }
      break;
    }
    float* const slots = p.slots + (size_t)worker * 2 * at_slot_floats(D, R);
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
      for (int nr = 0; nr < NR; nr++) {
        const int rr = it.row0 + (mt * NR + nr) * 8 + r;
        if (!whole) {
          write_slot(slots + (begins ? at_slot_floats(D, R) : 0), mt, nr);
        } else if (covered && rr < it.nrows) {
          // (a row that is no number stays one)
          const float back = ref[mt][nr] * (1.f / AT_P_SCALE);
          const float f = l[mt][nr] > 0.f ? back / l[mt][nr] : l[mt][nr] != l[mt][nr] ? NAN : 0.f;
          const long long at = ((long long)(it.tbase + rr / p.G) * p.n_heads + it.head * p.G + rr % p.G) * D + DW * part + 2 * c;
#pragma unroll
          for (int n2 = 0; n2 < NV; n2++) {
            const float2 x = pair(mt, nr, n2, f);
            if (QMV_CHECK(in_range(at + 8 * n2, 2, p.out_len, p.kv.err))) store2(p.out, at + 8 * n2, p.dtype, x.x, x.y);
          }
        }
      }
    }
    if (begins && part == 0 && lane == 0) {
      AttendJoin j{};
      j.first = worker;
      j.last = whole || !covered ? worker - 1 : (int)divide(u + it.tiles - 1, share);
      j.tbase = it.tbase;
      j.row0 = it.row0;
      j.nrows = it.nrows;
      j.head = it.head;
      // (starts that descend can name more items than there is room for, or than 32 bits count)
      if ((unsigned)it.id < (unsigned)p.max_items) p.joins[it.id] = j;
    }
    u += seg;
    if (u >= u1) break;
  }
  // After a wait that ran out, copies that nobody waits for may be in flight:
  // the CTA keeps its shared memory a while longer than any copy takes.
  if (*const_cast<volatile int*>(&stop)) {
    const long long t0 = clock64();
    while (clock64() - t0 < 1 << 24) {
    }
  }
}

// Joins the parts of an item: slot 1 of its first worker, slot 0 of the others,
// in that order (whatever the timing: the result is reproducible).  A
// row is the work of JW warps: each goes over every JW-th part with its lanes
// over the columns, AHEAD parts on their way at a time, and the JW results are
// added in order.  One warp a row, eight rows a block, where there are many
// items (of few parts each); 16 warps, one row a block, where the blocks of a
// few items leave SMs to spare (one sequence of 131072 tokens and 8 kv heads:
// 147 parts an item).
__host__ __device__ constexpr int join_rows(int JW) { return JW == 1 ? 8 : 1; }
template <int D, int R, int JW>
__global__ void __launch_bounds__(join_rows(JW) * JW * 32, JW == 1 ? 1 : 2) kv_join_kernel(const AttendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int SLOT = at_slot_floats(D, R), ROWS = join_rows(JW), AHEAD = JW == 1 ? 8 : 4;
  __shared__ float sm[ROWS][JW][2];
  __shared__ float sx[ROWS][JW][JW > 1 ? D : 1];
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) % JW, rb = threadIdx.x / (32 * JW);
  const int n_items = *p.n_items;
  const AttendJoin j = p.joins[blockIdx.x];
  if ((int)blockIdx.x >= n_items || j.last < j.first) return;
  const int row = blockIdx.y * ROWS + rb, rr = j.row0 + row, parts = j.last - j.first + 1;
  constexpr int E = D / 32;
  float M, L, acc[E];
  join_row<E, AHEAD>(
      (parts - w + JW - 1) / JW,
      [&](int i, float2& st, float (&x)[E]) {
        const int k = w + i * JW;
        const float* s = p.slots + ((size_t)(j.first + k) * 2 + (k == 0 ? 1 : 0)) * SLOT;
        st = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < E; e++) x[e] = 0.f;
        if (!QMV_CHECK(in_range(s - p.slots, SLOT, p.slots_len, p.kv.err))) return;
        st = *reinterpret_cast<const float2*>(s + 2 * row);
#pragma unroll
        for (int q = 0; q < E / 2; q++) {
          const float2 v = *reinterpret_cast<const float2*>(s + 2 * R + row * D + 64 * q + 2 * lane);
          x[2 * q] = v.x;
          x[2 * q + 1] = v.y;
        }
      },
      M, L, acc);
  if constexpr (JW > 1) {
    if (lane == 0) {
      sm[rb][w][0] = M;
      sm[rb][w][1] = L;
    }
#pragma unroll
    for (int e = 0; e < D / 32; e++) sx[rb][w][64 * (e >> 1) + 2 * lane + (e & 1)] = acc[e];
    __syncthreads();
    if (w != 0) return;
    join_row<E, 4>(
        JW,
        [&](int i, float2& st, float (&x)[E]) {
          st = make_float2(sm[rb][i][0], sm[rb][i][1]);
#pragma unroll
          for (int e = 0; e < E; e++) x[e] = sx[rb][i][64 * (e >> 1) + 2 * lane + (e & 1)];
        },
        M, L, acc);
  }
  if (rr >= j.nrows) return;
  const float inv = L > 0.f ? 1.f / L : L != L ? NAN : 0.f;
  const long long at = ((long long)(j.tbase + rr / p.G) * p.n_heads + j.head * p.G + rr % p.G) * D + 2 * lane;
#pragma unroll
  for (int q = 0; q < D / 64; q++)
    if (QMV_CHECK(in_range(at + 64 * q, 2, p.out_len, p.kv.err)))
      store2(p.out, at + 64 * q, p.dtype, acc[2 * q] * inv, acc[2 * q + 1] * inv);
}

// Shared memory of a CTA.
template <int D, int P, int MT, bool HALF>
static size_t attend_smem(int n_seq) {
  constexpr int groups = at_warps(D, MT, HALF) / at_split(D);
  const size_t exchange = at_split(D) > 1 ? at_split(D) * at_exchange_bytes(HALF ? 2 : 1) : 0;
  return (size_t)(n_seq + 1) * (sizeof(long long) + sizeof(int)) + 256 +
         groups * (exchange + AT_RING * (at_stage_bytes(D, P) + sizeof(uint64_t)));
}

template <int D, int P, int MT, bool HALF, bool CL>
static cudaError_t launch_attend(AttendParams& p, cudaStream_t stream) {
  const size_t smem = attend_smem<D, P, MT, HALF>(p.kv.n_seq);
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(configured.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kv_attend_kernel<D, P, MT, HALF, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             device_smem_optin() - 1024);
    if (e != cudaSuccess) return e;
    configured.fetch_or(1ull << dev);
  }
  const int sms = device_sm_count(), grid = sms < AT_MAX_CTAS ? sms : AT_MAX_CTAS;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  constexpr int R = at_rows(MT, HALF);
  if constexpr (CL) {
    make_config(cfg, attr, dim3(p.max_items * p.cluster), dim3(at_warps(D, MT, HALF) * 32), smem, stream, true);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv_attend_kernel<D, P, MT, HALF, CL>, p);
  }
  make_config(cfg, attr, dim3(grid), dim3(at_warps(D, MT, HALF) * 32), smem, stream, true);
  // (exactly as many where a token is an item by itself; else at most)
  const long long each = (p.G + R - 1) / R;
  p.max_items = (int)(p.kv.H * (p.sel || !p.kv.starts
                                    ? each * p.kv.n_tok
                                    : ((long long)p.kv.n_tok * p.G + R - 1) / R + p.kv.n_seq));
  e = cudaLaunchKernelEx(&cfg, kv_attend_kernel<D, P, MT, HALF, CL>, p);
  if (e != cudaSuccess) return e;
  const bool few = (long long)p.max_items * R <= (D == 256 ? 2ll : 4ll) * sms;  // the blocks of 16 warps fit at once
  const int jw = few ? 16 : 1;
  make_config(cfg, attr, dim3(p.max_items, R / join_rows(jw)), dim3(join_rows(jw) * jw * 32), 0, stream, true);
  return few ? cudaLaunchKernelEx(&cfg, kv_join_kernel<D, R, 16>, p)
             : cudaLaunchKernelEx(&cfg, kv_join_kernel<D, R, 1>, p);
}

template <int D, int MT, bool HALF, bool CL>
static cudaError_t launch_attend_p(AttendParams& p, cudaStream_t stream) {
  switch (p.kv.P) {
    case 16: return launch_attend<D, 16, MT, HALF, CL>(p, stream);
    case 32: return launch_attend<D, 32, MT, HALF, CL>(p, stream);
    default: return launch_attend<D, 64, MT, HALF, CL>(p, stream);
  }
}
// Rows that share a kv head, on average (with page lists a token's own).
static long long attend_rows(const AttendParams& p) {
  return p.sel ? p.G : ((long long)p.kv.n_tok * p.G + p.kv.n_seq - 1) / p.kv.n_seq;
}

// Row fragments of a warp.
static int attend_mt(const AttendParams& p, int D, bool half) { return D == 64 && !half && attend_rows(p) > at_rows(1, half) ? 2 : 1; }

template <int D, bool HALF, bool CL>
static cudaError_t launch_attend_d(AttendParams& p, cudaStream_t stream) {
  if constexpr (D == 64 && !HALF)  // (else a second set of fragments and sums would not fit the registers)
    if (attend_mt(p, D, HALF) == 2) return launch_attend_p<D, 2, HALF, CL>(p, stream);
  return launch_attend_p<D, 1, HALF, CL>(p, stream);
}

template <bool HALF, bool CL>
static cudaError_t launch_attend_as(AttendParams& p, int D, cudaStream_t stream) {
  switch (D) {
    case 64: return launch_attend_d<64, HALF, CL>(p, stream);
    case 128: return launch_attend_d<128, HALF, CL>(p, stream);
    case 192: return launch_attend_d<192, HALF, CL>(p, stream);
    default: return launch_attend_d<256, HALF, CL>(p, stream);
  }
}

}  // namespace qmv
