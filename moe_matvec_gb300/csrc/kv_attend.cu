// Attention over the paged 8-bit cache.
//
// out = softmax(scale q K^T) V for the rows (token, query head) that share a
// kv head.  Every byte of K and V is read once per item = (sequence, kv head,
// up to 8 MT of its rows); up to about 16 rows the kernel is bound by that
// read.  The units of work are tiles of 64 tokens of an item; the CTAs (one
// per SM) take equal contiguous shares of all units of the batch, so ragged
// lengths and single long sequences fill the GPU alike, and an item that
// crosses shares leaves partial results that a second kernel joins in order.
//
// In a CTA the tiles go to the consumer warps in turn, each warp with its own
// running maximum, sum and accumulator, merged when the share leaves the item.
// The page records of a tile (scales, K and V codes: one bulk copy per page)
// land in a ring of stages.  A planner warp works out ahead which records the
// tiles need (32 tiles at a time, a lane each) into a ring of plans; the warp
// that has emptied a stage starts the copies of the tile that comes into it
// next.  So no thread waits for stages to become free, and the fixed cost of a
// copy (about 300 ns for one thread that waits, posts the bytes and copies,
// against 350 ns of HBM time for a 16 KB tile) is spread over the warps.
//
// A consumer's arithmetic (mma.sync m16n8k16, f16 operands, fp32 sums): the
// rows of A are 8 query rows in two f16 parts, q = hi + lo, rows 0-7 hi and
// 8-15 lo, so one MMA gives both products and the padding that 8 rows would
// leave in a 16-row operand does the work of fp32 precision.  B holds codes,
// exact in f16.  The order of the contraction is free, so each lane takes the
// 16-byte pieces that the record layout puts in its reach: for S = q K^T lane
// (r, c) = (lane / 4, lane % 4) reads dimensions 64 h + 16 c .. + 15 of token
// 16 (r / 2) + 2 j + r % 2 of the tile (MMA column r of group j), and S then
// leaves lane c with tokens 16 c .. 16 c + 15 of row r: exactly the slots whose
// V codes are 16 contiguous bytes of dimension 8 n + r.  No shuffle or
// transposition lies between the two products.
#include <limits.h>

#include <atomic>

#include "float_io.cuh"
#include "kv_cache.cuh"
#include "kv_launch.h"
#include "launch.h"

namespace qmv {

#ifndef AT_W
#define AT_W(D, MT) ((D) > 192 ? 6 : 7)
#define AT_SP(D, MT) ((D) > 192 ? 2 : 1)
#define AT_IL(D, MT) 4
#endif
constexpr int AT_TILE = 64;        // tokens of a unit
constexpr int AT_MAX_STAGES = 32;  // the planner stays 32 to 64 tiles ahead
constexpr int AT_PLANS = 64;       // ring of plans, in two halves
constexpr int AT_MAX_CTAS = 320;
constexpr int AT_MAX_MT = 2;
// Softmax weights enter f16 times 2^6 and may exceed 1 by 2^8 (a running
// maximum is only followed when it is left behind by more than that) and, by
// the reference scale, by 2: below 2^15, and 22 bits down to 2^-9 of the
// largest, an error of 2^-31 of it below that.
constexpr float AT_P_SCALE = 64.f;
constexpr float AT_LAZY = 8.f;

// Consumer warps beside the planner warp, and how many of them share a tile
// (each takes 64 / at_split of its tokens).  The quarters of an SM hold whole
// warps: 8 of up to 255 registers a thread, 12 of up to 168 or 16 of up to 128.
__host__ __device__ constexpr int at_warps(int D, int MT) { return AT_W(D, MT); }
__host__ __device__ constexpr int at_split(int D, int MT) { return AT_SP(D, MT); }
// shared-memory bytes from one page record to the next: a lane's V piece of
// page c / (P / 16) must fall into another bank group than its neighbours'
__host__ __device__ constexpr int at_rec_stride(int D, int P) {
  return kv_page_bytes(D, P) + (P == 16 ? 16 : P == 32 ? 48 : 0);
}
__host__ __device__ constexpr int at_stage_bytes(int D, int P) { return AT_TILE / P * at_rec_stride(D, P); }
__host__ __device__ constexpr int at_merge_floats(int D, int MT) { return at_warps(D, MT) * 8 * MT * (D + 8 + 2); }

// A partial result in the workspace: m and l of each row, then the rows.
__host__ __device__ constexpr int at_slot_floats(int D, int MT) { return 8 * MT * (D + 2); }
// What the join needs of CTA c's item that begins in its share and ends in a
// later one's (last < 0: there is none).
struct AttendJoin {
  int last, tbase, row0, nrows, head, pad[3];
};

struct AttendParams {
  KvParams kv;
  const void* q;
  void* out;
  long long q_stride;
  float scale_log2;  // scale * log2(e)
  int dtype, G, n_heads, causal, window;
  const int32_t* sel;
  int n_sel, stages;
  AttendJoin* joins;
  float* slots;  // [CTA][2]
#ifdef QMV_DEBUG
  long long q_len, out_len, sel_len;
#endif
};

struct AttendItem {
  int s, tbase, nrows, row0, head;  // rows row0 .. of the item's row space; row r: token tbase + r / G
  int len;                          // of the sequence
  int tile0, tiles;                 // first tile, units
  int k;                            // the unit asked for
};

// Tiles of a sequence that any of its tokens may see.
__device__ __forceinline__ void seq_tiles(const AttendParams& p, const KvSeq& q, int& tile0, int& tiles) {
  tile0 = p.window > 0 ? max(q.len - q.n - p.window + 1, 0) / AT_TILE : 0;
  tiles = max((q.len + AT_TILE - 1) / AT_TILE - tile0, 1);
}

// Unit u of the batch (base: prefix sums of the sequences' units, or of their
// first tokens when each token has its own pages).
template <int MT>
__device__ __forceinline__ AttendItem locate(const AttendParams& p, const long long* base, const KvSeq* seqs,
                                             long long u) {
  AttendItem it;
  const int H = p.kv.H, R = 8 * MT;
  int lo = 0, hi = p.kv.n_seq;  // base[lo] <= key < base[hi]
  if (p.sel) {
    const int tiles = (p.n_sel * p.kv.P + AT_TILE - 1) / AT_TILE, n_rt = (p.G + R - 1) / R;
    const long long item = u / tiles;
    it.k = (int)(u - item * tiles);
    it.tiles = tiles;
    it.tile0 = 0;
    it.row0 = (int)(item % n_rt) * R;
    const long long th = item / n_rt;
    it.head = (int)(th % H);
    it.tbase = (int)(th / H);
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seqs[mid].t0 <= it.tbase) lo = mid; else hi = mid;
    }
    it.nrows = p.G;
  } else {
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (base[mid] <= u) lo = mid; else hi = mid;
    }
    const KvSeq q = seqs[lo];
    seq_tiles(p, q, it.tile0, it.tiles);
    it.nrows = q.n * p.G;
    const int n_rt = (it.nrows + R - 1) / R;
    const long long local = u - base[lo], item = local / it.tiles;
    it.k = (int)(local - item * it.tiles);
    it.row0 = (int)(item % n_rt) * R;
    it.head = (int)(item / n_rt);
    it.tbase = q.t0;
  }
  it.s = lo;
  it.len = seqs[lo].len;
  return it;
}

// The item after `it`, from its first unit.
template <int MT>
__device__ __forceinline__ void next_item(const AttendParams& p, const KvSeq* seqs, AttendItem& it) {
  it.k = 0;
  it.row0 += 8 * MT;
  if (it.row0 < it.nrows) return;
  it.row0 = 0;
  if (++it.head < p.kv.H) return;
  it.head = 0;
  if (p.sel) {
    it.tbase++;
    while (it.s + 1 < p.kv.n_seq && seqs[it.s + 1].t0 <= it.tbase) it.s++;
  } else {
    do {
      if (++it.s >= p.kv.n_seq) return;  // there is none: the caller is at its last unit
    } while (seqs[it.s].n == 0);
    const KvSeq q = seqs[it.s];
    seq_tiles(p, q, it.tile0, it.tiles);
    it.nrows = q.n * p.G;
    it.tbase = q.t0;
  }
  it.len = seqs[it.s].len;
}

// What a tile is made of: for each of its pages the record's byte offset in
// the cache or -1, and the page's index in the sequence or -1.
struct AttendPlan {
  long long rec[4];
  int idx[4];
  uint32_t bytes, pad[3];
};

// Position of row r's token (the row space of `it`).
__device__ __forceinline__ int row_pos(const AttendParams& p, const AttendItem& it, const KvSeq& q, int r) {
  return q.len - q.n + (it.tbase - q.t0) + r / p.G;
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
__device__ __forceinline__ void store4(void* base, long long at, int dt, const float (&v)[4]) {
  if (dt == QMV_DT_F32) store_vec<4>(static_cast<float*>(base) + at, v);
  else if (dt == QMV_DT_F16) store_vec<4>(static_cast<__half*>(base) + at, v);
  else store_vec<4>(static_cast<__nv_bfloat16*>(base) + at, v);
}

template <int D, int P, int MT>
__global__ void __launch_bounds__((at_warps(D, MT) + 1) * 32, 1) kv_attend_kernel(const AttendParams p) {
  constexpr int W = at_warps(D, MT), SP = at_split(D, MT), NG = W / SP, NJ = 8 / SP;
  // independent products in flight: a chain of MMAs into one accumulator waits
  // for each of them
  constexpr int IL = AT_IL(D, MT);
  constexpr int R = 8 * MT, KS = D / 16, NV = D / 8, MSTRIDE = D + 8;
  constexpr int ppt = AT_TILE / P, rec_stride = at_rec_stride(D, P), stage_bytes = ppt * rec_stride;
  extern __shared__ __align__(128) uint8_t smem[];
  const int S = p.stages, n_seq = p.kv.n_seq;
  // stages | merge rows | merge stats | meta | barriers | prefix sums | sequences
  uint8_t* cur = smem + (size_t)S * stage_bytes;
  float* merge = reinterpret_cast<float*>(cur);
  float* mstat = merge + W * R * MSTRIDE;  // [W][R][2]
  cur += at_merge_floats(D, MT) * sizeof(float);
  AttendPlan* plans = reinterpret_cast<AttendPlan*>(cur);
  cur += AT_PLANS * sizeof(AttendPlan);
  uint64_t* full = reinterpret_cast<uint64_t*>(cur);
  cur += AT_PLANS * sizeof(uint64_t);
  long long* base = reinterpret_cast<long long*>(cur);
  KvSeq* seqs = reinterpret_cast<KvSeq*>(base + n_seq + 1);
  __shared__ long long wtot[W + 1];
  __shared__ uint64_t plan_full[2], plan_done[2];  // of the halves of the ring of plans
  __shared__ int stop;                             // a wait ran out: no copy is started any more

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < AT_PLANS; i++) mbar_init(&full[i], 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(&plan_full[i], 1);
      mbar_init(&plan_done[i], AT_PLANS / 2);
    }
    stop = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (tid == 0) p.joins[blockIdx.x].last = -1;
  // the sequences, and the prefix sums of their units
  long long total = 0;
  for (int c = 0; c < n_seq; c += (W + 1) * 32) {
    const int s = c + tid;
    long long units = 0;
    if (s < n_seq) {
      const KvSeq q = kv_seq(p.kv, s);
      seqs[s] = q;
      int t0, tiles;
      seq_tiles(p, q, t0, tiles);
      units = (long long)((q.n * p.G + R - 1) / R) * p.kv.H * tiles;
    }
    long long inc = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wtot[warp] = inc;
    __syncthreads();
    long long before = total;
#pragma unroll
    for (int i = 0; i <= W; i++) {
      if (i < warp) before += wtot[i];
      total += wtot[i];
    }
    if (s < n_seq) base[s] = before + inc - units;
    __syncthreads();
  }
  if (p.sel) {
    const int tiles = (p.n_sel * P + AT_TILE - 1) / AT_TILE;
    total = (long long)p.kv.n_tok * p.kv.H * ((p.G + R - 1) / R) * tiles;
  }
  const long long share = (total + gridDim.x - 1) / gridDim.x;
  const long long u0 = blockIdx.x * share, u1 = min(total, u0 + share);
  if (u0 >= u1) return;
  if (tid == 0) base[n_seq] = total;
  __syncthreads();

  const int units = (int)(u1 - u0);
  if (warp == W) {
    // ---- planner: lane i plans unit 32 b + i of the share
    for (int b = 0; 32 * b < units; b++) {
      AttendPlan plan;
      plan.bytes = 0;
#pragma unroll
      for (int i = 0; i < 4; i++) plan.rec[i] = plan.idx[i] = -1;
      if (32 * b + lane < units) {
        const AttendItem it = locate<MT>(p, base, seqs, u0 + 32 * b + lane);
        const KvSeq q = seqs[it.s];
        const int rows = min(it.row0 + R, it.nrows) - 1;
        // positions that some row of the item may see: [vis0, vis1)
        const int vis1 = p.causal ? row_pos(p, it, q, rows) + 1 : it.len;
        const int vis0 = p.window > 0 ? row_pos(p, it, q, it.row0) - p.window + 1 : 0;
#pragma unroll
        for (int i = 0; i < ppt; i++) {
          int pg;
          if (p.sel) {
            const int j = it.k * ppt + i;
            const long long at = ((long long)it.tbase * p.kv.H + it.head) * p.n_sel + j;
            pg = j < p.n_sel && QMV_CHECK(in_range(at, 1, p.sel_len, p.kv.err)) ? p.sel[at] : -1;
            if (pg >= p.kv.max_pages) {
              set_error(p.kv.err, QMV_DEVERR_PAGE);
              pg = -1;
            }
            // a token that no sequence covers has no pages
            if (it.tbase < q.t0 || it.tbase >= q.t0 + q.n) pg = -1;
          } else {
            pg = (it.tile0 + it.k) * ppt + i;
          }
          const long long pos = (long long)pg * P;
          if (pg < 0 || pos >= vis1 || pos >= it.len || pos + P <= vis0) continue;
          const int id = kv_page(p.kv, it.s, pg);
          if (id < 0) continue;
          plan.rec[i] = ((long long)id * p.kv.H + it.head) * kv_page_bytes(D, P);
          plan.idx[i] = pg;
          plan.bytes += kv_page_bytes(D, P);
        }
      }
      if (b >= 2 && !mbar_wait(&plan_done[b & 1], (b / 2 - 1) & 1, p.kv.err)) break;
      plans[(32 * b + lane) % AT_PLANS] = plan;
      __syncwarp();
      if (lane == 0) mbar_arrive(&plan_full[b & 1]);
    }
    return;
  }

  // ---- consumers
  const int r = lane >> 2, c = lane & 3;
  const uint64_t policy = policy_evict_first();
  bool dead = false;
  // Barriers are waited for by parity, so a warp may wait for a phase only once
  // the phase before it is known to be complete.  The tiles' barriers belong to
  // the plans (unit m: plan and barrier m % 64), not to the stages, whose
  // successive tiles different warps wait for: when unit m's half of the plans
  // is posted, every unit of the half's former content has been consumed, unit
  // m - 64 among them; and the halves are posted in order, a warp that works on
  // one having seen the one before.
  int posted = -1;  // the last half (of 32 units) known to be posted
  auto planned = [&](int m) {
    if (m >> 5 <= posted) return true;
    if (mbar_wait(&plan_full[(m >> 5) & 1], (m >> 6) & 1, p.kv.err)) {
      posted = m >> 5;
      return true;
    }
    dead = true;
    stop = 1;
    return false;
  };
  // Starts the copies of unit m of the share into stage t, which nothing reads
  // any more (by whole warps; lane 0 posts the bytes and copies).
  auto fill = [&](int m, int t) {
    if (!planned(m)) return;
    if (lane == 0 && *const_cast<volatile int*>(&stop) == 0) {
      const AttendPlan& plan = plans[m % AT_PLANS];
      uint64_t* const bar = &full[m % AT_PLANS];
      mbar_arrive_expect_tx(bar, plan.bytes);
      constexpr uint32_t rb = kv_page_bytes(D, P);
#pragma unroll
      for (int k = 0; k < ppt; k++) {
        const long long at = plan.rec[k];
        if (at < 0) continue;
        uint8_t* dst = smem + t * stage_bytes + k * rec_stride;
        if (QMV_CHECK(in_range(at, rb, p.kv.pages_len, p.kv.err)) && QMV_CHECK(smem_in_range(dst, rb, p.kv.err)))
          bulk_copy_g2s_hint(dst, p.kv.pages + at, rb, bar, policy);
        else
          mbar_complete_tx(bar, rb);
      }
    }
  };
  // SP warps form a group that works on one tile at a time
  const int group = warp / SP, part = warp % SP;
  if (part == 0)
    for (int m = group; m < min(S, units) && !dead; m += NG) fill(m, m);
  long long u = u0;
  int n = group, st = group % S;  // the group's next unit of the share and its stage
  const int st_step = NG % S;
  AttendItem it = locate<MT>(p, base, seqs, u);
  for (; u < u1; next_item<MT>(p, seqs, it)) {
    const KvSeq sq = seqs[it.s];
    const int seg = (int)min((long long)(it.tiles - it.k), u1 - u);  // units of this item in the share
    // q of the lane's rows as A fragments
    uint32_t qa[MT][KS][4];
    float qs[MT];
    int lim[MT], low[MT];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      const int row = it.row0 + 8 * mt + r;
      const bool live = row < it.nrows;
      const int pos = live ? row_pos(p, it, sq, row) : -1;
      lim[mt] = live ? (p.causal ? min(pos + 1, it.len) : it.len) : 0;
      low[mt] = p.window > 0 ? pos - p.window + 1 : INT_MIN;
      const long long at = (long long)(it.tbase + row / p.G) * p.q_stride + (long long)(it.head * p.G + row % p.G) * D;
      float v[KS][4], amax = 0.f;
#pragma unroll
      for (int k = 0; k < KS; k++) {
        const int d0 = 64 * (k >> 2) + 16 * c + 4 * (k & 3);
        v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.f;
        if (live && QMV_CHECK(in_range(at + d0, 4, p.q_len, p.kv.err))) load4(p.q, at + d0, p.dtype, v[k]);
#pragma unroll
        for (int e = 0; e < 4; e++) amax = fmaxf(amax, fabsf(v[k][e]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // the row over a power of two near its largest magnitude (exact), so that
      // two f16 parts hold 22 bits of it
      const int e = min(max((int)(__float_as_uint(amax) >> 23), 1), 253);
      const float down = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e)
      // (the sign of the scale goes into q: a larger product is then a larger logit)
      const float down1 = p.scale_log2 < 0.f ? -down : down;
      qs[mt] = __uint_as_float((uint32_t)e << 23) * fabsf(p.scale_log2);
#pragma unroll
      for (int k = 0; k < KS; k++) {
        split_f16(v[k][0] * down1, v[k][1] * down1, qa[mt][k][0], qa[mt][k][1]);
        split_f16(v[k][2] * down1, v[k][3] * down1, qa[mt][k][2], qa[mt][k][3]);
      }
    }
    float o[MT][NV][4], m[MT], l[MT], vref = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      m[mt] = -INFINITY;
      l[mt] = 0.f;
#pragma unroll
      for (int n = 0; n < NV; n++) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    }

    const int seg_end = (int)(u - u0) + seg;
    for (; n < seg_end; n += NG) {
      if (!dead && planned(n) && !mbar_wait(&full[n % AT_PLANS], (n / AT_PLANS) & 1, p.kv.err)) {
        dead = true;
        stop = 1;
      }
      // a warp whose wait ran out computes nothing more, but keeps meeting the
      // others at the barriers
      if (!dead) {
        const uint8_t* stage = smem + st * stage_bytes;
        // the lane's 16 tokens: a piece of one page
        const int sub = 16 * c / P, idx = plans[n % AT_PLANS].idx[sub];
        const uint8_t* rec = stage + sub * rec_stride;
        float dk = 0.f, dv = 0.f;
        if (idx >= 0) {
          const float2 sc = *reinterpret_cast<const float2*>(rec);
          dk = sc.x;
          dv = sc.y;
        }
        // (of them the warp's: 2 NJ from 16 c + 2 NJ part on)
        const int pos0 = idx < 0 ? INT_MAX - 64 : idx * P + (16 * c) % P + 2 * NJ * part;

        // S = q K^T, group j: tokens 2 j, 2 j + 1 of the lane's, row r
        float s[MT][NJ][2];
        {
          const int ksub = 16 * (r >> 1) / P, kt = (16 * (r >> 1)) % P + (r & 1);
          const uint8_t* krow = stage + ksub * rec_stride + KV_HEADER + kt * 64 + 16 * c + 128 * NJ * part;
#pragma unroll
          for (int jg = 0; jg < NJ; jg += IL) {
            float acc[MT][IL][4];
#pragma unroll
            for (int h = 0; h < D / 64; h++) {
              uint32_t w[IL][4];
#pragma unroll
              for (int i = 0; i < IL; i++) load_words<4>(krow + h * P * 64 + (jg + i) * 128, w[i]);
#pragma unroll
              for (int k = 0; k < 4; k++) {
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
                s[mt][jg + i][0] = acc[mt][i][0] + acc[mt][i][2];
                s[mt][jg + i][1] = acc[mt][i][1] + acc[mt][i][3];
              }
            }
          }
        }
        // tiles at an end of some row's range: products out of it become -inf
        bool inside = true;
#pragma unroll
        for (int mt = 0; mt < MT; mt++) inside = inside && pos0 >= low[mt] && pos0 + 2 * NJ <= lim[mt];
        if (!__all_sync(0xffffffffu, inside)) {
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
#pragma unroll
            for (int j = 0; j < NJ; j++) {
#pragma unroll
              for (int e = 0; e < 2; e++)
                if (pos0 + 2 * j + e >= lim[mt] || pos0 + 2 * j + e < low[mt]) s[mt][j][e] = -INFINITY;
            }
          }
        }
        // values share one reference scale per warp: raised when a page's is over twice it
        float vmax = fmaxf(dv, __shfl_xor_sync(0xffffffffu, dv, 1));
        vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2));
        float vfix = 1.f;
        if (vmax > 2.f * vref) {
          vfix = vref / vmax;
          vref = vmax;
        }
        const float vrel = vref > 0.f ? __fdividef(dv, vref) * AT_P_SCALE : 0.f;
        uint32_t pa[MT][NJ / 2][4];
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
          // the lane's 16 products share one factor to logits in powers of two
          // (not 0: a masked product is -inf)
          const float f = fmaxf(qs[mt] * dk, 0x1p-120f);
          float mx = s[mt][0][0];
#pragma unroll
          for (int j = 0; j < NJ; j++) mx = fmaxf(mx, fmaxf(s[mt][j][0], s[mt][j][1]));
          mx *= f;
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          float fix = vfix;
          if (mx > m[mt] + AT_LAZY || (m[mt] == -INFINITY && mx > m[mt])) {
            const float alpha = ex2(m[mt] - mx);
            fix *= alpha;
            l[mt] *= alpha;
            m[mt] = mx;
          }
          if (__any_sync(0xffffffffu, fix != 1.f)) {
#pragma unroll
            for (int n2 = 0; n2 < NV; n2++) {
              o[mt][n2][0] *= fix, o[mt][n2][1] *= fix, o[mt][n2][2] *= fix, o[mt][n2][3] *= fix;
            }
          }
          const float ms = m[mt] == -INFINITY ? 0.f : m[mt];
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < NJ; j++) {
            const float a = ex2(fmaf(s[mt][j][0], f, -ms)), b = ex2(fmaf(s[mt][j][1], f, -ms));
            sum += a + b;
            split_f16(a * vrel, b * vrel, pa[mt][j >> 1][2 * (j & 1)], pa[mt][j >> 1][2 * (j & 1) + 1]);
          }
          l[mt] += sum;
        }
        // O += P V: k-step kk holds the lane's tokens 4 kk .. + 3
        const uint8_t* vrow = rec + KV_HEADER + P * D + r * P + (16 * c) % P + 2 * NJ * part;
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
              for (int mt = 0; mt < MT; mt++) mma16816(o[mt][ng + i], pa[mt][kk], b0, b1);
            }
          }
        }
      }
      if constexpr (SP > 1) named_sync(2 + group, SP * 32);  // the group has read the tile
      else __syncwarp();
      if (part == 0) {
        if (lane == 0) mbar_arrive(&plan_done[(n >> 5) & 1]);
        if (!dead && n + S < units) fill(n + S, st);
      }
      st += st_step;
      if (st >= S) st -= S;
    }

    // ---- the warps' results of the segment, merged in warp order
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      l[mt] += __shfl_xor_sync(0xffffffffu, l[mt], 1);
      l[mt] += __shfl_xor_sync(0xffffffffu, l[mt], 2);
      if (l[mt] != l[mt]) m[mt] = NAN;  // a row that is no number stays one (its maximum ignores it)
      const int row = warp * R + 8 * mt + r;
      const float back = vref * (1.f / AT_P_SCALE);
      float* dst = merge + row * MSTRIDE + 2 * c;
#pragma unroll
      for (int n2 = 0; n2 < NV; n2++)
        *reinterpret_cast<float2*>(dst + 8 * n2) =
            make_float2((o[mt][n2][0] + o[mt][n2][2]) * back, (o[mt][n2][1] + o[mt][n2][3]) * back);
      if (c == 0) {
        mstat[2 * row] = m[mt];
        mstat[2 * row + 1] = l[mt];
      }
    }
    named_sync(1, W * 32);
    const bool begins = it.k == 0, ends = it.k + seg == it.tiles;
    float* slot = p.slots + (size_t)(2 * blockIdx.x + (begins ? 1 : 0)) * at_slot_floats(D, MT);
    for (int i = tid; i < R * D / 4; i += W * 32) {
      const int row = i / (D / 4), col = 4 * (i % (D / 4));
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; w++) M = fmaxf(M, mstat[2 * (w * R + row)]);
      float acc[4] = {0.f, 0.f, 0.f, 0.f}, L = 0.f;
#pragma unroll
      for (int w = 0; w < W; w++) {
        const float mw = mstat[2 * (w * R + row)];
        if (mw == -INFINITY) continue;  // no visible token in this warp's tiles
        const float f = ex2(mw - M);
        const float4 x = *reinterpret_cast<const float4*>(merge + (w * R + row) * MSTRIDE + col);
        L = fmaf(mstat[2 * (w * R + row) + 1], f, L);
        acc[0] = fmaf(x.x, f, acc[0]);
        acc[1] = fmaf(x.y, f, acc[1]);
        acc[2] = fmaf(x.z, f, acc[2]);
        acc[3] = fmaf(x.w, f, acc[3]);
      }
      if (begins && ends) {
        if (it.row0 + row < it.nrows && it.tbase + (it.row0 + row) / p.G < sq.t0 + sq.n && it.tbase >= sq.t0) {
          const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
          for (int e = 0; e < 4; e++) acc[e] = L > 0.f ? acc[e] * inv : (M != M || L != L ? NAN : 0.f);
          const int rr = it.row0 + row;
          const long long at = ((long long)(it.tbase + rr / p.G) * p.n_heads + it.head * p.G + rr % p.G) * D + col;
          if (QMV_CHECK(in_range(at, 4, p.out_len, p.kv.err))) store4(p.out, at, p.dtype, acc);
        }
      } else {
        if (col == 0) {
          slot[2 * row] = M;
          slot[2 * row + 1] = L;
        }
        *reinterpret_cast<float4*>(slot + 2 * R + row * D + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      }
    }
    if (begins && !ends && tid == 0) {
      const long long item_end = u + it.tiles;
      const bool covered = it.tbase >= sq.t0 && it.tbase < sq.t0 + sq.n;
      AttendJoin j{};
      j.last = covered ? (int)((item_end - 1) / share) : -1;
      j.tbase = it.tbase;
      j.row0 = it.row0;
      j.nrows = it.nrows;
      j.head = it.head;
      p.joins[blockIdx.x] = j;
    }
    named_sync(1, W * 32);  // the merge area may be written again
    u += seg;
  }
  // After a wait that ran out, copies that nobody waits for may be in flight:
  // the CTA keeps its shared memory a while longer than any copy takes.
  if (*const_cast<volatile int*>(&stop)) {
    const long long t0 = clock64();
    while (clock64() - t0 < 1 << 24) {
    }
  }
}

// Joins the partial results of the item that begins in CTA c's share and ends
// in a later one's: slot 1 of c, slot 0 of c + 1 .. last, in that order.  One
// block per (c, row).
template <int D, int MT>
__global__ void __launch_bounds__(D / 4) kv_join_kernel(const AttendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int R = 8 * MT, SLOT = at_slot_floats(D, MT);
  const int c = blockIdx.x, row = blockIdx.y;
  const AttendJoin j = p.joins[c];
  const int rr = j.row0 + row;
  if (j.last <= c || rr >= j.nrows) return;
  const int parts = j.last - c + 1, col = 4 * threadIdx.x;
  float M = -INFINITY, acc[4] = {0.f, 0.f, 0.f, 0.f}, L = 0.f;
  // CHUNK parts at a time, all on their way together (8 kv heads of one
  // sequence share 152 SMs in 19 parts each)
  constexpr int CHUNK = 20;
  for (int i0 = 0; i0 < parts; i0 += CHUNK) {
    float2 st[CHUNK];
    float4 xs[CHUNK];
#pragma unroll
    for (int i = 0; i < CHUNK; i++) {
      const int k = min(i0 + i, parts - 1);
      const float* s = p.slots + (size_t)(2 * (c + k) + (k == 0 ? 1 : 0)) * SLOT;
      st[i] = *reinterpret_cast<const float2*>(s + 2 * row);
      xs[i] = *reinterpret_cast<const float4*>(s + 2 * R + row * D + col);
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < CHUNK; i++)
      if (i0 + i < parts) top = fmaxf(top, st[i].x);
    const float back = M == -INFINITY ? 0.f : ex2(M - top);
    M = top;
    L *= back;
#pragma unroll
    for (int e = 0; e < 4; e++) acc[e] *= back;
#pragma unroll
    for (int i = 0; i < CHUNK; i++) {
      if (i0 + i >= parts) continue;
      const float f = st[i].x == -INFINITY ? 0.f : ex2(st[i].x - M);
      L = fmaf(st[i].y, f, L);
      acc[0] = fmaf(xs[i].x, f, acc[0]);
      acc[1] = fmaf(xs[i].y, f, acc[1]);
      acc[2] = fmaf(xs[i].z, f, acc[2]);
      acc[3] = fmaf(xs[i].w, f, acc[3]);
    }
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
  for (int e = 0; e < 4; e++) acc[e] = L > 0.f ? acc[e] * inv : (M != M || L != L ? NAN : 0.f);
  const long long at = ((long long)(j.tbase + rr / p.G) * p.n_heads + j.head * p.G + rr % p.G) * D + col;
  if (QMV_CHECK(in_range(at, 4, p.out_len, p.kv.err))) store4(p.out, at, p.dtype, acc);
}

size_t kv_attend_ws_bytes(int D) {
  return (size_t)AT_MAX_CTAS * (sizeof(AttendJoin) + 2 * at_slot_floats(D, AT_MAX_MT) * sizeof(float));
}

template <int D, int P, int MT>
static cudaError_t launch_attend(AttendParams& p, cudaStream_t stream) {
  const size_t fixed = at_merge_floats(D, MT) * sizeof(float) + (size_t)(p.kv.n_seq + 1) * sizeof(long long) +
                       (size_t)p.kv.n_seq * sizeof(KvSeq) + AT_PLANS * (sizeof(AttendPlan) + sizeof(uint64_t)) + 256;
  const size_t per_stage = at_stage_bytes(D, P);
  int stages = (int)(((size_t)device_smem_optin() - 1024 - fixed) / per_stage);
  if (stages > AT_MAX_STAGES) stages = AT_MAX_STAGES;
  if (stages < 2) return cudaErrorInvalidConfiguration;
  p.stages = stages;
  const size_t smem = fixed + (size_t)stages * per_stage;
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(configured.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kv_attend_kernel<D, P, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             device_smem_optin() - 1024);
    if (e != cudaSuccess) return e;
    configured.fetch_or(1ull << dev);
  }
  const int sms = device_sm_count(), grid = sms < AT_MAX_CTAS ? sms : AT_MAX_CTAS;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3(grid), dim3((at_warps(D, MT) + 1) * 32), smem, stream, true);
  e = cudaLaunchKernelEx(&cfg, kv_attend_kernel<D, P, MT>, p);
  if (e != cudaSuccess) return e;
  make_config(cfg, attr, dim3(grid, 8 * MT), dim3(D / 4), 0, stream, true);
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, MT>, p);
}

template <int D, int MT>
static cudaError_t launch_attend_p(AttendParams& p, cudaStream_t stream) {
  switch (p.kv.P) {
    case 16: return launch_attend<D, 16, MT>(p, stream);
    case 32: return launch_attend<D, 32, MT>(p, stream);
    default: return launch_attend<D, 64, MT>(p, stream);
  }
}
template <int D>
static cudaError_t launch_attend_d(AttendParams& p, cudaStream_t stream) {
  if constexpr (D <= 128) {
    // rows that share a kv head, on average (with a page list a token's own)
    const long long rows = p.sel ? p.G : ((long long)p.kv.n_tok * p.G + p.kv.n_seq - 1) / p.kv.n_seq;
    if (rows > 8) return launch_attend_p<D, 2>(p, stream);
  }
  return launch_attend_p<D, 1>(p, stream);
}

cudaError_t launch_kv_attend(const KvParams& kv, int D, const AttendArgs& a, cudaStream_t stream) {
  AttendParams p{};
  p.kv = kv;
  p.q = a.q;
  p.out = a.out;
  p.q_stride = a.q_stride;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.dtype = a.dtype;
  p.n_heads = a.n_heads;
  p.G = a.n_heads / kv.H;
  p.causal = a.causal;
  p.window = a.window;
  p.sel = a.sel;
  p.n_sel = a.n_sel;
  p.joins = static_cast<AttendJoin*>(a.ws);
  p.slots = reinterpret_cast<float*>(p.joins + AT_MAX_CTAS);
  QMV_DEBUG_ONLY(p.q_len = (long long)(kv.n_tok - 1) * a.q_stride + (long long)a.n_heads * D;
                 p.out_len = output_extent((long long)kv.n_tok * a.n_heads * D);
                 p.sel_len = a.sel ? (long long)kv.n_tok * kv.H * a.n_sel : 0;)
  switch (D) {
    case 64: return launch_attend_d<64>(p, stream);
    case 128: return launch_attend_d<128>(p, stream);
    case 192: return launch_attend_d<192>(p, stream);
    default: return launch_attend_d<256>(p, stream);
  }
}

}  // namespace qmv
