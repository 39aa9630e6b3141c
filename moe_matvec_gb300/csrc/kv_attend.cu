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
// In a CTA one producer warp brings each tile's page records (scales, K and V
// codes: one bulk copy per page) into a ring of stages; the tiles go to the
// consumer warps in turn, each warp with its own running maximum, sum and
// accumulator, merged when the share leaves the item.
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

constexpr int AT_TILE = 64;        // tokens of a unit
constexpr int AT_MAX_STAGES = 32;  // the producer looks ahead by its 32 lanes
constexpr int AT_MAX_CTAS = 320;
constexpr int AT_MAX_MT = 1;
constexpr float AT_P_SCALE = 16384.f;  // softmax weights enter f16 times 2^14, far from its subnormals

// Consumer warps beside the producer warp: as many as the registers of q and
// the accumulators allow (the four quarters of an SM hold whole warps: 12
// warps of up to 168 registers a thread, or 8 of up to 255)
__host__ __device__ constexpr int at_warps(int D) { return D > 128 ? 7 : 11; }
// shared-memory bytes from one page record to the next: a lane's V piece of
// page c / (P / 16) must fall into another bank group than its neighbours'
__host__ __device__ constexpr int at_rec_stride(int D, int P) {
  return kv_page_bytes(D, P) + (P == 16 ? 16 : P == 32 ? 48 : 0);
}
__host__ __device__ constexpr int at_stage_bytes(int D, int P) { return AT_TILE / P * at_rec_stride(D, P); }
__host__ __device__ constexpr int at_merge_floats(int D, int MT) { return at_warps(D) * 8 * MT * (D + 8 + 2); }

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
  int n, len;                       // of the sequence
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
  it.n = seqs[lo].n;
  it.len = seqs[lo].len;
  return it;
}

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

// (x, y) as two f16 pairs, hi + lo
__device__ __forceinline__ void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
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

template <int D, int MT>
__global__ void __launch_bounds__((at_warps(D) + 1) * 32, 1) kv_attend_kernel(const AttendParams p) {
  constexpr int W = at_warps(D), R = 8 * MT, KS = D / 16, NV = D / 8, MSTRIDE = D + 8;
  extern __shared__ __align__(128) uint8_t smem[];
  const int P = p.kv.P, ppt = AT_TILE / P, S = p.stages, n_seq = p.kv.n_seq;
  const int rec_stride = at_rec_stride(D, P), stage_bytes = ppt * rec_stride;
  // stages | merge rows | merge stats | meta | barriers | prefix sums | sequences
  uint8_t* cur = smem + (size_t)S * stage_bytes;
  float* merge = reinterpret_cast<float*>(cur);
  float* mstat = merge + W * R * MSTRIDE;  // [W][R][2]
  cur += at_merge_floats(D, MT) * sizeof(float);
  int* meta = reinterpret_cast<int*>(cur);  // [S][4]: the sequence's page index of each page of the tile, or -1
  cur += S * 16;
  uint64_t* full = reinterpret_cast<uint64_t*>(cur);
  uint64_t* empty = full + S;
  cur += 2 * S * sizeof(uint64_t);
  long long* base = reinterpret_cast<long long*>(cur);
  KvSeq* seqs = reinterpret_cast<KvSeq*>(base + n_seq + 1);
  __shared__ long long wtot[W + 1];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < S; i++) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
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

  if (warp == W) {
    // ---- producer: lane i prepares unit u + i, then the copies go out in order
    const uint64_t policy = policy_evict_first();
    for (long long ub = u0; ub < u1; ub += 32) {
      const long long u = ub + lane;
      int page[4] = {-1, -1, -1, -1}, idx[4] = {-1, -1, -1, -1};
      int head = 0;
      uint32_t bytes = 0;
      if (u < u1) {
        const AttendItem it = locate<MT>(p, base, seqs, u);
        const KvSeq q = seqs[it.s];
        head = it.head;
        const int rows = min(it.row0 + R, it.nrows) - 1;
        // positions that some row of the item may see: [vis0, vis1)
        const int vis1 = p.causal ? row_pos(p, it, q, rows) + 1 : it.len;
        const int vis0 = p.window > 0 ? row_pos(p, it, q, it.row0) - p.window + 1 : 0;
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
          page[i] = id;
          idx[i] = pg;
          bytes += kv_page_bytes(D, P);
        }
      }
      bool dead = false;
      for (int i = 0; i < 32; i++) {
        if (lane == i && u < u1 && !dead) {
          const long long n = u - u0;
          const int st = (int)(n % S);
          const uint32_t use = (uint32_t)(n / S);
          if (use > 0 && !mbar_wait(&empty[st], (use - 1) & 1, p.kv.err)) dead = true;
          if (!dead) {
            *reinterpret_cast<int4*>(meta + 4 * st) = make_int4(idx[0], idx[1], idx[2], idx[3]);
            mbar_arrive_expect_tx(&full[st], bytes);
#pragma unroll
            for (int k = 0; k < 4; k++) {
              if (page[k] < 0) continue;
              const long long at = ((long long)page[k] * p.kv.H + head) * kv_page_bytes(D, P);
              uint8_t* dst = smem + (size_t)st * stage_bytes + k * rec_stride;
              if (QMV_CHECK(in_range(at, kv_page_bytes(D, P), p.kv.pages_len, p.kv.err)) &&
                  QMV_CHECK(smem_in_range(dst, kv_page_bytes(D, P), p.kv.err)))
                bulk_copy_g2s_hint(dst, p.kv.pages + at, kv_page_bytes(D, P), &full[st], policy);
              else
                mbar_complete_tx(&full[st], kv_page_bytes(D, P));
            }
          }
        }
        __syncwarp();
        dead = __any_sync(0xffffffffu, dead);
      }
      if (dead) break;
    }
    return;
  }

  // ---- consumers
  const int r = lane >> 2, c = lane & 3;
  const uint32_t smem0 = smem_u32(smem);
  bool dead = false;
  long long u = u0;
  while (u < u1) {
    const AttendItem it = locate<MT>(p, base, seqs, u);
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
      qs[mt] = __uint_as_float((uint32_t)e << 23) * p.scale_log2;
#pragma unroll
      for (int k = 0; k < KS; k++) {
        split_f16(v[k][0] * down, v[k][1] * down, qa[mt][k][0], qa[mt][k][1]);
        split_f16(v[k][2] * down, v[k][3] * down, qa[mt][k][2], qa[mt][k][3]);
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

    const int first = (int)(u - u0);  // the share's unit number of the segment's first tile
    for (int i = (warp - first % W + W) % W; i < seg; i += W) {
      const int n = first + i, st = n % S;
      if (!dead && !mbar_wait(&full[st], (uint32_t)(n / S) & 1, p.kv.err)) dead = true;
      if (dead) break;
      const uint32_t stage = smem0 + st * stage_bytes;
      // the lane's 16 tokens: a piece of one page
      const int sub = 16 * c / P, idx = meta[4 * st + sub];
      const uint32_t rec = stage + sub * rec_stride;
      float dk = 0.f, dv = 0.f;
      if (idx >= 0) {
        const float2 sc = *reinterpret_cast<const float2*>(smem + (size_t)st * stage_bytes + sub * rec_stride);
        dk = sc.x;
        dv = sc.y;
      }
      const int pos0 = idx < 0 ? INT_MAX - 64 : idx * P + (16 * c) % P;

      // S = q K^T, group j: tokens 16 c + 2 j, + 1 of row r
      float s[MT][8][2];
      {
        const int ksub = 16 * (r >> 1) / P, kt = (16 * (r >> 1)) % P + (r & 1);
        const uint32_t krow = stage + ksub * rec_stride + KV_HEADER + kt * 64 + 16 * c;
#pragma unroll
        for (int j = 0; j < 8; j++) {
          float acc[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; mt++) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
#pragma unroll
          for (int h = 0; h < D / 64; h++) {
            const uint4 kw = lds128(krow + h * P * 64 + j * 128);
            const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
              uint32_t b0, b1;
              codes_to_f16(w[k], b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; mt++) mma16816(acc[mt], qa[mt][4 * h + k], b0, b1);
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            const float f = qs[mt] * dk;
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const int pos = pos0 + 2 * j + e;
              s[mt][j][e] = pos < lim[mt] && pos >= low[mt] ? (acc[mt][e] + acc[mt][2 + e]) * f : -INFINITY;
            }
          }
        }
      }
      // values share one reference scale per warp, the largest so far
      float vmax = fmaxf(dv, __shfl_xor_sync(0xffffffffu, dv, 1));
      vmax = fmaxf(fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2)), vref);
      const float vfix = vmax > 0.f ? vref / vmax : 1.f;
      const float vrel = vmax > 0.f ? dv / vmax * AT_P_SCALE : 0.f;
      vref = vmax;
      uint32_t pa[MT][4][4];
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; j++) mx = fmaxf(mx, fmaxf(s[mt][j][0], s[mt][j][1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[mt], mx), ms = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2(m[mt] - ms), fix = alpha * vfix;
        m[mt] = mn;
        l[mt] *= alpha;
        if (__any_sync(0xffffffffu, fix != 1.f)) {
#pragma unroll
          for (int n2 = 0; n2 < NV; n2++) {
            o[mt][n2][0] *= fix, o[mt][n2][1] *= fix, o[mt][n2][2] *= fix, o[mt][n2][3] *= fix;
          }
        }
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float a = ex2(s[mt][j][0] - ms), b = ex2(s[mt][j][1] - ms);
          sum += a + b;
          split_f16(a * vrel, b * vrel, pa[mt][j >> 1][2 * (j & 1)], pa[mt][j >> 1][2 * (j & 1) + 1]);
        }
        l[mt] += sum;
      }
      // O += P V: k-step kk holds tokens 16 c + 4 kk .. + 3
      const uint32_t vrow = rec + KV_HEADER + P * D + r * P + (16 * c) % P;
#pragma unroll
      for (int n2 = 0; n2 < NV; n2++) {
        const uint4 vw = lds128(vrow + n2 * 8 * P);
        const uint32_t w[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
        for (int kk = 0; kk < 4; kk++) {
          uint32_t b0, b1;
          codes_to_f16(w[kk], b0, b1);
#pragma unroll
          for (int mt = 0; mt < MT; mt++) mma16816(o[mt][n2], pa[mt][kk], b0, b1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
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
  auto part = [&](int i) { return p.slots + (size_t)(2 * (c + i) + (i == 0 ? 1 : 0)) * SLOT; };
  float M = -INFINITY;
#pragma unroll 8
  for (int i = 0; i < parts; i++) M = fmaxf(M, part(i)[2 * row]);
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, L = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; i++) {
    const float* s = part(i);
    const float m = s[2 * row], l = s[2 * row + 1];
    const float4 x = *reinterpret_cast<const float4*>(s + 2 * R + row * D + col);
    const float f = m == -INFINITY ? 0.f : ex2(m - M);
    L = fmaf(l, f, L);
    acc[0] = fmaf(x.x, f, acc[0]);
    acc[1] = fmaf(x.y, f, acc[1]);
    acc[2] = fmaf(x.z, f, acc[2]);
    acc[3] = fmaf(x.w, f, acc[3]);
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

template <int D, int MT>
static cudaError_t launch_attend(AttendParams& p, cudaStream_t stream) {
  const size_t fixed = at_merge_floats(D, MT) * sizeof(float) + (size_t)(p.kv.n_seq + 1) * sizeof(long long) +
                       (size_t)p.kv.n_seq * sizeof(KvSeq) + 256;
  const size_t per_stage = at_stage_bytes(D, p.kv.P) + 16 + 2 * sizeof(uint64_t);
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
    e = cudaFuncSetAttribute(kv_attend_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             device_smem_optin() - 1024);
    if (e != cudaSuccess) return e;
    configured.fetch_or(1ull << dev);
  }
  const int sms = device_sm_count(), grid = sms < AT_MAX_CTAS ? sms : AT_MAX_CTAS;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3(grid), dim3((at_warps(D) + 1) * 32), smem, stream, true);
  e = cudaLaunchKernelEx(&cfg, kv_attend_kernel<D, MT>, p);
  if (e != cudaSuccess) return e;
  make_config(cfg, attr, dim3(grid, 8 * MT), dim3(D / 4), 0, stream, true);
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, MT>, p);
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
    case 64: return launch_attend<64, 1>(p, stream);
    case 128: return launch_attend<128, 1>(p, stream);
    case 192: return launch_attend<192, 1>(p, stream);
    default: return launch_attend<256, 1>(p, stream);
  }
}

}  // namespace qmv
