// Writing tokens into the paged 8-bit cache, and reading them back.
#include <type_traits>

#include "float_io.cuh"
#include "kv_cache.cuh"
#include "kv_launch.h"
#include "launch.h"

namespace qmv {

// The (sequence, page) that an item of the grid stands for; every thread
// returns the same answer, s = -1 for an item that stands for nothing.
// Sequence s of the batch owns items starts[s] / P + 2 s .. starts[s+1] / P +
// 2 (s + 1), at least as many as its new tokens can touch pages ((n - 2) / P +
// 2 for n of them, in the worst place), so the sequence is found from starts
// alone, where prefix sums of the touched pages would need every sequence and
// the block's barriers.
struct KvItem {
  int s, page;  // page: index in the sequence
  KvSeq seq;
};
__device__ __forceinline__ KvItem kv_item(const KvParams& p, int item) {
  KvItem r;
  if (!p.starts) {
    r.s = item;
    r.seq = kv_seq(p, item);
    r.page = max(r.seq.len - 1, 0) >> p.log_p;
    return r;
  }
  auto first_item = [&](int s) { return (p.starts[s] >> p.log_p) + 2 * s; };
  const int lo = last_seq_at_most(p.n_seq, item, first_item);
  r.s = lo;
  r.seq = kv_seq(p, lo);
  const int first = max(r.seq.len - r.seq.n, 0) >> p.log_p;
  r.page = first + max(item - first_item(lo), 0);
  // (page 0 of an empty sequence stays: some block sees to its tokens)
  if (r.seq.n < 1 || r.page > max(r.seq.len - 1, 0) >> p.log_p) r.s = -1;
  return r;
}

// The activation rule's scale, its reciprocal and code.
// (the branch-free forms where they are exact, the IEEE operations else)
__device__ __forceinline__ float rule_scale(float amax) {
  return amax >= 127.0f * 0x1p-126f && amax < INFINITY ? div127_rn(amax) : __fdiv_rn(amax, 127.0f);
}
__device__ __forceinline__ float rule_inv(float d) {
  return d >= 0x1p-126f && d <= 0x1p126f ? rcp_rn(d) : d > 0.f ? __frcp_rn(d) : 0.f;
}
__device__ __forceinline__ int rule_code(float x, float inv) {
  // the conversion takes +-inf to the ends of the int range and NaN to 0
  return min(max(__float2int_rn(__fmul_rn(x, inv)), -127), 127);
}

// Four values' codes as the bytes code + 128.  Where the scale is 0 or large
// enough that |x| / d stays below 127.5 whatever the roundings, adding 1.5 *
// 2^23 + 128 leaves the integer, rounded half to even, in the low mantissa
// bits; else the rule as it is written (`plain`).
__device__ __forceinline__ bool rule_is_plain(float d) { return d > 0.f && !(d >= 0x1p-100f && d < INFINITY); }
template <bool PLAIN>
__device__ __forceinline__ uint32_t rule_bytes(const float (&v)[4], float inv) {
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; j++)
    q[j] = PLAIN ? (uint32_t)(rule_code(v[j], inv) + 128)
                 : __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.0f + 128.0f));
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

// Byte j of w (code + 128) as the float code, exactly: 2^23 + byte, less 2^23 + 128.
__device__ __forceinline__ float byte_code(uint32_t w, int j) {
  return __fsub_rn(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + j)), 8388608.0f + 128.0f);
}

// The codes of four packed bytes (code + 128) under a grown scale.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    o |= (uint32_t)((__float2int_rn(__fmul_rn(byte_code(w, i), ratio)) + 128) & 0xFF) << (8 * i);
  }
  return o;
}
// the same for the first n of the four (the others unchanged)
__device__ __forceinline__ uint32_t rescale4_first(uint32_t w, float ratio, int n) {
  if (n >= 4) return rescale4(w, ratio);
  const uint32_t keep = n <= 0 ? 0xFFFFFFFFu : 0xFFFFFFFFu << (8 * n);
  return (rescale4(w, ratio) & ~keep) | (w & keep);
}

// Four vectors of four values, element (t, j) = token t, dimension j, as four
// words of one dimension's four tokens each.
__device__ __forceinline__ void transpose4(const uint32_t (&w)[4], uint32_t (&o)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  o[0] = __byte_perm(a, b, 0x5410);
  o[1] = __byte_perm(a, b, 0x7632);
  o[2] = __byte_perm(c, d, 0x5410);
  o[3] = __byte_perm(c, d, 0x7632);
}

// Half a CTA takes the keys of a (page, head), the other half the values; a
// thread takes four dimensions of groups of four consecutive slots.  The
// page's new tokens are read once into registers (T as it came); their largest
// magnitude gives the scale; if an old scale has to grow, the old codes are
// rewritten; then the codes are stored, the values' transposed in shared memory
// so that they leave in 16-byte pieces.
// NQ: groups of four slots a thread holds.  Prompts take 256 threads (512 for
// wider heads, whose values would take too many registers): the fewer,
// the smaller the share of finding the page and its scale.  Single tokens (ONE)
// take 128, a group being one slot.  At prompt sizes neither HBM (3.0 TB/s read
// and written) nor the issue slots (62%) are full: a CTA loads its page and then
// packs it, five warps a scheduler, and loads are what they wait for most (2.0
// warps per issue).  Ragged prompts of up to 6000 bfloat16 tokens, 6 sequences, 8
// heads of 128 (122 MB): 29 us, 4.2 TB/s.  Single tokens are bound by latency
// (lens, table, scale, codes one after another): 64 sequences 3.3 us.
template <int DT, int D, bool ONE>
struct AppendShape {
  static constexpr int THREADS = ONE ? 128 : D * sizeof(typename Elem<DT>::type) > 256 ? 512 : 256, HALF = THREADS / 2, COLS = D / 4, TG = HALF / COLS;
  static constexpr int SLOTS = ONE ? 1 : 4;                      // of a group
  static constexpr int NQ = ONE ? 1 : (64 / SLOTS + TG - 1) / TG;  // groups a thread
};

template <int DT, int D, bool ONE>
__global__ void __launch_bounds__(AppendShape<DT, D, ONE>::THREADS, ONE ? 1 : 768 / AppendShape<DT, D, ONE>::THREADS)
    kv_append_kernel(const KvParams p, const void* kx, const void* vx, long long k_stride, long long v_stride) {
  using T = typename Elem<DT>::type;
  using Shape = AppendShape<DT, D, ONE>;
  constexpr int HALF = Shape::HALF, COLS = Shape::COLS, TG = Shape::TG, NQ = Shape::NQ, SLOTS = Shape::SLOTS;
  static_assert(COLS <= HALF, "a thread takes four dimensions");
  using Raw = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;  // four values
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float red[Shape::THREADS / 32];
  __shared__ float lo_s[TG][D], hi_s[TG][D];
  // the values' codes, 16 words of four slots per dimension: word q of dimension
  // dd at q ^ (dd / 4 % 16), so that the lanes' stores fall into different banks
  __shared__ __align__(16) uint32_t vt[ONE ? 4 : D * 16];
  const KvItem it = kv_item(p, (int)(blockIdx.x / (unsigned)p.H));
  if (it.s < 0) return;
  const int head = (int)(blockIdx.x % (unsigned)p.H), P = p.P;  // a token's heads side by side
  const int pos0 = it.seq.len - it.seq.n, page0 = it.page * P;
  const int lo = max(max(pos0, 0) - page0, 0), hi = min(it.seq.len - page0, P);  // the new slots
  if (pos0 < 0 && it.seq.len > 0 && threadIdx.x == 0) set_error(p.err, QMV_DEVERR_BATCH);  // tokens before the first
  if (hi <= lo) return;  // an empty sequence
  const long long tok0 = (long long)it.seq.t0 + page0 - pos0;  // call's token of slot 0
  const int part = threadIdx.x / HALF, u = threadIdx.x % HALF;
  const int col = u % COLS, tg = u / COLS;
  const long long stride = part ? v_stride : k_stride;
  const T* x = static_cast<const T*>(part ? vx : kx) + (long long)head * D + 4 * col;
  // slots of the thread's group q: first_slot(q) .. + SLOTS - 1
  auto first_slot = [&](int q) { return ONE ? lo : 4 * (tg + q * TG); };
  const bool mine = tg < TG && (!ONE || tg == 0);  // the thread has slots
  auto is_new = [&](int t) { return t >= lo && t < hi; };
  // a slot that is not new takes the nearest new one's values: the extremes stay
  // those of the new tokens
  Raw raw[NQ][SLOTS];
  const T* const x0 = x + tok0 * stride;
#pragma unroll
  for (int q = 0; q < NQ; q++) {
#pragma unroll
    for (int i = 0; i < SLOTS; i++) {
      const int t = min(max(first_slot(q) + i, lo), hi - 1);
      raw[q][i] = Raw{};
      if (mine && QMV_CHECK(in_range(tok0 + t, 1, p.n_tok, p.err))) raw[q][i] = *reinterpret_cast<const Raw*>(x0 + t * stride);
    }
  }
  const int phys = kv_page(p, it.s, it.page);
  if (phys < 0) return;
  const int rec_bytes = kv_page_bytes(D, P);
  const long long rec_at = ((long long)phys * p.H + head) * rec_bytes;
  if (!QMV_CHECK(in_range(rec_at, rec_bytes, p.pages_len, p.err))) return;
  uint8_t* rec = p.pages + rec_at;
  float* scales = reinterpret_cast<float*>(rec);
  const float d_old = lo > 0 ? scales[part] : 0.f;
  auto values = [&](const Raw& r, float (&v)[4]) {
    const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = to_float(e[j]);
  };

  float amax = 0.f;
#pragma unroll
  for (int q = 0; q < NQ; q++) {
#pragma unroll
    for (int i = 0; i < SLOTS; i++) {
      float v[4];
      values(raw[q][i], v);
#pragma unroll
      for (int j = 0; j < 4; j++) amax = fmaxf(amax, fabsf(v[j]));
    }
  }
  if (p.bounds && part == 0 && tg < TG) {  // (ONE: a thread of another group has none)
    float mn[4], mx[4];
#pragma unroll
    for (int j = 0; j < 4; j++) mn[j] = INFINITY, mx[j] = -INFINITY;
#pragma unroll
    for (int q = 0; q < NQ; q++) {
#pragma unroll
      for (int i = 0; i < SLOTS; i++) {
        float v[4];
        values(raw[q][i], v);
        if (mine) {
#pragma unroll
          for (int j = 0; j < 4; j++) {
            mn[j] = fminf(mn[j], v[j]);
            mx[j] = fmaxf(mx[j], v[j]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      lo_s[tg][4 * col + j] = mn[j];
      hi_s[tg][4 * col + j] = mx[j];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < HALF / 32; i++) amax = fmaxf(amax, red[part * (HALF / 32) + i]);
  const float d = fmaxf(d_old, rule_scale(amax));
  const float inv = rule_inv(d);
  uint8_t* codes = rec + KV_HEADER + part * P * D;

  const bool grown = lo > 0 && d > d_old;
  const float ratio = lo > 0 && d > 0.f ? __fdiv_rn(d_old, d) : 0.f;
  if (grown) {
    if (part == 0) {  // slots [0, lo) of each group of 64 dimensions: contiguous
      for (int i = u; i < (D / 64) * lo * 4; i += HALF) {
        uint4* c = reinterpret_cast<uint4*>(codes + (size_t)(i / (lo * 4)) * P * 64) + i % (lo * 4);
        uint4 w = *c;
        w.x = rescale4(w.x, ratio), w.y = rescale4(w.y, ratio), w.z = rescale4(w.z, ratio), w.w = rescale4(w.w, ratio);
        *c = w;
      }
    } else {  // the first lo bytes of each dimension
      const int n16 = (lo + 15) / 16;
      for (int i = u; i < D * n16; i += HALF) {
        const int dd = i % D, c16 = i / D, left = lo - 16 * c16;
        uint4* c = reinterpret_cast<uint4*>(codes + dd * P) + c16;
        uint4 w = *c;
        w.x = rescale4_first(w.x, ratio, left), w.y = rescale4_first(w.y, ratio, left - 4);
        w.z = rescale4_first(w.z, ratio, left - 8), w.w = rescale4_first(w.w, ratio, left - 12);
        *c = w;
      }
    }
  }
  // the codes of each slot's four dimensions, code + 128 in each byte
  uint32_t packed[NQ][SLOTS];
  auto pack = [&](auto plain) {
#pragma unroll
    for (int q = 0; q < NQ; q++) {
#pragma unroll
      for (int i = 0; i < SLOTS; i++) {
        float v[4];
        values(raw[q][i], v);
        packed[q][i] = rule_bytes<decltype(plain)::value>(v, inv);
      }
    }
  };
  if (rule_is_plain(d)) pack(std::true_type{});
  else pack(std::false_type{});
  if constexpr (!ONE) {
    if (part == 1 && tg < TG) {
#pragma unroll
      for (int q = 0; q < NQ; q++) {
        const int t = first_slot(q);
        if (t >= P) continue;
        uint32_t o[4];
        transpose4(packed[q], o);
#pragma unroll
        for (int j = 0; j < 4; j++) vt[(4 * col + j) * 16 + ((t >> 2) ^ (col & 15))] = o[j];
      }
    }
  }
  __syncthreads();  // old codes rewritten (values: pieces shared with new slots), both scales read
  if (u == 0) scales[part] = d;
  if (part == 0) {
#pragma unroll
    for (int q = 0; q < NQ; q++) {
#pragma unroll
      for (int i = 0; i < SLOTS; i++) {
        const int t = first_slot(q) + i;
        if (mine && is_new(t))
          *reinterpret_cast<uint32_t*>(codes + ((size_t)(4 * col / 64) * P + t) * 64 + 4 * col % 64) = packed[q][i];
      }
    }
    if (p.bounds) {
      const int bb = kv_bounds_bytes(D);
      const long long at = ((long long)phys * p.H + head) * bb;
      if (QMV_CHECK(in_range(at, bb, p.bounds_len, p.err))) {
        uint8_t* b = p.bounds + at;
        if (u == 0) *reinterpret_cast<float*>(b) = d;
        int8_t* bl = reinterpret_cast<int8_t*>(b + KV_HEADER);
        for (int dd = u; dd < D; dd += HALF) {
          float a = lo_s[0][dd], z = hi_s[0][dd];
#pragma unroll
          for (int g = 1; g < TG; g++) {
            a = fminf(a, lo_s[g][dd]);
            z = fmaxf(z, hi_s[g][dd]);
          }
          // the code is monotone in x: the extremes' codes are the codes' extremes
          int ca = rule_code(a, inv), cz = rule_code(z, inv);
          if (lo > 0) {
            ca = min(ca, __float2int_rn(__fmul_rn((float)bl[dd], ratio)));
            cz = max(cz, __float2int_rn(__fmul_rn((float)bl[D + dd], ratio)));
          }
          bl[dd] = (int8_t)ca;
          bl[D + dd] = (int8_t)cz;
        }
      }
    }
  } else if constexpr (ONE) {
    if (tg == 0) {
      const uint32_t w = packed[0][0];
#pragma unroll
      for (int j = 0; j < 4; j++) codes[(4 * col + j) * P + lo] = (uint8_t)(w >> (8 * j));
    }
  } else {
    // 16 slots of a dimension a thread; single bytes where some are not new
    const int c0 = lo / 16, nc = (hi - 1) / 16 - c0 + 1;
    for (int i = u; i < D * 4; i += HALF) {
      const int dd = i / 4, c = i % 4, k = dd / 4 % 16;
      if (c < c0 || c >= c0 + nc) continue;
      uint4 w = *reinterpret_cast<const uint4*>(vt + dd * 16 + 4 * (c ^ (k >> 2)));
      if (k & 1) w = make_uint4(w.y, w.x, w.w, w.z);
      if (k & 2) w = make_uint4(w.z, w.w, w.x, w.y);
      const int a = max(lo, 16 * c), z = min(hi, 16 * c + 16);
      uint8_t* const dst = codes + dd * P + 16 * c;
      if (z - a == 16) {
        *reinterpret_cast<uint4*>(dst) = w;
      } else {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 16; j++)
          if (16 * c + j >= a && 16 * c + j < z) dst[j] = (uint8_t)(ws[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
}

// The values of the call's tokens: one CTA per (page, head).  A thread takes
// the codes of one 16-byte store of a token (keys), or, in pairs of
// dimensions, 16 slots (values: 16-byte loads, the stores of a warp side by
// side).  The same prompts read back: 24 us, 5.2 TB/s.
constexpr int KV_THREADS = 256;
template <int DT, int D>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const KvParams p, typename Elem<DT>::type* ko,
                                                             typename Elem<DT>::type* vo
                                                                 QMV_DEBUG_ONLY(, long long out_len)) {
  using T = typename Elem<DT>::type;
  pdl_launch_dependents();
  pdl_wait();
  const KvItem it = kv_item(p, (int)(blockIdx.x / (unsigned)p.H));
  if (it.s < 0) return;
  const int head = (int)(blockIdx.x % (unsigned)p.H), P = p.P;  // a token's heads side by side
  const int pos0 = it.seq.len - it.seq.n, page0 = it.page * P;
  const int lo = max(max(pos0, 0) - page0, 0), hi = min(it.seq.len - page0, P);
  const long long tok0 = (long long)it.seq.t0 + page0 - pos0;
  const long long row = (long long)p.H * D;
  if (pos0 < 0 && page0 == 0) {  // the call's tokens before the sequence's first
    if (it.seq.len > 0 && threadIdx.x == 0) set_error(p.err, QMV_DEVERR_BATCH);
    for (long long i = threadIdx.x; i < (long long)-pos0 * D; i += KV_THREADS) {
      const long long at = (it.seq.t0 + i / D) * row + (long long)head * D + i % D;
      if (!QMV_CHECK(in_range(at, 1, out_len, p.err))) continue;
      from_float(0.f, ko[at]);
      from_float(0.f, vo[at]);
    }
  }
  if (hi <= lo) return;
  const int phys = kv_page(p, it.s, it.page);
  const int rec_bytes = kv_page_bytes(D, P);
  const long long rec_at = ((long long)max(phys, 0) * p.H + head) * rec_bytes;
  if (!QMV_CHECK(in_range(rec_at, rec_bytes, p.pages_len, p.err))) return;
  const uint8_t* rec = p.pages + rec_at;
  const float dk = phys < 0 ? 0.f : reinterpret_cast<const float*>(rec)[0];
  const float dv = phys < 0 ? 0.f : reinterpret_cast<const float*>(rec)[1];
  const uint8_t* kc = rec + KV_HEADER;
  const uint8_t* vc = kc + P * D;
  constexpr int N = 16 / sizeof(T), PIECES = D / N;
  for (int i = threadIdx.x; i < (hi - lo) * PIECES; i += KV_THREADS) {
    const int t = lo + i / PIECES, e = i % PIECES * N;
    const uint32_t* c = reinterpret_cast<const uint32_t*>(kc + ((size_t)(e / 64) * P + t) * 64 + e % 64);
    float v[N];
#pragma unroll
    for (int k = 0; k < N / 4; k++) {
      const uint32_t w = c[k];
#pragma unroll
      for (int j = 0; j < 4; j++) v[4 * k + j] = dk * byte_code(w, j);
    }
    const long long at = (tok0 + t) * row + (long long)head * D + e;
    if (QMV_CHECK(in_range(at, N, out_len, p.err))) store_vec<N, T>(ko + at, v);
  }
  const int c0 = lo / 16, nc = (hi - 1) / 16 - c0 + 1;
  for (int i = threadIdx.x; i < D / 2 * nc; i += KV_THREADS) {
    const int dd = 2 * (i % (D / 2)), c = c0 + i / (D / 2);
    const uint4 a = *reinterpret_cast<const uint4*>(vc + dd * P + 16 * c);
    const uint4 b = *reinterpret_cast<const uint4*>(vc + (dd + 1) * P + 16 * c);
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
    const long long at = (tok0 + 16 * c) * row + (long long)head * D + dd;
    T* const out = vo + at;
    auto store = [&](int k) {
      T pair[2];
      from_float(dv * byte_code(wa[k >> 2], k & 3), pair[0]);
      from_float(dv * byte_code(wb[k >> 2], k & 3), pair[1]);
      if (!QMV_CHECK(in_range(at + k * row, 2, out_len, p.err))) return;
      if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(out + k * row) = make_float2(pair[0], pair[1]);
      else *reinterpret_cast<uint32_t*>(out + k * row) = *reinterpret_cast<const uint32_t*>(pair);
    };
    if (16 * c >= lo && 16 * c + 16 <= hi) {
#pragma unroll
      for (int k = 0; k < 16; k++) store(k);
    } else {
#pragma unroll
      for (int k = 0; k < 16; k++)
        if (16 * c + k >= lo && 16 * c + k < hi) store(k);
    }
  }
}

// Blocks of a call: items (see kv_item) times heads.
static unsigned grid_of(const KvParams& p) {
  const long long items = p.starts ? (long long)p.n_tok / p.P + 2ll * p.n_seq : p.n_seq;
  return (unsigned)(items * p.H);
}

template <int DT, int D>
static cudaError_t append_as(const KvParams& p, const void* k, long long ks, const void* v, long long vs,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  const bool one = !p.starts;
  make_config(cfg, attr, dim3(grid_of(p)), dim3(one ? AppendShape<DT, D, true>::THREADS : AppendShape<DT, D, false>::THREADS),
              0, stream, true);
  return one ? cudaLaunchKernelEx(&cfg, kv_append_kernel<DT, D, true>, p, k, v, ks, vs)
             : cudaLaunchKernelEx(&cfg, kv_append_kernel<DT, D, false>, p, k, v, ks, vs);
}
template <int DT, int D>
static cudaError_t read_as(const KvParams& p, void* k, void* v, cudaStream_t stream) {
  using T = typename Elem<DT>::type;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3(grid_of(p)), dim3(KV_THREADS), 0, stream, true);
  return cudaLaunchKernelEx(&cfg, kv_read_kernel<DT, D>, p, static_cast<T*>(k), static_cast<T*>(v)
                            QMV_DEBUG_ONLY(, output_extent((long long)p.n_tok * p.H * D)));
}

template <int DT>
static cudaError_t append_dt(const KvParams& p, int D, const void* k, long long ks, const void* v, long long vs,
                             cudaStream_t stream) {
  switch (D) {
    case 64: return append_as<DT, 64>(p, k, ks, v, vs, stream);
    case 128: return append_as<DT, 128>(p, k, ks, v, vs, stream);
    case 192: return append_as<DT, 192>(p, k, ks, v, vs, stream);
    default: return append_as<DT, 256>(p, k, ks, v, vs, stream);
  }
}
cudaError_t launch_kv_append(const KvParams& p, int dtype, int D, const void* k, long long ks, const void* v,
                             long long vs, cudaStream_t stream) {
  switch (dtype) {
    case QMV_DT_F16: return append_dt<QMV_DT_F16>(p, D, k, ks, v, vs, stream);
    case QMV_DT_BF16: return append_dt<QMV_DT_BF16>(p, D, k, ks, v, vs, stream);
    default: return append_dt<QMV_DT_F32>(p, D, k, ks, v, vs, stream);
  }
}

template <int DT>
static cudaError_t read_dt(const KvParams& p, int D, void* k, void* v, cudaStream_t stream) {
  switch (D) {
    case 64: return read_as<DT, 64>(p, k, v, stream);
    case 128: return read_as<DT, 128>(p, k, v, stream);
    case 192: return read_as<DT, 192>(p, k, v, stream);
    default: return read_as<DT, 256>(p, k, v, stream);
  }
}
cudaError_t launch_kv_read(const KvParams& p, int dtype, int D, void* k, void* v, cudaStream_t stream) {
  switch (dtype) {
    case QMV_DT_F16: return read_dt<QMV_DT_F16>(p, D, k, v, stream);
    case QMV_DT_BF16: return read_dt<QMV_DT_BF16>(p, D, k, v, stream);
    default: return read_dt<QMV_DT_F32>(p, D, k, v, stream);
  }
}

}  // namespace qmv
