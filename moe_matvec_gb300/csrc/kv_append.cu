// Writing tokens into the paged 8-bit cache, and reading them back.
#include "float_io.cuh"
#include "kv_cache.cuh"
#include "kv_launch.h"
#include "launch.h"

namespace qmv {

constexpr int KV_THREADS = 256;

// The (sequence, page) that block `item` of the grid works on: sequences take
// as many consecutive blocks as their new tokens touch pages.  Every thread
// returns the same answer; s = -1 past the last.
struct KvItem {
  int s, page;  // page: index in the sequence
  KvSeq seq;
};
// at least one for a sequence with tokens in the call, so that some block
// sees to the tokens of an empty one
__device__ __forceinline__ int touched_pages(const KvSeq& q, int P) {
  if (q.n < 1) return 0;
  return max(q.len - 1, 0) / P - max(q.len - q.n, 0) / P + 1;
}
__device__ __forceinline__ KvItem kv_item(const KvParams& p, int item) {
  KvItem r;
  if (!p.starts) {
    r.s = item;
    r.seq = kv_seq(p, item);
    r.page = max(r.seq.len - 1, 0) / p.P;
    return r;
  }
  // chunks of one sequence per thread, an exclusive scan of the page counts
  __shared__ int wsum[KV_THREADS / 32];
  __shared__ int found[2];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (tid == 0) found[0] = -1;
  int base = 0;
  for (int c = 0; c < p.n_seq; c += KV_THREADS) {
    const int s = c + tid;
    const int cnt = s < p.n_seq ? touched_pages(kv_seq(p, s), p.P) : 0;
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[w] = inc;
    __syncthreads();
    int before = base, total = 0;
#pragma unroll
    for (int i = 0; i < KV_THREADS / 32; i++) {
      if (i < w) before += wsum[i];
      total += wsum[i];
    }
    const int lo = before + inc - cnt;
    if (item >= lo && item < lo + cnt) {
      found[0] = s;
      found[1] = item - lo;
    }
    base += total;
    __syncthreads();
    if (found[0] >= 0 || item < base) break;
  }
  r.s = found[0];
  r.page = 0;
  r.seq = KvSeq{0, 0, 0};
  if (r.s >= 0) {
    r.seq = kv_seq(p, r.s);
    r.page = max(r.seq.len - r.seq.n, 0) / p.P + found[1];
  }
  return r;
}

// The activation rule's scale, its reciprocal and code.
__device__ __forceinline__ float rule_inv(float d) { return d > 0.f ? __frcp_rn(d) : 0.f; }
__device__ __forceinline__ int rule_code(float x, float inv) {
  // the conversion takes +-inf to the ends of the int range and NaN to 0
  return min(max(__float2int_rn(__fmul_rn(x, inv)), -127), 127);
}

// The codes of four packed bytes (code + 128) under a grown scale.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int c = (int)((w >> (8 * i)) & 0xFF) - 128;
    o |= (uint32_t)((__float2int_rn(__fmul_rn((float)c, ratio)) + 128) & 0xFF) << (8 * i);
  }
  return o;
}
// the same for the first n of the four (the others unchanged)
__device__ __forceinline__ uint32_t rescale4_first(uint32_t w, float ratio, int n) {
  if (n >= 4) return rescale4(w, ratio);
  const uint32_t keep = n <= 0 ? 0xFFFFFFFFu : 0xFFFFFFFFu << (8 * n);
  return (rescale4(w, ratio) & ~keep) | (w & keep);
}

// One CTA per (page, head) that the call's tokens touch; threads 0-127 take
// the keys, 128-255 the values.  Pass 1 reads the page's new tokens for the
// largest magnitude (and, for the bounds, the extremes of each dimension);
// if an old scale has to grow, the old codes are rewritten; pass 2 reads the
// tokens again (from L1 / L2) and stores their codes.  HBM-bound at the
// prompt sizes, latency at single tokens: then a CTA reads 2 D values and
// writes 2 D bytes.
template <int DT, int D>
__global__ void __launch_bounds__(KV_THREADS) kv_append_kernel(const KvParams p, const void* kx, const void* vx,
                                                               long long k_stride, long long v_stride) {
  using T = typename Elem<DT>::type;
  pdl_launch_dependents();
  pdl_wait();
  constexpr int HALF = KV_THREADS / 2, COLS = D / 4, TG = HALF / COLS;
  static_assert(COLS <= HALF, "a thread takes four dimensions");
  __shared__ float red[KV_THREADS / 32];
  __shared__ float lo_s[TG][D], hi_s[TG][D];
  const KvItem it = kv_item(p, blockIdx.x);
  if (it.s < 0) return;
  const int head = blockIdx.y, P = p.P;
  const int pos0 = it.seq.len - it.seq.n, page0 = it.page * P;
  const int lo = max(max(pos0, 0) - page0, 0), hi = min(it.seq.len - page0, P);  // the new slots
  if (pos0 < 0 && it.seq.len > 0 && threadIdx.x == 0) set_error(p.err, QMV_DEVERR_BATCH);  // tokens before the first
  if (hi <= lo) return;  // an empty sequence
  const int phys = kv_page(p, it.s, it.page);
  if (phys < 0) return;
  const long long tok0 = (long long)it.seq.t0 + page0 - pos0;                    // call's token of slot 0
  const int part = threadIdx.x / HALF, u = threadIdx.x % HALF;
  const int col = u % COLS, tg = u / COLS;
  const long long stride = part ? v_stride : k_stride;
  const T* x = static_cast<const T*>(part ? vx : kx) + (long long)head * D;
  const int rec_bytes = kv_page_bytes(D, P);
  const long long rec_at = ((long long)phys * p.H + head) * rec_bytes;
  if (!QMV_CHECK(in_range(rec_at, rec_bytes, p.pages_len, p.err))) return;
  uint8_t* rec = p.pages + rec_at;
  float* scales = reinterpret_cast<float*>(rec);
  const float d_old = lo > 0 ? scales[part] : 0.f;

  float amax = 0.f, mn[4], mx[4];
#pragma unroll
  for (int j = 0; j < 4; j++) mn[j] = INFINITY, mx[j] = -INFINITY;
  if (tg < TG) {
#pragma unroll 4
    for (int t = lo + tg; t < hi; t += TG) {
      float v[4];
      if (!QMV_CHECK(in_range(tok0 + t, 1, p.n_tok, p.err))) continue;
      load_vec<4>(x + (tok0 + t) * stride + 4 * col, v);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        amax = fmaxf(amax, fabsf(v[j]));
        mn[j] = fminf(mn[j], v[j]);
        mx[j] = fmaxf(mx[j], v[j]);
      }
    }
    if (p.bounds && part == 0) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        lo_s[tg][4 * col + j] = mn[j];
        hi_s[tg][4 * col + j] = mx[j];
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < HALF / 32; i++) amax = fmaxf(amax, red[part * (HALF / 32) + i]);
  const float d = fmaxf(d_old, __fdiv_rn(amax, 127.0f));
  const float inv = rule_inv(d);
  uint8_t* codes = rec + KV_HEADER + part * P * D;

  const bool grown = lo > 0 && d > d_old;
  const float ratio = d > 0.f ? __fdiv_rn(d_old, d) : 0.f;
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
  __syncthreads();  // old codes rewritten (values: chunks shared with new slots), both scales read
  if (u == 0) scales[part] = d;
  if (part == 0) {
    if (tg < TG) {
#pragma unroll 4
      for (int t = lo + tg; t < hi; t += TG) {
        float v[4];
        if (!QMV_CHECK(in_range(tok0 + t, 1, p.n_tok, p.err))) continue;
        load_vec<4>(x + (tok0 + t) * stride + 4 * col, v);
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) w |= (uint32_t)(rule_code(v[j], inv) + 128) << (8 * j);
        *reinterpret_cast<uint32_t*>(codes + ((size_t)(4 * col / 64) * P + t) * 64 + 4 * col % 64) = w;
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
  } else {
    // a thread takes one dimension of 16 slots: 16-byte stores where all are new
    const int c0 = lo / 16, nc = (hi - 1) / 16 - c0 + 1;
    for (int i = u; i < D * nc; i += HALF) {
      const int dd = i % D, c = c0 + i / D;
      const int a = max(lo, 16 * c), z = min(hi, 16 * c + 16);
      if (!QMV_CHECK(in_range(tok0 + a, z - a, p.n_tok, p.err))) continue;
      if (z - a == 16) {
        uint32_t w[4];
        float v[16];
#pragma unroll
        for (int k = 0; k < 16; k++) v[k] = to_float(x[(tok0 + 16 * c + k) * stride + dd]);
#pragma unroll
        for (int k = 0; k < 4; k++) {
          w[k] = 0;
#pragma unroll
          for (int j = 0; j < 4; j++) w[k] |= (uint32_t)(rule_code(v[4 * k + j], inv) + 128) << (8 * j);
        }
        reinterpret_cast<uint4*>(codes + dd * P)[c] = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        for (int t = a; t < z; t++)
          codes[dd * P + t] = (uint8_t)(rule_code(to_float(x[(tok0 + t) * stride + dd]), inv) + 128);
      }
    }
  }
}

// The values of the call's tokens: one CTA per (page, head); a thread takes
// 16 dimensions of a token (keys) or 16 slots of a dimension (values).
template <int DT, int D>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const KvParams p, typename Elem<DT>::type* ko,
                                                             typename Elem<DT>::type* vo
                                                                 QMV_DEBUG_ONLY(, long long out_len)) {
  using T = typename Elem<DT>::type;
  pdl_launch_dependents();
  pdl_wait();
  const KvItem it = kv_item(p, blockIdx.x);
  if (it.s < 0) return;
  const int head = blockIdx.y, P = p.P;
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
  for (int i = threadIdx.x; i < (hi - lo) * (D / 16); i += KV_THREADS) {
    const int t = lo + i / (D / 16), c = i % (D / 16);
    const uint4 q = *reinterpret_cast<const uint4*>(kc + ((size_t)(c / 4) * P + t) * 64 + 16 * (c % 4));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; k++) v[k] = dk * (float)((int)((w[k >> 2] >> (8 * (k & 3))) & 0xFF) - 128);
    const long long at = (tok0 + t) * row + (long long)head * D + 16 * c;
    if (QMV_CHECK(in_range(at, 16, out_len, p.err))) store_vec<16, T>(ko + at, v);
  }
  const int c0 = lo / 16, nc = (hi - 1) / 16 - c0 + 1;
  for (int i = threadIdx.x; i < D * nc; i += KV_THREADS) {
    const int dd = i % D, c = c0 + i / D;
    const uint4 q = reinterpret_cast<const uint4*>(vc + dd * P)[c];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 16; k++) {
      const int t = 16 * c + k;
      const long long at = (tok0 + t) * row + (long long)head * D + dd;
      if (t >= lo && t < hi && QMV_CHECK(in_range(at, 1, out_len, p.err)))
        from_float(dv * (float)((int)((w[k >> 2] >> (8 * (k & 3))) & 0xFF) - 128), vo[at]);
    }
  }
}

// Blocks that the batch's touched pages take at most: a sequence of n new
// tokens touches at most (n + P - 2) / P + 1 pages, and never more than n.
static unsigned item_bound(const KvParams& p) {
  if (!p.starts) return (unsigned)p.n_seq;
  const long long a = (long long)p.n_tok / p.P + 2ll * p.n_seq, b = p.n_tok;
  return (unsigned)(a < b ? a : b);
}

template <int DT, int D>
static cudaError_t append_as(const KvParams& p, const void* k, long long ks, const void* v, long long vs,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3(item_bound(p), p.H), dim3(KV_THREADS), 0, stream, true);
  return cudaLaunchKernelEx(&cfg, kv_append_kernel<DT, D>, p, k, v, ks, vs);
}
template <int DT, int D>
static cudaError_t read_as(const KvParams& p, void* k, void* v, cudaStream_t stream) {
  using T = typename Elem<DT>::type;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3(item_bound(p), p.H), dim3(KV_THREADS), 0, stream, true);
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
