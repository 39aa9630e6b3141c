// Root-mean-square norm with the residual's addition, its result as floats
// and / or in the library's Q8 activation layout, and the values that such
// activations stand for.
#include "float_io.cuh"
#include "launch.h"
#include "qmv_core.cuh"

namespace qmv {

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if one of them is
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

// The activation rule on a lane's eight values of a block (four lanes a
// block, as quant_units): codes in two words, scale, sum.  A block whose
// largest magnitude is 0 or at least 2^-100 rounds by adding and taking away
// 1.5 * 2^23: the sum's low mantissa bits are then the integer, rounded half to
// even, in two's complement (the exact product is below 127.5).  Other blocks,
// among them those with a NaN (whose code is 0), take the IEEE operations and the
// clamp.
__device__ __forceinline__ void quant8(const float (&v)[8], uint32_t& w0, uint32_t& w1, float& d, int& sum) {
  float m = max_nan(max_nan(fabsf(v[0]), fabsf(v[1]), fabsf(v[2])), max_nan(fabsf(v[3]), fabsf(v[4]), fabsf(v[5])),
                    max_nan(fabsf(v[6]), fabsf(v[7])));
  m = max_nan(m, __shfl_xor_sync(FULL, m, 1));
  m = max_nan(m, __shfl_xor_sync(FULL, m, 2));
  uint32_t q[8];
  if (!__any_sync(FULL, m != 0.0f && !(m >= 0x1p-100f && m < INFINITY))) {
    d = div127_rn(m);
    const float id = m > 0.0f ? rcp_rn(fmaxf(d, 0x1p-126f)) : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) q[k] = __float_as_uint(__fadd_rn(__fmul_rn(v[k], id), 12582912.0f));
  } else {
    m = fabsf(v[0]);
#pragma unroll
    for (int k = 1; k < 8; k++) m = fmaxf(m, fabsf(v[k]));
    m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));
    m = fmaxf(m, __shfl_xor_sync(FULL, m, 2));
    d = __fdiv_rn(m, 127.0f);
    const float id = d > 0.0f ? __frcp_rn(d) : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) q[k] = (uint32_t)min(max(__float2int_rn(__fmul_rn(v[k], id)), -127), 127);
  }
  w0 = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  w1 = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
  sum = __dp4a((int)w1, 0x01010101, __dp4a((int)w0, 0x01010101, 0));
  sum += __shfl_xor_sync(FULL, sum, 1);
  sum += __shfl_xor_sync(FULL, sum, 2);
}

// The blockDim.x threads of a row hold its K values s = x + r in registers
// (eight a thread and step, NV steps), so x and r are read once and everything
// else follows without another read:
//   rstd = 1 / sqrt(sum s^2 / K + eps),  y = (s rstd) w,  q8(y).
// s, the sum and y are fp32; only the stores round (s and y to T).  blockDim.y
// rows share a CTA so that short rows still fill it.  CTAs go over the rows in
// strides of the grid: the next row's x and r are on their way while this one
// is summed and stored, and w is read once per CTA.
// VEC: eight consecutive values a thread (K % 8 == 0, rows 16-byte aligned),
// which is also the activation rule's four lanes per block of 32; else single
// values, consecutive threads taking consecutive ones.
//
// Bound by HBM for many rows: 4096 x 5120 bfloat16 with the residual, the
// float and the Q8 result (194 MB): 32 us, 6.1 TB/s (and the codes read back 44
// us, 57 with one row a CTA).  One row of 5120: 2.7 us, the latency of a load, two
// barriers and the stores.  Without VEC by the number of loads and stores: 2000 x
// 4097 bfloat16 22 us, 1.5 TB/s (4096: 6.4 us).
template <int DT, bool VEC, int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) rms_norm_kernel(const NormParams p) {
  using T = typename Elem<DT>::type;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, nt = blockDim.x, wpr = nt >> 5;
  // value j of step i of this thread
  auto at_of = [&](int i, int j) { return VEC ? (i * nt + tid) * 8 + j : (i * 8 + j) * nt + tid; };
  auto load = [&](const T* src, long long first, long long len, T (&raw)[8], int i) {
    if constexpr (VEC) {
      const int e = at_of(i, 0);
      if (e < p.K && QMV_CHECK(in_range(first + e, 8, len, p.err))) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; k++)
          reinterpret_cast<uint4*>(raw)[k] = reinterpret_cast<const uint4*>(src + first + e)[k];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (at_of(i, j) < p.K && QMV_CHECK(in_range(first + at_of(i, j), 1, len, p.err))) raw[j] = src[first + at_of(i, j)];
    }
    (void)len;
  };
  auto load_w = [&](int i, float (&w)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j++) w[j] = 0.f;
    if constexpr (VEC) {
      if (at_of(i, 0) < p.K) load_vec<8>(p.w + at_of(i, 0), w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (at_of(i, j) < p.K) w[j] = p.w[at_of(i, j)];
    }
  };
  const T* x = static_cast<const T*>(p.x);
  const T* r = static_cast<const T*>(p.r);
  T* res = static_cast<T*>(p.res);
  T* y = static_cast<T*>(p.y);
  const long long stride = (long long)gridDim.x * blockDim.y;
  const long long row0 = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  struct alignas(16) Raw {
    T v[8];
  };
  Raw nx[NV], nr[NV];
  auto fetch_step = [&](long long row, int i) {
#pragma unroll
    for (int j = 0; j < 8; j++) from_float(0.f, nx[i].v[j]), from_float(0.f, nr[i].v[j]);
    if (row < p.rows) {
      load(x, row * p.ldx, QMV_EXTENT(p.x_len), nx[i].v, i);
      if (r) load(r, row * p.K, QMV_EXTENT(p.n), nr[i].v, i);
    }
  };
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; i++) fetch_step(row, i);
  };
  // Rows of over 16384 values: fetched and summed a step at a time (the raw values
  // of eight steps do not fit the registers beside their floats: 512 x 32768
  // bfloat16 24 us, now 21), in partial sums of eight (64 squares a thread one after
  // another lose many small ones beside a large one; so at most 16 roundings).
  constexpr bool LONG = NV == NORM_MAX_STEPS;
  constexpr bool AHEAD = NV <= 2;   // the next row on its way (registers)
  constexpr bool KEEP_W = NV <= 2;  // else w is read again for every row
  if constexpr (AHEAD) fetch(row0);
  float w[KEEP_W ? NV : 1][8];
  if constexpr (KEEP_W) {
#pragma unroll
    for (int i = 0; i < NV; i++) load_w(i, w[i]);
  }
  __shared__ float part[2][32];  // one per warp of the CTA (a row's warps are neighbours), by turns
  int turn = 0;
  // every row of the CTA makes the same number of steps
  for (long long first = (long long)blockIdx.x * blockDim.y; first < p.rows; first += stride, turn ^= 1) {
    const long long row = first + threadIdx.y;
    if constexpr (!AHEAD && !LONG) fetch(row);
    float v[NV][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      if constexpr (LONG) fetch_step(row, i);
      float eight = 0.f;
      float& into = LONG ? eight : sum;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        v[i][j] = to_float(nx[i].v[j]);
        if (r) v[i][j] += to_float(nr[i].v[j]);
        into = fmaf(v[i][j], v[i][j], into);
      }
      if constexpr (LONG) sum += eight;
    }
    if constexpr (AHEAD)
      if (first + stride < p.rows) fetch(row + stride);
    sum = warp_sum(sum);
    const int warp0 = threadIdx.y * wpr;
    if ((tid & 31) == 0) part[turn][warp0 + (tid >> 5)] = sum;
    __syncthreads();
    sum = (tid & 31) < wpr ? part[turn][warp0 + (tid & 31)] : 0.f;
    sum = warp_sum(sum);
    if (row >= p.rows) continue;
    const float rstd = rsqrtf(fmaf(sum, p.inv_k, p.eps));  // at most 2 units in the last place off
    const long long base = row * p.K;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      float(&wi)[8] = w[KEEP_W ? i : 0];
      if constexpr (!KEEP_W) load_w(i, wi);
      if constexpr (VEC) {
        const int e = at_of(i, 0);
        if (e < p.K) {
          if (res && QMV_CHECK(in_range(base + e, 8, p.out_len, p.err))) store_vec<8>(res + base + e, v[i]);
#pragma unroll
          for (int j = 0; j < 8; j++) v[i][j] = (v[i][j] * rstd) * wi[j];
          if (y && QMV_CHECK(in_range(base + e, 8, p.out_len, p.err))) store_vec<8>(y + base + e, v[i]);
        }
        // K % 256 == 0 here: a warp is whole or past the row
        if (p.q && at_of(i, 0) - 8 * (tid & 31) < p.K) {
          uint32_t w0, w1;
          float dd;
          int ss;
          quant8(v[i], w0, w1, dd, ss);
          const int lane = tid & 31, sub = lane >> 2, li = lane & 3;
          const long long g = (base + at_of(i, 0) - 8 * lane) >> 8;
          if (QMV_CHECK(in_range(g * 256 + act_pos(sub, 8 * li), 8, p.out_len, p.err)))
            *reinterpret_cast<uint2*>(p.q + g * 256 + act_pos(sub, 8 * li)) = make_uint2(w0, w1);
          if (li == 0 && QMV_CHECK(in_range(g * 8 + sub, 1, p.out_len / 32, p.err))) {
            p.d[g * 8 + sub] = dd;
            p.s[g * 8 + sub] = ss;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const int e = at_of(i, j);
          if (e < p.K && QMV_CHECK(in_range(base + e, 1, p.out_len, p.err))) {
            if (res) from_float(v[i][j], res[base + e]);
            if (y) from_float((v[i][j] * rstd) * wi[j], y[base + e]);
          }
        }
      }
    }
  }
}

template <int DT, bool VEC>
static cudaError_t launch_norm_as(const NormParams& p, cudaStream_t stream, bool pdl) {
  // Threads of a row: few rows, where latency counts, have one for every eight
  // values (up to 1024 threads); with more than four rows an SM each takes two
  // steps of eight, which halves the share of the row's sums and barrier.
  // Short rows share CTAs of about 256 threads.
  const int units = (p.K + 7) / 8;
  int steps = p.rows > 4ll * device_sm_count() && units >= 256 ? 2 : 1;
  if (units > 1024) steps = units <= 2048 ? 4 : NORM_MAX_STEPS;  // 512 threads at most from two steps on
  const int nt = ((units + steps - 1) / steps + 31) / 32 * 32;
  const int ny = p.rows > device_sm_count() && nt < 256 ? 256 / nt : 1;
  long long ctas = (p.rows + ny - 1) / ny;
  // as many CTAs as the SMs hold at once (registers: 64 a thread, from two steps on about 96)
  const int per_sm = (steps == 1 ? 1024 : 640) / (nt * ny);
  const long long cap = (long long)device_sm_count() * (per_sm > 1 ? per_sm : 1);
  if (ctas > cap) ctas = cap;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3((unsigned)ctas), dim3(nt, ny), 0, stream, pdl);
  switch (steps) {
    case 1: return cudaLaunchKernelEx(&cfg, rms_norm_kernel<DT, VEC, 1>, p);
    case 2: return cudaLaunchKernelEx(&cfg, rms_norm_kernel<DT, VEC, 2>, p);
    case 4: return cudaLaunchKernelEx(&cfg, rms_norm_kernel<DT, VEC, 4>, p);
    default: return cudaLaunchKernelEx(&cfg, rms_norm_kernel<DT, VEC, NORM_MAX_STEPS>, p);
  }
}

template <int DT>
static cudaError_t launch_norm_dt(const NormParams& p, bool vec, cudaStream_t stream, bool pdl) {
  return vec ? launch_norm_as<DT, true>(p, stream, pdl) : launch_norm_as<DT, false>(p, stream, pdl);
}

cudaError_t launch_rms_norm(int dtype, const NormParams& p, bool vec, cudaStream_t stream, bool pdl) {
  switch (dtype) {
    case QMV_DT_F16: return launch_norm_dt<QMV_DT_F16>(p, vec, stream, pdl);
    case QMV_DT_BF16: return launch_norm_dt<QMV_DT_BF16>(p, vec, stream, pdl);
    default: return launch_norm_dt<QMV_DT_F32>(p, vec, stream, pdl);
  }
}

// The values d q of activations in the Q8 layout: a thread takes the codes of
// one 16-byte store (4 or 8 values of a half block, contiguous in both).  Bound
// by HBM: 4096 x 5120 to bfloat16 (68 MB) in 13 us.
template <int DT>
__global__ void __launch_bounds__(256) act_dequant_kernel(const int8_t* __restrict__ q, const float* __restrict__ d,
                                                          long long chunks, typename Elem<DT>::type* __restrict__ out
                                                              QMV_DEBUG_ONLY(, unsigned* err, long long out_len)) {
  constexpr int N = 16 / sizeof(typename Elem<DT>::type);
  pdl_launch_dependents();
  pdl_wait();
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < chunks;
       i += (long long)gridDim.x * blockDim.x) {
    const long long at = i * N;
    const int e = (int)at & 255;  // the first value's place in its group of 256
    if (!QMV_CHECK(in_range(at, N, out_len, err))) continue;
    const int8_t* c = q + (at - e) + act_pos(e >> 5, e & 31);
    const float s = d[at >> 5];
    uint32_t w[N / 4];
    if constexpr (N == 8) {
      const uint2 t = *reinterpret_cast<const uint2*>(c);
      w[0] = t.x, w[1] = t.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(c);
    }
    float v[N];
#pragma unroll
    for (int k = 0; k < N; k++) {
      // code + 128 in the low byte of 2^23 + .., less 2^23 + 128: the code, exactly
      const uint32_t b = __byte_perm(w[k >> 2] ^ 0x80808080u, 0x4B000000u, 0x7440 + (k & 3));
      v[k] = s * __fsub_rn(__uint_as_float(b), 8388608.0f + 128.0f);
    }
    store_vec<N>(out + at, v);
  }
}

template <int DT>
static cudaError_t dequant_as(const int8_t* q, const float* d, long long n, void* out, cudaStream_t stream, bool pdl) {
  using T = typename Elem<DT>::type;
  const long long chunks = n * (long long)sizeof(T) / 16;
  long long ctas = (chunks + 255) / 256;
  const long long cap = 64ll * device_sm_count();
  if (ctas > cap) ctas = cap;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3((unsigned)ctas), dim3(256), 0, stream, pdl);
  return cudaLaunchKernelEx(&cfg, act_dequant_kernel<DT>, q, d, chunks, static_cast<T*>(out)
                            QMV_DEBUG_ONLY(, device_error_word(), output_extent(n)));
}

cudaError_t launch_act_dequant(int dtype, const int8_t* q, const float* d, long long n, void* out, cudaStream_t stream,
                               bool pdl) {
  switch (dtype) {
    case QMV_DT_F16: return dequant_as<QMV_DT_F16>(q, d, n, out, stream, pdl);
    case QMV_DT_BF16: return dequant_as<QMV_DT_BF16>(q, d, n, out, stream, pdl);
    default: return dequant_as<QMV_DT_F32>(q, d, n, out, stream, pdl);
  }
}

}  // namespace qmv
