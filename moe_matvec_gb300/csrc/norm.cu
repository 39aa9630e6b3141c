// Root-mean-square norm with the residual's addition, its result as floats
// and / or in the library's Q8 activation layout, and the values that such
// activations stand for.
#include "float_io.cuh"
#include "launch.h"
#include "qmv_core.cuh"

namespace qmv {

// One row s = x + r of K values is held in registers by the blockDim.x
// threads of a row (eight values a thread and step, NV steps), so x and r are
// read once and everything else follows without another read:
//   rstd = 1 / sqrt(sum s^2 / K + eps),  y = (s rstd) w,  q8(y).
// s, the sum and y are fp32; only the stores round (s and y to T).  blockDim.y
// rows share a CTA so that short rows still fill it.
// VEC: eight consecutive values a thread (K % 8 == 0, rows 16-byte aligned),
// which is also the activation rule's four lanes per block of 32; else single
// values, consecutive threads taking consecutive ones.
template <int DT, bool VEC, int NV>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p) {
  using T = typename Elem<DT>::type;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, nt = blockDim.x, wpr = nt >> 5;
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = p.r ? static_cast<const T*>(p.r) + row * p.K : nullptr;
  float v[NV][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; i++) {
#pragma unroll
    for (int j = 0; j < 8; j++) v[i][j] = 0.f;
    if constexpr (VEC) {
      const int e = (i * nt + tid) * 8;
      if (live && e < p.K && QMV_CHECK(in_range(row * p.ldx + e, 8, p.x_len, p.err))) {
        load_vec<8>(x + e, v[i]);
        if (r && QMV_CHECK(in_range(row * p.K + e, 8, p.n, p.err))) {
          float a[8];
          load_vec<8>(r + e, a);
#pragma unroll
          for (int j = 0; j < 8; j++) v[i][j] += a[j];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int e = (i * 8 + j) * nt + tid;
        if (live && e < p.K && QMV_CHECK(in_range(row * p.ldx + e, 1, p.x_len, p.err))) {
          v[i][j] = to_float(x[e]);
          if (r && QMV_CHECK(in_range(row * p.K + e, 1, p.n, p.err))) v[i][j] += to_float(r[e]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; j++) sum = fmaf(v[i][j], v[i][j], sum);
  }
  // w of one step; with a single step it is read while the row's sum is formed
  auto load_w = [&](int i, float (&w)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j++) w[j] = 0.f;
    if constexpr (VEC) {
      const int e = (i * nt + tid) * 8;
      if (e < p.K && QMV_CHECK(in_range(e, 8, p.K, p.err))) load_vec<8>(p.w + e, w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int e = (i * 8 + j) * nt + tid;
        if (e < p.K && QMV_CHECK(in_range(e, 1, p.K, p.err))) w[j] = p.w[e];
      }
    }
  };
  float w[8];
  if constexpr (NV == 1) load_w(0, w);
  sum = warp_sum(sum);
  __shared__ float part[32];  // one per warp of the CTA; a row's warps are neighbours
  const int warp0 = threadIdx.y * wpr;
  if ((tid & 31) == 0) part[warp0 + (tid >> 5)] = sum;
  __syncthreads();
  sum = (tid & 31) < wpr ? part[warp0 + (tid & 31)] : 0.f;
  sum = warp_sum(sum);
  if (!live) return;
  const float rstd = 1.0f / sqrtf(sum / (float)p.K + p.eps);
  T* res = static_cast<T*>(p.res);
  T* y = static_cast<T*>(p.y);
#pragma unroll
  for (int i = 0; i < NV; i++) {
    if constexpr (VEC) {
      const int e = (i * nt + tid) * 8;
      const long long at = row * p.K + e;
      if (e < p.K) {
        if (res && QMV_CHECK(in_range(at, 8, p.out_len, p.err))) store_vec<8>(res + at, v[i]);
        if constexpr (NV > 1) load_w(i, w);
#pragma unroll
        for (int j = 0; j < 8; j++) v[i][j] = (v[i][j] * rstd) * w[j];
        if (y && QMV_CHECK(in_range(at, 8, p.out_len, p.err))) store_vec<8>(y + at, v[i]);
      }
      // K % 256 == 0 here: a warp is whole or past the row
      if (p.q && (i * nt + (tid & ~31)) * 8 < p.K) {
        const float4 f[1][2] = {{make_float4(v[i][0], v[i][1], v[i][2], v[i][3]),
                                 make_float4(v[i][4], v[i][5], v[i][6], v[i][7])}};
        uint32_t w0[1], w1[1];
        float dd[1];
        int ss[1];
        quant_units<1>(f, w0, w1, dd, ss);
        const int lane = tid & 31, sub = lane >> 2, li = lane & 3;
        const long long g = (row * p.K + (i * nt + (tid & ~31)) * 8) / 256;
        if (QMV_CHECK(in_range(g * 256 + act_pos(sub, 8 * li), 8, p.out_len, p.err)))
          *reinterpret_cast<uint2*>(p.q + g * 256 + act_pos(sub, 8 * li)) = make_uint2(w0[0], w1[0]);
        if (li == 0 && QMV_CHECK(in_range(g * 8 + sub, 1, p.out_len / 32, p.err))) {
          p.d[g * 8 + sub] = dd[0];
          p.s[g * 8 + sub] = ss[0];
        }
      }
    } else {
      if constexpr (NV > 1) load_w(i, w);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int e = (i * 8 + j) * nt + tid;
        if (e < p.K && QMV_CHECK(in_range(row * p.K + e, 1, p.out_len, p.err))) {
          if (res) from_float(v[i][j], res[row * p.K + e]);
          if (y) from_float((v[i][j] * rstd) * w[j], y[row * p.K + e]);
        }
      }
    }
  }
}

template <int DT>
static cudaError_t launch_norm_dt(const NormParams& p, bool vec, cudaStream_t stream, bool pdl) {
  // threads of a row: enough for eight values each, at most 1024; short rows
  // share CTAs of about 256 threads once there are more rows than SMs
  const int units = (p.K + 7) / 8;
  int nt = (units + 31) / 32 * 32;
  if (nt > 1024) nt = 1024;
  int ny = p.rows > device_sm_count() && nt < 256 ? 256 / nt : 1;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3((unsigned)((p.rows + ny - 1) / ny)), dim3(nt, ny), 0, stream, pdl);
  if (units <= nt)
    return vec ? cudaLaunchKernelEx(&cfg, rms_norm_kernel<DT, true, 1>, p)
               : cudaLaunchKernelEx(&cfg, rms_norm_kernel<DT, false, 1>, p);
  return vec ? cudaLaunchKernelEx(&cfg, rms_norm_kernel<DT, true, NORM_MAX_STEPS>, p)
             : cudaLaunchKernelEx(&cfg, rms_norm_kernel<DT, false, NORM_MAX_STEPS>, p);
}

cudaError_t launch_rms_norm(int dtype, const NormParams& p, bool vec, cudaStream_t stream, bool pdl) {
  switch (dtype) {
    case QMV_DT_F16: return launch_norm_dt<QMV_DT_F16>(p, vec, stream, pdl);
    case QMV_DT_BF16: return launch_norm_dt<QMV_DT_BF16>(p, vec, stream, pdl);
    default: return launch_norm_dt<QMV_DT_F32>(p, vec, stream, pdl);
  }
}

// The values d q of activations in the Q8 layout: a thread takes the 16
// consecutive codes of one half block (bytes of the group in act_pos order).
template <int DT>
__global__ void __launch_bounds__(256) act_dequant_kernel(const int8_t* __restrict__ q, const float* __restrict__ d,
                                                          long long halves, typename Elem<DT>::type* __restrict__ out
                                                              QMV_DEBUG_ONLY(, unsigned* err, long long out_len)) {
  pdl_launch_dependents();
  pdl_wait();
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < halves;
       i += (long long)gridDim.x * blockDim.x) {
    const long long g = i >> 4;
    // the thread's half block in order of the values: block (i & 15) / 2
    const int blk = (int)(i & 15) >> 1, half = (int)i & 1;
    if (!QMV_CHECK(in_range(g * 256 + blk * 32 + half * 16, 16, out_len, err))) continue;
    const uint4 c = *reinterpret_cast<const uint4*>(q + g * 256 + act_pos(blk, 16 * half));
    const float s = d[g * 8 + blk];
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; k++) v[k] = s * (float)(int8_t)(w[k >> 2] >> (8 * (k & 3)));
    store_vec<16>(out + g * 256 + blk * 32 + half * 16, v);
  }
}

cudaError_t launch_act_dequant(int dtype, const int8_t* q, const float* d, long long n, void* out, cudaStream_t stream,
                               bool pdl) {
  const long long halves = n / 16;
  long long ctas = (halves + 255) / 256;
  const long long cap = 8ll * device_sm_count();
  if (ctas > cap) ctas = cap;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  make_config(cfg, attr, dim3((unsigned)ctas), dim3(256), 0, stream, pdl);
  switch (dtype) {
    case QMV_DT_F16:
      return cudaLaunchKernelEx(&cfg, act_dequant_kernel<QMV_DT_F16>, q, d, halves, static_cast<__half*>(out)
                                QMV_DEBUG_ONLY(, device_error_word(), output_extent(n)));
    case QMV_DT_BF16:
      return cudaLaunchKernelEx(&cfg, act_dequant_kernel<QMV_DT_BF16>, q, d, halves, static_cast<__nv_bfloat16*>(out)
                                QMV_DEBUG_ONLY(, device_error_word(), output_extent(n)));
    default:
      return cudaLaunchKernelEx(&cfg, act_dequant_kernel<QMV_DT_F32>, q, d, halves, static_cast<float*>(out)
                                QMV_DEBUG_ONLY(, device_error_word(), output_extent(n)));
  }
}

}  // namespace qmv
