// Launchers of the head norm and rotation, adapter, expert selection and log
// probability kernels (every size already checked).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qmv {

// Heads of one kind (queries or keys): tokens xs / ys elements apart.
struct RopeHeads {
  const void* x;
  void* y;
  long long xs, ys;
  const float* w;  // or nullptr: no norm
  int n;
#ifdef QMV_DEBUG
  long long x_len, y_len;
#endif
};
struct RopeParams {
  RopeHeads q, k;
  const float* freq;
  const uint8_t* axis;   // or nullptr
  const int32_t* pos;    // or nullptr: lens, starts
  const int32_t* lens;
  const int32_t* starts; // or nullptr
  int D, R, n_axes, n_seq, n_tok;
  float eps, scale;
  unsigned* err;
};
cudaError_t launch_norm_rope(int dtype, bool interleaved, const RopeParams& p, cudaStream_t stream);

// The arguments of moe_route_select.
constexpr int ROUTE_MAX_GROUPS = 32;
struct RouteParams {
  const void* logits;
  const float* bias;  // or nullptr
  int32_t* ids;
  float* gates;
  long long ld;
  int E, size, n_tok, top_k, gating, groups, keep, group_top, renorm;  // size: experts of a group
  float scale;
#ifdef QMV_DEBUG
  unsigned* err;
  long long logits_len, ids_len;
#endif
};
cudaError_t launch_route_select(int dtype, const RouteParams& p, cudaStream_t stream);

// The arguments of qmv_logprobs.
struct LogprobsParams {
  const void* logits;
  const int32_t* tokens;
  float *logp, *lse, *entropy;
  int32_t* top_ids;
  float* top_logp;
  long long ld, rows;
  int V, n_given, n_top;
  float scale;
  unsigned* err;
#ifdef QMV_DEBUG
  long long logits_len, rows_len, given_len, top_len;
#endif
};
cudaError_t launch_logprobs(int dtype, const LogprobsParams& p, cudaStream_t stream);

// The arguments of qmv_lora_run.
struct LoraParams {
  const void* A;         // [n][r][K]
  const void* B;         // [n][M][r]
  const int32_t* ranks;  // or nullptr: r
  const float* scales;   // or nullptr: 1
  const int32_t* ids;
  const float* x;
  const float* res;
  float* y;
  float* part;           // [splits][n_tok][r]
  long long M;
  int K, n, r, n_tok, splits, window;  // window: columns of a split
  unsigned* err;
#ifdef QMV_DEBUG
  long long a_len, b_len, x_len, part_len, y_len;
#endif
};
int lora_splits(long long K, int n_tok, int r, int dtype);
cudaError_t launch_lora(int dtype, LoraParams p, cudaStream_t stream);

}  // namespace qmv
