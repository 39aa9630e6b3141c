// Launchers of the cache, attention and page selection kernels (head_dim,
// page_tokens and every size already checked).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qmv {

struct KvParams;

cudaError_t launch_kv_append(const KvParams& p, int dtype, int D, const void* k, long long ks, const void* v,
                             long long vs, cudaStream_t stream);
cudaError_t launch_kv_read(const KvParams& p, int dtype, int D, void* k, void* v, cudaStream_t stream);

struct AttendArgs {
  int dtype;
  const void* q;
  long long q_stride;
  void* out;
  int n_heads;
  float scale;
  int causal, window;
  const int32_t* sel;  // or nullptr
  int n_sel;
  void* ws;
};
size_t kv_attend_ws_bytes(int D, int H, int G, int n_tok, int n_seq);
cudaError_t launch_kv_attend(const KvParams& p, int D, const AttendArgs& a, cudaStream_t stream);

struct SelectArgs {
  int dtype;
  const void* q;
  long long q_stride;
  int n_heads;
  int32_t* ids;
  int n_sel;
  void* ws;
};
size_t kv_select_ws_bytes(int H, int n_tok, int max_pages);
cudaError_t launch_kv_select(const KvParams& p, int D, const SelectArgs& a, cudaStream_t stream);

}  // namespace qmv
