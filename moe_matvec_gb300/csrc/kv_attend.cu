// Attention over the paged 8-bit cache: workspace and dispatch (the kernels are
// in kv_attend.cuh, instantiated in kv_attend_split.cu and kv_attend_half.cu).
#include "kv_attend.cuh"

namespace qmv {

cudaError_t launch_attend_split(AttendParams& p, int D, cudaStream_t stream);
cudaError_t launch_attend_half(AttendParams& p, int D, cudaStream_t stream);

// Items of a batch at most: with page lists every token has its own.
static long long max_items(int H, int G, int n_tok, int n_seq, int R) {
  return (long long)H * ((long long)n_tok * ((G + R - 1) / R) + n_seq);
}
static size_t slots_bytes(int D) {
  size_t most = 0;
  for (int i = 0; i < (D == 64 ? 4 : 2); i++) {
    const int mt = 1 + i / 2;
    const bool half = i % 2;
    const size_t b = (size_t)AT_MAX_CTAS * at_warps(D, mt, half) / at_split(D) * 2 * at_slot_floats(D, at_rows(mt, half)) * sizeof(float);
    if (b > most) most = b;
  }
  return most;
}
// slots | number of items | joins
size_t kv_attend_ws_bytes(int D, int H, int G, int n_tok, int n_seq) {
  return slots_bytes(D) + 256 + (size_t)max_items(H, G, n_tok, n_seq, 8) * sizeof(AttendJoin);
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
  p.window = a.window < 1 << 27 ? a.window : 1 << 27;  // (beyond any position: no sum below leaves 32 bits)
  p.sel = a.sel;
  p.n_sel = a.n_sel;
  p.slots = static_cast<float*>(a.ws);
  p.n_items = reinterpret_cast<int*>(static_cast<uint8_t*>(a.ws) + slots_bytes(D));
  p.joins = reinterpret_cast<AttendJoin*>(reinterpret_cast<uint8_t*>(p.n_items) + 256);
  QMV_DEBUG_ONLY(p.q_len = (long long)(kv.n_tok - 1) * a.q_stride + (long long)a.n_heads * D;
                 p.out_len = output_extent((long long)kv.n_tok * a.n_heads * D);
                 p.sel_len = a.sel ? (long long)kv.n_tok * kv.H * a.n_sel : 0;
                 p.slots_len = (long long)(slots_bytes(D) / sizeof(float));)
  return a.dtype != QMV_DT_F32 && attend_rows(p) > 8 ? launch_attend_half(p, D, stream) : launch_attend_split(p, D, stream);
}

}  // namespace qmv
