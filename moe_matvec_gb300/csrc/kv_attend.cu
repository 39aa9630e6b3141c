// Attention over the paged 8-bit cache: workspace and dispatch (the kernels are
// in kv_attend.cuh, instantiated in kv_attend_split.cu and kv_attend_half.cu).
#include "kv_attend.cuh"

namespace qmv {

cudaError_t launch_attend_split(AttendParams& p, int D, cudaStream_t stream);
cudaError_t launch_attend_half(AttendParams& p, int D, cudaStream_t stream);
cudaError_t launch_attend_split_cluster(AttendParams& p, int D, cudaStream_t stream);
cudaError_t launch_attend_half_cluster(AttendParams& p, int D, cudaStream_t stream);

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

int attend_resident_clusters(int c);

// CTAs of a cluster per item, or 0 for equal shares over the GPU and a second
// kernel.  A cluster saves that kernel, its launch and the prefix sum of the
// batch, about as much as CL_TILES tiles of a warp take, but its warps get as many
// tiles as its own sequence has: with page lists a number the host knows, else at
// most what the table can hold (against one tile for the shares: how much of the
// table is in use is not known here).  All clusters have to be resident at once.
// Measured, shares / clusters: one sequence of 1000 tokens 9.5 / 8.2 us, 32 of 500
// 10.9 / 7.3, 64 listed pages of 16 sequences (8 tiles a warp, 7 in equal shares)
// 32 / 28; where warps would get 5 tiles more than by shares (200 listed pages of 4
// sequences, with append and selection) clusters lose, 31 / 34.
constexpr int CL_TILES = 1;
static int clusters_for(AttendParams& p, int D, bool half) {
  const int mt = attend_mt(p, D, half), R = at_rows(mt, half), workers = at_warps(D, mt, half) / at_split(D);
  const bool several = p.kv.starts && !p.sel;  // tokens a sequence
  const long long items = several ? p.kv.H * ((long long)p.kv.n_tok * p.G / R + p.kv.n_seq)
                                  : (long long)p.kv.n_tok * p.kv.H * ((p.G + R - 1) / R);
  const long long slots = (long long)(p.sel ? p.n_sel : p.kv.max_pages) * p.kv.P;
  long long tiles = (slots + AT_TILE - 1) / AT_TILE;
  const long long seen = p.window + (several ? p.kv.n_tok : 1);  // positions, at most
  if (p.window > 0 && !p.sel && seen / AT_TILE + 2 < tiles) tiles = seen / AT_TILE + 2;
  int c = 1;
  while (c < 8 && c * workers < tiles && items <= attend_resident_clusters(2 * c)) c *= 2;
  if (items > attend_resident_clusters(c)) return 0;
  p.max_items = (int)items;
  const long long here = (tiles + c * workers - 1) / (c * workers);
  const long long all = p.sel ? (items * tiles + workers * device_sm_count() - 1) / (workers * device_sm_count()) : 1;
  return here <= all + CL_TILES ? c : 0;
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
  const bool half = a.dtype != QMV_DT_F32 && attend_rows(p) > 8;
  p.cluster = clusters_for(p, D, half);
  if (p.cluster) return half ? launch_attend_half_cluster(p, D, stream) : launch_attend_split_cluster(p, D, stream);
  return half ? launch_attend_half(p, D, stream) : launch_attend_split(p, D, stream);
}

}  // namespace qmv
