// C ABI of the head norm and rotation, adapter, expert selection and log
// probability entry points (declared in include/qmv.h): argument checking and
// dispatch.
#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "step_launch.h"

namespace qmv {

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool dtype_ok(int dt) { return dt >= QMV_DT_F32 && dt <= QMV_DT_BF16; }
static int dtype_bytes(int dt) { return dt == QMV_DT_F32 ? 4 : 2; }
static int status(cudaError_t e) { return e == cudaSuccess ? QMV_OK : QMV_ERR_CUDA; }

// Heads of one kind, [n_tok][n][D] with tokens xs / ys elements apart.
static int check_heads(int dtype, int D, int n_tok, const RopeHeads& h) {
  if (h.n < 1 || h.n > 16384) return QMV_ERR_SHAPE;
  if (!h.x || !h.y) return QMV_ERR_NULL;
  const long long row = (long long)h.n * D, far = 1ll << 40;
  if (h.xs < row || h.xs > far || h.ys < row || h.ys > far) return QMV_ERR_SHAPE;
  if (h.x == h.y && h.xs != h.ys && n_tok > 1) return QMV_ERR_SHAPE;
  if (!al16(h.x) || !al16(h.y) || !al16(h.w) || h.xs * dtype_bytes(dtype) % 16 || h.ys * dtype_bytes(dtype) % 16)
    return QMV_ERR_ALIGN;
  return QMV_OK;
}

// Rows of `len` bytes, `step` bytes apart (step >= len), one a token.
struct Rows {
  const char* at;
  long long step, len;
};
static long long floor_div(long long a, long long b) { return a / b - (a % b < 0); }
// Whether a row of a and a row of b have a byte in common.
static bool meet(const Rows& a, const Rows& b, int n) {
  const long long d = reinterpret_cast<intptr_t>(b.at) - reinterpret_cast<intptr_t>(a.at);  // of the first rows
  if (d >= (n - 1) * a.step + a.len || -d >= (n - 1) * b.step + b.len) return false;
  if (n == 1) return true;
  if (a.step == b.step) {  // parts of one buffer's rows: row j of b lies d + (j - i) step after row i of a
    const long long m = floor_div(d, a.step), r = d - m * a.step;
    return (r < a.len && m > -n && m < n) || (a.step - r < b.len && m + 1 > -n && m + 1 < n);
  }
  for (long long i = 0; i < n; i++) {  // (rows of two steps among one another: row by row)
    const long long x = i * a.step - d, first = floor_div(x - b.len, b.step) + 1, last = floor_div(x + a.len - 1, b.step);
    if (first < n && last >= 0 && first <= last) return true;
  }
  return false;
}
// Heads are read by other warps while results are written: results take exactly the
// place of their own input, or lie apart from both inputs and one another.
static bool results_apart(int dtype, int D, int n_tok, const RopeHeads& q, const RopeHeads& k) {
  const long long e = dtype_bytes(dtype);
  auto in = [&](const RopeHeads& h) { return Rows{static_cast<const char*>(h.x), h.xs * e, h.n * D * e}; };
  auto out = [&](const RopeHeads& h) { return Rows{static_cast<const char*>(h.y), h.ys * e, h.n * D * e}; };
  if (q.y != q.x && meet(in(q), out(q), n_tok)) return false;
  if (!k.n) return true;
  return (k.y == k.x || !meet(in(k), out(k), n_tok)) && !meet(in(k), out(q), n_tok) && !meet(in(q), out(k), n_tok) &&
         !meet(out(q), out(k), n_tok);
}

static int check_lora(const qmv_lora* l, int64_t K, int n_tok) {
  if (!l) return QMV_ERR_NULL;
  if (!dtype_ok(l->dtype)) return QMV_ERR_FORMAT;
  if (l->n_adapters < 1 || l->n_adapters > (1 << 20) || l->rank < 4 || l->rank > QMV_MAX_RANK || l->rank % 4 || K < 8 ||
      K > (1 << 20) || K % 8)
    return QMV_ERR_SHAPE;
  if (n_tok < 1 || n_tok > QMV_MAX_TOKENS) return QMV_ERR_NTOK;
  return QMV_OK;
}

}  // namespace qmv

using namespace qmv;

extern "C" {

int qmv_norm_rope(const qmv_rope* rope, int dtype, const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                  int n_heads, const float* q_w, const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride,
                  int n_kv_heads, const float* k_w, float eps, const int32_t* pos, const int32_t* lens,
                  const int32_t* starts, int n_seq, int n_tok, cudaStream_t stream) {
  if (!rope) return QMV_ERR_NULL;
  if (!dtype_ok(dtype)) return QMV_ERR_FORMAT;
  const int D = rope->head_dim, R = rope->rotary_dim;
  if (D < 2 || D > 256 || D % 2 || R < 2 || R > D || R % 2 || rope->n_axes < 1 || rope->n_axes > 4 ||
      !std::isfinite(rope->scale) || !(eps >= 0.f) || std::isinf(eps))
    return QMV_ERR_SHAPE;
  if (n_tok < 1 || n_tok > QMV_MAX_BATCH_TOKENS) return QMV_ERR_NTOK;
  if (!rope->freq) return QMV_ERR_NULL;
  if (!al16(rope->freq) || !al16(rope->axis)) return QMV_ERR_ALIGN;
  RopeParams p{};
  p.q.x = q, p.q.y = q_out, p.q.xs = q_stride, p.q.ys = q_out_stride, p.q.w = q_w, p.q.n = n_heads;
  p.k.x = k, p.k.y = k_out, p.k.xs = k_stride, p.k.ys = k_out_stride, p.k.w = k_w, p.k.n = n_kv_heads;
  int rc = check_heads(dtype, D, n_tok, p.q);
  if (rc) return rc;
  if (n_kv_heads != 0 || k || k_out) {
    if ((rc = check_heads(dtype, D, n_tok, p.k))) return rc;
  }
  if (pos) {
    if (lens || starts) return QMV_ERR_SHAPE;  // one or the other
    if (!al16(pos)) return QMV_ERR_ALIGN;
  } else {
    if (!lens) return QMV_ERR_NULL;
    if (!al16(lens) || !al16(starts)) return QMV_ERR_ALIGN;
    if (starts && (n_seq < 1 || n_seq > QMV_MAX_SEQS)) return QMV_ERR_SHAPE;
    if (!starts && n_seq != n_tok) return QMV_ERR_NTOK;
  }
  if (!results_apart(dtype, D, n_tok, p.q, p.k)) return QMV_ERR_SHAPE;
  if ((rc = check_device())) return rc;
  p.freq = rope->freq;
  p.axis = rope->axis;
  p.pos = pos;
  p.lens = lens;
  p.starts = starts;
  p.D = D;
  p.R = R;
  p.n_axes = rope->n_axes;
  p.n_seq = n_seq;
  p.n_tok = n_tok;
  p.eps = eps;
  p.scale = rope->scale;
  p.err = device_error_word();
  QMV_DEBUG_ONLY(p.q.x_len = (n_tok - 1) * q_stride + (long long)n_heads * D;
                 p.q.y_len = output_extent((n_tok - 1) * q_out_stride + (long long)n_heads * D);
                 p.k.x_len = (n_tok - 1) * k_stride + (long long)n_kv_heads * D;
                 p.k.y_len = output_extent((n_tok - 1) * k_out_stride + (long long)n_kv_heads * D);)
  return status(launch_norm_rope(dtype, rope->interleaved != 0, p, stream));
}

size_t qmv_lora_workspace_bytes(const qmv_lora* l, int64_t K, int n_tok) {
  if (check_lora(l, K, n_tok)) return 0;
  return (size_t)lora_splits(K, n_tok, l->rank, l->dtype) * n_tok * l->rank * sizeof(float);
}

int qmv_lora_run(const qmv_lora* l, const int32_t* ids, const float* x, const float* res, float* y, int64_t K, int64_t M,
                 int n_tok, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = check_lora(l, K, n_tok);
  if (rc) return rc;
  if (M < 1 || M > (1 << 30)) return QMV_ERR_SHAPE;
  if (!l->A || !l->B || !ids || !x || !res || !y || !ws) return QMV_ERR_NULL;
  if (!al16(l->A) || !al16(l->B) || !al16(l->ranks) || !al16(l->scales) || !al16(ids) || !al16(x) || !al16(res) ||
      !al16(y) || !al16(ws))
    return QMV_ERR_ALIGN;
  const size_t need = qmv_lora_workspace_bytes(l, K, n_tok);
  if (ws_bytes < need) return QMV_ERR_WORKSPACE;
  // y is res, or has nothing of res and x, and the workspace has nothing of the three
  // (other CTAs read res, x and the workspace meanwhile)
  auto of = [](const void* p, long long bytes) { return Rows{static_cast<const char*>(p), 0, bytes}; };
  const Rows ry = of(y, n_tok * M * 4), rr = of(res, n_tok * M * 4), rx = of(x, n_tok * K * 4), rw = of(ws, need);
  if ((y != res && meet(ry, rr, 1)) || meet(ry, rx, 1) || meet(rw, ry, 1) || meet(rw, rr, 1) || meet(rw, rx, 1))
    return QMV_ERR_SHAPE;
  if ((rc = check_device())) return rc;
  LoraParams p{};
  p.A = l->A;
  p.B = l->B;
  p.ranks = l->ranks;
  p.scales = l->scales;
  p.ids = ids;
  p.x = x;
  p.res = res;
  p.y = y;
  p.part = static_cast<float*>(ws);
  p.M = M;
  p.K = (int)K;
  p.n = l->n_adapters;
  p.r = l->rank;
  p.n_tok = n_tok;
  p.err = device_error_word();
  QMV_DEBUG_ONLY(p.a_len = (long long)p.n * p.r * K; p.b_len = (long long)p.n * p.r * M;
                 p.x_len = n_tok * K; p.part_len = (long long)qmv_lora_workspace_bytes(l, K, n_tok) / 4;
                 p.y_len = output_extent(n_tok * M);)
  return status(launch_lora(l->dtype, p, stream));
}

int moe_route_select(int dtype, const void* logits, int64_t ld, const float* bias, int n_experts, int n_tok, int top_k,
                     int gating, int n_groups, int keep, int group_top, int renorm, float scale, int32_t* ids,
                     float* gates, cudaStream_t stream) {
  if (!dtype_ok(dtype)) return QMV_ERR_FORMAT;
  if (n_experts < 1 || n_experts > 512 || n_groups < 1 || n_groups > ROUTE_MAX_GROUPS || n_experts % n_groups ||
      keep < 1 || keep > n_groups || ld < n_experts || ld > (1ll << 40) || !std::isfinite(scale) ||
      (gating != QMV_GATING_SOFTMAX && gating != QMV_GATING_SIGMOID))
    return QMV_ERR_SHAPE;
  const int size = n_experts / n_groups;
  if (keep < n_groups && (group_top < 1 || group_top > 2 || group_top > size)) return QMV_ERR_SHAPE;
  if (n_tok < 1 || n_tok > QMV_MAX_PREFILL_TOKENS || top_k < 1 || top_k > QMV_MAX_TOPK) return QMV_ERR_NTOK;
  if (top_k > keep * size) return QMV_ERR_SHAPE;
  if (!logits || !ids || !gates) return QMV_ERR_NULL;
  if (!al16(logits) || !al16(bias) || !al16(ids) || !al16(gates)) return QMV_ERR_ALIGN;
  int rc = check_device();
  if (rc) return rc;
  RouteParams p{};
  p.logits = logits;
  p.bias = bias;
  p.ids = ids;
  p.gates = gates;
  p.ld = ld;
  p.E = n_experts;
  p.n_tok = n_tok;
  p.top_k = top_k;
  p.gating = gating;
  p.groups = keep < n_groups ? n_groups : 1;
  p.keep = keep < n_groups ? keep : 1;
  p.group_top = group_top;
  p.renorm = renorm != 0;
  p.scale = scale;
  QMV_DEBUG_ONLY(p.err = device_error_word(); p.logits_len = (n_tok - 1) * ld + n_experts;
                 p.ids_len = output_extent((long long)n_tok * top_k);)
  return status(launch_route_select(dtype, p, stream));
}

int qmv_logprobs(int dtype, const void* logits, int64_t ld, int64_t rows, int64_t V, float scale, const int32_t* tokens,
                 int n_given, float* logp, float* lse, float* entropy, int n_top, int32_t* top_ids, float* top_logp,
                 cudaStream_t stream) {
  if (!dtype_ok(dtype)) return QMV_ERR_FORMAT;
  if (rows < 1 || rows > (1 << 24) || V < 1 || V > (1 << 28) || ld < V || ld > (1ll << 40) || n_given < 0 ||
      n_given > QMV_MAX_GIVEN || n_top < 0 || n_top > QMV_MAX_TOP || !(scale >= 0x1p-100f) || scale > 0x1p126f)
    return QMV_ERR_SHAPE;
  if (!logits || (n_given && (!tokens || !logp)) || (n_top && (!top_ids || !top_logp)) ||
      (!n_given && !n_top && !lse && !entropy))
    return QMV_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype) || !al16(tokens) || !al16(logp) || !al16(lse) || !al16(entropy) || !al16(top_ids) || !al16(top_logp))
    return QMV_ERR_ALIGN;
  int rc = check_device();
  if (rc) return rc;
  LogprobsParams p{};
  p.logits = logits;
  p.tokens = tokens;
  p.logp = logp;
  p.lse = lse;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_logp = top_logp;
  p.ld = ld;
  p.rows = rows;
  p.V = (int)V;
  p.n_given = n_given;
  p.n_top = n_top;
  p.scale = scale;
  p.err = device_error_word();
  QMV_DEBUG_ONLY(p.logits_len = (rows - 1) * ld + V; p.rows_len = output_extent(rows);
                 p.given_len = output_extent(rows * n_given); p.top_len = output_extent(rows * n_top);)
  return status(launch_logprobs(dtype, p, stream));
}

}  // extern "C"
