// C ABI of the norm, cache, attention and page selection entry points
// (declared in include/qmv.h): argument checking and dispatch.
#include <cmath>

#include "kv_cache.cuh"
#include "kv_launch.h"
#include "launch.h"

namespace qmv {

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool dtype_ok(int dt) { return dt >= QMV_DT_F32 && dt <= QMV_DT_BF16; }
static int dtype_bytes(int dt) { return dt == QMV_DT_F32 ? 4 : 2; }
static int status(cudaError_t e) { return e == cudaSuccess ? QMV_OK : QMV_ERR_CUDA; }

static int check_cache(const qmv_kv_cache* c) {
  if (!c) return QMV_ERR_NULL;
  if (qmv_kv_page_bytes(c->head_dim, c->page_tokens) < 0 || c->n_kv_heads < 1 || c->n_kv_heads > 1024 ||
      c->n_pages < 1)
    return QMV_ERR_SHAPE;
  return QMV_OK;
}

static int check_batch(const qmv_kv_cache* c, const qmv_kv_batch* b, int max_tok) {
  int rc = check_cache(c);
  if (rc) return rc;
  if (!b) return QMV_ERR_NULL;
  if (b->n_seq < 1 || b->n_seq > QMV_MAX_SEQS || b->max_pages < 1 || b->max_pages > KV_MAX_PAGES)
    return QMV_ERR_SHAPE;
  if (b->n_tok < 1 || b->n_tok > max_tok || (!b->starts && b->n_tok != b->n_seq)) return QMV_ERR_NTOK;
  if (!b->table || !b->lens || !c->pages) return QMV_ERR_NULL;
  if (!al16(b->table) || !al16(b->lens) || !al16(b->starts) || !al16(c->pages) || !al16(c->bounds))
    return QMV_ERR_ALIGN;
  return QMV_OK;
}

// A token's rows of `row` elements, `stride` elements apart.
static int check_rows(int dtype, const void* x, long long row, long long stride) {
  if (!x) return QMV_ERR_NULL;
  if (stride < row || stride > (1ll << 40)) return QMV_ERR_SHAPE;
  if (!al16(x) || stride * dtype_bytes(dtype) % 16) return QMV_ERR_ALIGN;
  return QMV_OK;
}

static KvParams params(const qmv_kv_cache* c, const qmv_kv_batch* b) {
  KvParams p{};
  p.pages = static_cast<uint8_t*>(c->pages);
  p.bounds = static_cast<uint8_t*>(c->bounds);
  p.table = b->table;
  p.lens = b->lens;
  p.starts = b->starts;
  p.H = c->n_kv_heads;
  p.P = c->page_tokens;
  p.log_p = c->page_tokens == 16 ? 4 : c->page_tokens == 32 ? 5 : 6;
  p.n_pages = c->n_pages;
  p.n_seq = b->n_seq;
  p.max_pages = b->max_pages;
  p.n_tok = b->n_tok;
  p.err = device_error_word();
  QMV_DEBUG_ONLY(p.pages_len = (long long)c->n_pages * c->n_kv_heads * kv_page_bytes(c->head_dim, c->page_tokens);
                 p.bounds_len = c->bounds ? (long long)c->n_pages * c->n_kv_heads * kv_bounds_bytes(c->head_dim) : 0;
                 p.table_len = (long long)b->n_seq * b->max_pages;)
  return p;
}

}  // namespace qmv

using namespace qmv;

extern "C" {

int qmv_rms_norm(int dtype, const void* x, int64_t ldx, const void* r, const float* w, float eps, int64_t rows,
                 int64_t K, void* res, void* y, int8_t* q, float* d, int32_t* sum, cudaStream_t stream) {
  if (!dtype_ok(dtype)) return QMV_ERR_FORMAT;
  if (K < 1 || K > QMV_MAX_NORM || rows < 1 || rows > (1 << 24) || ldx < K || ldx > (1ll << 40) || !(eps >= 0.f) ||
      std::isinf(eps) || (q && K % 256))
    return QMV_ERR_SHAPE;
  if (!x || !w || (!res && !y && !q) || (q && (!d || !sum)) || (!q && (d || sum))) return QMV_ERR_NULL;
  if (!al16(x) || !al16(r) || !al16(w) || !al16(res) || !al16(y) || !al16(q) || !al16(d) || !al16(sum))
    return QMV_ERR_ALIGN;
  const bool vec = K % 8 == 0 && ldx * dtype_bytes(dtype) % 16 == 0;
  if (q && !vec) return QMV_ERR_ALIGN;
  int rc = check_device();
  if (rc) return rc;
  NormParams p{};
  p.x = x;
  p.r = r;
  p.w = w;
  p.res = res;
  p.y = y;
  p.q = q;
  p.d = d;
  p.s = sum;
  p.ldx = ldx;
  p.rows = rows;
  p.K = (int)K;
  p.eps = eps;
  p.inv_k = 1.0f / (float)K;
  QMV_DEBUG_ONLY(p.err = device_error_word(); p.x_len = (rows - 1) * ldx + K; p.n = rows * K;
                 p.out_len = output_extent(rows * K);)
  return status(launch_rms_norm(dtype, p, vec, stream, true));
}

int qmv_dequantize_act(int dtype, const int8_t* q, const float* d, int64_t rows, int64_t K, void* out,
                       cudaStream_t stream) {
  if (!dtype_ok(dtype)) return QMV_ERR_FORMAT;
  if (K < 1 || K > (1 << 20) || K % 256 || rows < 1 || rows > (1 << 24)) return QMV_ERR_SHAPE;
  if (!q || !d || !out) return QMV_ERR_NULL;
  if (!al16(q) || !al16(d) || !al16(out)) return QMV_ERR_ALIGN;
  int rc = check_device();
  if (rc) return rc;
  return status(launch_act_dequant(dtype, q, d, rows * K, out, stream, true));
}

int64_t qmv_kv_page_bytes(int head_dim, int page_tokens) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 192 && head_dim != 256) return QMV_ERR_SHAPE;
  if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64) return QMV_ERR_SHAPE;
  return kv_page_bytes(head_dim, page_tokens);
}

int64_t qmv_kv_bounds_bytes(int head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 192 && head_dim != 256) return QMV_ERR_SHAPE;
  return kv_bounds_bytes(head_dim);
}

int qmv_kv_append(const qmv_kv_cache* c, const qmv_kv_batch* b, int dtype, const void* k, int64_t k_stride,
                  const void* v, int64_t v_stride, cudaStream_t stream) {
  if (!dtype_ok(dtype)) return QMV_ERR_FORMAT;
  int rc = check_batch(c, b, QMV_MAX_BATCH_TOKENS);
  if (rc) return rc;
  const long long row = (long long)c->n_kv_heads * c->head_dim;
  if ((rc = check_rows(dtype, k, row, k_stride)) || (rc = check_rows(dtype, v, row, v_stride))) return rc;
  if ((rc = check_device())) return rc;
  return status(launch_kv_append(params(c, b), dtype, c->head_dim, k, k_stride, v, v_stride, stream));
}

int qmv_kv_read(const qmv_kv_cache* c, const qmv_kv_batch* b, int dtype, void* k, void* v, cudaStream_t stream) {
  if (!dtype_ok(dtype)) return QMV_ERR_FORMAT;
  int rc = check_batch(c, b, 1 << 24);
  if (rc) return rc;
  if (!k || !v) return QMV_ERR_NULL;
  if (!al16(k) || !al16(v)) return QMV_ERR_ALIGN;
  if ((rc = check_device())) return rc;
  return status(launch_kv_read(params(c, b), dtype, c->head_dim, k, v, stream));
}

size_t qmv_kv_attend_workspace_bytes(const qmv_kv_cache* c, int n_heads, int n_tok, int n_seq) {
  if (check_cache(c) || n_heads < 1 || n_heads % c->n_kv_heads || n_tok < 1 || n_seq < 1) return 0;
  return kv_attend_ws_bytes(c->head_dim, c->n_kv_heads, n_heads / c->n_kv_heads, n_tok, n_seq);
}

int qmv_kv_attend(const qmv_kv_cache* c, const qmv_kv_batch* b, int dtype, const void* q, int64_t q_stride, void* out,
                  int n_heads, float scale, int causal, int window, const int32_t* pages, int n_sel, void* ws,
                  size_t ws_bytes, cudaStream_t stream) {
  if (!dtype_ok(dtype)) return QMV_ERR_FORMAT;
  int rc = check_batch(c, b, QMV_MAX_BATCH_TOKENS);
  if (rc) return rc;
  if (n_heads < 1 || n_heads > 16384 || n_heads % c->n_kv_heads || !std::isfinite(scale) || window < 0 ||
      (pages && (n_sel < 1 || n_sel > KV_MAX_PAGES)))
    return QMV_ERR_SHAPE;
  if ((rc = check_rows(dtype, q, (long long)n_heads * c->head_dim, q_stride))) return rc;
  if (!out || !ws) return QMV_ERR_NULL;
  if (!al16(out) || !al16(ws) || !al16(pages)) return QMV_ERR_ALIGN;
  if (ws_bytes < qmv_kv_attend_workspace_bytes(c, n_heads, b->n_tok, b->n_seq)) return QMV_ERR_WORKSPACE;
  if ((rc = check_device())) return rc;
  AttendArgs a{dtype, q, q_stride, out, n_heads, scale, causal, window, pages, n_sel, ws};
  return status(launch_kv_attend(params(c, b), c->head_dim, a, stream));
}

size_t qmv_kv_select_workspace_bytes(const qmv_kv_cache* c, const qmv_kv_batch* b) {
  if (check_cache(c) || !b || b->n_tok < 1 || b->max_pages < 1) return 0;
  return kv_select_ws_bytes(c->n_kv_heads, b->n_tok, b->max_pages);
}

int qmv_kv_select(const qmv_kv_cache* c, const qmv_kv_batch* b, int dtype, const void* q, int64_t q_stride, int n_heads,
                  int32_t* ids, int n_sel, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!dtype_ok(dtype)) return QMV_ERR_FORMAT;
  int rc = check_batch(c, b, QMV_MAX_BATCH_TOKENS);
  if (rc) return rc;
  if (n_heads < 1 || n_heads > 16384 || n_heads % c->n_kv_heads || n_heads / c->n_kv_heads > 256 || n_sel < 1 ||
      n_sel > KV_MAX_PAGES)
    return QMV_ERR_SHAPE;
  if ((rc = check_rows(dtype, q, (long long)n_heads * c->head_dim, q_stride))) return rc;
  if (!c->bounds || !ids || !ws) return QMV_ERR_NULL;
  if (!al16(ids) || !al16(ws)) return QMV_ERR_ALIGN;
  if (ws_bytes < kv_select_ws_bytes(c->n_kv_heads, b->n_tok, b->max_pages)) return QMV_ERR_WORKSPACE;
  if ((rc = check_device())) return rc;
  SelectArgs a{dtype, q, q_stride, n_heads, ids, n_sel, ws};
  return status(launch_kv_select(params(c, b), c->head_dim, a, stream));
}

}  // extern "C"
