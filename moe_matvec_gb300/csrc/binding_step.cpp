// CPython binding of the head norm and rotation, adapter, expert selection and
// log probability entry points, in the manner of binding.cpp.
#include "binding_util.h"

#include <c10/cuda/CUDACachingAllocator.h>

#include <algorithm>
#include <initializer_list>
#include <vector>

namespace {

struct Abi {
  decltype(&qmv_norm_rope) norm_rope;
  decltype(&qmv_lora_run) lora_run;
  decltype(&qmv_lora_workspace_bytes) lora_workspace_bytes;
  decltype(&moe_route_select) route_select;
  decltype(&qmv_logprobs) logprobs;
} abi{};

// (error class, addresses of the functions of Abi in order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    void* p[5];
    for (int i = 0; i < 5; i++) p[i] = reinterpret_cast<void*>(integer(a[i + 1]));
    Py_XDECREF(qmv_error);
    Py_INCREF(a[0]);
    qmv_error = a[0];
    abi.norm_rope = reinterpret_cast<decltype(abi.norm_rope)>(p[0]);
    abi.lora_run = reinterpret_cast<decltype(abi.lora_run)>(p[1]);
    abi.lora_workspace_bytes = reinterpret_cast<decltype(abi.lora_workspace_bytes)>(p[2]);
    abi.route_select = reinterpret_cast<decltype(abi.route_select)>(p[3]);
    abi.logprobs = reinterpret_cast<decltype(abi.logprobs)>(p[4]);
    Py_RETURN_NONE;
  });
}

// The kernels run on the current device, so a call's tensors have to live there.
struct Here {
  mutable int dev = -1;  // looked up once a call
  void operator()(const at::Tensor& t) const {
    on_device(t);
    if (dev < 0) dev = c10::cuda::current_device();
    if (t.device().index() != dev)
      value_error("tensor on " + t.device().str() + ", but the current device is cuda:" + std::to_string(dev));
  }
};

// A descriptor's tensors: `mark` is their device's index + 1, as api.py keeps it in the
// reserved field (0: not known).
void there(const Here& here, int32_t mark, const char* what) {
  if (mark > 0 && mark - 1 != here.dev)
    value_error(std::string(what) + " has its tensors on cuda:" + std::to_string(mark - 1) + ", but the current device is cuda:" +
                std::to_string(here.dev));
}

// An optional tensor of this type and shape: its address or NULL.
void* maybe(const Here& here, PyObject* o, at::ScalarType type, at::IntArrayRef shape, const char* what) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, what);
  void* p = typed(t, type, shape, what);
  here(t);
  return p;
}

// New memory on the current device for work on st (without the dispatcher, which
// takes a microsecond of a small call); as fresh(), kept until that work is done.
c10::Storage memory(int64_t bytes, cudaStream_t st) {
  c10::Allocator* a = c10::GetAllocator(c10::DeviceType::CUDA);
  c10::Storage s(c10::Storage::use_byte_size_t(), (size_t)bytes, a->allocate((size_t)bytes), a, true);
  if (st != c10::cuda::getCurrentCUDAStream().stream()) {
    const c10::DeviceIndex dev = c10::cuda::current_device();
    c10::cuda::CUDACachingAllocator::recordStream(s.data_ptr(), c10::cuda::getStreamFromExternal(st, dev));
  }
  return s;
}
at::Tensor over(const c10::Storage& memory, int64_t byte, at::IntArrayRef shape, at::ScalarType type) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(memory), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                   c10::scalarTypeToTypeMeta(type));
  impl->set_storage_offset(byte / (int64_t)c10::elementSize(type));
  impl->set_sizes_contiguous(shape);
  return at::Tensor(std::move(impl));
}

// A result of one call: given, or a part of the memory that the new ones share.
struct Part {
  PyObject* given;
  at::ScalarType type;
  std::vector<int64_t> shape;
  const char* what;
  at::Tensor t;
  int64_t bytes() const {
    int64_t b = (int64_t)c10::elementSize(type);
    for (int64_t s : shape) b *= s;
    return (b + 15) / 16 * 16;
  }
};
// New results of up to eight megabytes are one allocation (which costs the host more
// than all else of a small call); larger ones have one each, so that none keeps
// another's memory.
void allot(const Here& here, std::initializer_list<Part*> parts, cudaStream_t st) {
  int64_t all = 0;
  int fresh_ones = 0;
  for (Part* p : parts) {
    if (p->given != Py_None) {
      p->t = tensor(p->given, p->what);
      typed(p->t, p->type, p->shape, p->what);
      here(p->t);
    } else {
      all += p->bytes();
      fresh_ones++;
    }
  }
  const bool one = fresh_ones > 1 && all <= 8 << 20;
  c10::Storage shared;
  if (one) shared = memory(all, st);
  int64_t at = 0;
  for (Part* p : parts) {
    if (p->given != Py_None) continue;
    p->t = one ? over(shared, at, p->shape, p->type) : over(memory(p->bytes(), st), 0, p->shape, p->type);
    at += p->bytes();
  }
}

// The address and token stride of [n_tok][heads][D], heads and dimensions
// contiguous.
void* heads_of(const Here& here, const at::Tensor& t, int64_t D, const char* what, int64_t& stride) {
  if (t.dim() != 3 || t.size(2) != D)
    value_error(std::string(what) + ": [n_tok][heads][" + std::to_string(D) + "] wanted, got " + text(t.sizes()));
  here(t);
  if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != D))
    value_error(std::string(what) + ": the heads and dimensions of a token must be contiguous");
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) value_error(std::string(what) + ": too large");
  stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * D;
  return t.data_ptr();
}

// Rows of values [n][K], the values of a row contiguous.
void* rows_of(const Here& here, const at::Tensor& t, const char* what, int64_t& ld) {
  if (t.dim() != 2) value_error(std::string(what) + ": a matrix wanted, got " + text(t.sizes()));
  here(t);
  if (t.size(1) > 1 && t.stride(1) != 1) value_error(std::string(what) + ": the values of a row must be contiguous");
  ld = t.size(0) > 1 ? t.stride(0) : t.size(1);
  return t.data_ptr();
}

// (rope, q, k, q_w, k_w, eps, pos, lens, starts, q_out, k_out, stream) -> (q_out, k_out)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Here here;
    const qmv_rope* rope = reinterpret_cast<const qmv_rope*>(integer(a[0]));
    const int64_t D = rope->head_dim;
    const at::Tensor& q = tensor(a[1], "q");
    const int dt = dtype_code(q.scalar_type());
    int64_t qs, ks = 0, qos, kos = 0, kv = 0;
    void *qp = heads_of(here, q, D, "q", qs), *kp = nullptr;
    there(here, rope->reserved, "rope");
    const int64_t n_tok = q.size(0);
    const bool has_k = a[2] != Py_None;
    if (has_k) {
      const at::Tensor& k = tensor(a[2], "k");
      kp = heads_of(here, k, D, "k", ks);
      if (k.scalar_type() != q.scalar_type() || k.size(0) != n_tok) value_error("q and k must be of one type and length");
      kv = k.size(1);
    } else if (a[10] != Py_None) {
      value_error("k_out without k");
    }
    const float* qw = static_cast<const float*>(maybe(here, a[3], at::kFloat, {D}, "q_w"));
    const float* kw = static_cast<const float*>(maybe(here, a[4], at::kFloat, {D}, "k_w"));
    const float eps = (float)real(a[5]);
    if ((a[6] != Py_None) == (a[7] != Py_None)) value_error("positions are given by pos or by lens (and starts)");
    if (a[6] != Py_None && a[8] != Py_None) value_error("starts goes with lens");
    const int32_t *pos = static_cast<const int32_t*>(maybe(here, a[6], at::kInt, {n_tok, rope->n_axes}, "pos")), *lens = nullptr,
                  *starts = nullptr;
    int64_t n_seq = 0;
    if (a[7] != Py_None) {
      const at::Tensor& t = tensor(a[7], "lens");
      if (t.dim() != 1 || t.numel() > INT32_MAX) value_error("lens: [n_seq] wanted");
      n_seq = t.numel();
      lens = ints(t);
      here(t);
      starts = static_cast<const int32_t*>(maybe(here, a[8], at::kInt, {n_seq + 1}, "starts"));
    }
    const cudaStream_t st = stream_of(a[11]);
    // given outputs may be strided like q and k
    auto out = [&](PyObject* o, int64_t heads, const char* what, int64_t& stride) -> void* {
      const at::Tensor& t = tensor(o, what);
      void* p = heads_of(here, t, D, what, stride);
      if (t.scalar_type() != q.scalar_type() || t.size(0) != n_tok || t.size(1) != heads)
        value_error(std::string(what) + ": the type and shape of its input wanted");
      return p;
    };
    Part qo{Py_None, q.scalar_type(), {n_tok, q.size(1), D}, "q_out", {}}, ko{Py_None, q.scalar_type(), {n_tok, kv, D}, "k_out", {}};
    void *qop, *kop = nullptr;
    const bool new_q = a[9] == Py_None, new_k = has_k && a[10] == Py_None;
    if (new_q && new_k) allot(here, {&qo, &ko}, st);
    else if (new_q) allot(here, {&qo}, st);
    else if (new_k) allot(here, {&ko}, st);
    if (new_q) qop = qo.t.data_ptr(), qos = q.size(1) * D;
    else qo.t = tensor(a[9], "q_out"), qop = out(a[9], q.size(1), "q_out", qos);
    if (new_k) kop = ko.t.data_ptr(), kos = kv * D;
    else if (has_k) ko.t = tensor(a[10], "k_out"), kop = out(a[10], kv, "k_out", kos);
    check(called([&] {
            return abi.norm_rope(rope, dt, qp, qs, qop, qos, (int)q.size(1), qw, kp, ks, kop, kos, (int)kv, kw, eps, pos,
                                 lens, starts, (int)n_seq, (int)n_tok, st);
          }),
          "qmv_norm_rope");
    return Py_BuildValue("(NN)", wrap(qo.t), wrap(ko.t));
  });
}

// (lora, K, M, ids, x, r, out, ws, stream) -> out
PyObject* lora_run(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Here here;
    const qmv_lora* l = reinterpret_cast<const qmv_lora*>(integer(a[0]));
    const int64_t K = integer(a[1]), M = integer(a[2]);
    const at::Tensor &ids = tensor(a[3], "ids"), &x = tensor(a[4], "x"), &r = tensor(a[5], "r");
    if (ids.dim() != 1) value_error("ids: [n_tok] wanted");
    const int64_t n_tok = ids.size(0);
    if (n_tok > INT32_MAX) value_error("too many tokens");
    const int32_t* ip = ints(ids);
    const float* xp = static_cast<const float*>(typed(x, at::kFloat, {n_tok, K}, "x"));
    const float* rp = static_cast<const float*>(typed(r, at::kFloat, {n_tok, M}, "r"));
    here(x);
    here(ids);
    here(r);
    there(here, l->reserved, "lora");
    const cudaStream_t st = stream_of(a[8]);
    Part out{a[6], at::kFloat, {n_tok, M}, "out", {}};
    allot(here, {&out}, st);
    c10::Storage scratch;
    void* ws;
    size_t ws_bytes;
    if (a[7] == Py_None) {
      ws_bytes = std::max<size_t>(16, abi.lora_workspace_bytes(l, K, (int)n_tok));
      scratch = memory((int64_t)ws_bytes, st);
      ws = scratch.mutable_data();
    } else {
      const at::Tensor& t = tensor(a[7], "ws");
      ws = ptr(t);
      here(t);
      ws_bytes = t.nbytes();
    }
    check(called([&] {
            return abi.lora_run(l, ip, xp, rp, static_cast<float*>(out.t.data_ptr()), K, M, (int)n_tok, ws, ws_bytes, st);
          }),
          "qmv_lora_run");
    return wrap(out.t);
  });
}

// (logits, top_k, gating, bias, groups, keep, group_top, renorm, scale, ids, gates, stream) -> (ids, gates)
PyObject* route_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Here here;
    const at::Tensor& logits = tensor(a[0], "logits");
    const int dt = dtype_code(logits.scalar_type());
    int64_t ld;
    const void* lp = rows_of(here, logits, "logits", ld);
    const int64_t n_tok = logits.size(0), E = logits.size(1);
    if (n_tok > INT32_MAX || E > INT32_MAX) value_error("logits: too large");
    const int top_k = as_int(a[1]);
    const float* bias = static_cast<const float*>(maybe(here, a[3], at::kFloat, {E}, "bias"));
    const int renorm = PyObject_IsTrue(a[7]);
    if (renorm < 0) throw Raised{};
    const float scale = (float)real(a[8]);
    const cudaStream_t st = stream_of(a[11]);
    if (top_k < 1 || top_k > QMV_MAX_TOPK) check(QMV_ERR_NTOK, "moe_route_select");
    Part ids{a[9], at::kInt, {n_tok, top_k}, "ids", {}}, gates{a[10], at::kFloat, {n_tok, top_k}, "gates", {}};
    allot(here, {&ids, &gates}, st);
    const int gating = as_int(a[2]), groups = as_int(a[4]), keep = as_int(a[5]), group_top = as_int(a[6]);
    check(called([&] {
            return abi.route_select(dt, lp, ld, bias, (int)E, (int)n_tok, top_k, gating, groups, keep, group_top, renorm,
                                    scale, static_cast<int32_t*>(ids.t.data_ptr()), static_cast<float*>(gates.t.data_ptr()),
                                    st);
          }),
          "moe_route_select");
    return Py_BuildValue("(NN)", wrap(ids.t), wrap(gates.t));
  });
}

// (logits, tokens, n_top, scale, logp, lse, entropy, ids, top, stream) -> (logp, lse, entropy, ids, top)
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Here here;
    const at::Tensor& logits = tensor(a[0], "logits");
    const int dt = dtype_code(logits.scalar_type());
    int64_t ld;
    const void* lp = rows_of(here, logits, "logits", ld);
    const int64_t rows = logits.size(0), V = logits.size(1);
    int64_t given = 0;
    const int32_t* tokens = nullptr;
    if (a[1] != Py_None) {
      const at::Tensor& t = tensor(a[1], "tokens");
      if (t.dim() != 2 || t.size(0) != rows) value_error("tokens: [rows][n_given] wanted, got " + text(t.sizes()));
      given = t.size(1);
      if (given < 1 || given > QMV_MAX_GIVEN) check(QMV_ERR_SHAPE, "qmv_logprobs");
      tokens = ints(t);
      here(t);
    }
    const int n_top = as_int(a[2]);
    if (n_top < 0 || n_top > QMV_MAX_TOP) check(QMV_ERR_SHAPE, "qmv_logprobs");
    const float scale = (float)real(a[3]);
    const cudaStream_t st = stream_of(a[9]);
    if ((!given && a[4] != Py_None) || (!n_top && (a[7] != Py_None || a[8] != Py_None)))
      value_error("an output for a result that was not asked for");
    Part logp{a[4], at::kFloat, {rows, given}, "logp", {}}, lse{a[5], at::kFloat, {rows}, "lse", {}},
        entropy{a[6], at::kFloat, {rows}, "entropy", {}}, ids{a[7], at::kInt, {rows, n_top}, "ids", {}},
        top{a[8], at::kFloat, {rows, n_top}, "top", {}};
    if (given && n_top) allot(here, {&logp, &lse, &entropy, &ids, &top}, st);
    else if (given) allot(here, {&logp, &lse, &entropy}, st);
    else if (n_top) allot(here, {&lse, &entropy, &ids, &top}, st);
    else allot(here, {&lse, &entropy}, st);
    auto at_or_null = [](const Part& p) { return p.t.defined() ? p.t.data_ptr() : nullptr; };
    check(called([&] {
            return abi.logprobs(dt, lp, ld, rows, V, scale, tokens, (int)given, static_cast<float*>(at_or_null(logp)),
                                static_cast<float*>(at_or_null(lse)), static_cast<float*>(at_or_null(entropy)), n_top,
                                static_cast<int32_t*>(at_or_null(ids)), static_cast<float*>(at_or_null(top)), st);
          }),
          "qmv_logprobs");
    return Py_BuildValue("(NNNNN)", wrap(logp.t), wrap(lse.t), wrap(entropy.t), wrap(ids.t), wrap(top.t));
  });
}

PyMethodDef methods[] = {QMV_METHOD(bind),         QMV_METHOD(norm_rope), QMV_METHOD(lora_run),
                         QMV_METHOD(route_select), QMV_METHOD(logprobs),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding_step", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding_step(void) { return PyModule_Create(&module); }
