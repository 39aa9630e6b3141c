// CPython binding of the norm, cache, attention and page selection entry
// points: tensors are checked, results allocated and the C ABI called without
// going through Python for each of these steps.  (A decode step makes these
// calls for every layer: the ctypes form of kv_attend took 10 us of the Grace
// host, of which the launches are 4.)  The functions of the C ABI come as
// addresses from the loaded library, so the same binding drives the release and
// the range-checked build.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/core/TensorImpl.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <exception>
#include <string>

#include "qmv.h"

namespace {

struct Abi {
  decltype(&qmv_rms_norm) rms_norm;
  decltype(&qmv_dequantize_act) dequantize_act;
  decltype(&qmv_kv_append) kv_append;
  decltype(&qmv_kv_read) kv_read;
  decltype(&qmv_kv_attend) kv_attend;
  decltype(&qmv_kv_attend_workspace_bytes) kv_attend_workspace_bytes;
  decltype(&qmv_kv_select) kv_select;
  decltype(&qmv_kv_select_workspace_bytes) kv_select_workspace_bytes;
} abi{};
PyObject* qmv_error = nullptr;  // the binding's exception class (code, call)

// A Python error is set.
struct Raised {};

[[noreturn]] void value_error(const std::string& s) {
  PyErr_SetString(PyExc_ValueError, s.c_str());
  throw Raised{};
}

void check(int rc, const char* what) {
  if (rc == 0) return;
  PyObject* e = PyObject_CallFunction(qmv_error, "is", rc, what);
  if (e) {
    PyErr_SetObject(qmv_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: a tensor wanted", what);
    throw Raised{};
  }
  return THPVariable_Unpack(o);
}

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return QMV_DT_F32;
    case at::kHalf: return QMV_DT_F16;
    case at::kBFloat16: return QMV_DT_BF16;
    default: value_error(std::string("float32, float16 or bfloat16 tensor wanted, got ") + c10::toString(t));
  }
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); i++) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

void on_device(const at::Tensor& t) {
  if (!t.is_cuda()) value_error("tensor must be on a CUDA device");
}

// The address of a contiguous CUDA tensor.
void* ptr(const at::Tensor& t) {
  on_device(t);
  if (!t.is_contiguous()) value_error("tensor must be contiguous");
  return t.data_ptr();
}

// The address of a contiguous CUDA tensor of this type and shape.
void* typed(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, const char* what) {
  if (t.scalar_type() != type || t.sizes() != shape)
    value_error(std::string(what) + ": " + c10::toString(type) + " " + text(shape) + " wanted, got " +
                c10::toString(t.scalar_type()) + " " + text(t.sizes()));
  return ptr(t);
}

// The stream of a call: the given one's handle, or torch's current one.
cudaStream_t stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (PyErr_Occurred()) throw Raised{};
  return reinterpret_cast<cudaStream_t>(v);
}

// A new tensor for work on st.  The allocator takes memory for used on the
// current stream: it is told where that is another one, so that memory dropped
// early (a workspace always is) goes to nobody before the work is done.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like, cudaStream_t st) {
  at::Tensor t = at::empty(shape, like.options().dtype(type));
  const c10::DeviceIndex dev = t.device().index();
  if (st != c10::cuda::getCurrentCUDAStream(dev).stream()) t.record_stream(c10::cuda::getStreamFromExternal(st, dev).unwrap());
  return t;
}

// A tensor of its own type over part of buf's memory (which it keeps): results
// that belong together share one allocation, which costs the host more than
// all else of a small call.
at::Tensor piece(const at::Tensor& buf, int64_t byte, at::IntArrayRef shape, at::ScalarType type) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                   c10::scalarTypeToTypeMeta(type));
  impl->set_storage_offset(byte / (int64_t)c10::elementSize(type));
  impl->set_sizes_contiguous(shape);
  return at::Tensor(std::move(impl));
}

// A given result, checked, or a new one on like's device.
at::Tensor result(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const at::Tensor& like, cudaStream_t st, const char* what) {
  if (o == Py_None) {
    on_device(like);
    return fresh(shape, type, like, st);
  }
  const at::Tensor& t = tensor(o, what);
  typed(t, type, shape, what);
  return t;
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int as_int(PyObject* o) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error("integer out of range");
  return (int)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

const qmv_kv_cache* cache_of(PyObject* o) { return reinterpret_cast<const qmv_kv_cache*>(integer(o)); }

const int32_t* ints(const at::Tensor& t) {
  if (t.scalar_type() != at::kInt) value_error(std::string("int32 tensor wanted, got ") + c10::toString(t.scalar_type()));
  return static_cast<const int32_t*>(ptr(t));
}

qmv_kv_batch batch_of(PyObject* table_o, PyObject* lens_o, PyObject* starts_o, int64_t n_tok) {
  const at::Tensor &table = tensor(table_o, "table"), &lens = tensor(lens_o, "lens");
  if (table.dim() != 2) value_error("table: [n_seq][max_pages] wanted");
  const int64_t n_seq = table.size(0);
  const bool ragged = starts_o != Py_None;
  if (lens.dim() != 1 || lens.size(0) != n_seq ||
      (ragged && (tensor(starts_o, "starts").dim() != 1 || tensor(starts_o, "starts").size(0) != n_seq + 1)))
    value_error("lens [" + std::to_string(n_seq) + "] and starts [" + std::to_string(n_seq + 1) +
                "] wanted for a table of " + std::to_string(n_seq) + " sequences");
  if (n_tok > INT32_MAX || n_seq > INT32_MAX || table.size(1) > INT32_MAX) value_error("batch too large");
  qmv_kv_batch b{};
  b.table = ints(table);
  b.lens = ints(lens);
  b.starts = ragged ? ints(tensor(starts_o, "starts")) : nullptr;
  b.n_seq = (int32_t)n_seq;
  b.max_pages = (int32_t)table.size(1);
  b.n_tok = (int32_t)n_tok;
  return b;
}

// The address and token stride of [n_tok][heads][D], heads and dimensions
// contiguous.
const void* rows(const at::Tensor& t, const qmv_kv_cache* c, int64_t heads, const char* what, int64_t& stride) {
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != c->head_dim)
    value_error(std::string(what) + ": [n_tok][" + std::to_string(heads) + "][" + std::to_string(c->head_dim) +
                "] wanted, got " + text(t.sizes()));
  on_device(t);
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != t.size(2)))
    value_error(std::string(what) + ": the heads and dimensions of a token must be contiguous");
  stride = t.size(0) > 1 ? t.stride(0) : heads * t.size(2);
  return t.data_ptr();
}

template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", want, got);
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <class F>
int called(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

// (error class, addresses of the functions of Abi in order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    void* p[8];
    for (int i = 0; i < 8; i++) p[i] = reinterpret_cast<void*>(integer(a[i + 1]));
    Py_XDECREF(qmv_error);
    Py_INCREF(a[0]);
    qmv_error = a[0];
    abi.rms_norm = reinterpret_cast<decltype(abi.rms_norm)>(p[0]);
    abi.dequantize_act = reinterpret_cast<decltype(abi.dequantize_act)>(p[1]);
    abi.kv_append = reinterpret_cast<decltype(abi.kv_append)>(p[2]);
    abi.kv_read = reinterpret_cast<decltype(abi.kv_read)>(p[3]);
    abi.kv_attend = reinterpret_cast<decltype(abi.kv_attend)>(p[4]);
    abi.kv_attend_workspace_bytes = reinterpret_cast<decltype(abi.kv_attend_workspace_bytes)>(p[5]);
    abi.kv_select = reinterpret_cast<decltype(abi.kv_select)>(p[6]);
    abi.kv_select_workspace_bytes = reinterpret_cast<decltype(abi.kv_select_workspace_bytes)>(p[7]);
    Py_RETURN_NONE;
  });
}

PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

// (x, w, eps, r, want: 1 float, 2 q8, 3 both, y, q8, res, stream) -> (y, q8, res)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
    if (x.dim() != 2) value_error("x: [n][K] wanted");
    const int dt = dtype_code(x.scalar_type());
    on_device(x);
    const int64_t rows_n = x.size(0), K = x.size(1);
    if (K > 1 && x.stride(1) != 1) value_error("x: the values of a row must be contiguous");
    const int want = as_int(a[4]);
    void* wp = typed(w, at::kFloat, {K}, "w");
    void* rp = a[3] == Py_None ? nullptr : typed(tensor(a[3], "r"), x.scalar_type(), x.sizes(), "r");
    const cudaStream_t st = stream_of(a[8]);
    at::Tensor y, q, d, s, res;
    // New results of up to a megabyte are one allocation (y | codes, scales, sums
    // | res); larger ones two or three, so that none keeps another's memory.
    const bool new_y = a[5] == Py_None && (want & 1), new_q = a[6] == Py_None && (want & 2), new_res = a[7] == Py_None && rp;
    if (new_q && K % 256) check(QMV_ERR_SHAPE, "qmv_rms_norm");
    // (K % 256 == 0 keeps the parts 16-byte aligned)
    const int64_t codes = rows_n * K, scales = codes / 8, floats = (codes * (int64_t)c10::elementSize(x.scalar_type()) + 255) / 256 * 256;
    const int64_t at_q = new_y ? floats : 0, at_res = at_q + (new_q ? codes + 2 * scales : 0), all = at_res + (new_res ? floats : 0);
    const bool one = new_y + new_q + new_res > 1 && all <= 1 << 20;
    const at::Tensor shared = one ? fresh({all}, at::kByte, x, st) : at::Tensor();
    if (one && new_y) y = piece(shared, 0, x.sizes(), x.scalar_type());
    else if (a[5] != Py_None || new_y) y = result(a[5], x.scalar_type(), x.sizes(), x, st, "y");
    if (a[6] != Py_None) {
      if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 3) value_error("q8: a tuple (q, d, s) wanted");
      q = result(PyTuple_GET_ITEM(a[6], 0), at::kChar, x.sizes(), x, st, "q8");
      d = result(PyTuple_GET_ITEM(a[6], 1), at::kFloat, {rows_n, K / 32}, x, st, "q8");
      s = result(PyTuple_GET_ITEM(a[6], 2), at::kInt, {rows_n, K / 32}, x, st, "q8");
    } else if (new_q) {
      const at::Tensor buf = one ? shared : fresh({codes + 2 * scales}, at::kByte, x, st);
      const int64_t from = one ? at_q : 0;
      q = piece(buf, from, x.sizes(), at::kChar);
      d = piece(buf, from + codes, {rows_n, K / 32}, at::kFloat);
      s = piece(buf, from + codes + scales, {rows_n, K / 32}, at::kInt);
    }
    if (one && new_res) res = piece(shared, at_res, x.sizes(), x.scalar_type());
    else if (a[7] != Py_None || new_res) res = result(a[7], x.scalar_type(), x.sizes(), x, st, "res");
    const float eps = (float)real(a[2]);
    auto at_or_null = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    const int64_t ld = rows_n > 1 ? x.stride(0) : K;
    check(called([&] {
            return abi.rms_norm(dt, x.data_ptr(), ld, rp, static_cast<const float*>(wp), eps, rows_n, K, at_or_null(res),
                                at_or_null(y), static_cast<int8_t*>(at_or_null(q)), static_cast<float*>(at_or_null(d)),
                                static_cast<int32_t*>(at_or_null(s)), st);
          }),
          "qmv_rms_norm");
    PyObject* q8 = q.defined() ? Py_BuildValue("(NNN)", wrap(q), wrap(d), wrap(s)) : Py_NewRef(Py_None);
    return Py_BuildValue("(NNN)", wrap(y), q8, wrap(res));
  });
}

// (q, d, dtype, out, stream) -> out
PyObject* dequantize_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &d = tensor(a[1], "d");
    if (q.dim() != 2) value_error("q: [n][K] wanted");
    if (!THPDtype_Check(a[2])) value_error("a torch dtype wanted");
    at::ScalarType t = reinterpret_cast<THPDtype*>(a[2])->scalar_type;
    if (a[3] != Py_None) t = tensor(a[3], "out").scalar_type();
    const int dt = dtype_code(t);
    const int64_t rows_n = q.size(0), K = q.size(1);
    const void* qp = typed(q, at::kChar, q.sizes(), "q");
    const void* dp = typed(d, at::kFloat, {rows_n, K / 32}, "d");
    const cudaStream_t st = stream_of(a[4]);
    at::Tensor out = result(a[3], t, q.sizes(), q, st, "out");
    check(called([&] {
            return abi.dequantize_act(dt, static_cast<const int8_t*>(qp), static_cast<const float*>(dp), rows_n, K,
                                      out.data_ptr(), st);
          }),
          "qmv_dequantize_act");
    return wrap(out);
  });
}

// (cache, k, v, table, lens, starts, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const qmv_kv_cache* c = cache_of(a[0]);
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    int64_t ks, vs;
    const void* kp = rows(k, c, c->n_kv_heads, "k", ks);
    const void* vp = rows(v, c, c->n_kv_heads, "v", vs);
    if (v.scalar_type() != k.scalar_type() || v.size(0) != k.size(0)) value_error("k and v must be of one type and length");
    const int dt = dtype_code(k.scalar_type());
    const qmv_kv_batch b = batch_of(a[3], a[4], a[5], k.size(0));
    const cudaStream_t st = stream_of(a[6]);
    check(called([&] { return abi.kv_append(c, &b, dt, kp, ks, vp, vs, st); }), "qmv_kv_append");
    Py_RETURN_NONE;
  });
}

// (cache, table, lens, starts, n_tok, dtype, k, v, stream) -> (k, v)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const qmv_kv_cache* c = cache_of(a[0]);
    const at::Tensor &table = tensor(a[1], "table"), &lens = tensor(a[2], "lens");
    if (a[4] == Py_None && a[3] != Py_None) value_error("n_tok is needed with starts");
    const int64_t n_tok = a[4] == Py_None ? lens.numel() : integer(a[4]);
    if (n_tok < 0) value_error("n_tok is negative");
    if (!THPDtype_Check(a[5])) value_error("a torch dtype wanted");
    at::ScalarType t = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    if (a[6] != Py_None) t = tensor(a[6], "k").scalar_type();
    const int dt = dtype_code(t);
    const int64_t shape[3] = {n_tok, c->n_kv_heads, c->head_dim};
    const qmv_kv_batch b = batch_of(a[1], a[2], a[3], n_tok);
    const cudaStream_t st = stream_of(a[8]);
    at::Tensor k, v;
    if (a[6] == Py_None && a[7] == Py_None) {
      on_device(table);
      const int64_t bytes = n_tok * c->n_kv_heads * c->head_dim * (int64_t)c10::elementSize(t);
      const at::Tensor buf = fresh({2 * bytes}, at::kByte, table, st);
      k = piece(buf, 0, shape, t);
      v = piece(buf, bytes, shape, t);
    } else {
      k = result(a[6], t, shape, table, st, "k");
      v = result(a[7], t, shape, table, st, "v");
    }
    check(called([&] { return abi.kv_read(c, &b, dt, k.data_ptr(), v.data_ptr(), st); }), "qmv_kv_read");
    return Py_BuildValue("(NN)", wrap(k), wrap(v));
  });
}

at::Tensor workspace(PyObject* o, size_t bytes, const at::Tensor& like, cudaStream_t st) {
  if (o == Py_None) return fresh({(int64_t)(bytes < 16 ? 16 : bytes)}, at::kByte, like, st);
  const at::Tensor& t = tensor(o, "ws");
  ptr(t);
  return t;
}

// (cache, q, table, lens, starts, scale, causal, window, pages, ws, out, stream) -> out
PyObject* kv_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const qmv_kv_cache* c = cache_of(a[0]);
    const at::Tensor& q = tensor(a[1], "q");
    if (q.dim() != 3) value_error("q: [n_tok][n_heads][D] wanted");
    int64_t qs;
    const void* qp = rows(q, c, q.size(1), "q", qs);
    const int dt = dtype_code(q.scalar_type());
    const int64_t n_tok = q.size(0), heads = q.size(1);
    if (heads > INT32_MAX) value_error("too many heads");
    const qmv_kv_batch b = batch_of(a[2], a[3], a[4], n_tok);
    const float scale = a[5] == Py_None ? 1.0f / std::sqrt((float)c->head_dim) : (float)real(a[5]);
    const int causal = PyObject_IsTrue(a[6]), window = as_int(a[7]);
    if (causal < 0) throw Raised{};
    const int32_t* pages = nullptr;
    int n_sel = 0;
    if (a[8] != Py_None) {
      const at::Tensor& t = tensor(a[8], "pages");
      if (t.dim() != 3 || t.size(0) != n_tok || t.size(1) != c->n_kv_heads || t.size(2) > INT32_MAX)
        value_error("pages: [" + std::to_string(n_tok) + "][" + std::to_string(c->n_kv_heads) + "][n_sel] wanted, got " +
                    text(t.sizes()));
      // (an empty tensor has no address, which would mean all pages)
      if (t.size(2) < 1) check(QMV_ERR_SHAPE, "qmv_kv_attend");
      pages = ints(t);
      n_sel = (int)t.size(2);
    }
    const cudaStream_t st = stream_of(a[11]);
    at::Tensor out = result(a[10], q.scalar_type(), q.sizes(), q, st, "out");
    at::Tensor ws =
        workspace(a[9], a[9] == Py_None ? abi.kv_attend_workspace_bytes(c, (int)heads, b.n_tok, b.n_seq) : 0, q, st);
    check(called([&] {
            return abi.kv_attend(c, &b, dt, qp, qs, out.data_ptr(), (int)heads, scale, causal, window, pages, n_sel,
                                 ws.data_ptr(), ws.nbytes(), st);
          }),
          "qmv_kv_attend");
    return wrap(out);
  });
}

// (cache, q, table, lens, starts, n_sel, ws, ids, stream) -> ids
PyObject* kv_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const qmv_kv_cache* c = cache_of(a[0]);
    const at::Tensor& q = tensor(a[1], "q");
    if (q.dim() != 3) value_error("q: [n_tok][n_heads][D] wanted");
    int64_t qs;
    const void* qp = rows(q, c, q.size(1), "q", qs);
    const int dt = dtype_code(q.scalar_type());
    const int n_sel = as_int(a[5]);
    if (n_sel < 1) check(QMV_ERR_SHAPE, "qmv_kv_select");
    if (q.size(1) > INT32_MAX) value_error("too many heads");
    const qmv_kv_batch b = batch_of(a[2], a[3], a[4], q.size(0));
    const int64_t shape[3] = {q.size(0), c->n_kv_heads, n_sel};
    const cudaStream_t st = stream_of(a[8]);
    at::Tensor ids = result(a[7], at::kInt, shape, q, st, "ids");
    at::Tensor ws = workspace(a[6], a[6] == Py_None ? abi.kv_select_workspace_bytes(c, &b) : 0, q, st);
    check(called([&] {
            return abi.kv_select(c, &b, dt, qp, qs, (int)q.size(1), static_cast<int32_t*>(ids.data_ptr()), n_sel,
                                 ws.data_ptr(), ws.nbytes(), st);
          }),
          "qmv_kv_select");
    return wrap(ids);
  });
}

#define QMV_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {QMV_METHOD(bind),     QMV_METHOD(rms_norm),  QMV_METHOD(dequantize_act), QMV_METHOD(kv_append),
                         QMV_METHOD(kv_read),  QMV_METHOD(kv_attend), QMV_METHOD(kv_select),      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
