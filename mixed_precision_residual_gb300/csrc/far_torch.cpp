// Binding of the per-head and block-scaled operators to PyTorch tensors: the same functions as
// heads.py and block.py document, checked and allocated here.  A decode step makes each of
// these calls for a few tokens, where its time is the host's: about 20 us of interpreted
// checks, ctypes conversions and two allocations before a kernel of 3 us; here 3.5 (the product), 4 (a
// matrix quantised), 4.5 (qk_norm_rope) and 5 (the norm), 9 for qk_norm_rope's gradients.
// Every function takes its arguments by position and enqueues on the tensors' device, on that
// device's current stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "far.h"

namespace {

PyObject* g_far_error = nullptr;     // the package's FarError
PyObject* g_out_of_memory = nullptr;  // torch.OutOfMemoryError

struct Refused {  // a Python exception to raise
  PyObject* type;
  std::string text;
};
[[noreturn]] void refuse(const char* text) { throw Refused{PyExc_ValueError, text}; }

struct Status {  // a status of the library
  int code;
};
void check(int status) {
  if (status != FAR_OK) throw Status{status};
}

// f() without Python's lock: an allocation may wait for the device, and a launch for room in its queue, either of which
// may itself wait for a host function that needs the lock.  One region a call, at its end: 0.2 us.
template <class F>
auto unlocked(const F& f) {
  struct Lock {
    PyThreadState* state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return f();
}

using at::Tensor;
constexpr auto kE4M3 = at::ScalarType::Float8_e4m3fn;

const Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, "expected a tensor"};
  return THPVariable_Unpack(o);
}
// an argument that may be None
const Tensor* maybe(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }
// a whole number (a float, as an index, is refused)
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}

int code_of(at::ScalarType t) {
  switch (t) {
    case at::ScalarType::Float: return FAR_F32;
    case at::ScalarType::Half: return FAR_F16;
    case at::ScalarType::BFloat16: return FAR_BF16;
    default: throw Status{FAR_ERR_DTYPE};
  }
}
int dtypes(const Tensor& act, const Tensor& w) { return FAR_DTYPES(code_of(act.scalar_type()), code_of(w.scalar_type())); }

// The one CUDA device of all tensors given, made current for the call's duration, and its stream.
struct Place {
  c10::cuda::OptionalCUDAGuard guard;
  c10::Device device{c10::kCPU};
  void* stream = nullptr;
  Place(std::initializer_list<const Tensor*> ts) {
    bool any = false;
    for (const Tensor* t : ts) {
      if (!t) continue;
      if (!t->is_cuda()) refuse("tensors must be on a CUDA device");
      if (!any) device = t->device();
      else if (t->device() != device) refuse("tensors must be on one device");
      any = true;
    }
    guard.set_device(device);
    stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  }
  Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return Tensor(at::detail::empty_cuda(shape, t, device, std::nullopt));
  }
};

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

// ---------------------------------------------------------------------------
// heads
// ---------------------------------------------------------------------------

struct Heads {
  void* p = nullptr;
  int64_t ts = 0, hs = 0;
};
Heads heads(const Tensor* t) {
  Heads r;
  if (!t) return r;
  const auto sizes = t->sizes(), strides = t->strides();
  const int64_t n = t->dim();
  int64_t lead = 1, run = -1;
  for (int64_t i = n - 3; i >= 0; --i) {
    if (sizes[i] != 1) {
      if (run < 0) r.ts = strides[i];
      else if (strides[i] != run && t->numel() > 0)
        refuse("the leading axes do not collapse to one stride: call once a sequence, or copy");
      run = strides[i] * sizes[i];
    }
    lead *= sizes[i];
  }
  if (strides[n - 1] != 1 && sizes[n - 1] > 1) refuse("the values of a head must be contiguous");
  if (lead <= 1) r.ts = 0;
  r.hs = sizes[n - 2] > 1 ? strides[n - 2] : 0;
  r.p = t->data_ptr();
  return r;
}

struct Sizes {
  int64_t tokens = 1, q = 0, k = 0, dim = 0;
};
Sizes sizes_of(const Tensor& q, const Tensor* k) {
  if (q.dim() < 3) refuse("q and k are [..., heads, head_dim]");
  const int64_t n = q.dim();
  Sizes s;
  for (int64_t i = 0; i < n - 2; ++i) s.tokens *= q.size(i);
  s.q = q.size(n - 2);
  s.dim = q.size(n - 1);
  if (k) {
    bool same = k->dim() == n && k->size(n - 1) == s.dim;
    for (int64_t i = 0; same && i < n - 2; ++i) same = k->size(i) == q.size(i);
    if (!same) refuse("q and k must agree but in their number of heads");
    if (k->scalar_type() != q.scalar_type()) refuse("q and k must share a dtype");
    s.k = k->size(n - 2);
  }
  return s;
}

int weights(const Tensor& q, const Tensor* k, const Tensor* qw, const Tensor* kw, int64_t dim) {
  if (!qw || qw->numel() != dim || !qw->is_contiguous() || (k && (!kw || kw->numel() != dim || !kw->is_contiguous())))
    refuse("a weight is a contiguous [head_dim] tensor");
  if (k && kw->scalar_type() != qw->scalar_type()) refuse("q_weight and k_weight must share a dtype");
  return dtypes(q, *qw);
}

void table_and_positions(const Tensor& table, const Tensor& pos, int64_t tokens) {
  if (table.dim() != 2 || table.scalar_type() != at::ScalarType::Float || !table.is_contiguous())
    refuse("table must be a contiguous float32 [rows, rot_dim] tensor (rope_table)");
  if ((pos.scalar_type() != at::ScalarType::Long && pos.scalar_type() != at::ScalarType::Int) || !pos.is_contiguous())
    refuse("positions must be a contiguous int32 or int64 tensor");
  if (pos.numel() != tokens) refuse("one position for each token");
}

using Shape = c10::SmallVector<int64_t, 6>;

// an output given (checked) or one to make, without Python's lock, before the call; None where there is no input
struct Out {
  Tensor t;
  PyObject* given = nullptr;
  Shape shape;
  at::ScalarType type = at::ScalarType::Float;
  bool wanted = false;
  void make(const Place& place) {
    if (wanted) t = place.empty(shape, type);
  }
  const Tensor* get() const { return t.defined() ? &t : nullptr; }
  PyObject* object() const {
    if (given) return Py_NewRef(given);
    if (!t.defined()) return Py_NewRef(Py_None);
    return THPVariable_Wrap(t);
  }
};
Out fresh(at::IntArrayRef shape, at::ScalarType type) {
  Out r;
  r.shape.assign(shape.begin(), shape.end());
  r.type = type;
  r.wanted = true;
  return r;
}
Out output(const Tensor* in, PyObject* o) {
  Out r;
  if (!in) {
    if (o != Py_None) refuse("an output without its input");
    return r;
  }
  if (o == Py_None) return fresh(in->sizes(), in->scalar_type());
  r.t = tensor(o);
  if (r.t.sizes() != in->sizes() || r.t.scalar_type() != in->scalar_type())
    refuse("an output has its input's shape and dtype");
  r.given = o;
  return r;
}

PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
  return t;
}

// q, k, q_weight, k_weight, eps, table, positions, interleaved, q_out, k_out
PyObject* qk_norm_rope_(PyObject* const* a) {
  const Tensor& q = tensor(a[0]);
  const Tensor *k = maybe(a[1]), *qw = maybe(a[2]), *kw = maybe(a[3]);
  const Tensor &table = tensor(a[5]), &pos = tensor(a[6]);
  const Sizes s = sizes_of(q, k);
  const int code = weights(q, k, qw, kw, s.dim);
  table_and_positions(table, pos, s.tokens);
  const Place place{&q, k, qw, kw, &table, &pos, maybe(a[8]), maybe(a[9])};
  Out yq = output(&q, a[8]), yk = output(k, a[9]);
  const Heads x = heads(&q), xk = heads(k);
  const float eps = (float)real(a[4]);
  const int pairs = (int)integer(a[7]);
  check(unlocked([&] {
    yq.make(place);
    yk.make(place);
    const Heads y = heads(yq.get()), z = heads(yk.get());
    return qk_norm_rope(x.p, x.ts, x.hs, xk.p, xk.ts, xk.hs, ptr(qw), k ? ptr(kw) : nullptr, eps,
                        static_cast<const float*>(table.data_ptr()), table.size(0), pos.data_ptr(),
                        (int)pos.element_size(), y.p, y.ts, y.hs, z.p, z.ts, z.hs, s.tokens, s.q, s.k, s.dim,
                        table.size(1), pairs, code, place.stream);
  }));
  return tuple({yq.object(), yk.object()});
}

// q, k, table, positions, interleaved, transpose, q_out, k_out
PyObject* rope_(PyObject* const* a) {
  const Tensor& q = tensor(a[0]);
  const Tensor* k = maybe(a[1]);
  const Tensor &table = tensor(a[2]), &pos = tensor(a[3]);
  const Sizes s = sizes_of(q, k);
  const int act = code_of(q.scalar_type());
  table_and_positions(table, pos, s.tokens);
  const Place place{&q, k, &table, &pos, maybe(a[6]), maybe(a[7])};
  Out yq = output(&q, a[6]), yk = output(k, a[7]);
  const Heads x = heads(&q), xk = heads(k);
  const int pairs = (int)integer(a[4]), transpose = (int)integer(a[5]);
  check(unlocked([&] {
    yq.make(place);
    yk.make(place);
    const Heads y = heads(yq.get()), z = heads(yk.get());
    return rope(x.p, x.ts, x.hs, xk.p, xk.ts, xk.hs, static_cast<const float*>(table.data_ptr()), table.size(0),
                pos.data_ptr(), (int)pos.element_size(), y.p, y.ts, y.hs, z.p, z.ts, z.hs, s.tokens, s.q, s.k, s.dim,
                table.size(1), pairs, transpose, act, place.stream);
  }));
  return tuple({yq.object(), yk.object()});
}

// dq_out, dk_out, q, k, q_weight, k_weight, eps, table, positions, interleaved, dq, dk, workspace
PyObject* qk_norm_rope_backward_(PyObject* const* a) {
  const Tensor& q = tensor(a[2]);
  const Tensor *gq = maybe(a[0]), *gk = maybe(a[1]), *k = maybe(a[3]), *qw = maybe(a[4]), *kw = maybe(a[5]);
  const Tensor &table = tensor(a[7]), &pos = tensor(a[8]);
  const Sizes s = sizes_of(q, k);
  const int code = weights(q, k, qw, kw, s.dim);
  table_and_positions(table, pos, s.tokens);
  auto like = [](const Tensor* g, const Tensor* x) {
    return (g != nullptr) == (x != nullptr) && (!g || (g->sizes() == x->sizes() && g->scalar_type() == x->scalar_type()));
  };
  if (!like(gq, &q) || !like(gk, k)) refuse("an output's gradient has its input's shape and dtype");
  const Tensor* ws = maybe(a[12]);
  const Place place{&q, k, qw, kw, &table, &pos, gq, gk, maybe(a[10]), maybe(a[11]), ws};
  Out yq = output(&q, a[10]), yk = output(k, a[11]);
  if (ws && !ws->is_contiguous()) refuse("workspace must be contiguous");
  const int64_t bytes = ws ? ws->numel() * (int64_t)ws->element_size() : far_qk_backward_workspace_bytes(s.dim);
  if (bytes < 0) throw Status{(int)-bytes};
  const Heads g = heads(gq), h = heads(gk), x = heads(&q), xk = heads(k);
  const float eps = (float)real(a[6]);
  const int pairs = (int)integer(a[9]);
  Tensor dqw, dkw, own;
  check(unlocked([&] {
    yq.make(place);
    yk.make(place);
    dqw = place.empty({s.dim}, at::ScalarType::Float);
    if (k) dkw = place.empty({s.dim}, at::ScalarType::Float);
    if (s.q == 0) dqw.zero_();  // (the C entry point leaves the arguments of a half without heads alone)
    if (k && s.k == 0) dkw.zero_();
    if (!ws) own = place.empty({bytes}, at::ScalarType::Byte);
    const Heads y = heads(yq.get()), z = heads(yk.get());
    return qk_norm_rope_backward(g.p, g.ts, g.hs, h.p, h.ts, h.hs, x.p, x.ts, x.hs, xk.p, xk.ts, xk.hs, ptr(qw),
                                 k ? ptr(kw) : nullptr, eps, static_cast<const float*>(table.data_ptr()), table.size(0),
                                 pos.data_ptr(), (int)pos.element_size(), y.p, y.ts, y.hs, z.p, z.ts, z.hs,
                                 static_cast<float*>(dqw.data_ptr()), k ? static_cast<float*>(dkw.data_ptr()) : nullptr,
                                 (ws ? *ws : own).data_ptr(), bytes, s.tokens, s.q, s.k, s.dim, table.size(1), pairs,
                                 code, place.stream);
  }));
  return tuple({yq.object(), yk.object(), THPVariable_Wrap(dqw), k ? THPVariable_Wrap(dkw) : Py_NewRef(Py_None)});
}

// ---------------------------------------------------------------------------
// blocks of 128
// ---------------------------------------------------------------------------

int64_t blocks(int64_t n) { return (n + 127) / 128; }

struct Rows {
  int64_t rows, cols, stride;
};
Rows rows_of(const Tensor& t, const char* refusal = "non-contiguous tensors must be 2-D with contiguous rows") {
  const int64_t c = t.dim() ? t.size(-1) : 0;
  if (t.is_contiguous()) {
    int64_t r = 1;
    for (int64_t i = 0; i + 1 < t.dim(); ++i) r *= t.size(i);
    return {r, c, c};
  }
  if (t.dim() != 2 || (t.stride(1) != 1 && c != 1)) refuse(refusal);
  return {t.size(0), c, t.size(0) > 1 ? t.stride(0) : c};
}

Shape with_last(const Tensor& t, int64_t last) {
  Shape s(t.sizes().begin(), t.sizes().end());
  s.back() = last;
  return s;
}

Out codes(PyObject* o, at::IntArrayRef shape) {
  if (o == Py_None) return fresh(shape, kE4M3);
  Out r;
  r.t = tensor(o);
  r.given = o;
  if (r.t.sizes() != shape || (r.t.scalar_type() != kE4M3 && r.t.scalar_type() != at::ScalarType::Byte) ||
      !r.t.is_contiguous())
    refuse("q must be a contiguous float8_e4m3fn (or uint8) tensor of the output's shape");
  return r;
}
Out scales(PyObject* o, at::IntArrayRef shape) {
  if (o == Py_None) return fresh(shape, at::ScalarType::Float);
  Out r;
  r.t = tensor(o);
  r.given = o;
  if (r.t.sizes() != shape || r.t.scalar_type() != at::ScalarType::Float || !r.t.is_contiguous())
    refuse("scale must be a contiguous float32 tensor, one value a block");
  return r;
}

// x, residual (or None), weight, eps, q, scale, residual_out
PyObject* norm_quant_block_(PyObject* const* a) {
  const Tensor &x = tensor(a[0]), &w = tensor(a[2]);
  const Tensor* r = maybe(a[1]);
  if (x.dim() < 1) refuse("x is [..., hidden]");
  if (!w.is_contiguous() || w.numel() != x.size(-1)) refuse("weight must be a contiguous [hidden] tensor");
  const int code = dtypes(x, w);
  if (r && (r->sizes() != x.sizes() || r->scalar_type() != x.scalar_type()))
    refuse("x and residual must share a shape and a dtype");
  const Place place{&x, r, &w, maybe(a[4]), maybe(a[5]), maybe(a[6])};
  Out res = output(r, a[6]);
  Out q = codes(a[4], x.sizes()), sc = scales(a[5], with_last(x, blocks(x.size(-1))));
  const Rows X = rows_of(x);
  const int64_t r_stride = r ? rows_of(*r).stride : 0;
  const float eps = (float)real(a[3]);
  check(unlocked([&] {
    res.make(place);
    q.make(place);
    sc.make(place);
    float* sp = static_cast<float*>(sc.t.data_ptr());
    if (!r)
      return rmsnorm_quant_block(x.data_ptr(), X.stride, w.data_ptr(), eps, q.t.data_ptr(), sp, X.rows, X.cols, code,
                                 place.stream);
    return fused_add_rmsnorm_quant_block(x.data_ptr(), X.stride, r->data_ptr(), r_stride, w.data_ptr(), eps,
                                         q.t.data_ptr(), sp, res.t.data_ptr(), rows_of(res.t).stride, X.rows, X.cols,
                                         code, place.stream);
  }));
  if (!r) return tuple({q.object(), sc.object()});
  return tuple({q.object(), sc.object(), res.object()});
}

// x, block (0 rows, 1 tiles), transpose, q, scale
PyObject* quant_block_fp8_(PyObject* const* a) {
  const Tensor& x = tensor(a[0]);
  if (x.dim() != 2) refuse("x must be a matrix");
  const int act = code_of(x.scalar_type());
  const int block = (int)integer(a[1]), transpose = (int)integer(a[2]);
  const Place place{&x, maybe(a[3]), maybe(a[4])};
  const Rows X = rows_of(x, "x must have contiguous rows");
  const int64_t r = transpose ? X.cols : X.rows, c = transpose ? X.rows : X.cols;
  Out q = codes(a[3], {r, c}), s = scales(a[4], {block == FAR_BLOCK_ROW ? r : blocks(r), blocks(c)});
  check(unlocked([&] {
    q.make(place);
    s.make(place);
    return quant_block_fp8(x.data_ptr(), X.stride, q.t.data_ptr(), static_cast<float*>(s.t.data_ptr()), X.rows, X.cols,
                           block, transpose, act, place.stream);
  }));
  return tuple({q.object(), s.object()});
}

bool is_codes(const Tensor& t) { return t.scalar_type() == kE4M3 || t.scalar_type() == at::ScalarType::Byte; }

// x, x_scale, wt, wt_scale, out_dtype, out
PyObject* gemm_fp8_block_(PyObject* const* a) {
  const Tensor &x = tensor(a[0]), &xs = tensor(a[1]), &w = tensor(a[2]), &ws = tensor(a[3]);
  if (!is_codes(x) || !is_codes(w)) refuse("x and wt hold E4M3 codes (float8_e4m3fn or uint8)");
  if (x.dim() < 2 || w.dim() != 2 || x.size(-1) != w.size(1)) refuse("x is [..., k] and wt [n, k]");
  if (!THPDtype_Check(a[4])) throw Refused{PyExc_TypeError, "out_dtype is a torch.dtype"};
  const at::ScalarType ot = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
  const int od = code_of(ot);
  const int64_t n = w.size(0), k = w.size(1), kb = blocks(k);
  if (xs.sizes() != at::IntArrayRef(with_last(x, kb)) || xs.scalar_type() != at::ScalarType::Float || !xs.is_contiguous())
    refuse("x_scale must be a contiguous float32 [..., ceil(k / 128)] tensor");
  if (ws.scalar_type() != at::ScalarType::Float || !ws.is_contiguous() || ws.dim() != 2 || ws.size(1) != kb)
    refuse("wt_scale must be a contiguous float32 [.., ceil(k / 128)] tensor");
  if (ws.size(0) != blocks(n) && ws.size(0) != n) refuse("wt_scale has one row for each 128 rows of wt, or one for each");
  // (n = 1 has one of either: the same numbers)
  const int block = ws.size(0) == blocks(n) ? FAR_BLOCK_TILE : FAR_BLOCK_ROW;
  const Place place{&x, &xs, &w, &ws, maybe(a[5])};
  Out out = fresh(with_last(x, n), ot);
  if (a[5] != Py_None) {
    out.t = tensor(a[5]);
    out.given = a[5];
    out.wanted = false;
    if (out.t.sizes() != at::IntArrayRef(out.shape) || out.t.scalar_type() != ot) refuse("out has shape [..., n] and out_dtype");
  }
  int64_t m = 1;
  for (int64_t i = 0; i + 1 < x.dim(); ++i) m *= x.size(i);
  const int64_t ldx = k ? rows_of(x).stride : 0, ldw = k ? rows_of(w).stride : 0;
  check(unlocked([&] {
    out.make(place);
    return gemm_fp8_block(x.data_ptr(), ldx, static_cast<const float*>(xs.data_ptr()), w.data_ptr(), ldw,
                          static_cast<const float*>(ws.data_ptr()), block, out.t.data_ptr(), rows_of(out.t).stride, m, n,
                          k, od, place.stream);
  }));
  return out.object();
}

// ---------------------------------------------------------------------------
// the module
// ---------------------------------------------------------------------------

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& e) {
    if (e.type) PyErr_SetString(e.type, e.text.c_str());
  } catch (const Status& e) {
    if (PyObject* v = PyObject_CallFunction(g_far_error, "i", e.code)) {
      PyErr_SetObject(g_far_error, v);
      Py_DECREF(v);
    }
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// (FarError, OutOfMemoryError): the classes that the calls raise
PyObject* init_errors(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "expected two classes");
    return nullptr;
  }
  Py_XSETREF(g_far_error, Py_NewRef(args[0]));
  Py_XSETREF(g_out_of_memory, Py_NewRef(args[1]));
  Py_RETURN_NONE;
}

#define FAR_ENTRY(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<name##_, n>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAR_ENTRY(qk_norm_rope, 10),
                           FAR_ENTRY(rope, 8),
                           FAR_ENTRY(qk_norm_rope_backward, 13),
                           FAR_ENTRY(norm_quant_block, 7),
                           FAR_ENTRY(quant_block_fp8, 5),
                           FAR_ENTRY(gemm_fp8_block, 6),
                           {"init_errors", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&init_errors)), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_far_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__far_torch(void) { return PyModule_Create(&g_module); }
