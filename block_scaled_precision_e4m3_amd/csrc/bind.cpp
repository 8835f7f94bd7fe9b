// The usual calls of the torch wrappers without Python's share of their cost.
//
// Each function here takes the wrapper's arguments, and if they are what the
// entry point takes as they stand (tensors of the current device, the right
// shapes, types and layouts, on the current stream) allocates the outputs, makes
// the C-ABI call and returns them.  In every other case it returns None and has
// done nothing: the wrapper then goes through its own checks, which say what is
// wrong.  A status other than MXG_OK goes to the package's function for that
// (on_status), which raises it.  Host time per call, through ctypes and through
// here: product 8.1 and 3.6 us, quantise 8.2 and 4.0, rotation 8.3 and 3.7,
// norm 12.1 and 4.4, its backward pass 21.9 and 8.7.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPStream.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mxgemm.h"

namespace {

using at::Tensor;

constexpr unsigned kTrusted = MXG_TRUSTED_POINTERS;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tensor of an argument; null for None and for anything else (*other).
const Tensor* tensor(PyObject* o, bool* other) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    *other = true;
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

int dt_of(at::ScalarType t) {
  return t == at::kFloat ? MXG_DT_F32 : t == at::kBFloat16 ? MXG_DT_BF16 : t == at::kHalf ? MXG_DT_F16 : -1;
}
int fmt_of(at::ScalarType t) {
  return t == at::kFloat8_e4m3fn ? MXG_FMT_E4M3 : t == at::kFloat8_e5m2 ? MXG_FMT_E5M2 : -1;
}

// Whether t is dense memory of device `dev`.
bool on(const Tensor& t, int dev) { return t.is_cuda() && t.layout() == at::kStrided && t.get_device() == dev; }

// A contiguous float32 operand of that shape.
bool floats(const Tensor& t, at::IntArrayRef shape, int dev) {
  return t.scalar_type() == at::kFloat && t.sizes() == shape && t.is_contiguous() && on(t, dev);
}

bool current(int dev) {
  int now = -1;
  return dev >= 0 && hipGetDevice(&now) == hipSuccess && now == dev;
}

void* stream_of(int dev) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }

// A new contiguous tensor on like's device, without the dispatcher on the way to the allocator.
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), c10::nullopt);
}

PyObject* none() { Py_RETURN_NONE; }

// Whether the call's result needs a history, which the wrapper gives it.
bool history(std::initializer_list<const Tensor*> all) {
  if (!at::GradMode::is_enabled()) return false;
  for (const Tensor* t : all)
    if (t && t->requires_grad()) return true;
  return false;
}

// A tensor of the caller's that the call has written: autograd must not take it for what it was.
void changed(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A flag argument: what Python takes for true (nothing that raises).
bool truth(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) PyErr_Clear();
  return t == 1;
}

// An integer argument; false for anything else, or one past 64 bits.
bool integer(PyObject* o, int64_t* value) {
  if (!PyLong_Check(o)) return false;
  *value = PyLong_AsLongLong(o);
  if (*value == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// The package's function that raises a status.
PyObject* raise_status = nullptr;
PyObject* refused(int status) {
  if (!raise_status) return none();
  PyObject* r = PyObject_CallFunction(raise_status, "i", status);
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, "mxgemm: a call failed");
  return nullptr;
}

// Rows of a (rows, columns) or (L, rows, columns) tensor: as the wrapper has it.
struct Rows {
  int64_t l = 1, m = 0, k = 0, ld = 0;
  bool ok = false;
};
Rows rows_of(const Tensor& t) {
  Rows r;
  const int64_t n = t.dim();
  if (n != 2 && n != 3) return r;
  r.l = n == 3 ? t.size(0) : 1;
  r.m = t.size(n - 2);
  r.k = t.size(n - 1);
  r.ld = r.m > 1 ? t.stride(n - 2) : n == 3 && r.l > 1 ? t.stride(0) : r.k;
  r.ok = r.ld >= r.k && (r.k <= 1 || t.stride(n - 1) == 1) &&
         (n == 2 || r.l <= 1 || r.m * r.k == 0 || t.stride(0) == r.m * r.ld);
  return r;
}

// quantize(x, fmt, rows, cols, square, pow2)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return none();
  bool other = false;
  const Tensor* x = tensor(a[0], &other);
  int64_t fmt = 0;
  if (!x || !integer(a[1], &fmt)) return none();
  const bool rows = truth(a[2]), cols = truth(a[3]), square = truth(a[4]), pow2 = truth(a[5]);
  const int dt = dt_of(x->scalar_type());
  if (dt < 0 || (fmt != MXG_FMT_E4M3 && fmt != MXG_FMT_E5M2) || (!rows && !cols)) return none();
  const int dev = x->is_cuda() ? x->get_device() : -1;
  const Rows r = rows_of(*x);
  if (!r.ok || !current(dev) || !on(*x, dev)) return none();
  const int64_t kb = cdiv(r.k, 128), mb = cdiv(r.m, 128);
  const at::ScalarType f8 = fmt == MXG_FMT_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2;
  const bool batched = x->dim() == 3;
  auto make = [&](int64_t p, int64_t q, at::ScalarType type) {
    return batched ? fresh({r.l, p, q}, type, *x) : fresh({p, q}, type, *x);
  };
  Tensor q, s, qt, st;
  if (rows) {
    q = make(r.m, cdiv(r.k, 16) * 16, f8);
    s = square ? make(mb, kb, at::kFloat) : make(kb, r.m, at::kFloat);
  }
  if (cols) {
    qt = make(r.k, cdiv(r.m, 16) * 16, f8);
    st = square ? make(kb, mb, at::kFloat) : make(mb, r.k, at::kFloat);
  }
  const unsigned flags = (square ? MXG_QUANT_SQUARE : 0u) | (pow2 ? MXG_QUANT_POW2 : 0u) | kTrusted;
  const int status = mxgemm_block128_quantize(
      x->data_ptr(), r.ld, rows ? q.data_ptr() : nullptr, rows ? s.data_ptr<float>() : nullptr,
      cols ? qt.data_ptr() : nullptr, cols ? st.data_ptr<float>() : nullptr, r.m, r.k, r.l, dt, (int)fmt, flags,
      stream_of(dev));
  if (status != MXG_OK) return refused(status);
  PyObject* out = PyTuple_New(4);
  if (!out) return nullptr;
  const Tensor* all[4] = {&q, &s, &qt, &st};
  for (int i = 0; i < 4; ++i) {
    PyObject* o = all[i]->defined() ? THPVariable_Wrap(*all[i]) : none();
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i, o);
  }
  return out;
}

// gemm(a, sa, b, sb, b_block, c_dtype, c, accumulate)
PyObject* gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 8) return none();
  bool other = false;
  const Tensor *a = tensor(v[0], &other), *sa = tensor(v[1], &other), *b = tensor(v[2], &other), *sb = tensor(v[3], &other),
               *given = tensor(v[6], &other);
  int64_t block = 0;
  if (other || !a || !sa || !b || !sb || !integer(v[4], &block)) return none();
  const bool accumulate = truth(v[7]);
  const int fa = fmt_of(a->scalar_type()), fb = fmt_of(b->scalar_type());
  if (fa < 0 || fb < 0 || (block != 1 && block != 128) || (accumulate && !given) || history({given})) return none();
  const int64_t nd = a->dim();
  if ((nd != 2 && nd != 3) || b->dim() != nd || (nd == 3 && a->size(0) != b->size(0))) return none();
  const int64_t l = nd == 3 ? a->size(0) : 1, m = a->size(nd - 2), k = a->size(nd - 1), cols = b->size(nd - 2);
  const int dev = a->is_cuda() ? a->get_device() : -1;
  if (b->size(nd - 1) != k || !current(dev) || !on(*a, dev) || !on(*b, dev) || !a->is_contiguous() || !b->is_contiguous())
    return none();
  const int64_t kb = cdiv(k, 128), s0 = block == 1 ? kb : cdiv(cols, 128), s1 = block == 1 ? cols : kb;
  const int64_t want_a[3] = {l, kb, m}, want_b[3] = {l, s0, s1};
  if (!floats(*sa, {want_a + 3 - nd, (size_t)nd}, dev) || !floats(*sb, {want_b + 3 - nd, (size_t)nd}, dev)) return none();
  at::ScalarType type = at::kBFloat16;
  if (v[5] != Py_None) {
    if (!THPDtype_Check(v[5])) return none();
    type = reinterpret_cast<THPDtype*>(v[5])->scalar_type;
  }
  int64_t ldc = cols;
  if (given) {
    if (v[5] != Py_None && given->scalar_type() != type) return none();
    type = given->scalar_type();
    const Rows r = rows_of(*given);
    if (!r.ok || given->dim() != nd || r.l != l || r.m != m || r.k != cols || !on(*given, dev)) return none();
    ldc = r.ld;
  }
  const int ct = dt_of(type);
  if (ct < 0) return none();
  Tensor c = given ? *given : nd == 3 ? fresh({l, m, cols}, type, *a) : fresh({m, cols}, type, *a);
  Tensor ws;
  const size_t need = mxgemm_block128_workspace_bytes(m, cols, k, l, ct);
  if (need) ws = fresh({(int64_t)need}, at::kByte, *a);
  const unsigned flags = (block == 1 ? MXG_B128_B_ROWS : 0u) | (accumulate ? MXG_B128_ACCUMULATE : 0u) | kTrusted;
  const int status =
      mxgemm_block128(a->data_ptr(), sa->data_ptr<float>(), b->data_ptr(), sb->data_ptr<float>(), c.data_ptr(), ldc, m,
                      cols, k, l, fa, fb, ct, flags, need ? ws.data_ptr() : nullptr, need, stream_of(dev));
  if (status != MXG_OK) return refused(status);
  if (given) {
    changed(*given);
    Py_INCREF(v[6]);
    return v[6];
  }
  return THPVariable_Wrap(c);
}

// Heads (T, H, D) with contiguous features.
bool heads(const Tensor& t, int dev) { return t.dim() == 3 && (t.size(2) <= 1 || t.stride(2) == 1) && on(t, dev); }

// The rotary arguments cos, sin, positions, layout, rot_offset of a call on T tokens.
struct Rotary {
  const float *cos = nullptr, *sin = nullptr;
  const void* pos = nullptr;
  int64_t rot = 0, rows = 0, off = 0;
  int layout = -1;
  unsigned flags = kTrusted;
};
bool rotary(PyObject* const* v, int64_t T, int dev, Rotary* r) {
  bool other = false;
  const Tensor *cos = tensor(v[0], &other), *sin = tensor(v[1], &other), *pos = tensor(v[2], &other);
  if (other || !PyUnicode_Check(v[3]) || !integer(v[4], &r->off)) return false;
  if (PyUnicode_CompareWithASCIIString(v[3], "half") == 0) r->layout = MXG_ROPE_HALF;
  else if (PyUnicode_CompareWithASCIIString(v[3], "interleaved") == 0) r->layout = MXG_ROPE_INTERLEAVED;
  else if (PyUnicode_CompareWithASCIIString(v[3], "interleaved_to_half") == 0) r->layout = MXG_ROPE_INTERLEAVED_TO_HALF;
  else return false;
  if (!cos || !sin) return !cos && !sin && !pos;
  if (cos->dim() != 2 || !floats(*cos, cos->sizes(), dev) || !floats(*sin, cos->sizes(), dev)) return false;
  r->cos = cos->data_ptr<float>();
  r->sin = sin->data_ptr<float>();
  r->rows = cos->size(0);
  r->rot = 2 * cos->size(1);
  if (pos) {
    if (pos->dim() != 1 || pos->size(0) != T || !pos->is_contiguous() || !on(*pos, dev)) return false;
    if (pos->scalar_type() == at::kLong) r->flags |= MXG_ROPE_POS64;
    else if (pos->scalar_type() != at::kInt) return false;
    r->pos = pos->data_ptr();
  }
  return true;
}

// rope(x, cos, sin, positions, layout, rot_offset, transpose, out)
PyObject* rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 8) return none();
  bool other = false;
  const Tensor *x = tensor(v[0], &other), *given = tensor(v[7], &other);
  if (other || !x || history({x, given})) return none();
  const int dev = x->is_cuda() ? x->get_device() : -1, dt = dt_of(x->scalar_type());
  Rotary r;
  if (dt < 0 || !current(dev) || !heads(*x, dev) || !rotary(v + 1, x->size(0), dev, &r)) return none();
  if (given && (!heads(*given, dev) || given->sizes() != x->sizes() || given->scalar_type() != x->scalar_type())) return none();
  const Tensor y = given ? *given : fresh(x->sizes(), x->scalar_type(), *x);
  const int64_t strides[4] = {x->stride(0), x->stride(1), y.stride(0), y.stride(1)};
  const int status = mxgemm_rope(x->data_ptr(), y.data_ptr(), r.cos, r.sin, r.pos, strides, x->size(0), x->size(1),
                                 x->size(2), r.rot, r.off, r.rows, r.layout, dt,
                                 r.flags | (truth(v[6]) ? MXG_ROPE_TRANSPOSE : 0u), stream_of(dev));
  if (status != MXG_OK) return refused(status);
  if (given) {
    changed(*given);
    Py_INCREF(v[7]);
    return v[7];
  }
  return THPVariable_Wrap(y);
}

// What the norm's forward and backward share: q, k, their weights and the rotation.
struct Norm {
  const Tensor *q, *k, *wq, *wk;
  int dev, dt, wdt;
  Rotary r;
};
bool norm(PyObject* q, PyObject* k, PyObject* wq, PyObject* wk, PyObject* const* rot, Norm* s) {
  bool other = false;
  s->q = tensor(q, &other);
  s->k = tensor(k, &other);
  s->wq = tensor(wq, &other);
  s->wk = tensor(wk, &other);
  if (other || !s->q || !s->wq || (s->k && !s->wk)) return false;
  const Tensor& Q = *s->q;
  s->dev = Q.is_cuda() ? Q.get_device() : -1;
  s->dt = dt_of(Q.scalar_type());
  s->wdt = dt_of(s->wq->scalar_type());
  if (s->dt < 0 || (s->wdt != s->dt && s->wdt != MXG_DT_F32) || !current(s->dev) || !heads(Q, s->dev)) return false;
  const Tensor* w[2] = {s->wq, s->k ? s->wk : nullptr};
  for (const Tensor* t : w)
    if (t && (t->dim() != 1 || t->size(0) != Q.size(2) || t->scalar_type() != s->wq->scalar_type() || !t->is_contiguous() ||
              !on(*t, s->dev)))
      return false;
  if (s->k && (!heads(*s->k, s->dev) || s->k->size(0) != Q.size(0) || s->k->size(2) != Q.size(2) ||
               s->k->scalar_type() != Q.scalar_type()))
    return false;
  return rotary(rot, Q.size(0), s->dev, &s->r);
}
void put(int64_t* strides, const Tensor* t) {
  strides[0] = t ? t->stride(0) : 0;
  strides[1] = t ? t->stride(1) : 0;
}
void* data(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

PyObject* pack(std::initializer_list<const Tensor*> all) {
  PyObject* out = PyTuple_New((Py_ssize_t)all.size());
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* t : all) {
    PyObject* o = t ? THPVariable_Wrap(*t) : none();
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, layout, rot_offset, eps)
PyObject* qk_norm_rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Norm s;
  if (n != 10 || !norm(v[0], v[1], v[2], v[3], v + 4, &s) || history({s.q, s.k, s.wq, s.wk})) return none();
  const double eps = PyFloat_AsDouble(v[9]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return none();
  }
  const Tensor &q = *s.q, yq = fresh(q.sizes(), q.scalar_type(), q);
  Tensor yk;
  if (s.k) yk = fresh(s.k->sizes(), q.scalar_type(), q);
  const Tensor* k_out = s.k ? &yk : nullptr;
  int64_t strides[8];
  put(strides, &q);
  put(strides + 2, s.k);
  put(strides + 4, &yq);
  put(strides + 6, k_out);
  const int status = mxgemm_qk_norm_rope(
      q.data_ptr(), data(s.k), yq.data_ptr(), data(k_out), s.wq->data_ptr(), s.k ? data(s.wk) : nullptr, s.r.cos, s.r.sin,
      s.r.pos, strides, q.size(0), q.size(1), s.k ? s.k->size(1) : 0, q.size(2), s.r.rot, s.r.off, s.r.rows, (float)eps,
      s.r.layout, s.dt, s.wdt, s.r.flags, stream_of(s.dev));
  if (status != MXG_OK) return refused(status);
  return pack({&yq, k_out});
}

// qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, cos, sin, positions, layout, rot_offset, eps)
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Norm s;
  if (n != 12 || !norm(v[2], v[3], v[4], v[5], v + 6, &s)) return none();
  bool other = false;
  const Tensor *dq = tensor(v[0], &other), *dk = tensor(v[1], &other);
  const double eps = PyFloat_AsDouble(v[11]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return none();
  }
  const Tensor& q = *s.q;
  if (other || !dq || (dk != nullptr) != (s.k != nullptr) || !heads(*dq, s.dev) || dq->sizes() != q.sizes() ||
      dq->scalar_type() != q.scalar_type() ||
      (dk && (!heads(*dk, s.dev) || dk->sizes() != s.k->sizes() || dk->scalar_type() != q.scalar_type())))
    return none();
  const int64_t T = q.size(0), D = q.size(2);
  const Tensor xq = fresh(q.sizes(), q.scalar_type(), q), dwq = fresh({D}, at::kFloat, q);
  Tensor xk, dwk;
  if (s.k) {
    xk = fresh(s.k->sizes(), q.scalar_type(), q);
    dwk = fresh({D}, at::kFloat, q);
  }
  const size_t need = mxgemm_qk_norm_rope_backward_workspace_bytes(T, D);
  const Tensor ws = fresh({(int64_t)need}, at::kByte, q);
  const Tensor* k_out = s.k ? &xk : nullptr;
  int64_t strides[12];
  const Tensor* order[6] = {dq, dk, &q, s.k, &xq, k_out};
  for (int i = 0; i < 6; ++i) put(strides + 2 * i, order[i]);
  const int status = mxgemm_qk_norm_rope_backward(
      dq->data_ptr(), data(dk), q.data_ptr(), data(s.k), xq.data_ptr(), data(k_out), dwq.data_ptr<float>(),
      s.k ? dwk.data_ptr<float>() : nullptr, s.wq->data_ptr(), s.k ? data(s.wk) : nullptr, s.r.cos, s.r.sin, s.r.pos,
      strides, T, q.size(1), s.k ? s.k->size(1) : 0, D, s.r.rot, s.r.off, s.r.rows, (float)eps, s.r.layout, s.dt, s.wdt,
      s.r.flags, ws.data_ptr(), need, stream_of(s.dev));
  if (status != MXG_OK) return refused(status);
  return pack({&xq, k_out, &dwq, s.k ? &dwk : nullptr});
}

// C++ exceptions (an allocation that fails) become Python's.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(self, args, n);
  END_HANDLE_TH_ERRORS
}

// on_status(f): f(status) raises what a call's status stands for.
PyObject* on_status(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(raise_status, f);
  return none();
}

PyMethodDef methods[] = {
    {"on_status", on_status, METH_O, nullptr},
    {"quantize", (PyCFunction)(void*)guarded<quantize>, METH_FASTCALL, nullptr},
    {"gemm", (PyCFunction)(void*)guarded<gemm>, METH_FASTCALL, nullptr},
    {"rope", (PyCFunction)(void*)guarded<rope>, METH_FASTCALL, nullptr},
    {"qk_norm_rope", (PyCFunction)(void*)guarded<qk_norm_rope>, METH_FASTCALL, nullptr},
    {"qk_norm_rope_backward", (PyCFunction)(void*)guarded<qk_norm_rope_backward>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
