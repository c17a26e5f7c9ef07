// The common call of the packed-layer blocks from Python: checks the tensors, allocates the output and
// calls the C entry point on torch's current stream.  A single token's layer product takes 4 us on
// the device; through ctypes and tensor attributes its call took 9 us of the host.  Whatever is out of
// the ordinary (another device, a type, shape or stride to refuse) returns None, and binding.py decides, so no
// check is left out here and every message is written there.  A refusal by the library returns its status.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>

#include "dit.h"

namespace {

using LinearFn = decltype(&dit_op_linear_fused);
using AttentionFn = decltype(&dit_op_attention_packed);
using RotaryFn = decltype(&dit_op_rotary);
LinearFn linear_fn = nullptr;
AttentionFn attention_fn = nullptr;
RotaryFn rotary_fn = nullptr;

#define NOT_HERE Py_RETURN_NONE

// the entry points wait for a full launch queue, so other threads run meanwhile
#define CALL(rc, ...)       \
  dit_status rc;            \
  Py_BEGIN_ALLOW_THREADS    \
  rc = __VA_ARGS__;         \
  Py_END_ALLOW_THREADS

// the tensor behind o, or null; None is an absent tensor where `optional`
bool tensor(PyObject* o, const at::Tensor** t, bool optional = false) {
  *t = nullptr;
  if (o == Py_None) return optional;
  if (!THPVariable_CheckExact(o)) return false;
  *t = &THPVariable_Unpack(o);
  return (*t)->is_cuda() && (*t)->layout() == c10::kStrided;
}

int code_of(at::ScalarType t) {
  return t == at::kFloat ? DIT_DTYPE_F32 : t == at::kBFloat16 ? DIT_DTYPE_BF16 : t == at::kHalf ? DIT_DTYPE_FP16 : -1;
}

// stride between the rows of a matrix whose rows are contiguous, or -1
int64_t row_stride(const at::Tensor& t) {
  if (t.is_contiguous()) return t.size(1);
  if (t.size(1) != 1 && t.stride(1) != 1) return -1;
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// token and head stride of [tokens, heads, features]; those of a length-1 axis are free
bool head_strides(const at::Tensor& t, long long* s) {
  const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
  if (t.is_contiguous()) {
    s[0] = h * d, s[1] = d;
    return true;
  }
  if (d != 1 && t.stride(2) != 1) return false;
  s[1] = h > 1 ? t.stride(1) : (d + 7) / 8 * 8;
  s[0] = n > 1 ? t.stride(0) : h * s[1];
  return true;
}

bool fits(int64_t v) { return v <= INT_MAX; }

dit_stream_t current_stream() { return reinterpret_cast<dit_stream_t>(c10::cuda::getCurrentCUDAStream().stream()); }

// linear(x, w, bias, act, residual, out, out_dtype)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor *x, *w, *b, *r, *o;
  if (n != 7 || linear_fn == nullptr || !tensor(a[0], &x) || !tensor(a[1], &w) || !tensor(a[2], &b, true) ||
      !tensor(a[4], &r, true) || !tensor(a[5], &o, true))
    NOT_HERE;
  const int act = static_cast<int>(PyLong_AsLong(a[3]));
  if (act < 0 || x->dim() != 2 || w->dim() != 2 || x->size(1) != w->size(1) || x->scalar_type() != w->scalar_type()) NOT_HERE;
  const int64_t M = x->size(0), K = x->size(1), N = w->size(0);
  at::ScalarType ot = o ? o->scalar_type() : x->scalar_type();
  if (a[6] != Py_None) {
    if (!THPDtype_Check(a[6])) NOT_HERE;
    const at::ScalarType want = reinterpret_cast<THPDtype*>(a[6])->scalar_type;
    if (o && want != ot) NOT_HERE;
    ot = want;
  }
  const int code = code_of(x->scalar_type()), ocode = code_of(ot);
  const int64_t ldx = row_stride(*x), ldw = row_stride(*w);
  const c10::DeviceIndex dev = c10::cuda::current_device();
  if (code <= 0 || ocode < 0 || ldx < 0 || ldw < 0 || !fits(M) || !fits(N) || !fits(K) || x->get_device() != dev ||
      w->get_device() != dev)
    NOT_HERE;
  if (b && (b->dim() != 1 || b->size(0) != N || b->scalar_type() != at::kFloat || !b->is_contiguous() || b->get_device() != dev))
    NOT_HERE;
  int64_t ldr = 0, ldy = N;
  if (r) {
    if (r->dim() != 2 || r->size(0) != M || r->size(1) != N || r->scalar_type() != ot || (r->stride(1) != 1 && N > 1) ||
        r->get_device() != dev)
      NOT_HERE;
    ldr = r->stride(0);
  }
  at::Tensor fresh;
  if (o) {
    if (o->dim() != 2 || o->size(0) != M || o->size(1) != N || o->get_device() != dev || (ldy = row_stride(*o)) < 0) NOT_HERE;
  } else {
    fresh = at::empty({M, N}, x->options().dtype(ot));
    o = &fresh;
  }
  const dit_stream_t stream = current_stream();
  CALL(rc, linear_fn(code, x->const_data_ptr(), ldx, w->const_data_ptr(), ldw, b ? static_cast<const float*>(b->const_data_ptr()) : nullptr,
                act, r ? r->const_data_ptr() : nullptr, ldr, o->mutable_data_ptr(), ldy, ocode, static_cast<int>(M),
                static_cast<int>(N), static_cast<int>(K), nullptr, stream));
  if (rc != DIT_OK) return PyLong_FromLong(rc);
  return THPVariable_Wrap(*o);
  END_HANDLE_TH_ERRORS
}

// attention(q, k, v, cu_q, cu_k, max_q, max_k, causal, scale, out, return_lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor *q, *k, *v, *cq, *ck, *o;
  if (n != 11 || attention_fn == nullptr || !tensor(a[0], &q) || !tensor(a[1], &k) || !tensor(a[2], &v) || !tensor(a[3], &cq) ||
      !tensor(a[4], &ck) || !tensor(a[9], &o, true) || !PyLong_Check(a[5]) || !PyLong_Check(a[6]))
    NOT_HERE;
  int over = 0;
  const long long max_q = PyLong_AsLongLongAndOverflow(a[5], &over), max_k = over ? -1 : PyLong_AsLongLongAndOverflow(a[6], &over);
  const int causal = PyObject_IsTrue(a[7]), want_lse = PyObject_IsTrue(a[10]);
  if (over || max_q < 0 || max_k < 0 || !fits(max_q) || !fits(max_k) || causal < 0 || want_lse < 0) {
    PyErr_Clear();
    NOT_HERE;
  }
  const at::ScalarType t = q->scalar_type();
  const int code = code_of(t);
  if (q->dim() != 3 || k->dim() != 3 || v->sizes() != k->sizes() || code <= 0 || k->scalar_type() != t || v->scalar_type() != t ||
      k->size(2) != q->size(2) || cq->dim() != 1 || cq->size(0) < 1 || ck->sizes() != cq->sizes() || cq->scalar_type() != at::kInt ||
      ck->scalar_type() != at::kInt || !cq->is_contiguous() || !ck->is_contiguous())
    NOT_HERE;
  const int64_t tq = q->size(0), h = q->size(1), d = q->size(2), tk = k->size(0), hk = k->size(1), seqs = cq->size(0) - 1;
  const c10::DeviceIndex dev = c10::cuda::current_device();
  if (q->get_device() != dev || k->get_device() != dev || v->get_device() != dev || cq->get_device() != dev ||
      ck->get_device() != dev || !fits(tq) || !fits(tk) || !fits(h) || !fits(d) || !fits(seqs))
    NOT_HERE;
  if (d < 1 || (a[8] != Py_None && !PyFloat_Check(a[8]))) NOT_HERE;
  const double scale = a[8] == Py_None ? std::pow(static_cast<double>(d), -0.5) : PyFloat_AS_DOUBLE(a[8]);
  long long s[8];
  if (!head_strides(*q, s) || !head_strides(*k, s + 2) || !head_strides(*v, s + 4)) NOT_HERE;
  at::Tensor fresh, lse;
  if (o) {
    if (o->sizes() != q->sizes() || o->scalar_type() != t || o->get_device() != dev || !head_strides(*o, s + 6)) NOT_HERE;
  } else {
    fresh = at::empty({tq, h, d}, q->options());
    o = &fresh;
    s[6] = h * d, s[7] = d;
  }
  if (want_lse) lse = at::empty({h, tq}, q->options().dtype(at::kFloat));
  const dit_stream_t stream = current_stream();
  CALL(rc, attention_fn(
      code, q->const_data_ptr(), k->const_data_ptr(), v->const_data_ptr(), o->mutable_data_ptr(),
      want_lse ? static_cast<float*>(lse.mutable_data_ptr()) : nullptr, static_cast<const int*>(cq->const_data_ptr()),
      static_cast<const int*>(ck->const_data_ptr()), static_cast<int>(seqs), static_cast<int>(tq), static_cast<int>(tk),
      static_cast<int>(max_q), static_cast<int>(max_k), static_cast<int>(h), static_cast<int>(hk), static_cast<int>(d), s,
      static_cast<float>(scale), causal, nullptr, stream));
  if (rc != DIT_OK) return PyLong_FromLong(rc);
  if (!want_lse) return THPVariable_Wrap(*o);
  return Py_BuildValue("(NN)", THPVariable_Wrap(*o), THPVariable_Wrap(lse));
  END_HANDLE_TH_ERRORS
}

// rotary(plan address, head_dim, axes, interleaved, x, positions, out, transpose)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor *x, *p, *o;
  if (n != 8 || rotary_fn == nullptr || !tensor(a[4], &x) || !tensor(a[5], &p) || !tensor(a[6], &o, true)) NOT_HERE;
  const dit_rotary* plan = static_cast<const dit_rotary*>(PyLong_AsVoidPtr(a[0]));
  const int64_t head_dim = PyLong_AsLong(a[1]), axes = PyLong_AsLong(a[2]);
  const int inter = PyObject_IsTrue(a[3]), transpose = PyObject_IsTrue(a[7]);
  if (inter < 0 || transpose < 0) {
    PyErr_Clear();
    NOT_HERE;
  }
  const bool wide = p->scalar_type() == at::kLong;
  const int code = code_of(x->scalar_type());
  const c10::DeviceIndex dev = c10::cuda::current_device();
  if (plan == nullptr || x->dim() != 3 || x->size(2) != head_dim || code < 0 || (!wide && p->scalar_type() != at::kInt) ||
      !p->is_contiguous() || !fits(x->size(0)) || !fits(x->size(1)) || x->get_device() != dev || p->get_device() != dev)
    NOT_HERE;
  const int64_t tokens = x->size(0);
  if (!(p->dim() == 2 && p->size(0) == tokens && p->size(1) == axes) && !(p->dim() == 1 && axes == 1 && p->size(0) == tokens))
    NOT_HERE;
  long long xs[2], ys[2];
  if (!head_strides(*x, xs)) NOT_HERE;
  at::Tensor fresh;
  if (o) {
    if (o->sizes() != x->sizes() || o->scalar_type() != x->scalar_type() || o->get_device() != dev || !head_strides(*o, ys)) NOT_HERE;
  } else {
    fresh = at::empty(x->sizes(), x->options());
    o = &fresh;
    ys[0] = x->size(1) * head_dim, ys[1] = head_dim;
  }
  const dit_stream_t stream = current_stream();
  CALL(rc, rotary_fn(plan, code, x->const_data_ptr(), xs[0], xs[1], p->const_data_ptr(), wide, o->mutable_data_ptr(),
                                  ys[0], ys[1], static_cast<int>(tokens), static_cast<int>(x->size(1)), static_cast<int>(head_dim),
                                  inter, transpose, stream));
  if (rc != DIT_OK) return PyLong_FromLong(rc);
  return THPVariable_Wrap(*o);
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the three entry points)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) Py_RETURN_NONE;
  linear_fn = reinterpret_cast<LinearFn>(PyLong_AsVoidPtr(a[0]));
  attention_fn = reinterpret_cast<AttentionFn>(PyLong_AsVoidPtr(a[1]));
  rotary_fn = reinterpret_cast<RotaryFn>(PyLong_AsVoidPtr(a[2]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
                         {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
                         {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)), METH_FASTCALL, nullptr},
                         {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotary)), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
