// The calls of attention to states of another length and of a decode step behind
// a prefix without the interpreter, as kv4_py.cpp's: arguments that are in order
// are looked over, outputs allocated and the entry point called; anything else comes
// back as None and cross.py says what is wrong or does it, an entry point's error as
// its number.  (Attention of 32 tokens over 1500 states: 25 us a call through ctypes,
// 10 so, 10 on the GPU.)
#include "py_tensors.h"

namespace {

decltype(&sfa_cross_workspace_size) cross_size;
decltype(&sfa_cross_forward) forward_entry;
decltype(&sfa_cross_backward) backward_entry;
decltype(&sfa_prefix_workspace_size) prefix_size;
decltype(&sfa_prefix_decode) prefix_entry;

// t [B, H, T, 64] with dense rows that do not overlap: its strides.
bool view(const Tensor* t, int64_t* s) {
  if (!t || t->dim() != 4 || t->size(3) != 64 || t->stride(3) != 1) return false;
  for (int i = 0; i < 3; ++i) {
    if (!fits(t->size(i))) return false;
    s[i] = t->stride(i);
    if (t->size(i) > 1 && (s[i] < 64 || s[i] * t->element_size() % 16)) return false;
  }
  return true;
}

// q, k, v and the lengths of a call into d: q, or null.
const Tensor* describe(PyObject* const* a, PyObject* q_len, PyObject* kv_len, int index, sfa_cross_desc* d) {
  const Tensor *const q = index >= 0 ? tensor(a[0], index) : nullptr, *const k = q ? tensor(a[1], index) : nullptr,
               *const v = k ? tensor(a[2], index) : nullptr;
  if (!v || !view(q, d->q_stride) || !view(k, d->k_stride) || !view(v, d->v_stride) || v->sizes() != k->sizes() ||
      q->size(0) != k->size(0) || k->scalar_type() != q->scalar_type() || v->scalar_type() != q->scalar_type() || !code(q->scalar_type(), &d->dtype))
    return nullptr;
  d->B = (int32_t)q->size(0);
  d->Hq = (int32_t)q->size(1);
  d->Tq = (int32_t)q->size(2);
  d->Hkv = (int32_t)k->size(1);
  d->Tk = (int32_t)k->size(2);
  d->D = 64;
  if (q_len != Py_None && !(d->q_len = ints(q_len, index, d->B))) return nullptr;
  if (kv_len != Py_None && !(d->kv_len = ints(kv_len, index, d->B))) return nullptr;
  return q;
}

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* const r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, a);
  PyTuple_SET_ITEM(r, 1, b);
  return r;
}

// forward(q, k, v, q_len, kv_len): o, lse
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  sfa_cross_desc d = {};
  const int index = n == 5 ? current(a[0]) : -1;
  const Tensor* const q = describe(a, a[3], a[4], index, &d);
  if (!q) SLOW;
  size_t bytes = 0;
  int rc = cross_size(&d, 0, &bytes);
  if (rc) return PyLong_FromLong(rc);
  const Tensor o = empty(q->sizes(), q->scalar_type(), index), lse = empty({d.B, d.Hq, d.Tq}, at::kFloat, index);
  Tensor ws;
  if (bytes) ws = empty({(int64_t)bytes}, at::kByte, index);
  const void *const qp = q->data_ptr(), *const kp = THPVariable_Unpack(a[1]).data_ptr(), *const vp = THPVariable_Unpack(a[2]).data_ptr();
  void *const op = o.data_ptr(), *const wp = bytes ? ws.data_ptr() : nullptr;
  float* const lp = static_cast<float*>(lse.data_ptr());
  rc = enqueue([&](void* s) { return forward_entry(&d, qp, kp, vp, op, lp, wp, bytes, s); }, index);
  if (rc) return PyLong_FromLong(rc);
  return pair(THPVariable_Wrap(o), THPVariable_Wrap(lse));
  END_HANDLE_TH_ERRORS
}

// backward(q, k, v, o, lse, do, q_len, kv_len): dq, dk, dv
PyObject* backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  sfa_cross_desc d = {};
  const int index = n == 8 ? current(a[0]) : -1;
  const Tensor* const q = n == 8 ? describe(a, a[6], a[7], index, &d) : nullptr;
  if (!q) SLOW;
  const Tensor *const o = dense(a[3], index, q->scalar_type(), q->sizes()), *const lse = dense(a[4], index, at::kFloat, {d.B, d.Hq, d.Tq}),
               *const go = dense(a[5], index, q->scalar_type(), q->sizes());
  if (!o || !lse || !go) SLOW;
  size_t bytes = 0;
  int rc = cross_size(&d, 1, &bytes);
  if (rc) return PyLong_FromLong(rc);
  const Tensor &k = THPVariable_Unpack(a[1]), &v = THPVariable_Unpack(a[2]);
  const Tensor dq = empty(q->sizes(), q->scalar_type(), index), dk = empty(k.sizes(), q->scalar_type(), index),
               dv = empty(k.sizes(), q->scalar_type(), index), ws = empty({(int64_t)bytes}, at::kByte, index);
  const void *const qp = q->data_ptr(), *const kp = k.data_ptr(), *const vp = v.data_ptr(), *const op = o->data_ptr(), *const gp = go->data_ptr();
  const float* const lp = static_cast<const float*>(lse->data_ptr());
  void *const dqp = dq.data_ptr(), *const dkp = dk.data_ptr(), *const dvp = dv.data_ptr(), *const wp = ws.data_ptr();
  rc = enqueue([&](void* s) { return backward_entry(&d, qp, kp, vp, op, lp, gp, dqp, dkp, dvp, wp, bytes, s); }, index);
  if (rc) return PyLong_FromLong(rc);
  PyObject* const r = PyTuple_New(3);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(dq));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(dk));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(dv));
  return r;
  END_HANDLE_TH_ERRORS
}

// Stride between the heads of t [Hkv, P, 64], each of which is dense.
bool heads(const Tensor* t, at::ScalarType type, const sfa_prefix_desc& d, int64_t* stride) {
  if (!t || t->scalar_type() != type || t->dim() != 3 || t->size(0) != d.Hkv || t->size(1) != d.P || t->size(2) != 64) return false;
  *stride = t->stride(0);
  if (t->is_contiguous() || d.P == 0) return true;
  return t->stride(2) == 1 && (d.P == 1 || t->stride(1) == 64) &&
         (d.Hkv == 1 || (*stride >= 64LL * d.P && *stride * t->element_size() % 16 == 0));
}

// prefix(q, k_new, v_new, prefix_k, prefix_v, k_cache, v_cache, pos, rope): o, lse
PyObject* prefix(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  sfa_prefix_desc d = {};
  const int index = n == 9 ? current(a[0]) : -1;
  const Tensor *const q = index >= 0 ? tensor(a[0], index) : nullptr, *const kc = q ? tensor(a[5], index) : nullptr,
               *const pk = kc ? tensor(a[3], index) : nullptr;
  if (!pk || kc->dim() != 4 || !kc->is_contiguous() || pk->dim() != 3 || kc->size(3) != 64 || !code(q->scalar_type(), &d.dtype) ||
      kc->scalar_type() != q->scalar_type())
    SLOW;
  for (int i = 0; i < 3; ++i)
    if (!fits(kc->size(i))) SLOW;
  if (!fits(pk->size(1)) || !rows(q, &d.q_stride)) SLOW;
  const at::ScalarType type = q->scalar_type();
  d.B = (int32_t)kc->size(0);
  d.Hkv = (int32_t)kc->size(1);
  d.T = (int32_t)kc->size(2);
  d.P = (int32_t)pk->size(1);
  d.Hq = (int32_t)q->size(1);
  d.D = 64;
  const Tensor* const vc = dense(a[6], index, type, kc->sizes());
  const int32_t* const pos = ints(a[7], index, d.B);
  if (!vc || !pos || q->size(0) != d.B || !heads(pk, type, d, &d.prefix_k_stride) || !heads(tensor(a[4], index), type, d, &d.prefix_v_stride)) SLOW;
  const bool news = a[1] != Py_None;
  const Tensor *const kn = news ? tensor(a[1], index) : nullptr, *const vn = news ? tensor(a[2], index) : nullptr;
  d.k_stride = d.v_stride = 64LL * d.Hkv;
  if (news ? !rows(kn, &d.k_stride) || !rows(vn, &d.v_stride) || kn->size(0) != d.B || kn->size(1) != d.Hkv || vn->sizes() != kn->sizes() ||
                 kn->scalar_type() != type || vn->scalar_type() != type
           : a[2] != Py_None)
    SLOW;
  if (a[8] != Py_None) {
    const Tensor* const t = tensor(a[8], index);
    if (!t || t->scalar_type() != at::kFloat || t->dim() != 3 || t->size(1) != 32 || t->size(2) != 2 || !t->is_contiguous() || !fits(t->size(0))) SLOW;
    d.rope = static_cast<const float*>(t->data_ptr());
    d.rope_T = (int32_t)t->size(0);
  }
  size_t bytes = 0;
  int rc = prefix_size(&d, &bytes);
  if (rc) return PyLong_FromLong(rc);
  const Tensor o = empty({d.B, d.Hq, 64}, type, index), lse = empty({d.B, d.Hq}, at::kFloat, index), ws = empty({(int64_t)bytes}, at::kByte, index);
  const Tensor& pv = THPVariable_Unpack(a[4]);
  const void *const qp = q->data_ptr(), *const knp = news ? kn->data_ptr() : nullptr, *const vnp = news ? vn->data_ptr() : nullptr;
  const void *const pkp = d.P ? pk->data_ptr() : nullptr, *const pvp = d.P ? pv.data_ptr() : nullptr;
  void *const kcp = kc->data_ptr(), *const vcp = vc->data_ptr(), *const op = o.data_ptr(), *const wp = ws.data_ptr();
  float* const lp = static_cast<float*>(lse.data_ptr());
  rc = enqueue([&](void* s) { return prefix_entry(&d, qp, knp, vnp, pkp, pvp, kcp, vcp, pos, op, lp, wp, bytes, s); }, index);
  if (rc) return PyLong_FromLong(rc);
  return pair(THPVariable_Wrap(o), THPVariable_Wrap(lse));
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the workspace size, forward, backward, prefix size, prefix)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind takes five addresses");
  void* p[5];
  for (int i = 0; i < 5; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(a[i]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "a null address");
  cross_size = reinterpret_cast<decltype(cross_size)>(p[0]);
  forward_entry = reinterpret_cast<decltype(forward_entry)>(p[1]);
  backward_entry = reinterpret_cast<decltype(backward_entry)>(p[2]);
  prefix_size = reinterpret_cast<decltype(prefix_size)>(p[3]);
  prefix_entry = reinterpret_cast<decltype(prefix_entry)>(p[4]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {METHOD(forward), METHOD(backward), METHOD(prefix), METHOD(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cross", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cross() { return PyModule_Create(&module); }
