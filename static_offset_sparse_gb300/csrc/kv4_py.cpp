// The calls of the paged 4-bit cache's Python names: arguments looked over,
// outputs allocated and the entry point called without the interpreter, whose
// share of a call is three times what the GPU takes for a small one (attention
// of 32 rows of 23 keys: 17.5 us a call through ctypes, 5.7 so, 4.3 on the GPU;
// a plan 22 and 5.2, a write and a read of 32 rows 20 and 7).  Only what is in
// order is done here.  Anything else (wrong types or shapes, another device than
// the current one, a workspace of the caller's) comes back as None, and kv4.py
// says what is wrong or does it; an entry point's error comes back as its number.
#include "py_tensors.h"

namespace {

decltype(&sfa_kv4_plan) plan_entry;
decltype(&sfa_kv4_append) append_entry;
decltype(&sfa_kv4_read) read_entry;
decltype(&sfa_kv4_workspace_size) size_entry;
decltype(&sfa_kv4_attend) attend_entry;

// Pages, rows a page and KV heads of a cache into d; its address, or null.
uint8_t* pool(PyObject* o, int index, sfa_kv4_desc* d) {
  const Tensor* t = tensor(o, index);
  if (!t || t->scalar_type() != at::kByte || t->dim() != 3 || !t->is_contiguous()) return nullptr;
  const int64_t width = t->size(2);
  if (width != 72 * 16 && width != 72 * 32 && width != 72 * 64 && width != 72 * 128) return nullptr;
  if (!fits(t->size(0)) || !fits(t->size(1))) return nullptr;
  d->n_pages = (int32_t)t->size(0);
  d->Hkv = (int32_t)t->size(1);
  d->page = (int32_t)(width / 72);
  d->D = 64;
  return static_cast<uint8_t*>(t->data_ptr());
}

bool rope_table(PyObject* o, int index, sfa_kv4_desc* d) {
  if (o == Py_None) return true;
  const Tensor* t = tensor(o, index);
  if (!t || t->scalar_type() != at::kFloat || t->dim() != 3 || t->size(1) != 32 || t->size(2) != 2 || !t->is_contiguous() ||
      !fits(t->size(0)))
    return false;
  d->rope = static_cast<const float*>(t->data_ptr());
  d->rope_T = (int32_t)t->size(0);
  return true;
}

bool scales(PyObject* k, PyObject* v, sfa_kv4_desc* d) {
  if (!PyFloat_CheckExact(k) || !PyFloat_CheckExact(v)) return false;
  const double ks = PyFloat_AS_DOUBLE(k), vs = PyFloat_AS_DOUBLE(v);
  d->kscale = (float)ks;
  d->vscale = (float)vs;
  return ks > 0.0 && ks <= 3.4e38 && vs > 0.0 && vs <= 3.4e38;
}

// n int32 from `offset` on of a buffer that several outputs share.
Tensor part(const Tensor& buffer, int64_t offset, int64_t n) {
  auto impl = c10::make_intrusive<at::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(), buffer.dtype());
  impl->set_sizes_contiguous({n});
  impl->set_storage_offset(offset);
  return Tensor(std::move(impl));
}

// attend(q, cache, block_table, seq_lens, cu_q, (address, number, ..) of dist, rope, kscale, vscale, o, lse, ws)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  sfa_kv4_desc d = {};
  const int index = n == 12 ? current(a[0]) : -1;
  const Tensor* const q = index >= 0 ? tensor(a[0], index) : nullptr;
  uint8_t* const cache = q ? pool(a[1], index, &d) : nullptr;
  const Tensor* const table = cache ? tensor(a[2], index) : nullptr;
  if (!table || table->scalar_type() != at::kInt || table->dim() != 2 || !table->is_contiguous() || !fits(table->size(0)) ||
      !fits(table->size(1)) || !rows(q, &d.q_stride) || !code(q->scalar_type(), &d.dtype) || !scales(a[7], a[8], &d) ||
      !rope_table(a[6], index, &d))
    SLOW;
  d.R = (int32_t)table->size(0);
  d.max_pages = (int32_t)table->size(1);
  d.N = (int32_t)q->size(0);
  d.Hq = (int32_t)q->size(1);
  int32_t *const lens = ints(a[3], index, d.R), *const cu = a[4] == Py_None ? nullptr : ints(a[4], index, d.R + 1LL);
  if (!lens || (a[4] == Py_None ? d.N != d.R : !cu) || a[11] != Py_None) SLOW;
  if (a[5] != Py_None) {
    d.dist = static_cast<const int32_t*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[5], 0)));
    d.n_dist = (int32_t)PyLong_AsLong(PyTuple_GET_ITEM(a[5], 1));
  }
  const Tensor* const oo = a[9] == Py_None ? nullptr : dense(a[9], index, q->scalar_type(), q->sizes());
  const Tensor* const ll = a[10] == Py_None ? nullptr : dense(a[10], index, at::kFloat, {d.N, d.Hq});
  if ((a[9] != Py_None && !oo) || (a[10] != Py_None && !ll)) SLOW;
  const Tensor o = oo ? *oo : empty(q->sizes(), q->scalar_type(), index), lse = ll ? *ll : empty({d.N, d.Hq}, at::kFloat, index);
  size_t bytes = 0;
  int rc = size_entry(&d, &bytes);
  if (rc) return PyLong_FromLong(rc);
  Tensor ws;
  if (bytes) ws = empty({(int64_t)bytes}, at::kByte, index);
  const void* const qp = q->data_ptr();
  void *const op = o.data_ptr(), *const wp = bytes ? ws.data_ptr() : nullptr;
  float* const lp = static_cast<float*>(lse.data_ptr());
  const int32_t* const tp = static_cast<const int32_t*>(table->data_ptr());
  rc = enqueue([&](void* s) { return attend_entry(&d, qp, cache, tp, lens, cu, op, lp, wp, bytes, s); }, index);
  if (rc) return PyLong_FromLong(rc);
  PyObject* const r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, oo ? Py_NewRef(a[9]) : THPVariable_Wrap(o));
  PyTuple_SET_ITEM(r, 1, ll ? Py_NewRef(a[10]) : THPVariable_Wrap(lse));
  return r;
  END_HANDLE_TH_ERRORS
}

// append(k, v, cache, slots, pos, rope, kscale, vscale)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  sfa_kv4_desc d = {};
  const int index = n == 8 ? current(a[0]) : -1;
  const Tensor *const k = index >= 0 ? tensor(a[0], index) : nullptr, *const v = k ? tensor(a[1], index) : nullptr;
  uint8_t* const cache = v ? pool(a[2], index, &d) : nullptr;
  if (!cache || !rows(k, &d.k_stride) || !rows(v, &d.v_stride) || k->size(1) != d.Hkv || v->sizes() != k->sizes() ||
      v->scalar_type() != k->scalar_type() || !code(k->scalar_type(), &d.dtype) || !scales(a[6], a[7], &d) || !rope_table(a[5], index, &d))
    SLOW;
  d.N = (int32_t)k->size(0);
  const int32_t *const slots = ints(a[3], index, d.N), *const pos = ints(a[4], index, d.N);
  if (!slots || !pos) SLOW;
  const void *const kp = k->data_ptr(), *const vp = v->data_ptr();
  return PyLong_FromLong(enqueue([&](void* s) { return append_entry(&d, kp, vp, cache, slots, pos, s); }, index));
  END_HANDLE_TH_ERRORS
}

// read(cache, slots, kscale, vscale, bf16): new tensors
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  sfa_kv4_desc d = {};
  const int index = n == 5 ? current(a[0]) : -1;
  uint8_t* const cache = index >= 0 ? pool(a[0], index, &d) : nullptr;
  const Tensor* const t = cache ? tensor(a[1], index) : nullptr;
  if (!t || t->dim() != 1 || !fits(t->size(0)) || !scales(a[2], a[3], &d)) SLOW;
  d.N = (int32_t)t->size(0);
  const int32_t* const slots = ints(a[1], index, d.N);
  if (!slots) SLOW;
  const at::ScalarType type = a[4] == Py_True ? at::kBFloat16 : at::kFloat;
  code(type, &d.dtype);
  const Tensor k = empty({d.N, d.Hkv, 64}, type, index), v = empty({d.N, d.Hkv, 64}, type, index);
  void *const kp = k.data_ptr(), *const vp = v.data_ptr();
  const int rc = enqueue([&](void* s) { return read_entry(&d, cache, slots, kp, vp, s); }, index);
  if (rc) return PyLong_FromLong(rc);
  PyObject* const r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(k));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(v));
  return r;
  END_HANDLE_TH_ERRORS
}

// plan(n_new, seq_lens, block_table, free_pages, n_free, page, rows, seq_lens_out, n_free_out)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  sfa_kv4_desc d = {};
  const int index = n == 9 ? current(a[2]) : -1;
  const Tensor *const table = index >= 0 ? tensor(a[2], index) : nullptr, *const stack = table ? tensor(a[3], index) : nullptr;
  if (!stack || table->scalar_type() != at::kInt || table->dim() != 2 || !table->is_contiguous() || !fits(table->size(0)) ||
      !fits(table->size(1)) || stack->dim() != 1 || !fits(stack->size(0)) || !PyLong_CheckExact(a[5]) || !PyLong_CheckExact(a[6]))
    SLOW;
  const long long page = PyLong_AsLongLong(a[5]), N = PyLong_AsLongLong(a[6]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    SLOW;
  }
  if (!fits(page) || !fits(N)) SLOW;
  d.n_pages = (int32_t)stack->size(0);
  d.page = (int32_t)page;
  d.R = (int32_t)table->size(0);
  d.max_pages = (int32_t)table->size(1);
  d.N = (int32_t)N;
  int32_t *const fresh = ints(a[0], index, d.R), *const lens = ints(a[1], index, d.R), *const free_pages = ints(a[3], index, d.n_pages);
  int32_t* const n_free = ints(a[4], index, 1);
  int32_t *lens_out = a[7] == Py_None ? nullptr : ints(a[7], index, d.R), *left = a[8] == Py_None ? nullptr : ints(a[8], index, 1);
  if (!fresh || !lens || !free_pages || !n_free || (a[7] != Py_None && !lens_out) || (a[8] != Py_None && !left)) SLOW;
  const int64_t R = d.R;
  const Tensor own = empty({2 * R + 2 + 2 * N}, at::kInt, index);  // boundaries, slots, positions, lengths, pages left
  int32_t *const cp = static_cast<int32_t*>(own.data_ptr()), *const sp = cp + R + 1, *const pp = sp + N;
  int32_t* const tp = static_cast<int32_t*>(table->data_ptr());
  if (!lens_out) lens_out = pp + N;
  if (!left) left = pp + N + R;
  const int rc =
      enqueue([&](void* s) { return plan_entry(&d, fresh, lens, tp, free_pages, n_free, cp, sp, pp, lens_out, left, s); }, index);
  if (rc) return PyLong_FromLong(rc);
  PyObject* const r = PyTuple_New(5);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(part(own, 0, R + 1)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(part(own, R + 1, N)));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(part(own, R + 1 + N, N)));
  PyTuple_SET_ITEM(r, 3, a[7] == Py_None ? THPVariable_Wrap(part(own, R + 1 + 2 * N, R)) : Py_NewRef(a[7]));
  PyTuple_SET_ITEM(r, 4, a[8] == Py_None ? THPVariable_Wrap(part(own, 2 * R + 1 + 2 * N, 1)) : Py_NewRef(a[8]));
  return r;
  END_HANDLE_TH_ERRORS
}

// bind(addresses of plan, append, read, workspace_size, attend)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind takes five addresses");
  void* p[5];
  for (int i = 0; i < 5; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(a[i]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "a null address");
  plan_entry = reinterpret_cast<decltype(plan_entry)>(p[0]);
  append_entry = reinterpret_cast<decltype(append_entry)>(p[1]);
  read_entry = reinterpret_cast<decltype(read_entry)>(p[2]);
  size_entry = reinterpret_cast<decltype(size_entry)>(p[3]);
  attend_entry = reinterpret_cast<decltype(attend_entry)>(p[4]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {METHOD(plan), METHOD(append), METHOD(read), METHOD(attend), METHOD(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv4", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv4() { return PyModule_Create(&module); }
