// binding.cpp -- the packed and paged calls straight from Python: the checks
// that exact_io_aware_65_b200/__init__.py makes, on the tensors' own fields, the
// outputs' allocation, and the call into libfa.  A call that takes the Python
// checks and ctypes 11 to 30 us of the host takes 3.5 to 13.5 us this way (an append
// 10.5 and 3.5, a backward that makes its outputs 30 and 13.5); the smallest kernels
// take 2 us.
//
// A function here returns what its Python namesake returns; an int, the status
// of a call that the library refused; or None for anything out of the ordinary
// (a tensor that fails a check, another device than the current one): the
// Python code then makes its checks again, and reports or handles what it finds.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
// (first, as its own headers ask)
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "fa.h"

namespace {

struct Calls {
  decltype(&fa_fwd_packed) fwd;
  decltype(&fa_fwd_packed_workspace_size) fwd_size;
  decltype(&fa_bwd_packed) bwd;
  decltype(&fa_bwd_packed_workspace_size) bwd_size;
  decltype(&fa_paged_append) append;
  decltype(&fa_paged_decode) decode;
  decltype(&fa_paged_decode_workspace_size) decode_size;
  decltype(&fa_paged_evict) evict;
} fa;

// A tensor argument; null for None.  False: neither.
bool tensor(PyObject* o, const at::Tensor** t) {
  *t = nullptr;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  return true;
}

// What all of a call's tensors must share.
struct On {
  c10::Device device{c10::kCPU};
  // The call's device: the current one.
  bool take(const at::Tensor* t) {
    if (!t || !t->is_cuda()) return false;
    device = t->device();
    return device.index() == c10::cuda::current_device();
  }
  bool has(const at::Tensor* t) const { return t && t->device() == device && t->layout() == at::kStrided; }
  // contiguous, of this type and shape
  bool is(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape) const {
    return has(t) && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
};

// fa_rows of bf16 rows [n, h, d] (-1: any).
bool rows(const On& on, const at::Tensor* t, int64_t n, int64_t h, int64_t d, fa_rows* r) {
  if (!on.has(t) || t->scalar_type() != at::kBFloat16 || t->dim() != 3) return false;
  if ((n >= 0 && t->size(0) != n) || (h >= 0 && t->size(1) != h) || (d >= 0 && t->size(2) != d)) return false;
  // (the stride of a single row or head is never used)
  r->row_stride = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
  r->head_stride = t->size(1) > 1 ? t->stride(1) : t->size(2);
  r->data = t->data_ptr();
  return (t->stride(2) == 1 || t->size(2) <= 1) && ((r->row_stride | r->head_stride) & 7) == 0 &&
         (reinterpret_cast<uintptr_t>(r->data) & 15) == 0;
}

bool table(const On& on, const at::Tensor* t, int64_t B, const int** p, int64_t* width, int64_t* stride) {
  if (!on.has(t) || t->scalar_type() != at::kInt || t->dim() != 2 || t->size(0) <= 0 || t->size(1) <= 0) return false;
  if ((t->stride(1) != 1 && t->size(1) != 1) || (B >= 0 && t->size(0) != B)) return false;
  *p = t->data_ptr<int>();
  *width = t->size(1);
  *stride = t->size(0) > 1 ? t->stride(0) : t->size(1);
  return true;
}

bool cache(const On& on, const at::Tensor* k, const at::Tensor* v, const at::Tensor* pages, const at::Tensor* ks,
           const at::Tensor* vs, bool scales, fa_paged_cache* c) {
  if (!on.has(k) || !on.has(v) || k->dim() != 4 || k->scalar_type() != v->scalar_type()) return false;
  if (k->sizes() != v->sizes() || k->strides() != v->strides()) return false;
  const bool eight = k->scalar_type() == at::kFloat8_e4m3fn;
  if (!eight && k->scalar_type() != at::kBFloat16) return false;
  c->K = k->data_ptr();
  c->V = v->data_ptr();
  c->dtype = eight ? FA_CACHE_E4M3 : FA_CACHE_BF16;
  for (int i = 0; i < 4; ++i)
    if (k->size(i) > INT32_MAX) return false;
  c->num_pages = (int)k->size(0);
  c->Hkv = (int)k->size(1);
  c->page_size = (int)k->size(2);
  c->d = (int)k->size(3);
  c->page_stride = c->num_pages > 1 ? k->stride(0) : 0;
  c->head_stride = c->Hkv > 1 ? k->stride(1) : 0;
  c->row_stride = c->page_size > 1 ? k->stride(2) : 0;
  if (k->stride(3) != 1 && c->d > 1) return false;
  if ((c->page_stride | c->head_stride | c->row_stride) & (eight ? 15 : 7)) return false;
  if ((reinterpret_cast<uintptr_t>(c->K) | reinterpret_cast<uintptr_t>(c->V)) & 15) return false;
  c->k_scale = c->v_scale = nullptr;
  if (eight && scales) {
    if (!on.is(ks, at::kFloat, {c->Hkv}) || !on.is(vs, at::kFloat, {c->Hkv})) return false;
    c->k_scale = ks->data_ptr<float>();
    c->v_scale = vs->data_ptr<float>();
  } else if (ks || vs) {
    return false;
  }
  int64_t width;
  if (!table(on, pages, -1, &c->page_table, &width, &c->table_stride) || width > INT32_MAX || pages->size(0) > INT32_MAX)
    return false;
  c->B = (int)pages->size(0);
  c->max_pages = (int)width;
  return true;
}

// fp32 rows [B, Hkv, at least `least`].
bool weights(const On& on, const at::Tensor* t, int64_t B, int64_t H, int64_t least, float** p, int64_t* batch, int64_t* head) {
  if (!on.has(t) || t->scalar_type() != at::kFloat || t->dim() != 3 || t->size(0) != B || t->size(1) != H) return false;
  if (t->size(2) < least || (t->stride(2) != 1 && t->size(2) != 1)) return false;
  *p = t->data_ptr<float>();
  *batch = B > 1 ? t->stride(0) : 0;
  *head = H > 1 ? t->stride(1) : 0;
  return true;
}

// The caller's workspace, or a new one.
bool workspace(const On& on, const at::Tensor* given, size_t need, at::Tensor* own, void** p, size_t* bytes) {
  if (given) {
    if (!on.has(given) || !given->is_contiguous() || given->nbytes() < need) return false;
    *p = given->data_ptr();
    *bytes = given->nbytes();
    return true;
  }
  *p = nullptr;
  *bytes = 0;
  if (need == 0) return true;
  *own = on.empty({(int64_t)need}, at::kByte);
  *p = own->data_ptr();
  *bytes = need;
  return true;
}

bool number(PyObject* o, int64_t* v) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0;
}
// scale, or 1 / sqrt(d) for None
bool scale_of(PyObject* o, int64_t d, float* s) {
  if (o == Py_None) *s = (float)(1.0 / std::sqrt((double)d));
  else if (PyFloat_Check(o)) *s = (float)PyFloat_AS_DOUBLE(o);
  else return false;
  return true;
}

PyObject* answer(fa_status st, std::initializer_list<at::Tensor> out) {
  if (st != FA_OK) return PyLong_FromLong(st);
  PyObject* t = PyTuple_New((Py_ssize_t)out.size());
  Py_ssize_t i = 0;
  for (const at::Tensor& x : out) PyTuple_SET_ITEM(t, i++, THPVariable_Wrap(x));
  return t;
}

struct Packed {
  int64_t Tq, Tk, Hq, Hkv, d, B, kind;
  float scale;
  const int *cu_q, *cu_k;
  fa_rows q, k, v;
};
bool packed(On& on, const at::Tensor* Q, const at::Tensor* K, const at::Tensor* V, const at::Tensor* cq, const at::Tensor* ck,
            PyObject* kind, PyObject* scale, Packed* p) {
  if (!on.take(Q) || !rows(on, Q, -1, -1, -1, &p->q)) return false;
  p->Tq = Q->size(0);
  p->Hq = Q->size(1);
  p->d = Q->size(2);
  if (!rows(on, K, -1, -1, p->d, &p->k)) return false;
  p->Tk = K->size(0);
  p->Hkv = K->size(1);
  if (!rows(on, V, p->Tk, p->Hkv, p->d, &p->v)) return false;
  if (!on.has(cq) || cq->dim() != 1 || cq->size(0) < 2) return false;
  p->B = cq->size(0) - 1;
  if (!on.is(cq, at::kInt, {p->B + 1}) || !on.is(ck, at::kInt, {p->B + 1})) return false;
  p->cu_q = cq->data_ptr<int>();
  p->cu_k = ck->data_ptr<int>();
  if (p->Tq > INT32_MAX || p->Tk > INT32_MAX || p->Hq > INT32_MAX || p->Hkv > INT32_MAX || p->B > INT32_MAX) return false;
  return number(kind, &p->kind) && scale_of(scale, p->d, &p->scale);
}

#define TENSORS(n)                                    \
  const at::Tensor* t[n];                             \
  for (int i = 0; i < (n); ++i)                       \
    if (!tensor(a[i], &t[i])) Py_RETURN_NONE;
#define REQUIRE(x) \
  if (!(x)) Py_RETURN_NONE;

// (Q, K, V, cu_q, cu_k, O, LSE, workspace, kind, scale)
PyObject* fwd_packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REQUIRE(n == 10 && fa.fwd);
  TENSORS(8)
  On on;
  Packed p;
  REQUIRE(packed(on, t[0], t[1], t[2], t[3], t[4], a[8], a[9], &p));
  const at::Tensor O = t[5] ? *t[5] : on.empty({p.Tq, p.Hq, p.d}, at::kBFloat16);
  fa_rows o;
  REQUIRE(rows(on, &O, p.Tq, p.Hq, p.d, &o));
  REQUIRE(!t[6] || on.is(t[6], at::kFloat, {p.Hq, p.Tq}));
  const at::Tensor L = t[6] ? *t[6] : on.empty({p.Hq, p.Tq}, at::kFloat);
  at::Tensor own;
  void* ws;
  size_t wn;
  REQUIRE(workspace(on, t[7], fa.fwd_size((int)p.B, (int)p.Tq, (int)p.Hq, (int)p.Hkv, (int)p.d), &own, &ws, &wn));
  return answer(fa.fwd(&p.q, &p.k, &p.v, p.cu_q, p.cu_k, (int)p.B, (int)p.Tq, (int)p.Tk, (int)p.Hq, (int)p.Hkv, (int)p.d,
                       (int)p.kind, p.scale, &o, L.data_ptr<float>(), ws, wn, on.stream()),
                {O, L});
}

// (Q, K, V, cu_q, cu_k, O, dO, LSE, dQ, dK, dV, workspace, kind, scale, deterministic)
PyObject* bwd_packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REQUIRE(n == 15 && fa.bwd);
  TENSORS(12)
  On on;
  Packed p;
  int64_t det;
  REQUIRE(packed(on, t[0], t[1], t[2], t[3], t[4], a[12], a[13], &p) && number(a[14], &det));
  fa_rows o, g, dq, dk, dv;
  REQUIRE(rows(on, t[5], p.Tq, p.Hq, p.d, &o) && rows(on, t[6], p.Tq, p.Hq, p.d, &g));
  REQUIRE(on.is(t[7], at::kFloat, {p.Hq, p.Tq}));
  const at::Tensor dQ = t[8] ? *t[8] : on.empty({p.Tq, p.Hq, p.d}, at::kBFloat16);
  const at::Tensor dK = t[9] ? *t[9] : on.empty({p.Tk, p.Hkv, p.d}, at::kBFloat16);
  const at::Tensor dV = t[10] ? *t[10] : on.empty({p.Tk, p.Hkv, p.d}, at::kBFloat16);
  REQUIRE(rows(on, &dQ, p.Tq, p.Hq, p.d, &dq) && rows(on, &dK, p.Tk, p.Hkv, p.d, &dk) && rows(on, &dV, p.Tk, p.Hkv, p.d, &dv));
  at::Tensor own;
  void* ws;
  size_t wn;
  REQUIRE(workspace(on, t[11], fa.bwd_size((int)p.B, (int)p.Tq, (int)p.Tk, (int)p.Hq, (int)p.Hkv, (int)p.d), &own, &ws, &wn));
  return answer(fa.bwd(&p.q, &p.k, &p.v, &o, &g, t[7]->data_ptr<float>(), p.cu_q, p.cu_k, (int)p.B, (int)p.Tq, (int)p.Tk,
                       (int)p.Hq, (int)p.Hkv, (int)p.d, (int)p.kind, p.scale, (int)det, &dq, &dk, &dv, ws, wn, on.stream()),
                {dQ, dK, dV});
}

// (K, V, cu_seqlens, lens, k_cache, v_cache, page_table, k_scale, v_scale)
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REQUIRE(n == 9 && fa.append);
  TENSORS(9)
  On on;
  fa_paged_cache c;
  fa_rows k, v;
  REQUIRE(on.take(t[4]) && cache(on, t[4], t[5], t[6], t[7], t[8], true, &c));
  REQUIRE(rows(on, t[0], -1, c.Hkv, c.d, &k) && rows(on, t[1], t[0]->size(0), c.Hkv, c.d, &v));
  REQUIRE(t[0]->size(0) <= INT32_MAX && on.is(t[2], at::kInt, {c.B + 1}) && on.is(t[3], at::kInt, {c.B}));
  return answer(fa.append(&c, &k, &v, t[2]->data_ptr<int>(), t[3]->data_ptr<int>(), (int)t[0]->size(0), on.stream()), {});
}

// (Q, k_cache, v_cache, page_table, lens, k_scale, v_scale, weights, O, LSE, workspace, scale, accumulate)
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REQUIRE(n == 13 && fa.decode);
  TENSORS(11)
  On on;
  fa_paged_cache c;
  fa_rows q;
  float scale;
  int64_t add;
  REQUIRE(on.take(t[1]) && cache(on, t[1], t[2], t[3], t[5], t[6], true, &c));
  REQUIRE(rows(on, t[0], c.B, -1, c.d, &q) && scale_of(a[11], c.d, &scale) && number(a[12], &add));
  const int64_t Hq = t[0]->size(1), cap = (int64_t)c.max_pages * c.page_size;
  REQUIRE(Hq <= INT32_MAX && on.is(t[4], at::kInt, {c.B}));
  float* w = nullptr;
  int64_t wb = 0, wh = 0;
  REQUIRE(!t[7] || weights(on, t[7], c.B, c.Hkv, cap, &w, &wb, &wh));
  REQUIRE((!t[8] || on.is(t[8], at::kBFloat16, {c.B, Hq, c.d})) && (!t[9] || on.is(t[9], at::kFloat, {c.B, Hq})));
  const at::Tensor O = t[8] ? *t[8] : on.empty({c.B, Hq, c.d}, at::kBFloat16);
  const at::Tensor L = t[9] ? *t[9] : on.empty({c.B, Hq}, at::kFloat);
  at::Tensor own;
  void* ws;
  size_t wn;
  REQUIRE(workspace(on, t[10], fa.decode_size(c.B, (int)Hq, c.Hkv, c.d, cap, w != nullptr), &own, &ws, &wn));
  return answer(fa.decode(&c, &q, (int)Hq, t[4]->data_ptr<int>(), scale, w, wb, wh, (int)add, O.data_ptr(),
                          L.data_ptr<float>(), ws, wn, on.stream()),
                {O, L});
}

// (weights, k_cache, v_cache, page_table, lens, table_out, weights_out, kept, lens_out, budget, recent)
PyObject* paged_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REQUIRE(n == 11 && fa.evict);
  TENSORS(9)
  On on;
  fa_paged_cache c;
  int64_t budget, recent, wb, wh, ob, oh, width, stride;
  float *w, *wo;
  const int* out;
  REQUIRE(number(a[9], &budget) && number(a[10], &recent) && budget > 0 && budget <= INT32_MAX && recent >= 0 && recent <= budget);
  REQUIRE(on.take(t[1]) && cache(on, t[1], t[2], t[3], nullptr, nullptr, false, &c));
  const int64_t cap = (int64_t)c.max_pages * c.page_size;
  REQUIRE(weights(on, t[0], c.B, c.Hkv, cap, &w, &wb, &wh));
  REQUIRE(weights(on, t[6], c.B, c.Hkv, budget < cap ? budget : cap, &wo, &ob, &oh));
  REQUIRE(table(on, t[5], c.B, &out, &width, &stride) && width <= INT32_MAX && on.is(t[4], at::kInt, {c.B}));
  REQUIRE((!t[7] || on.is(t[7], at::kInt, {c.B, c.Hkv, budget})) && (!t[8] || on.is(t[8], at::kInt, {c.B})));
  const at::Tensor kept = t[7] ? *t[7] : on.empty({c.B, c.Hkv, budget}, at::kInt);
  const at::Tensor left = t[8] ? *t[8] : on.empty({c.B}, at::kInt);
  return answer(fa.evict(&c, t[4]->data_ptr<int>(), out, stride, (int)width, w, wb, wh, (int)budget, (int)recent, wo, ob, oh,
                         t[6]->size(2), kept.data_ptr<int>(), left.data_ptr<int>(), on.stream()),
                {kept, left});
}

// An exception from torch (an allocation that fails, say) as a Python one.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const c10::OutOfMemoryError&) {
    Py_RETURN_NONE;  // the Python code tries again, and torch raises its own error
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// use(handle): take the calls from this libfa (the handle of dlopen).
PyObject* use(PyObject*, PyObject* arg) {
  void* h = PyLong_AsVoidPtr(arg);
  if (PyErr_Occurred()) return nullptr;
  Calls c;
#define SYM(field, name) c.field = reinterpret_cast<decltype(c.field)>(dlsym(h, #name))
  SYM(fwd, fa_fwd_packed);
  SYM(fwd_size, fa_fwd_packed_workspace_size);
  SYM(bwd, fa_bwd_packed);
  SYM(bwd_size, fa_bwd_packed_workspace_size);
  SYM(append, fa_paged_append);
  SYM(decode, fa_paged_decode);
  SYM(decode_size, fa_paged_decode_workspace_size);
  SYM(evict, fa_paged_evict);
  if (!c.fwd || !c.fwd_size || !c.bwd || !c.bwd_size || !c.append || !c.decode || !c.decode_size || !c.evict) {
    PyErr_SetString(PyExc_RuntimeError, "libfa lacks a call of the binding");
    return nullptr;
  }
  fa = c;
  Py_RETURN_NONE;
}

#define CALL(name) {#name, (PyCFunction)(void (*)(void))guarded<name>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(fwd_packed), CALL(bwd_packed),  CALL(paged_append),      CALL(paged_decode),
                         CALL(paged_evict), {"use", use, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
