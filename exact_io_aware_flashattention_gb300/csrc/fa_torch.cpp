// Native marshalling of torch tensors into the rotary and paged-cache entry
// points (include/fa.h), for the calls a decoding loop makes thousands of
// times a second: 4-7 us of host time a call instead of 20-25 through Python
// and ctypes, several times what a small one takes on the GPU.
//
// Each function takes the arguments of its Python namesake (without stream),
// in order, and returns what that returns; None where it does not take the
// call (an argument of another kind, shape, type or device, another current
// device): Python then makes it itself and says what is wrong with it.  A
// status other than FA_OK comes back as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "fa.h"

namespace {

decltype(&fa_rope) p_rope = nullptr;
decltype(&fa_paged_append) p_append = nullptr;
decltype(&fa_paged_decode) p_decode = nullptr;
decltype(&fa_paged_decode_workspace_bytes) p_decode_ws = nullptr;
decltype(&fa_paged_evict) p_evict = nullptr;

using Shape = at::IntArrayRef;

// The device of a call's first tensor, if it is the current one.
struct Where {
  c10::Device device{c10::kCPU};
  void* stream = nullptr;
};
bool where(const at::Tensor& t, Where& w) {
  if (!t.is_cuda()) return false;
  w.device = t.device();
  if (w.device.index() != c10::cuda::current_device()) return false;
  w.stream = c10::cuda::getCurrentCUDAStream(w.device.index()).stream();
  return true;
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }
// None: absent (null), a tensor: itself; anything else: refused.
bool maybe(PyObject* o, const at::Tensor*& t) {
  t = nullptr;
  if (o == Py_None) return true;
  t = tensor(o);
  return t != nullptr;
}
bool integer(PyObject* o, int& x) {
  if (!PyLong_CheckExact(o)) return false;
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  x = (int)v;
  return !overflow && v == x;
}
bool boolean(PyObject* o, int& x) {
  x = o == Py_True;
  return o == Py_True || o == Py_False;
}

// A tensor of this type and shape on the call's device whose rows are
// contiguous, or that is contiguous altogether.
bool rows_of(const at::Tensor& t, const Where& w, at::ScalarType type, Shape shape) {
  return t.scalar_type() == type && t.is_cuda() && t.device() == w.device && t.layout() == c10::kStrided &&
         t.sizes() == shape && t.stride(-1) == 1;
}
bool dense(const at::Tensor& t, const Where& w, at::ScalarType type, Shape shape) {
  return t.scalar_type() == type && t.is_cuda() && t.device() == w.device && t.layout() == c10::kStrided &&
         t.sizes() == shape && t.is_contiguous();
}
bool fits(int64_t n) { return n >= 0 && n <= INT32_MAX; }

const long long* strides(const at::Tensor& t) { return reinterpret_cast<const long long*>(t.strides().data()); }
// On the current device, which is the call's.
at::Tensor empty(Shape shape, at::ScalarType type) {
  return at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                   type, std::nullopt);
}
int dtype_code(at::ScalarType t) { return t == at::kBFloat16 ? FA_BF16 : t == at::kHalf ? FA_FP16 : -1; }

PyObject* result(fa_status s, const at::Tensor& a) {
  return s == FA_OK ? THPVariable_Wrap(a) : PyLong_FromLong(s);
}
PyObject* result(fa_status s, const at::Tensor& a, const at::Tensor& b) {
  if (s != FA_OK) return PyLong_FromLong(s);
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}

// positions [n_axes, lead...], inv_freq and axes [n].
bool rotary(PyObject* const* o, PyObject* inter, const Where& w, int64_t d, Shape lead, fa_rotary& r) {
  const at::Tensor *pos = tensor(o[0]), *freq = tensor(o[1]), *axes = tensor(o[2]);
  int interleaved = 0;
  if (!pos || !freq || !axes || !boolean(inter, interleaved)) return false;
  if (pos->scalar_type() != at::kInt || !pos->is_cuda() || pos->device() != w.device || pos->dim() != (int64_t)lead.size() + 1 ||
      pos->sizes().slice(1) != lead || pos->stride(-1) != 1 || freq->dim() != 1)
    return false;
  const int64_t n = freq->size(0);
  if (n < 1 || 2 * n > d || !fits(pos->size(0)) || !dense(*freq, w, at::kDouble, n) || !dense(*axes, w, at::kInt, n))
    return false;
  r.positions = static_cast<const int*>(pos->const_data_ptr());
  r.axis_stride = pos->stride(0);
  r.batch_stride = lead.size() == 2 ? pos->stride(1) : 0;
  r.inv_freq = static_cast<const double*>(freq->const_data_ptr());
  r.axes = static_cast<const int*>(axes->const_data_ptr());
  r.n_axes = (int)pos->size(0);
  r.rot = (int)(2 * n);
  r.interleaved = interleaved;
  return true;
}

// k_cache, v_cache, block_table, seq_lens.
struct Cache {
  Where w;
  at::ScalarType type;
  fa_paged_kv kv;
  fa_page_table table;
  const int* lens;
  int64_t B;
  const at::Tensor* k;
};
bool page_table(PyObject* o, const Where& w, fa_page_table& p, int64_t& B) {
  const at::Tensor* t = tensor(o);
  if (!t || t->dim() != 2 || t->scalar_type() != at::kInt || !t->is_cuda() || t->device() != w.device || t->stride(1) != 1 ||
      !fits(t->size(0)) || !fits(t->size(1)))
    return false;
  p.pages = static_cast<const int*>(t->const_data_ptr());
  p.stride = t->stride(0);
  p.max_pages = (int)t->size(1);
  B = t->size(0);
  return true;
}
bool cache(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo, Cache& c) {
  const at::Tensor *k = tensor(ko), *v = tensor(vo), *lens = tensor(lo);
  if (!k || !v || !lens || k->dim() != 4 || !where(*k, c.w)) return false;
  c.type = k->scalar_type();
  c.k = k;
  const int code = dtype_code(c.type);
  if (code < 0 || !rows_of(*k, c.w, c.type, k->sizes()) || !rows_of(*v, c.w, c.type, k->sizes()) ||
      v->strides() != k->strides() || !page_table(to, c.w, c.table, c.B) || !dense(*lens, c.w, at::kInt, c.B))
    return false;
  for (int i = 0; i < 4; ++i)
    if (!fits(k->size(i))) return false;
  c.kv = fa_paged_kv{k->mutable_data_ptr(), v->mutable_data_ptr(), k->stride(0),      k->stride(1),      k->stride(2),
                     (int)k->size(0),       (int)k->size(2),       (int)k->size(1), (int)k->size(3), code};
  c.lens = static_cast<const int*>(lens->const_data_ptr());
  return true;
}
bool scores_of(PyObject* o, const Cache& c, float*& p) {
  const at::Tensor* t;
  p = nullptr;
  if (!maybe(o, t)) return false;
  if (!t) return true;
  if (!dense(*t, c.w, at::kFloat, c.k->sizes().slice(0, 3))) return false;
  p = static_cast<float*>(t->mutable_data_ptr());
  return true;
}

// An output that is given, or a new one.
bool output(PyObject* o, const Where& w, at::ScalarType type, Shape shape, bool whole, at::Tensor& t) {
  const at::Tensor* x;
  if (!maybe(o, x)) return false;
  if (!x) {
    t = empty(shape, type);
    return true;
  }
  if (!(whole ? dense(*x, w, type, shape) : rows_of(*x, w, type, shape))) return false;
  t = *x;
  return true;
}

// q, k, positions, inv_freq, axes, interleaved, inverse, q_out, k_out
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor *q, *k;
  Where w;
  int inverse;
  if (n != 9 || !(q = tensor(a[0])) || !maybe(a[1], k) || q->dim() != 4 || !where(*q, w) || !boolean(a[6], inverse) ||
      (!k && a[8] != Py_None))
    Py_RETURN_NONE;
  const at::ScalarType type = q->scalar_type();
  const int code = dtype_code(type);
  const int64_t B = q->size(0), N = q->size(2), d = q->size(3);
  if (code < 0 || !rows_of(*q, w, type, q->sizes()) || !fits(B) || !fits(q->size(1)) || !fits(N) || !fits(d))
    Py_RETURN_NONE;
  if (k && (k->dim() != 4 || !rows_of(*k, w, type, {B, k->size(1), N, d}) || !fits(k->size(1)))) Py_RETURN_NONE;
  const int64_t lead[2] = {B, N};
  fa_rotary r;
  if (!rotary(a + 2, a[5], w, d, Shape(lead, 2), r)) Py_RETURN_NONE;
  at::Tensor qo, ko;
  if (!output(a[7], w, type, q->sizes(), false, qo) || (k && !output(a[8], w, type, k->sizes(), false, ko))) Py_RETURN_NONE;
  fa_status s;
  const void* qp = q->const_data_ptr();
  void* qop = qo.mutable_data_ptr();
  const void* kp = k ? k->const_data_ptr() : nullptr;
  void* kop = k ? ko.mutable_data_ptr() : nullptr;
  Py_BEGIN_ALLOW_THREADS;
  s = p_rope(qp, strides(*q), qop, strides(qo), kp, k ? strides(*k) : nullptr, kop, k ? strides(ko) : nullptr, (int)B,
             (int)q->size(1), k ? (int)k->size(1) : 0, (int)N, (int)d, code, &r, inverse, w.stream);
  Py_END_ALLOW_THREADS;
  return k ? result(s, qo, ko) : result(s, qo);
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, block_table, seq_lens, k, v, cu_seqlens, q, positions,
// inv_freq, axes, interleaved, scores, q_out
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  const at::Tensor *k, *v, *cu, *q;
  float* scores;
  if (n != 14 || !cache(a[0], a[1], a[2], a[3], c) || !(k = tensor(a[4])) || !(v = tensor(a[5])) || !maybe(a[6], cu) ||
      !maybe(a[7], q) || !scores_of(a[12], c, scores) || k->dim() != 3)
    Py_RETURN_NONE;
  const int64_t T = k->size(0), Hkv = c.kv.Hkv, d = c.kv.d;
  if (T == 0 || !fits(T) || !rows_of(*k, c.w, c.type, {T, Hkv, d}) || !rows_of(*v, c.w, c.type, {T, Hkv, d}) ||
      (cu ? !dense(*cu, c.w, at::kInt, c.B + 1) : T != c.B))
    Py_RETURN_NONE;
  fa_rotary r;
  const bool turn = a[8] != Py_None || a[9] != Py_None || a[10] != Py_None;
  if (turn && !rotary(a + 8, a[11], c.w, d, T, r)) Py_RETURN_NONE;
  at::Tensor qo;
  int64_t Hq = 0;
  if (q) {
    if (q->dim() != 3 || !fits(Hq = q->size(1)) || !rows_of(*q, c.w, c.type, {T, Hq, d}) ||
        !output(a[13], c.w, c.type, {T, Hq, d}, false, qo))
      Py_RETURN_NONE;
  } else if (a[13] != Py_None) {
    Py_RETURN_NONE;
  }
  fa_status s;
  const void *kp = k->const_data_ptr(), *vp = v->const_data_ptr(), *qp = q ? q->const_data_ptr() : nullptr;
  void* qop = q ? qo.mutable_data_ptr() : nullptr;
  const int* cup = cu ? static_cast<const int*>(cu->const_data_ptr()) : nullptr;
  Py_BEGIN_ALLOW_THREADS;
  s = p_append(&c.kv, &c.table, c.lens, cup, (int)c.B, (int)T, kp, strides(*k), vp, strides(*v), qp, q ? strides(*q) : nullptr,
               qop, q ? strides(qo) : nullptr, (int)Hq, turn ? &r : nullptr, scores, c.w.stream);
  Py_END_ALLOW_THREADS;
  if (s != FA_OK) return PyLong_FromLong(s);
  // None would mean that the call was not taken: without q the answer is False.
  if (!q) Py_RETURN_FALSE;
  return THPVariable_Wrap(qo);
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, block_table, seq_lens, scale, window, scores, out, lse, workspace
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  const at::Tensor *q, *ws;
  float* scores;
  int window;
  if (n != 11 || !cache(a[1], a[2], a[3], a[4], c) || !(q = tensor(a[0])) || !integer(a[6], window) ||
      !scores_of(a[7], c, scores) || !maybe(a[10], ws) || q->dim() != 3)
    Py_RETURN_NONE;
  const int64_t B = c.B, Hq = q->size(1), d = c.kv.d;
  if (!fits(Hq) || !rows_of(*q, c.w, c.type, {B, Hq, d})) Py_RETURN_NONE;
  float scale;
  if (a[5] == Py_None) scale = (float)(1.0 / std::sqrt((double)d));
  else if (PyFloat_CheckExact(a[5])) scale = (float)PyFloat_AS_DOUBLE(a[5]);
  else Py_RETURN_NONE;
  at::Tensor o, lse;
  c10::DataPtr own;
  if (ws && (ws->dim() != 1 || !dense(*ws, c.w, at::kByte, ws->sizes()))) Py_RETURN_NONE;
  size_t bytes = ws ? (size_t)ws->numel() : 0;
  if (!ws) {
    bytes = p_decode_ws((int)B, (int)Hq, c.kv.Hkv, c.kv.d, c.kv.page_size, c.table.max_pages, scores != nullptr);
    if (bytes == 0) Py_RETURN_NONE;
    own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
  }
  if (!output(a[8], c.w, c.type, {B, Hq, d}, true, o) || !output(a[9], c.w, at::kFloat, {B, Hq}, true, lse)) Py_RETURN_NONE;
  fa_status s;
  const void* qp = q->const_data_ptr();
  void *op = o.mutable_data_ptr(), *lp = lse.mutable_data_ptr(), *wp = ws ? ws->mutable_data_ptr() : own.mutable_get();
  Py_BEGIN_ALLOW_THREADS;
  s = p_decode(qp, strides(*q), &c.kv, &c.table, c.lens, op, static_cast<float*>(lp), scores, (int)B, (int)Hq, window, scale,
               wp, bytes, c.w.stream);
  Py_END_ALLOW_THREADS;
  return result(s, o, lse);
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, scores, block_table, seq_lens, dst_table, budget, recent, sinks, new_lens, kept
PyObject* py_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  float* scores;
  fa_page_table dst;
  int64_t rows;
  int budget, recent, sinks;
  if (n != 11 || !cache(a[0], a[1], a[3], a[4], c) || !scores_of(a[2], c, scores) || !scores ||
      !page_table(a[5], c.w, dst, rows) || rows != c.B || !integer(a[6], budget) || !integer(a[7], recent) ||
      !integer(a[8], sinks) || budget < 1)
    Py_RETURN_NONE;
  at::Tensor lens, kept;
  if (!output(a[9], c.w, at::kInt, c.B, true, lens) || !output(a[10], c.w, at::kInt, {c.B, c.kv.Hkv, budget}, true, kept))
    Py_RETURN_NONE;
  fa_status s;
  void *lp = lens.mutable_data_ptr(), *kp = kept.mutable_data_ptr();
  Py_BEGIN_ALLOW_THREADS;
  s = p_evict(&c.kv, scores, &c.table, c.lens, &dst, static_cast<int*>(lp), static_cast<int*>(kp), (int)c.B, budget, recent,
              sinks, c.w.stream);
  Py_END_ALLOW_THREADS;
  return result(s, lens, kept);
  END_HANDLE_TH_ERRORS
}

// The addresses of fa_rope, fa_paged_append, fa_paged_decode,
// fa_paged_decode_workspace_bytes and fa_paged_evict in the loaded library.
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[5];
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind takes 5 addresses");
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "null address");
  }
  p_rope = reinterpret_cast<decltype(p_rope)>(p[0]);
  p_append = reinterpret_cast<decltype(p_append)>(p[1]);
  p_decode = reinterpret_cast<decltype(p_decode)>(p[2]);
  p_decode_ws = reinterpret_cast<decltype(p_decode_ws)>(p[3]);
  p_evict = reinterpret_cast<decltype(p_evict)>(p[4]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fastcall(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}
PyMethodDef methods[] = {{"bind", fastcall(py_bind), METH_FASTCALL, nullptr},
                         {"rope", fastcall(py_rope), METH_FASTCALL, nullptr},
                         {"paged_append", fastcall(py_append), METH_FASTCALL, nullptr},
                         {"paged_decode", fastcall(py_decode), METH_FASTCALL, nullptr},
                         {"paged_evict", fastcall(py_evict), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "fa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// FA_TORCH_KEY names the torch, Python and fa.h that this was compiled against;
// nothing here may be called with others (see native_key in _build.py).
PyMODINIT_FUNC PyInit_fa_torch() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "key", FA_TORCH_KEY) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
