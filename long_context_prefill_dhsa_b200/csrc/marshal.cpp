// Argument checks of the cache's calls (include/dhsa.h, 6 to 8) for the Python
// binding, which is called once per new token and layer: in Python the checks
// of ten tensors take 5 to 8 us, more than the launch.
//
// Each function takes what its namesake in binding.py takes and makes the call
// if everything is as it should be. It returns the call's result, or its
// status (an int) if the library refused, or None if an argument is not one
// that it takes as it is: binding.py then finds out what is wrong and says so,
// or mends it (another current device, a number that is not an int).
// Nothing is kept from one call to the next.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "dhsa.h"

namespace {

decltype(&dhsa_rotary_qkv) rotary_qkv = nullptr;
decltype(&dhsa_tree_attn) tree_attn = nullptr;
decltype(&dhsa_tree_attn_workspace_size) tree_ws = nullptr;
decltype(&dhsa_cache_evict) cache_evict = nullptr;
decltype(&dhsa_cache_evict_workspace_size) evict_ws = nullptr;

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// four dimensions that fit an int, bf16, on a GPU
bool is_rows(const at::Tensor* t) {
  if (!t || !t->is_cuda() || t->scalar_type() != at::kBFloat16 || t->dim() != 4) return false;
  for (int64_t n : t->sizes())
    if (n > INT_MAX) return false;
  return true;
}

// a dense tensor of the call, or None
bool dense(PyObject* o, at::ScalarType type, at::IntArrayRef shape, int device, void** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->scalar_type() != type || t->get_device() != device || t->sizes() != shape ||
      !t->is_contiguous())
    return false;
  *p = t->data_ptr();
  return true;
}

// [B, H, rows, d] with contiguous rows and any strides, or None
struct Rows {
  void* p = nullptr;
  int64_t strides[3];
  const int64_t* s = nullptr;      // null when dense
  bool read(PyObject* o, at::IntArrayRef shape, int device) {
    if (o == Py_None) return true;
    const at::Tensor* t = tensor(o);
    if (!is_rows(t) || t->get_device() != device || t->sizes() != shape) return false;
    if (!t->is_contiguous()) {
      if (t->stride(3) != 1) return false;
      for (int i = 0; i < 3; ++i) strides[i] = t->stride(i);
      s = strides;
    }
    p = t->data_ptr();
    return true;
  }
};

bool integer(PyObject* o, int* x) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (over || v < INT_MIN || v > INT_MAX) return false;
  *x = (int)v;
  return true;
}

// the call's workspace: the caller's, or a new one (in `own`)
bool workspace(PyObject* o, size_t size, int device, const at::Tensor& like, at::Tensor* own, void** p, size_t* bytes) {
  if (o == Py_None) {
    *own = at::empty({(int64_t)size}, like.options().dtype(at::kByte));
    *p = own->data_ptr();
    *bytes = size;
    return true;
  }
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->get_device() != device || !t->is_contiguous()) return false;
  *p = t->data_ptr();
  *bytes = t->nbytes();
  return true;
}

// None without a current error: the Python side takes over
PyObject* leave() {
  PyErr_Clear();
  Py_RETURN_NONE;
}
PyObject* given(PyObject* o, const at::Tensor& made) { return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(o); }

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    return leave();
  }
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[5];
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind: five addresses");
  for (int i = 0; i < 5; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(a[i]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "bind: null");
  rotary_qkv = reinterpret_cast<decltype(rotary_qkv)>(p[0]);
  tree_attn = reinterpret_cast<decltype(tree_attn)>(p[1]);
  tree_ws = reinterpret_cast<decltype(tree_ws)>(p[2]);
  cache_evict = reinterpret_cast<decltype(cache_evict)>(p[3]);
  evict_ws = reinterpret_cast<decltype(evict_ws)>(p[4]);
  Py_RETURN_NONE;
}

// Q K inv_freq V positions start n_new slots interleaved transpose factor Q_out K_out V_out pos_out
PyObject* py_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 15 || !rotary_qkv) return leave();
  return guarded([&]() -> PyObject* {
    PyObject *Q = a[0], *K = a[1], *V = a[3];
    const at::Tensor* ref = tensor(Q != Py_None ? Q : K != Py_None ? K : V);
    if (!is_rows(ref)) return leave();
    const int device = ref->get_device();
    if (device != c10::cuda::current_device()) return leave();
    const int64_t B = ref->size(0), T = ref->size(2), d = ref->size(3);
    const at::Tensor* kv = tensor(K != Py_None ? K : V);
    if (!kv && (K != Py_None || V != Py_None)) return leave();
    if (kv && kv->dim() != 4) return leave();
    const int64_t Hq = Q != Py_None ? ref->size(1) : 1, Hkv = kv ? kv->size(1) : 1;
    PyObject *Qo = a[11], *Ko = a[12], *Vo = a[13];
    if ((Q == Py_None && Qo != Py_None) || (K == Py_None && Ko != Py_None) || (V == Py_None && Vo != Py_None))
      return leave();
    if (a[4] != Py_None && a[5] != Py_None) return leave();
    int64_t cap = T;
    if (Ko != Py_None || Vo != Py_None) {
      const at::Tensor* o = tensor(Ko != Py_None ? Ko : Vo);
      if (!is_rows(o)) return leave();
      cap = o->size(2);
    }
    Rows q, k, v, ko, vo;
    if (!q.read(Q, {B, Hq, T, d}, device) || !k.read(K, {B, Hkv, T, d}, device) || !v.read(V, {B, Hkv, T, d}, device))
      return leave();
    at::Tensor mq, mk, mv;
    void *qo, *f, *positions, *start, *n_new, *slots, *pos_out;
    const at::Tensor* freq = tensor(a[2]);
    if (!freq || freq->numel() > INT_MAX / 2 || !dense(a[2], at::kDouble, {freq->numel()}, device, &f) ||
        !dense(Qo, at::kBFloat16, {B, Hq, T, d}, device, &qo) || !ko.read(Ko, {B, Hkv, cap, d}, device) ||
        !vo.read(Vo, {B, Hkv, cap, d}, device) || !dense(a[4], at::kInt, {B, T}, device, &positions) ||
        !dense(a[5], at::kInt, {B}, device, &start) || !dense(a[6], at::kInt, {B}, device, &n_new) ||
        !dense(a[7], at::kInt, {B}, device, &slots) || !dense(a[14], at::kInt, {B, Hkv, cap}, device, &pos_out))
      return leave();
    if (Q != Py_None && Qo == Py_None) qo = (mq = at::empty({B, Hq, T, d}, ref->options())).data_ptr();
    if (K != Py_None && Ko == Py_None) ko.p = (mk = at::empty({B, Hkv, cap, d}, ref->options())).data_ptr();
    if (V != Py_None && Vo == Py_None) vo.p = (mv = at::empty({B, Hkv, cap, d}, ref->options())).data_ptr();
    const int interleaved = PyObject_IsTrue(a[8]), transpose = PyObject_IsTrue(a[9]);
    const double factor = PyFloat_AsDouble(a[10]);
    if (interleaved < 0 || transpose < 0 || PyErr_Occurred()) return leave();
    void* stream = c10::cuda::getCurrentCUDAStream(device).stream();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = rotary_qkv(q.p, q.s, k.p, k.s, v.p, v.s, (int)B, (int)Hq, (int)Hkv, (int)T, (int)d,
                    static_cast<const double*>(f), 2 * (int)freq->numel(), interleaved, transpose, (float)factor,
                    static_cast<const int32_t*>(positions), static_cast<const int32_t*>(start),
                    static_cast<const int32_t*>(n_new), qo, ko.p, ko.s, vo.p, vo.s, static_cast<const int32_t*>(slots),
                    (int)cap, static_cast<int32_t*>(pos_out), stream);
    Py_END_ALLOW_THREADS;
    if (st) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, given(Qo, mq));
    PyTuple_SET_ITEM(r, 1, given(Ko, mk));
    PyTuple_SET_ITEM(r, 2, given(Vo, mv));
    return r;
  });
}

// Q K V lengths parents n_draft softmax_scale weight weight_out out lse workspace
PyObject* py_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12 || !tree_attn) return leave();
  return guarded([&]() -> PyObject* {
    const at::Tensor *Q = tensor(a[0]), *K = tensor(a[1]);
    if (!is_rows(Q) || !is_rows(K)) return leave();
    const int device = Q->get_device();
    if (device != c10::cuda::current_device()) return leave();
    const int64_t B = Q->size(0), Hq = Q->size(1), T = Q->size(2), d = Q->size(3), Hkv = K->size(1), cap = K->size(2);
    PyObject *w = a[7], *wo = a[8] != Py_None ? a[8] : a[7];
    if (w == Py_None && wo != Py_None) return leave();
    Rows k, v;
    void *q, *lengths, *parents, *n_draft, *weight, *weight_out, *out, *lse, *ws;
    size_t bytes;
    if (!dense(a[0], at::kBFloat16, {B, Hq, T, d}, device, &q) || !k.read(a[1], {B, Hkv, cap, d}, device) ||
        a[2] == Py_None || !v.read(a[2], {B, Hkv, cap, d}, device) || a[3] == Py_None ||
        !dense(a[3], at::kInt, {B}, device, &lengths) || !dense(a[4], at::kInt, {B, T}, device, &parents) ||
        !dense(a[5], at::kInt, {B}, device, &n_draft) || !dense(w, at::kFloat, {B, Hkv, cap}, device, &weight) ||
        !dense(wo, at::kFloat, {B, Hkv, cap}, device, &weight_out) ||
        !dense(a[9], at::kBFloat16, {B, Hq, T, d}, device, &out) || !dense(a[10], at::kFloat, {B, Hq, T}, device, &lse))
      return leave();
    const double scale = a[6] == Py_None ? 1.0 / std::sqrt((double)d) : PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) return leave();
    at::Tensor own, made;
    const size_t need = tree_ws((int)B, (int)Hq, (int)Hkv, (int)T, (int)cap, weight != nullptr);
    if (!workspace(a[11], need, device, *Q, &own, &ws, &bytes)) return leave();
    if (a[9] == Py_None) out = (made = at::empty({B, Hq, T, d}, Q->options())).data_ptr();
    void* stream = c10::cuda::getCurrentCUDAStream(device).stream();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = tree_attn(q, k.p, k.s, v.p, v.s, (int)B, (int)Hq, (int)Hkv, (int)T, (int)cap, (int)d,
                   static_cast<const int32_t*>(lengths), static_cast<const int32_t*>(parents),
                   static_cast<const int32_t*>(n_draft), (float)scale, out, static_cast<float*>(lse),
                   static_cast<const float*>(weight), static_cast<float*>(weight_out), ws, bytes, stream);
    Py_END_ALLOW_THREADS;
    return st ? PyLong_FromLong(st) : given(a[9], made);
  });
}

// K V weight pos lengths keep next_pos n_draft accept sinks recent weight_out pos_out lengths_out index workspace
PyObject* py_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 16 || !cache_evict) return leave();
  return guarded([&]() -> PyObject* {
    const at::Tensor* K = tensor(a[0]);
    if (!is_rows(K)) return leave();
    const int device = K->get_device();
    if (device != c10::cuda::current_device()) return leave();
    const int64_t B = K->size(0), Hkv = K->size(1), cap = K->size(2), d = K->size(3);
    int keep, sinks, recent;
    if (!integer(a[5], &keep) || !integer(a[9], &sinks) || !integer(a[10], &recent)) return leave();
    for (int i : {1, 2, 3, 4})
      if (a[i] == Py_None) return leave();
    Rows k, v;
    void *weight, *pos, *lengths, *next, *n_draft, *accept, *weight_out, *pos_out, *lengths_out, *index, *ws;
    size_t bytes;
    if (!k.read(a[0], {B, Hkv, cap, d}, device) || !v.read(a[1], {B, Hkv, cap, d}, device) ||
        !dense(a[2], at::kFloat, {B, Hkv, cap}, device, &weight) || !dense(a[3], at::kInt, {B, Hkv, cap}, device, &pos) ||
        !dense(a[4], at::kInt, {B}, device, &lengths) || !dense(a[6], at::kInt, {B}, device, &next) ||
        !dense(a[7], at::kInt, {B}, device, &n_draft) || !dense(a[8], at::kLong, {B}, device, &accept) ||
        !dense(a[11], at::kFloat, {B, Hkv, cap}, device, &weight_out) ||
        !dense(a[12], at::kInt, {B, Hkv, cap}, device, &pos_out) ||
        !dense(a[13], at::kInt, {B}, device, &lengths_out) ||
        !dense(a[14], at::kInt, {B, Hkv, keep < cap ? keep : cap}, device, &index))
      return leave();
    if (!weight_out) weight_out = weight;
    if (!pos_out) pos_out = pos;
    at::Tensor own, made;
    if (!workspace(a[15], evict_ws((int)B, (int)Hkv, (int)cap), device, *K, &own, &ws, &bytes)) return leave();
    if (!lengths_out) lengths_out = (made = at::empty({B}, K->options().dtype(at::kInt))).data_ptr();
    void* stream = c10::cuda::getCurrentCUDAStream(device).stream();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = cache_evict(k.p, k.s, v.p, v.s, static_cast<const float*>(weight), static_cast<const int32_t*>(pos), (int)B,
                     (int)Hkv, (int)cap, (int)d, static_cast<const int32_t*>(lengths),
                     static_cast<const int32_t*>(n_draft), static_cast<const int64_t*>(accept), keep, sinks, recent,
                     static_cast<const int32_t*>(next), static_cast<float*>(weight_out),
                     static_cast<int32_t*>(pos_out), static_cast<int32_t*>(lengths_out), static_cast<int32_t*>(index), ws,
                     bytes, stream);
    Py_END_ALLOW_THREADS;
    return st ? PyLong_FromLong(st) : given(a[13], made);
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FAST(bind)},
                         {"rotary_qkv", FAST(py_rotary)},
                         {"tree_attn", FAST(py_tree)},
                         {"cache_evict", FAST(py_evict)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
