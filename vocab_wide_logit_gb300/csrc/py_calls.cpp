// py_calls.cpp -- the serving head's calls on torch tensors without the interpreter.
//
// At decoding sizes a call is issued slower than it runs: through ctypes and
// torch's Python bindings one row of 1025 logits took 15 us to issue for 9 us on the
// device, most of it attribute lookups on tensors and argument conversion; this way
// it takes 5 us (a head of one token: 17 and 7 us). These functions check the usual
// arguments (dense rows, contiguous vectors, one current device, outputs to be made
// here), allocate the outputs and call the C entry point. They return None for
// anything else, which the Python wrapper then checks, reports or runs itself, and
// the status of a call that failed. They hold no state but the addresses of the
// entry points.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "dsample.h"

namespace {

decltype(&ds_sample_filtered) p_sample = nullptr;
decltype(&ds_quantize_rows) p_quantize = nullptr;
decltype(&ds_linear_i8_workspace) p_linear_ws = nullptr;
decltype(&ds_linear_i8) p_linear = nullptr;
decltype(&ds_head_i8_workspace) p_head_ws = nullptr;
decltype(&ds_head_i8) p_head = nullptr;

const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// A device matrix with dense rows, at least one.
struct Rows {
  const void* p;
  int64_t n, k, ld;
  int device;
};
bool rows(const at::Tensor* t, Rows* r) {
  if (!t || !t->is_cuda() || t->dim() != 2) return false;
  r->p = t->const_data_ptr();
  r->n = t->size(0);
  r->k = t->size(1);
  r->ld = r->n == 1 ? r->k : t->stride(0);
  r->device = t->get_device();
  return r->n > 0 && r->n <= INT32_MAX && r->k > 0 && r->k <= INT32_MAX && (r->k == 1 || t->stride(1) == 1) &&
         r->ld >= r->k && r->device == c10::cuda::current_device();
}

// A contiguous vector [n] on the device, or None where that is allowed.
bool vec(PyObject* o, int64_t n, at::ScalarType type, int device, bool optional, void** p) {
  *p = nullptr;
  if (o == Py_None) return optional;
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->dim() != 1 || t->size(0) != n || t->scalar_type() != type || t->get_device() != device ||
      !t->is_contiguous())
    return false;
  *p = t->data_ptr();
  return true;
}

bool code(at::ScalarType t, int32_t* c) {
  *c = t == at::kFloat ? DS_DTYPE_F32 : DS_DTYPE_BF16;
  return t == at::kFloat || t == at::kBFloat16;
}

at::TensorOptions on(int device, at::ScalarType t) {
  return at::TensorOptions().dtype(t).device(at::kCUDA, (c10::DeviceIndex)device);
}

void* stream(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

PyObject* both(at::Tensor first, at::Tensor second) {
  PyObject* a = THPVariable_Wrap(std::move(first));
  PyObject* b = a ? THPVariable_Wrap(std::move(second)) : nullptr;
  PyObject* r = b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

// sample(logits, temperature, u, top_k, top_p, min_p) -> (tokens, logprobs)
PyObject* sample(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Rows x;
  int32_t c;
  void *tau, *u, *k, *p, *mp;
  const at::Tensor* t = count == 6 && p_sample ? tensor(v[0]) : nullptr;
  if (!rows(t, &x) || !code(t->scalar_type(), &c) || !vec(v[1], x.n, at::kFloat, x.device, false, &tau) ||
      !vec(v[2], x.n, at::kFloat, x.device, false, &u) || !vec(v[3], x.n, at::kInt, x.device, true, &k) ||
      !vec(v[4], x.n, at::kFloat, x.device, true, &p) || !vec(v[5], x.n, at::kFloat, x.device, true, &mp))
    Py_RETURN_NONE;
  at::Tensor tok = at::empty({x.n}, on(x.device, at::kInt)), lp = at::empty({x.n}, on(x.device, at::kFloat));
  const ds_status rc = p_sample(x.p, c, (int32_t)x.n, (int32_t)x.k, x.ld, (const float*)tau, (const int32_t*)k,
                                (const float*)p, (const float*)mp, (const float*)u, (int32_t*)tok.data_ptr(),
                                (float*)lp.data_ptr(), nullptr, stream(x.device));
  return rc != DS_OK ? PyLong_FromLong(rc) : both(std::move(tok), std::move(lp));
  END_HANDLE_TH_ERRORS
}

// quantize(x, gain, eps) -> (q, scale)
PyObject* quantize(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Rows x;
  int32_t c;
  void* gain;
  const at::Tensor* t = count == 3 && p_quantize ? tensor(v[0]) : nullptr;
  if (!rows(t, &x) || !code(t->scalar_type(), &c) || !vec(v[1], x.k, at::kFloat, x.device, true, &gain)) Py_RETURN_NONE;
  const double eps = PyFloat_AsDouble(v[2]);
  if (PyErr_Occurred()) return nullptr;
  at::Tensor q = at::empty({x.n, x.k}, on(x.device, at::kChar)), scale = at::empty({x.n}, on(x.device, at::kFloat));
  const ds_status rc = p_quantize(x.p, c, (int32_t)x.n, (int32_t)x.k, x.ld, (const float*)gain, (float)eps,
                                  (int8_t*)q.data_ptr(), (float*)scale.data_ptr(), stream(x.device));
  return rc != DS_OK ? PyLong_FromLong(rc) : both(std::move(q), std::move(scale));
  END_HANDLE_TH_ERRORS
}

// The packed weight of a product: [N][K] bytes laid out by ds_pack_i8, its scales, the type code of the result.
struct Weight {
  const void* packed;
  const float* scale;
  int64_t N, K;
  int32_t out;
};
bool weight(PyObject* const* v, int device, Weight* w) {
  const at::Tensor *p = tensor(v[0]), *s = tensor(v[1]);
  w->N = PyLong_AsLong(v[2]);
  w->K = PyLong_AsLong(v[3]);
  w->out = (int32_t)PyLong_AsLong(v[4]);
  if (PyErr_Occurred() || !p || !s || !p->is_cuda() || p->get_device() != device || s->get_device() != device) {
    PyErr_Clear();
    return false;
  }
  w->packed = p->const_data_ptr();
  w->scale = (const float*)s->const_data_ptr();
  return true;
}
at::Tensor result(const Weight& w, int64_t n, int device) {
  return at::empty({n, w.N}, on(device, w.out == DS_DTYPE_F32 ? at::kFloat : at::kBFloat16));
}

// linear(a, a_scale, packed, w_scale, N, K, out code) -> out
PyObject* linear(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Rows a;
  Weight w;
  void* sa;
  const at::Tensor* t = count == 7 && p_linear ? tensor(v[0]) : nullptr;
  if (!rows(t, &a) || t->scalar_type() != at::kChar || !vec(v[1], a.n, at::kFloat, a.device, false, &sa) ||
      !weight(v + 2, a.device, &w) || a.k != w.K)
    Py_RETURN_NONE;
  at::Tensor out = result(w, a.n, a.device);
  const int64_t need = p_linear_ws((int32_t)a.n, (int32_t)w.N, (int32_t)w.K);
  at::Tensor ws = at::empty({need}, on(a.device, at::kByte));
  const ds_status rc =
      p_linear((const int8_t*)a.p, a.ld, (const float*)sa, w.packed, w.scale, (int32_t)a.n, (int32_t)w.N, (int32_t)w.K,
               out.data_ptr(), w.out, w.N, ws.data_ptr(), need, nullptr, stream(a.device));
  return rc != DS_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// head(hidden, gain, packed, w_scale, N, K, out code, eps) -> logits
PyObject* head(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Rows x;
  Weight w;
  int32_t c;
  void* gain;
  const at::Tensor* t = count == 8 && p_head ? tensor(v[0]) : nullptr;
  if (!rows(t, &x) || !code(t->scalar_type(), &c) || !vec(v[1], x.k, at::kFloat, x.device, true, &gain) ||
      !weight(v + 2, x.device, &w) || x.k != w.K)
    Py_RETURN_NONE;
  const double eps = PyFloat_AsDouble(v[7]);
  if (PyErr_Occurred()) return nullptr;
  at::Tensor out = result(w, x.n, x.device);
  const int64_t need = p_head_ws((int32_t)x.n, (int32_t)w.N, (int32_t)w.K);
  at::Tensor ws = at::empty({need}, on(x.device, at::kByte));
  const ds_status rc =
      p_head(x.p, c, (int32_t)x.n, (int32_t)x.k, x.ld, (const float*)gain, (float)eps, w.packed, w.scale, (int32_t)w.N,
             out.data_ptr(), w.out, w.N, ws.data_ptr(), need, nullptr, stream(x.device));
  return rc != DS_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the entry points)
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t count) {
  void* p[6];
  if (count != 6) {
    PyErr_SetString(PyExc_TypeError, "bind() takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(v[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_sample = reinterpret_cast<decltype(p_sample)>(p[0]);
  p_linear_ws = reinterpret_cast<decltype(p_linear_ws)>(p[1]);
  p_linear = reinterpret_cast<decltype(p_linear)>(p[2]);
  p_head_ws = reinterpret_cast<decltype(p_head_ws)>(p[3]);
  p_head = reinterpret_cast<decltype(p_head)>(p[4]);
  p_quantize = reinterpret_cast<decltype(p_quantize)>(p[5]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sample)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"head", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(head)), METH_FASTCALL, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize)), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ds_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ds_calls(void) { return PyModule_Create(&module); }
