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
decltype(&ds_score_tokens) p_score = nullptr;
decltype(&ds_score_tokens_grad) p_score_grad = nullptr;
decltype(&ds_add_adapters_workspace) p_adapters_ws = nullptr;
decltype(&ds_add_adapters) p_adapters = nullptr;

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

// A contiguous tensor [n] or [n][columns] within the memory of another of the same type: a quarter of what an allocation
// takes.
at::Tensor within(const at::Tensor& memory, int64_t first, at::ScalarType type, int64_t n, int64_t columns = -1) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(memory.storage()), memory.key_set(),
                                                   c10::scalarTypeToTypeMeta(type));
  impl->set_storage_offset(first);
  const int64_t sizes[2] = {n, columns};
  impl->set_sizes_contiguous(c10::IntArrayRef(sizes, columns < 0 ? 1 : 2));
  return at::Tensor(std::move(impl));
}

// score(logits, tokens, top) -> (logprobs, lse, entropy, ranks, top ids, top logprobs). Results of a type share their
// memory, the alternatives only where they are few: a program that keeps the log-probabilities alone keeps what is with them.
PyObject* score(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Rows x;
  int32_t c;
  void* tokens;
  const at::Tensor* t = count == 3 && p_score ? tensor(v[0]) : nullptr;
  if (!rows(t, &x) || !code(t->scalar_type(), &c) || !vec(v[1], x.n, at::kInt, x.device, false, &tokens) ||
      !PyLong_CheckExact(v[2]))
    Py_RETURN_NONE;
  const long top = PyLong_AsLong(v[2]);
  if (top < 0 || top > x.k || top > DS_SCORE_MAX_TOP) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const at::TensorOptions f = on(x.device, at::kFloat), i = on(x.device, at::kInt);
  const int64_t more = x.n * top;
  const bool few = more <= 2048;
  const at::Tensor fs = at::empty({3 * x.n + (few ? more : 0)}, f), is = at::empty({x.n + (few ? more : 0)}, i);
  at::Tensor r[6] = {within(fs, 0, at::kFloat, x.n),
                     within(fs, x.n, at::kFloat, x.n),
                     within(fs, 2 * x.n, at::kFloat, x.n),
                     within(is, 0, at::kInt, x.n),
                     few ? within(is, x.n, at::kInt, x.n, top) : at::empty({x.n, top}, i),
                     few ? within(fs, 3 * x.n, at::kFloat, x.n, top) : at::empty({x.n, top}, f)};
  const ds_status rc = p_score(x.p, c, (int32_t)x.n, (int32_t)x.k, x.ld, (const int32_t*)tokens, (int32_t)top,
                               (float*)r[0].data_ptr(), (float*)r[1].data_ptr(), (float*)r[2].data_ptr(),
                               (int32_t*)r[3].data_ptr(), (int32_t*)r[4].data_ptr(), (float*)r[5].data_ptr(), nullptr,
                               stream(x.device));
  if (rc != DS_OK) return PyLong_FromLong(rc);
  PyObject* all = PyTuple_New(6);
  for (int j = 0; all && j < 6; ++j) {
    PyObject* o = THPVariable_Wrap(std::move(r[j]));
    if (!o) {
      Py_CLEAR(all);
      break;
    }
    PyTuple_SET_ITEM(all, j, o);
  }
  return all;
  END_HANDLE_TH_ERRORS
}

// score_grad(logits, tokens, lse, entropy, g_logprobs, g_entropy) -> gradient
PyObject* score_grad(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Rows x;
  int32_t c;
  void *tokens, *lse, *entropy, *gl, *gh;
  const at::Tensor* t = count == 6 && p_score_grad ? tensor(v[0]) : nullptr;
  if (!rows(t, &x) || !code(t->scalar_type(), &c) || !vec(v[1], x.n, at::kInt, x.device, false, &tokens) ||
      !vec(v[2], x.n, at::kFloat, x.device, false, &lse) || !vec(v[3], x.n, at::kFloat, x.device, true, &entropy) ||
      !vec(v[4], x.n, at::kFloat, x.device, true, &gl) || !vec(v[5], x.n, at::kFloat, x.device, true, &gh) ||
      (!gl && !gh) || (gh && !entropy))
    Py_RETURN_NONE;
  at::Tensor out = at::empty({x.n, x.k}, on(x.device, t->scalar_type()));
  const ds_status rc = p_score_grad(x.p, c, (int32_t)x.n, (int32_t)x.k, x.ld, (const int32_t*)tokens, (const float*)lse,
                                    (const float*)entropy, (const float*)gl, (const float*)gh, out.data_ptr(), x.k,
                                    nullptr, stream(x.device));
  return rc != DS_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// A stack of adapters' factors on the device.
bool stack(const at::Tensor& t, int device) {
  return t.is_cuda() && t.get_device() == device && t.dim() == 3 && t.scalar_type() == at::kBFloat16 && t.is_contiguous() &&
         t.numel() > 0;
}

// adapters(base, hidden, a, b, scale, ids, gain, eps) -> base with the adapters' part
PyObject* adapters(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Rows base, x;
  int32_t c, xc;
  void *ids, *gain, *scale;
  const bool all = count == 8 && p_adapters;
  const at::Tensor *t = all ? tensor(v[0]) : nullptr, *h = all ? tensor(v[1]) : nullptr, *a = all ? tensor(v[2]) : nullptr,
                   *b = all ? tensor(v[3]) : nullptr;
  if (!rows(t, &base) || !code(t->scalar_type(), &c) || !rows(h, &x) || !code(h->scalar_type(), &xc) || !a || !b ||
      !stack(*a, base.device) || !stack(*b, base.device) || a->size(0) != b->size(0) || a->size(1) != b->size(2) ||
      x.n != base.n || x.k != a->size(2) || base.k != b->size(1) || a->size(0) > DS_ADAPTERS_MAX ||
      a->size(1) > DS_ADAPTERS_MAX_RANK || !vec(v[4], a->size(0), at::kFloat, base.device, false, &scale) || !vec(v[5], base.n, at::kInt, base.device, false, &ids) ||
      !vec(v[6], x.k, at::kFloat, base.device, true, &gain))
    Py_RETURN_NONE;
  const double eps = PyFloat_AsDouble(v[7]);
  if (PyErr_Occurred()) return nullptr;
  const int32_t L = (int32_t)a->size(0), R = (int32_t)a->size(1);
  const int64_t need = p_adapters_ws((int32_t)base.n, L, R);
  const int64_t size = c == DS_DTYPE_F32 ? 4 : 2, bytes = base.n * base.k * size, at = (bytes + 127) / 128 * 128;
  at::Tensor out, ws;
  void* work;
  if (8 * need <= bytes) {  // a small workspace behind the result, in one allocation
    ws = at::empty({(at + need) / size}, on(base.device, t->scalar_type()));
    out = within(ws, 0, t->scalar_type(), base.n, base.k);
    work = static_cast<char*>(ws.data_ptr()) + at;
  } else {
    out = at::empty({base.n, base.k}, on(base.device, t->scalar_type()));
    ws = at::empty({need}, on(base.device, at::kByte));
    work = ws.data_ptr();
  }
  const ds_status rc =
      p_adapters(base.p, c, (int32_t)base.n, (int32_t)base.k, base.ld, x.p, xc, (int32_t)x.k, x.ld, (const float*)gain,
                 (float)eps, a->const_data_ptr(), b->const_data_ptr(), (const float*)scale, L, R,
                 (const int32_t*)ids, out.data_ptr(), base.k, work, need, nullptr, stream(base.device));
  return rc != DS_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the entry points)
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t count) {
  void* p[10];
  if (count != 10) {
    PyErr_SetString(PyExc_TypeError, "bind() takes ten addresses");
    return nullptr;
  }
  for (int i = 0; i < 10; ++i) {
    p[i] = PyLong_AsVoidPtr(v[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_sample = reinterpret_cast<decltype(p_sample)>(p[0]);
  p_linear_ws = reinterpret_cast<decltype(p_linear_ws)>(p[1]);
  p_linear = reinterpret_cast<decltype(p_linear)>(p[2]);
  p_head_ws = reinterpret_cast<decltype(p_head_ws)>(p[3]);
  p_head = reinterpret_cast<decltype(p_head)>(p[4]);
  p_quantize = reinterpret_cast<decltype(p_quantize)>(p[5]);
  p_score = reinterpret_cast<decltype(p_score)>(p[6]);
  p_score_grad = reinterpret_cast<decltype(p_score_grad)>(p[7]);
  p_adapters_ws = reinterpret_cast<decltype(p_adapters_ws)>(p[8]);
  p_adapters = reinterpret_cast<decltype(p_adapters)>(p[9]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sample)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"head", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(head)), METH_FASTCALL, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize)), METH_FASTCALL, nullptr},
    {"score", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(score)), METH_FASTCALL, nullptr},
    {"score_grad", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(score_grad)), METH_FASTCALL, nullptr},
    {"adapters", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adapters)), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ds_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ds_calls(void) { return PyModule_Create(&module); }
