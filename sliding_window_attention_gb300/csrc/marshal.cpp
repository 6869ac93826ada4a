// Argument marshalling of the calls that a generation step or a short training
// step makes most often, for the Python binding (_native.py).  Nothing is
// computed here: a call looks at its tensors, allocates the outputs and the
// workspace and calls the C ABI on the current stream.
//
// The same in Python (attribute reads, three torch.empty, some thirty ctypes
// arguments) takes 20 to 31 us on the GB300's host, two to six times what the
// GPU needs for a step's tensors.  A function here returns None whenever
// something is not as it expects (another type, shape, layout, device, a
// stream of its own): the Python path then runs the call or says what is wrong.
// An int is the library's error code.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/swa_attn.h"

namespace {

// The library's entry points, as the binding loaded it.
decltype(&swa_attn_fwd_workspace_bytes_shared) g_shared_ws;
decltype(&swa_attn_fwd_shared) g_shared;
decltype(&swa_attn_qk_rope_fwd) g_rope;
decltype(&swa_attn_qk_rope_bwd_workspace_bytes) g_rope_bwd_ws;
decltype(&swa_attn_qk_rope_bwd) g_rope_bwd;
PyObject* g_out_of_memory;  // torch.OutOfMemoryError

// Thrown (and turned into None) where the Python path has to take the call.
struct NotThisWay {};

const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw NotThisWay{};
  return &THPVariable_Unpack(o);
}
const at::Tensor* tensor_or_null(PyObject* o) { return o == Py_None ? nullptr : tensor(o); }
long long integer(PyObject* o) {
  if (!PyLong_Check(o)) throw NotThisWay{};
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotThisWay{};
  }
  return v;
}
int int32(PyObject* o) {
  const long long v = integer(o);
  if (v != (int)v) throw NotThisWay{};
  return (int)v;
}
float real(PyObject* o) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) throw NotThisWay{};
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotThisWay{};
  }
  return (float)v;
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw NotThisWay{};
  }
  return v;
}
int dim32(int64_t v) {
  if (v != (int)v) throw NotThisWay{};
  return (int)v;
}

// A dense tensor of this type and shape on device `dev`.
void expect(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape, int dev) {
  if (t && (t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous() || t->get_device() != dev))
    throw NotThisWay{};
}
int current(const at::Tensor* t) {
  if (!t->is_cuda() || t->get_device() != c10::cuda::current_device()) throw NotThisWay{};
  return (int)t->get_device();
}
// Elements between the tokens of a bf16 [B, L, H, D] tensor whose heads are dense.
long long token_stride(const at::Tensor* t, int64_t B, int64_t L, int64_t D, int dev) {
  if (t->scalar_type() != at::kBFloat16 || t->dim() != 4 || t->size(0) != B || t->size(1) != L || t->size(3) != D ||
      t->get_device() != dev)
    throw NotThisWay{};
  const int64_t H = t->size(2), sb = t->stride(0), sl = t->stride(1);
  const int64_t tok = L > 1 ? sl : (B > 1 ? sb : H * D);
  if (t->stride(3) != 1 || (H > 1 && t->stride(2) != D) || (B > 1 && L > 1 && sb != L * sl) || tok < H * D || tok % 8)
    throw NotThisWay{};
  return tok;
}

template <typename T>
T* ptr(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
at::Tensor empty(at::IntArrayRef shape, const at::Tensor* like, at::ScalarType type) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like->device(), std::nullopt));
}
// The call's scratch: freed on return, to be used again behind the call on its stream.
c10::DataPtr scratch(size_t bytes) { return c10::cuda::CUDACachingAllocator::get()->allocate(bytes); }
PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Other threads may run Python while this one allocates and launches: a full
// launch queue makes it wait, and what the queue waits for may need Python.
template <typename F>
int unlocked(F&& f) {
  struct NoGil {
    PyThreadState* state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
  } no_gil;
  return f();
}

// Runs f with n arguments; no C++ exception leaves.
template <typename F>
PyObject* call(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const NotThisWay&) {
    Py_RETURN_NONE;
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {  // torch: a tensor without storage
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (q, k_prefix or None, v_prefix or None, k_own, v_own, own_len, window, scale, prefix_len or None, sinks or None)
// -> (o, lse)
PyObject* forward_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&]() -> PyObject* {
    const at::Tensor *q = tensor(a[0]), *kp = tensor_or_null(a[1]), *vp = tensor_or_null(a[2]), *ko = tensor(a[3]),
                     *vo = tensor(a[4]), *len = tensor(a[5]), *sinks = tensor_or_null(a[9]);
    if (q->dim() != 4 || !kp != !vp || (kp && kp->dim() != 3) || ko->dim() != 4) throw NotThisWay{};
    const int B = dim32(q->size(0)), Hq = dim32(q->size(1)), Lq = dim32(q->size(2)), D = dim32(q->size(3));
    const int Hkv = dim32(ko->size(1)), rows = dim32(ko->size(2)), prefix_rows = kp ? dim32(kp->size(1)) : 0;
    const int window = int32(a[6]), P = a[8] == Py_None ? prefix_rows : int32(a[8]);
    const float scale = real(a[7]);
    const int dev = current(q);
    expect(q, at::kBFloat16, {B, Hq, Lq, D}, dev);
    expect(kp, at::kBFloat16, {Hkv, prefix_rows, D}, dev);
    expect(vp, at::kBFloat16, {Hkv, prefix_rows, D}, dev);
    expect(ko, at::kBFloat16, {B, Hkv, rows, D}, dev);
    expect(vo, at::kBFloat16, {B, Hkv, rows, D}, dev);
    expect(len, at::kInt, {B}, dev);
    expect(sinks, at::kFloat, {Hq}, dev);
    const size_t bytes = g_shared_ws(B, Hq, Hkv, Lq, P, rows, D, window);
    at::Tensor o, lse;
    const int rc = unlocked([&] {
      o = empty(q->sizes(), q, at::kBFloat16);
      lse = empty({B, Hq, Lq}, q, at::kFloat);
      const c10::DataPtr ws = scratch(bytes);
      return g_shared(ptr<swa_bf16>(q), ptr<swa_bf16>(kp), ptr<swa_bf16>(vp), ptr<swa_bf16>(ko), ptr<swa_bf16>(vo),
                      ptr<int32_t>(len), ptr<float>(sinks), ptr<swa_bf16>(&o), ptr<float>(&lse), B, Hq, Hkv, Lq, P,
                      prefix_rows, rows, D, window, scale, ws.get(), bytes,
                      c10::cuda::getCurrentCUDAStream(dev).stream());
    });
    return rc ? PyLong_FromLong(rc) : tuple({o, lse});
  });
}

struct Rope {
  const at::Tensor *q, *k, *wq, *wk, *freq, *pos;
  int dev, B, L, D, Hq, Hkv, rot;
  long long q_tok, k_tok;
};
Rope rope(PyObject* q, PyObject* k, PyObject* wq, PyObject* wk, PyObject* freq, PyObject* pos) {
  Rope r;
  r.q = tensor(q);
  r.k = tensor_or_null(k);
  r.wq = tensor_or_null(wq);
  r.wk = tensor_or_null(wk);
  r.freq = tensor_or_null(freq);
  r.pos = tensor_or_null(pos);
  if (r.q->dim() != 4 || (r.freq && r.freq->dim() != 1)) throw NotThisWay{};
  r.dev = current(r.q);
  r.B = dim32(r.q->size(0));
  r.L = dim32(r.q->size(1));
  r.Hq = dim32(r.q->size(2));
  r.D = dim32(r.q->size(3));
  r.q_tok = token_stride(r.q, r.B, r.L, r.D, r.dev);
  r.k_tok = r.k ? token_stride(r.k, r.B, r.L, r.D, r.dev) : 0;
  r.Hkv = r.k ? dim32(r.k->size(2)) : 1;
  expect(r.wq, at::kFloat, {r.D}, r.dev);
  expect(r.wk, at::kFloat, {r.D}, r.dev);
  if (r.freq) expect(r.freq, at::kDouble, r.freq->sizes(), r.dev);
  expect(r.pos, at::kInt, {r.B, r.L}, r.dev);
  r.rot = r.freq ? dim32(2 * r.freq->size(0)) : 0;
  return r;
}

// (q, k or None, v or None, wq, wk, inv_freq, k_cache or None, v_cache, kv_len, eps, positions, pos0, weight_offset,
// interleaved) -> (q, k, v), the latter two None with caches
PyObject* qk_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 14, [&]() -> PyObject* {
    const Rope r = rope(a[0], a[1], a[3], a[4], a[5], a[10]);
    const at::Tensor *v = tensor_or_null(a[2]), *kc = tensor_or_null(a[6]), *vc = tensor_or_null(a[7]),
                     *len = tensor_or_null(a[8]);
    const long long v_tok = v ? token_stride(v, r.B, r.L, r.D, r.dev) : 0;
    const int Hkv = r.k ? r.Hkv : (v ? dim32(v->size(2)) : 1);
    if (v && v->size(2) != Hkv) throw NotThisWay{};
    at::Tensor q_out, k_out, v_out;
    int rows = r.L;
    if (len) {  // into caches
      if ((r.k && !kc) || (v && !vc)) throw NotThisWay{};
      const at::Tensor* c = r.k ? kc : (v ? vc : nullptr);
      if (c) {
        if (c->dim() != 4) throw NotThisWay{};
        rows = dim32(c->size(2));
      }
      if (r.k) expect(kc, at::kBFloat16, {r.B, Hkv, rows, r.D}, r.dev);
      if (v) expect(vc, at::kBFloat16, {r.B, Hkv, rows, r.D}, r.dev);
      expect(len, at::kInt, {r.B}, r.dev);
    }
    const int interleaved = truth(a[13]), pos0 = int32(a[11]);
    const float eps = real(a[9]), off = real(a[12]);
    const int rc = unlocked([&] {
      if (!len && r.k) k_out = empty({r.B, Hkv, r.L, r.D}, r.q, at::kBFloat16);
      if (!len && v) v_out = empty({r.B, Hkv, r.L, r.D}, r.q, at::kBFloat16);
      q_out = empty({r.B, r.Hq, r.L, r.D}, r.q, at::kBFloat16);
      swa_bf16* ko = r.k ? ptr<swa_bf16>(len ? kc : &k_out) : nullptr;
      swa_bf16* vo = v ? ptr<swa_bf16>(len ? vc : &v_out) : nullptr;
      return g_rope(ptr<swa_bf16>(r.q), ptr<swa_bf16>(r.k), ptr<swa_bf16>(v), r.q_tok, r.k_tok, v_tok,
                    ptr<float>(r.wq), ptr<float>(r.wk), ptr<double>(r.freq), ptr<int32_t>(r.pos), ptr<int32_t>(len),
                    ptr<swa_bf16>(&q_out), ko, vo, r.B, r.Hq, Hkv, r.L, r.D, rows, r.rot, interleaved, pos0, eps, off,
                    c10::cuda::getCurrentCUDAStream(r.dev).stream());
    });
    return rc ? PyLong_FromLong(rc) : tuple({q_out, k_out, v_out});
  });
}

// (q, k or None, wq, wk, inv_freq, dq, dk, dv or None, eps, positions, pos0, weight_offset, interleaved)
// -> (gradient of the fused projection, dwq, dwk)
PyObject* qk_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 13, [&]() -> PyObject* {
    const Rope r = rope(a[0], a[1], a[2], a[3], a[4], a[9]);
    const at::Tensor *dq = tensor(a[5]), *dk = r.k ? tensor(a[6]) : nullptr, *dv = tensor_or_null(a[7]);
    if (dv && dv->dim() != 4) throw NotThisWay{};
    const int Hkv = r.k ? r.Hkv : (dv ? dim32(dv->size(1)) : 1);
    expect(dq, at::kFloat, {r.B, r.Hq, r.L, r.D}, r.dev);
    expect(dk, at::kFloat, {r.B, Hkv, r.L, r.D}, r.dev);
    expect(dv, at::kFloat, {r.B, Hkv, r.L, r.D}, r.dev);
    const int Hk = r.k ? Hkv : 0, H = r.Hq + Hk + (dv ? Hkv : 0);
    const int interleaved = truth(a[12]), pos0 = int32(a[10]);
    const float eps = real(a[8]), off = real(a[11]);
    const size_t bytes = g_rope_bwd_ws(r.B, r.L, r.D);
    const long long tok = (long long)H * r.D;
    at::Tensor d, dwq, dwk;
    const int rc = unlocked([&] {
      d = empty({r.B, r.L, H, r.D}, r.q, at::kBFloat16);
      if (r.wq) dwq = empty({r.D}, r.q, at::kFloat);
      if (r.wk && r.k) dwk = empty({r.D}, r.q, at::kFloat);
      const c10::DataPtr ws = scratch(bytes);
      swa_bf16* out = ptr<swa_bf16>(&d);
      return g_rope_bwd(ptr<swa_bf16>(r.q), ptr<swa_bf16>(r.k), r.q_tok, r.k_tok, ptr<float>(r.wq), ptr<float>(r.wk),
                        ptr<double>(r.freq), ptr<int32_t>(r.pos), ptr<float>(dq), ptr<float>(dk), ptr<float>(dv), out,
                        Hk ? out + (size_t)r.Hq * r.D : nullptr, dv ? out + (size_t)(r.Hq + Hk) * r.D : nullptr, tok,
                        tok, tok, dwq.defined() ? ptr<float>(&dwq) : nullptr, dwk.defined() ? ptr<float>(&dwk) : nullptr,
                        r.B, r.Hq, Hkv, r.L, r.D, r.rot, interleaved, pos0, eps, off, ws.get(), bytes,
                        c10::cuda::getCurrentCUDAStream(r.dev).stream());
    });
    return rc ? PyLong_FromLong(rc) : tuple({d, dwq, dwk});
  });
}

// The five entry points' addresses, in the order of the globals above, and torch.OutOfMemoryError.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6 || !PyExceptionClass_Check(a[5])) {
    PyErr_SetString(PyExc_TypeError, "5 addresses and an exception class expected");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  g_shared_ws = reinterpret_cast<decltype(g_shared_ws)>(p[0]);
  g_shared = reinterpret_cast<decltype(g_shared)>(p[1]);
  g_rope = reinterpret_cast<decltype(g_rope)>(p[2]);
  g_rope_bwd_ws = reinterpret_cast<decltype(g_rope_bwd_ws)>(p[3]);
  g_rope_bwd = reinterpret_cast<decltype(g_rope_bwd)>(p[4]);
  Py_XSETREF(g_out_of_memory, Py_NewRef(a[5]));
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef kMethods[] = {
    {"bind", FAST(bind), METH_FASTCALL, nullptr},
    {"forward_shared", FAST(forward_shared), METH_FASTCALL, nullptr},
    {"qk_rope", FAST(qk_rope), METH_FASTCALL, nullptr},
    {"qk_rope_backward", FAST(qk_rope_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
