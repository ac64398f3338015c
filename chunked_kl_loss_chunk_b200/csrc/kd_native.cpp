// kd_native.cpp -- the short way from torch tensors to the post-training entry
// points of libkd (Python module _kd_native).
//
// A call on a small batch is bound by the host: checks, allocations and the
// marshalling of some twenty arguments through ctypes take 13 us beside 5 us of
// launch, and reading 580 tensors' addresses, sizes and types in Python 190 us.
// These functions do the same in C++.  They take the usual case only, tensors
// of the right type and shape on the current device and its current stream; for
// anything else they return None, and kd.py's own checks say what is wrong (or
// make the call on another device or stream).  Otherwise they return the call's
// outputs, or its kd_status if that is not KD_OK.
#define AT_PER_OPERATOR_HEADERS
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "kd.h"

namespace {

// Entry points of the library that kd.py has loaded (kd.bind).
struct {
  decltype(&kd_head_logprob_workspace_size) head_ws;
  decltype(&kd_head_logprob_fwd) head_fwd;
  decltype(&kd_head_logprob_bwd) head_bwd;
  decltype(&kd_policy_loss_workspace_size) policy_ws;
  decltype(&kd_policy_loss) policy;
  decltype(&kd_preference_loss_workspace_size) preference_ws;
  decltype(&kd_preference_loss) preference;
  decltype(&kd_grad_clip_workspace_size) clip_ws;
  decltype(&kd_grad_clip) clip;
} g_lib = {};

using at::ScalarType;
using at::Tensor;

// The tensor of a Python object: null for None, `bad` set for what is no plain tensor.
const Tensor* tensor_of(PyObject* o, bool* bad) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    *bad = true;
    return nullptr;
  }
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.unsafeGetTensorImpl()->is_python_dispatch()) *bad = true;
  return &t;
}

// An absent tensor, or a dense one of this type and shape on this device.
bool fits(const Tensor* t, ScalarType type, at::IntArrayRef shape, at::Device device) {
  return !t || (t->scalar_type() == type && t->sizes() == shape && t->device() == device &&
                t->is_contiguous());
}

template <typename T>
T* data(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

bool number(PyObject* o, double* v) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
  *v = PyFloat_AsDouble(o);
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();                       // an integer beyond a double
  return false;
}

bool on_current_device(const Tensor& t) {
  return t.is_cuda() && t.device().index() == c10::cuda::current_device();
}

void* current_stream(const Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
}

// A call's workspace: the given one (uint8 on the device), or one of `bytes`.
struct Workspace {
  Tensor own;
  void* at = nullptr;
  size_t bytes = 0;
  Workspace(const Tensor* given, size_t need, const Tensor& like) {
    if (given) {
      at = given->data_ptr();
      bytes = static_cast<size_t>(given->numel());
      return;
    }
    bytes = need < 1024 ? 1024 : need;
    own = at::empty({static_cast<int64_t>(bytes) + 1024}, like.options().dtype(at::kByte));
    at = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(own.data_ptr()) + 1023) &
                                 ~uintptr_t(1023));
  }
};

bool workspace_fits(const Tensor* ws, at::Device device) {
  return !ws || fits(ws, at::kByte, {ws->numel()}, device);
}

// Number of sequences of a batch, or -1: rows of a 2-D logp, or cu over a 1-D one.
int64_t sequences(const Tensor& logp, const Tensor* cu, const Tensor* mask) {
  if (!on_current_device(logp) || logp.scalar_type() != at::kFloat || !logp.is_contiguous())
    return -1;
  if (mask && !fits(mask, at::kBool, logp.sizes(), logp.device()) &&
      !fits(mask, at::kByte, logp.sizes(), logp.device()))
    return -1;
  if (!cu) return logp.dim() == 2 ? logp.size(0) : -1;
  if (logp.dim() != 1 || cu->dim() != 1 || cu->size(0) < 2 ||
      !fits(cu, at::kInt, cu->sizes(), logp.device()))
    return -1;
  return cu->size(0) - 1;
}

template <typename... T>
PyObject* outputs(const T&... t) {
  PyObject* items[] = {THPVariable_Wrap(t)...};
  PyObject* r = PyTuple_New(sizeof...(T));
  for (size_t i = 0; i < sizeof...(T); ++i) {
    if (!r || !items[i]) {
      for (size_t k = i; k < sizeof...(T); ++k) Py_XDECREF(items[k]);
      Py_XDECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, static_cast<Py_ssize_t>(i), items[i]);
  }
  return r;
}

// bind(addresses of the entry points, in the order of g_lib)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) {
    PyErr_SetString(PyExc_TypeError, "bind: 9 addresses are needed");
    return nullptr;
  }
  void* p[9];
  for (int i = 0; i < 9; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_lib.head_ws = reinterpret_cast<decltype(g_lib.head_ws)>(p[0]);
  g_lib.head_fwd = reinterpret_cast<decltype(g_lib.head_fwd)>(p[1]);
  g_lib.head_bwd = reinterpret_cast<decltype(g_lib.head_bwd)>(p[2]);
  g_lib.policy_ws = reinterpret_cast<decltype(g_lib.policy_ws)>(p[3]);
  g_lib.policy = reinterpret_cast<decltype(g_lib.policy)>(p[4]);
  g_lib.preference_ws = reinterpret_cast<decltype(g_lib.preference_ws)>(p[5]);
  g_lib.preference = reinterpret_cast<decltype(g_lib.preference)>(p[6]);
  g_lib.clip_ws = reinterpret_cast<decltype(g_lib.clip_ws)>(p[7]);
  g_lib.clip = reinterpret_cast<decltype(g_lib.clip)>(p[8]);
  Py_RETURN_NONE;
}

bool bound(Py_ssize_t n, Py_ssize_t want, bool have) {
  if (n == want && have) return true;
  PyErr_SetString(PyExc_TypeError, "_kd_native: wrong number of arguments, or not bound");
  return false;
}

// What both calls of the head take; false for what is not that.
struct Head {
  const Tensor *h, *W, *targets, *ws;
  int64_t T, d, V, chunk;
  double tau;
  int dtype;
};
bool head_of(PyObject* h, PyObject* W, PyObject* targets, PyObject* chunk, PyObject* tau,
             PyObject* ws, Head* x) {
  bool bad = false;
  x->h = tensor_of(h, &bad);
  x->W = tensor_of(W, &bad);
  x->targets = tensor_of(targets, &bad);
  x->ws = tensor_of(ws, &bad);
  if (bad || !x->h || !x->W || !x->targets || !PyLong_Check(chunk) || !number(tau, &x->tau))
    return false;
  if (!on_current_device(*x->h) || x->h->dim() != 2 || x->W->dim() != 2) return false;
  x->T = x->h->size(0);
  x->d = x->h->size(1);
  x->V = x->W->size(0);
  const bool bf16 = x->h->scalar_type() == at::kBFloat16;
  x->dtype = bf16 ? KD_DTYPE_BF16 : KD_DTYPE_F32;
  int overflow = 0;
  x->chunk = PyLong_AsLongLongAndOverflow(chunk, &overflow);
  return !overflow && (bf16 || x->h->scalar_type() == at::kFloat) && x->h->is_contiguous() &&
         fits(x->W, x->h->scalar_type(), {x->V, x->d}, x->h->device()) &&
         fits(x->targets, at::kInt, {x->T}, x->h->device()) &&
         workspace_fits(x->ws, x->h->device());
}

// The workspace as a tensor to hand on.
Tensor given_out(const Tensor* ws, const Workspace& w) {
  return ws ? *ws
            : w.own.narrow(0, static_cast<char*>(w.at) - static_cast<char*>(w.own.data_ptr()),
                           static_cast<int64_t>(w.bytes));
}

// head_logprobs(h, W, targets, chunk, temperature, use, ws)
PyObject* head_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!bound(n, 7, g_lib.head_fwd)) return nullptr;
  Head x;
  if (!head_of(a[0], a[1], a[2], a[3], a[4], a[6], &x)) Py_RETURN_NONE;
  const int use = static_cast<int>(PyLong_AsLong(a[5]));
  if (PyErr_Occurred()) return nullptr;
  Workspace w(x.ws, x.ws ? 0 : g_lib.head_ws(x.T, x.d, x.V, x.chunk, x.dtype, use), *x.h);
  const auto f32 = x.h->options().dtype(at::kFloat);
  Tensor logp = at::empty({x.T}, f32), lse = at::empty({x.T}, f32);
  const kd_status st = g_lib.head_fwd(
      x.h->data_ptr(), x.W->data_ptr(), x.dtype, x.T, x.d, x.V, data<const int32_t>(x.targets),
      x.chunk, static_cast<float>(x.tau), use == KD_HEAD_KEEP, logp.data_ptr<float>(),
      lse.data_ptr<float>(), w.at, w.bytes, current_stream(*x.h));
  if (st != KD_OK) return PyLong_FromLong(st);
  return outputs(logp, lse, given_out(x.ws, w));
  END_HANDLE_TH_ERRORS
}

// head_logprobs_bwd(h, W, targets, lse, kept_logp, grad_logp, grad_loss, chunk, temperature,
//                   need dH, need dW, dW in bf16, ws): new dH and dW
PyObject* head_logprobs_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!bound(n, 13, g_lib.head_bwd)) return nullptr;
  Head x;
  bool bad = false;
  const Tensor *lse = tensor_of(a[3], &bad), *kept = tensor_of(a[4], &bad);
  const Tensor *grad = tensor_of(a[5], &bad), *grad_loss = tensor_of(a[6], &bad);
  if (bad || !lse || !grad || !head_of(a[0], a[1], a[2], a[7], a[8], a[12], &x) ||
      (kept && !x.ws))
    Py_RETURN_NONE;
  const auto dev = x.h->device();
  if (!fits(lse, at::kFloat, {x.T}, dev) || !fits(kept, at::kFloat, {x.T}, dev) ||
      !fits(grad, at::kFloat, {x.T}, dev) ||
      (grad_loss && (grad_loss->numel() != 1 || !fits(grad_loss, at::kFloat, grad_loss->sizes(), dev))))
    Py_RETURN_NONE;
  const bool need_h = PyObject_IsTrue(a[9]), need_w = PyObject_IsTrue(a[10]);
  const bool w_bf16 = PyObject_IsTrue(a[11]);
  Workspace w(x.ws, x.ws ? 0 : g_lib.head_ws(x.T, x.d, x.V, x.chunk, x.dtype, KD_HEAD_BOTH), *x.h);
  Tensor dH, dW;
  if (need_h) dH = at::empty({x.T, x.d}, x.h->options());
  if (need_w) dW = at::empty({x.V, x.d}, x.h->options().dtype(w_bf16 ? at::kBFloat16 : at::kFloat));
  const kd_status st = g_lib.head_bwd(
      x.h->data_ptr(), x.W->data_ptr(), x.dtype, x.T, x.d, x.V, data<const int32_t>(x.targets),
      x.chunk, static_cast<float>(x.tau), data<const float>(lse), data<const float>(kept),
      data<const float>(grad), data<const float>(grad_loss), need_h ? dH.data_ptr() : nullptr,
      need_w ? dW.data_ptr() : nullptr, w_bf16 ? KD_DTYPE_BF16 : KD_DTYPE_F32, 0, w.at, w.bytes,
      current_stream(*x.h));
  if (st != KD_OK) return PyLong_FromLong(st);
  return outputs(dH, dW, given_out(x.ws, w));
  END_HANDLE_TH_ERRORS
}

// policy_loss(logp, old_logp, ref_logp, advantages, per_token, mask, cu_seqlens, clip_low,
//             clip_high, kl_coef, reduction, denom, grad, ws)
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!bound(n, 14, g_lib.policy)) return nullptr;
  bool bad = false;
  const Tensor *logp = tensor_of(a[0], &bad), *old = tensor_of(a[1], &bad);
  const Tensor *ref = tensor_of(a[2], &bad), *adv = tensor_of(a[3], &bad);
  const Tensor *mask = tensor_of(a[5], &bad), *cu = tensor_of(a[6], &bad);
  const Tensor* ws = tensor_of(a[13], &bad);
  double low, high, kl, denom;
  if (bad || !logp || !adv || !number(a[7], &low) || !number(a[8], &high) || !number(a[9], &kl) ||
      !number(a[11], &denom))
    Py_RETURN_NONE;
  const int64_t S = sequences(*logp, cu, mask);
  const bool per_token = PyObject_IsTrue(a[4]), grad = PyObject_IsTrue(a[12]);
  const auto dev = logp->device();
  if (S < 0 || !fits(old, at::kFloat, logp->sizes(), dev) ||
      !fits(ref, at::kFloat, logp->sizes(), dev) || !workspace_fits(ws, dev) ||
      !(per_token ? fits(adv, at::kFloat, logp->sizes(), dev) : fits(adv, at::kFloat, {S}, dev)))
    Py_RETURN_NONE;
  const int reduction = static_cast<int>(PyLong_AsLong(a[10]));
  if (PyErr_Occurred()) return nullptr;
  const int64_t N = logp->numel();
  Workspace w(ws, ws ? 0 : g_lib.policy_ws(S, N), *logp);
  Tensor loss = at::empty({}, logp->options()), stats = at::empty({4}, logp->options()), dlogp;
  if (grad) dlogp = at::empty(logp->sizes(), logp->options());
  const kd_status st = g_lib.policy(
      data<const float>(logp), data<const float>(old), data<const float>(ref),
      data<const float>(adv), per_token, data<const uint8_t>(mask), data<const int32_t>(cu), S, N,
      low, high, kl, reduction, denom, loss.data_ptr<float>(), stats.data_ptr<float>(),
      grad ? dlogp.data_ptr<float>() : nullptr, w.at, w.bytes, current_stream(*logp));
  if (st != KD_OK) return PyLong_FromLong(st);
  return outputs(loss, stats, dlogp);
  END_HANDLE_TH_ERRORS
}

// preference_loss(logp, ref_logp, mask, cu_seqlens, kind, beta, margin, label_smoothing,
//                 length_normalize, pairs_total (or None), grad, ws)
PyObject* preference_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!bound(n, 12, g_lib.preference)) return nullptr;
  bool bad = false;
  const Tensor *logp = tensor_of(a[0], &bad), *ref = tensor_of(a[1], &bad);
  const Tensor *mask = tensor_of(a[2], &bad), *cu = tensor_of(a[3], &bad);
  const Tensor* ws = tensor_of(a[11], &bad);
  double beta, margin, smoothing;
  if (bad || !logp || !number(a[5], &beta) || !number(a[6], &margin) ||
      !number(a[7], &smoothing) || (a[9] != Py_None && !PyLong_Check(a[9])))
    Py_RETURN_NONE;
  const int64_t S = sequences(*logp, cu, mask);
  if (S < 0 || S % 2 || !fits(ref, at::kFloat, logp->sizes(), logp->device()) ||
      !workspace_fits(ws, logp->device()))
    Py_RETURN_NONE;
  const bool normalize = PyObject_IsTrue(a[8]), grad = PyObject_IsTrue(a[10]);
  const int kind = static_cast<int>(PyLong_AsLong(a[4]));
  const int64_t total = a[9] == Py_None ? S / 2 : PyLong_AsLongLong(a[9]);
  if (PyErr_Occurred()) return nullptr;
  const int64_t N = logp->numel();
  Workspace w(ws, ws ? 0 : g_lib.preference_ws(S / 2, N), *logp);
  Tensor loss = at::empty({}, logp->options()), rewards = at::empty({S}, logp->options()), dlogp;
  if (grad) dlogp = at::empty(logp->sizes(), logp->options());
  const kd_status st = g_lib.preference(
      data<const float>(logp), data<const float>(ref), data<const uint8_t>(mask),
      data<const int32_t>(cu), S / 2, N, kind, beta, margin, smoothing, normalize, total,
      loss.data_ptr<float>(), rewards.data_ptr<float>(), grad ? dlogp.data_ptr<float>() : nullptr,
      w.at, w.bytes, current_stream(*logp));
  if (st != KD_OK) return PyLong_FromLong(st);
  return outputs(loss, rewards, dlogp);
  END_HANDLE_TH_ERRORS
}

// Addresses, sizes and types of a list of gradients on the current device; false for what is not
// one.
bool grad_list(PyObject* list, std::vector<void*>* at, std::vector<int64_t>* sizes,
               std::vector<int>* types, const Tensor** first) {
  const Py_ssize_t n = PyList_GET_SIZE(list);
  for (Py_ssize_t i = 0; i < n; ++i) {
    bool bad = false;
    const Tensor* t = tensor_of(PyList_GET_ITEM(list, i), &bad);
    if (bad || !t) return false;
    if (i == 0) {
      if (!on_current_device(*t)) return false;
      *first = t;
    }
    const bool bf16 = t->scalar_type() == at::kBFloat16;
    if ((!bf16 && t->scalar_type() != at::kFloat) || t->device() != (*first)->device() ||
        !t->is_contiguous())
      return false;
    at->push_back(t->data_ptr());
    sizes->push_back(t->numel());
    types->push_back(bf16 ? KD_DTYPE_BF16 : KD_DTYPE_F32);
  }
  return n > 0;
}

// clip_grad_norm(grads, out (list or None), max_norm, sumsq)
PyObject* clip_grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!bound(n, 4, g_lib.clip)) return nullptr;
  bool bad = false;
  const Tensor* sumsq = tensor_of(a[3], &bad);
  double max_norm;
  if (bad || !PyList_Check(a[0]) || (a[1] != Py_None && !PyList_Check(a[1])) ||
      !number(a[2], &max_norm))
    Py_RETURN_NONE;
  std::vector<void*> grads, outs;
  std::vector<int64_t> sizes, out_sizes;
  std::vector<int> types, out_types;
  const Tensor *first = nullptr, *first_out = nullptr;
  if (!grad_list(a[0], &grads, &sizes, &types, &first) ||
      !fits(sumsq, at::kDouble, {}, first->device()))
    Py_RETURN_NONE;
  if (a[1] != Py_None &&
      (!grad_list(a[1], &outs, &out_sizes, &out_types, &first_out) ||
       first_out->device() != first->device() || out_sizes != sizes || out_types != types))
    Py_RETURN_NONE;
  const int count = static_cast<int>(grads.size());
  Workspace w(nullptr, g_lib.clip_ws(count), *first);
  Tensor norm = at::empty({}, first->options().dtype(at::kFloat));
  const kd_status st =
      g_lib.clip(grads.data(), a[1] == Py_None ? grads.data() : outs.data(), sizes.data(),
                 types.data(), count, max_norm, data<const double>(sumsq), norm.data_ptr<float>(),
                 w.at, w.bytes, current_stream(*first));
  if (st != KD_OK) return PyLong_FromLong(st);
  return outputs(norm);
  END_HANDLE_TH_ERRORS
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);

PyMethodDef method(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL,
          nullptr};
}

PyMethodDef g_methods[] = {method("bind", bind),
                           method("head_logprobs", head_logprobs),
                           method("head_logprobs_bwd", head_logprobs_bwd),
                           method("policy_loss", policy_loss),
                           method("preference_loss", preference_loss),
                           method("clip_grad_norm", clip_grad_norm),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kd_native",
                        "Short way from torch tensors to libkd's post-training entry points.", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kd_native(void) { return PyModule_Create(&g_module); }
