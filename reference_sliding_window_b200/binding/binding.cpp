// The short way from Python into the calls whose kernels take no longer than
// marshalling their arguments through ctypes does (a turn of one step's queries
// and keys, the gradient of a short document): checks of the tensors, the
// results' and the workspace's allocation and the C call in one function.
//
// Every function takes the plain case only: torch.Tensor arguments that fit,
// results allocated here.  It returns None where something does not fit, without
// having done anything, and the caller's checks in Python then name the problem
// (or the C call takes the rarer case); the status of a refused C call as an
// int; or the results.  The library's functions come in by address, from the
// handle that ctypes opened, so both ways lead into the same library.

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/SmallVector.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include "rswa.h"

namespace {

decltype(&rswa_masked_backward) masked_backward;
decltype(&rswa_masked_backward_workspace_bytes) masked_backward_workspace_bytes;
decltype(&rswa_rotary_apply) rotary_apply;

// (masked_backward, masked_backward_workspace_bytes, rotary_apply): their addresses.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "bind takes 3 addresses");
    return nullptr;
  }
  void* f[3];
  for (int i = 0; i < 3; ++i) {
    f[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  masked_backward = reinterpret_cast<decltype(masked_backward)>(f[0]);
  masked_backward_workspace_bytes = reinterpret_cast<decltype(masked_backward_workspace_bytes)>(f[1]);
  rotary_apply = reinterpret_cast<decltype(rotary_apply)>(f[2]);
  Py_RETURN_NONE;
}

// The tensor of a torch.Tensor (or Parameter; not another subclass), or null.
const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool dtype_of(const at::Tensor& t, rswa_dtype* dt) {
  if (t.scalar_type() == at::kBFloat16) *dt = RSWA_BF16;
  else if (t.scalar_type() == at::kFloat) *dt = RSWA_F32;
  else return false;
  return true;
}

at::Tensor empty_cuda(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, like.device(), std::nullopt));
}

// A sequence of ints that fit int32.
bool ints(PyObject* o, c10::SmallVector<int32_t, 64>* out) {
  if (!PyTuple_Check(o) && !PyList_Check(o)) return false;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
  PyObject** items = PySequence_Fast_ITEMS(o);
  out->resize(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (!PyLong_CheckExact(items[i])) return false;
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(items[i], &overflow);
    if (overflow || v < INT32_MIN || v > INT32_MAX) return false;
    (*out)[i] = (int32_t)v;
  }
  return true;
}

bool int_of(PyObject* o, int* v) {
  if (!PyLong_CheckExact(o)) return false;
  int overflow = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (overflow || x < INT32_MIN || x > INT32_MAX) return false;
  *v = (int)x;
  return true;
}

// (dO, Q, K, V, O, lse, cu_seqlens, ref_lens, n, scale, flags) -> (dQ, dK, dV), a status, or None.
PyObject* backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 11) {
    PyErr_SetString(PyExc_TypeError, "backward takes 11 arguments");
    return nullptr;
  }
  const at::Tensor* t[6];
  for (int i = 0; i < 6; ++i)
    if (!(t[i] = tensor(args[i]))) Py_RETURN_NONE;
  const at::Tensor& Q = *t[1];
  rswa_dtype dt;
  if (!Q.is_cuda() || Q.dim() != 3 || !dtype_of(Q, &dt)) Py_RETURN_NONE;
  for (int i = 0; i < 5; ++i)
    if (t[i]->scalar_type() != Q.scalar_type() || t[i]->sizes() != Q.sizes() || t[i]->device() != Q.device() ||
        !t[i]->is_contiguous())
      Py_RETURN_NONE;
  const int64_t L = Q.size(0), H = Q.size(1), d = Q.size(2);
  const at::Tensor& lse = *t[5];
  if (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != H || lse.size(1) != L ||
      lse.device() != Q.device() || !lse.is_contiguous() || L > INT32_MAX || H > INT32_MAX || d > INT32_MAX)
    Py_RETURN_NONE;
  c10::SmallVector<int32_t, 64> cu, refs;
  int n, flags;
  if (!ints(args[6], &cu) || !ints(args[7], &refs) || !int_of(args[8], &n) || !int_of(args[10], &flags) ||
      refs.empty() || cu.size() != refs.size() + 1 || cu.back() != L)
    Py_RETURN_NONE;
  const double scale = PyFloat_AsDouble(args[9]);
  if (scale == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  HANDLE_TH_ERRORS  // (out of memory, say)
    const c10::cuda::OptionalCUDAGuard guard(Q.device());
    const int docs = (int)refs.size();
    const size_t bytes = masked_backward_workspace_bytes(cu.data(), refs.data(), docs, n, (int)H, (int)d, dt, flags);
    if (bytes == 0) Py_RETURN_NONE;
    at::Tensor g[3];
    for (at::Tensor& x : g) x = empty_cuda(Q.sizes(), Q.scalar_type(), Q);
    const at::Tensor ws = empty_cuda({(int64_t)bytes}, at::kByte, Q);
    const rswa_status st = masked_backward(
        t[0]->const_data_ptr(), Q.const_data_ptr(), t[2]->const_data_ptr(), t[3]->const_data_ptr(),
        t[4]->const_data_ptr(), lse.const_data_ptr<float>(), g[0].mutable_data_ptr(), g[1].mutable_data_ptr(),
        g[2].mutable_data_ptr(), cu.data(), refs.data(), docs, n, (int)H, (int)d, dt, (float)scale, flags,
        ws.mutable_data_ptr(), bytes, c10::cuda::getCurrentCUDAStream(Q.device().index()).stream());
    if (st != RSWA_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(3);
    if (!out) return nullptr;
    for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(out, i, THPVariable_Wrap(std::move(g[i])));
    return out;
  END_HANDLE_TH_ERRORS
}

// Whether x is [rows, heads, d] with contiguous heads; *stride: its rows' distance in elements.
bool rows_of(const at::Tensor& x, int64_t rows, int64_t d, int64_t* stride) {
  if (x.dim() != 3 || x.size(0) != rows || x.size(2) != d || x.stride(2) != 1 ||
      (x.size(1) > 1 && x.stride(1) != d) || x.size(1) > INT32_MAX)
    return false;
  *stride = rows > 1 ? x.stride(0) : x.size(1) * d;
  return true;
}

// (plan address, Q, K or None, positions or None, first, inverse) -> Q's result, the pair, a status, or None.
PyObject* rotary(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 6) {
    PyErr_SetString(PyExc_TypeError, "rotary takes 6 arguments");
    return nullptr;
  }
  const rswa_rotary* plan = static_cast<const rswa_rotary*>(PyLong_AsVoidPtr(args[0]));
  if (!plan) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null plan");
    return nullptr;
  }
  const at::Tensor *Q = tensor(args[1]), *K = args[2] == Py_None ? nullptr : tensor(args[2]),
                   *pos = args[3] == Py_None ? nullptr : tensor(args[3]);
  if (!Q || (!K && args[2] != Py_None) || (!pos && args[3] != Py_None)) Py_RETURN_NONE;
  rswa_dtype dt;
  int first;
  if (!Q->is_cuda() || Q->dim() != 3 || !dtype_of(*Q, &dt) || !int_of(args[4], &first)) Py_RETURN_NONE;
  const int inverse = PyObject_IsTrue(args[5]);
  if (inverse < 0) return nullptr;
  const int64_t rows = Q->size(0);
  int64_t sq = 0, sk = 0;
  if (rows < 1 || rows > INT32_MAX || !rows_of(*Q, rows, plan->d, &sq)) Py_RETURN_NONE;
  if (K && (K->scalar_type() != Q->scalar_type() || K->device() != Q->device() || !rows_of(*K, rows, plan->d, &sk)))
    Py_RETURN_NONE;
  if (pos && (pos->scalar_type() != at::kInt || pos->dim() != 1 || pos->size(0) != rows ||
              pos->device() != Q->device() || !pos->is_contiguous()))
    Py_RETURN_NONE;
  HANDLE_TH_ERRORS
    const c10::cuda::OptionalCUDAGuard guard(Q->device());
    at::Tensor q = empty_cuda(Q->sizes(), Q->scalar_type(), *Q), k;
    if (K) k = empty_cuda(K->sizes(), Q->scalar_type(), *Q);
    const int H = (int)Q->size(1), Hk = K ? (int)K->size(1) : 0;
    const rswa_status st = rotary_apply(
        plan, Q->const_data_ptr(), sq, H, q.mutable_data_ptr(), (long long)H * plan->d, K ? K->const_data_ptr() : nullptr,
        sk, Hk, K ? k.mutable_data_ptr() : nullptr, (long long)Hk * plan->d,
        pos ? static_cast<const int32_t*>(pos->const_data_ptr()) : nullptr, first, (int)rows, dt, inverse,
        c10::cuda::getCurrentCUDAStream(Q->device().index()).stream());
    if (st != RSWA_OK) return PyLong_FromLong(st);
    if (!K) return THPVariable_Wrap(std::move(q));
    PyObject* out = PyTuple_New(2);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(q)));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(k)));
    return out;
  END_HANDLE_TH_ERRORS
}

// (leaf) -> whether its gradient is added up on its device's default stream:
// an autograd graph made there still holds the leaf.
PyObject* accumulates_on_default_stream(PyObject*, PyObject* leaf) {
  const at::Tensor* t = THPVariable_Check(leaf) ? &THPVariable_Unpack(leaf) : nullptr;
  if (!t || !t->is_cuda()) Py_RETURN_FALSE;
  HANDLE_TH_ERRORS
    const auto node = torch::autograd::impl::try_get_grad_accumulator(*t);
    const auto stream = node ? node->stream() : std::nullopt;
    return PyBool_FromLong(stream && *stream == c10::cuda::getDefaultCUDAStream(t->device().index()).unwrap());
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(backward)), METH_FASTCALL, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotary)), METH_FASTCALL, nullptr},
    {"accumulates_on_default_stream", accumulates_on_default_stream, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
