// mx_torch.cpp -- the short way from torch tensors to the MXFP4 calls of
// include/wqbmm_mxfp4.h, as the Python module _mx_calls.
//
// Many of these calls run in a few microseconds, and in Python the checks, the
// outputs' allocation (1.5 us each) and ctypes took longer than that: 8.1 us to
// issue a quantisation and 7.3 a product, of which the launch itself takes 2.9;
// this way 4.8 and 3.9.  Each function takes the ordinary case, outputs allocated
// for the current stream of the current device, and returns None for anything
// else, a call that the library refuses among them: the wrappers of _mxfp4.py
// then take the long way, which says what is wrong.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/wqbmm_mxfp4.h"

namespace {

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return WQBMM_DTYPE_F16;
    case at::kBFloat16: return WQBMM_DTYPE_BF16;
    case at::kFloat: return WQBMM_DTYPE_F32;
    default: return -1;
  }
}

bool on_current_device(const at::Tensor& t) {
  return t.is_cuda() && t.layout() == at::kStrided && t.get_device() == c10::hip::current_device();
}

// A matrix with contiguous rows on the current device; the distance of its rows.
bool rows_of(const at::Tensor& t, int64_t* ld) {
  if (t.dim() != 2 || !on_current_device(t) || (t.stride(1) != 1 && t.size(1) > 1)) return false;
  *ld = t.size(0) <= 1 ? (t.size(1) + 7) / 8 * 8 : t.stride(0);
  return true;
}

bool is_bytes(const at::Tensor& t, int64_t numel) {
  return t.scalar_type() == at::kByte && on_current_device(t) && t.is_contiguous() && t.numel() == numel;
}

// The other way ends the outputs' history in an error.
bool needs_gradient(const at::Tensor& t) { return t.requires_grad() && at::GradMode::is_enabled(); }

void* stream_of(const at::Tensor& t) { return c10::hip::getCurrentHIPStream(t.get_device()).stream(); }

PyObject* other_way() { Py_RETURN_NONE; }

// quantize(x) -> (codes, scales)
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* x = n == 1 ? tensor(args[0]) : nullptr;
  int64_t ld;
  if (!x || !rows_of(*x, &ld)) return other_way();
  const int code = dtype_code(x->scalar_type());
  const int64_t M = x->size(0), K = x->size(1);
  if (code < 0 || K % 32 != 0) return other_way();
  const auto bytes = x->options().dtype(at::kByte);
  at::Tensor codes = at::empty({M, K / 2}, bytes), scales = at::empty({M, K / 32}, bytes);
  if (wqbmm_mxfp4_quantize(x->data_ptr(), code, M, K, ld, codes.data_ptr(), scales.data_ptr(), stream_of(*x)) !=
      WQBMM_OK)
    return other_way();
  PyObject* both = PyTuple_New(2);
  if (!both) return nullptr;
  PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(std::move(codes)));
  PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(std::move(scales)));
  return both;
  END_HANDLE_TH_ERRORS
}

// dequantize(codes, scales, code of the type) -> y
PyObject* dequantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* codes = n == 3 ? tensor(args[0]) : nullptr;
  const at::Tensor* scales = n == 3 ? tensor(args[1]) : nullptr;
  if (!codes || !scales || codes->dim() != 2 || scales->dim() != 2) return other_way();
  const int64_t M = codes->size(0), K = codes->size(1) * 2;
  if (scales->size(0) != M || scales->size(1) != K / 32 || K % 32 != 0 || !is_bytes(*codes, M * (K / 2)) ||
      !is_bytes(*scales, M * (K / 32)))
    return other_way();
  const long code = PyLong_AsLong(args[2]);
  if (code == -1 && PyErr_Occurred()) return nullptr;
  const at::ScalarType t = code == WQBMM_DTYPE_F16 ? at::kHalf : code == WQBMM_DTYPE_BF16 ? at::kBFloat16 : at::kFloat;
  at::Tensor y = at::empty({M, K}, codes->options().dtype(t));
  if (wqbmm_mxfp4_dequantize(codes->data_ptr(), scales->data_ptr(), M, K, y.data_ptr(), (int)code, K,
                             stream_of(*codes)) != WQBMM_OK)
    return other_way();
  return THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

// matmul(x, w_tiled, N, act) -> y
PyObject* matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* x = n == 4 ? tensor(args[0]) : nullptr;
  const at::Tensor* w = n == 4 ? tensor(args[1]) : nullptr;
  int64_t ld;
  if (!x || !w || !rows_of(*x, &ld) || !PyLong_Check(args[2]) || needs_gradient(*x)) return other_way();
  const int code = dtype_code(x->scalar_type());
  const long long N = PyLong_AsLongLong(args[2]);
  const long act = PyLong_AsLong(args[3]);
  if (PyErr_Occurred()) return nullptr;
  const int64_t M = x->size(0), K = x->size(1), bytes = wqbmm_mxfp4_tiled_weight_bytes(K, N);
  if (code < 0 || bytes < 0 || w->dim() != 1 || !is_bytes(*w, bytes)) return other_way();
  at::Tensor y = at::empty({M, N}, x->options());
  if (wqbmm_mxfp4_matmul(x->data_ptr(), code, ld, w->data_ptr(), M, K, N, y.data_ptr(), (int)act, stream_of(*x)) !=
      WQBMM_OK)
    return other_way();
  return THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

// moe(x, router, gate_up, down, I, k, renormalize) -> (y, ids, weights)
PyObject* moe(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor *x = nullptr, *router = nullptr, *gate_up = nullptr, *down = nullptr;
  if (n == 7) {
    x = tensor(args[0]);
    router = tensor(args[1]);
    gate_up = tensor(args[2]);
    down = tensor(args[3]);
  }
  int64_t ld;
  if (!x || !router || !gate_up || !down || !rows_of(*x, &ld) || !PyLong_Check(args[4]) || !PyLong_Check(args[5]) ||
      needs_gradient(*x) || needs_gradient(*router))
    return other_way();
  const int code = dtype_code(x->scalar_type());
  const long long I = PyLong_AsLongLong(args[4]), k = PyLong_AsLongLong(args[5]);
  const int renormalize = PyObject_IsTrue(args[6]);
  if (PyErr_Occurred()) return nullptr;
  const int64_t T = x->size(0), H = x->size(1);
  if (code < 0 || router->dim() != 2 || router->size(1) != H || router->scalar_type() != x->scalar_type() ||
      !on_current_device(*router) || !router->is_contiguous())
    return other_way();
  const int64_t E = router->size(0);
  if (I < 1 || I > (int64_t(1) << 24) || E < 1 || E > 256 || k < 1 || k > E) return other_way();
  const int64_t gb = wqbmm_mxfp4_tiled_weight_bytes(H, E * 2 * I), db = wqbmm_mxfp4_tiled_weight_bytes(I, E * H);
  if (gb < 0 || db < 0 || gate_up->dim() != 1 || down->dim() != 1 || !is_bytes(*gate_up, gb) || !is_bytes(*down, db))
    return other_way();
  at::Tensor y = at::empty({T, H}, x->options()), ids = at::empty({T, k}, x->options().dtype(at::kInt)),
             weights = at::empty({T, k}, x->options().dtype(at::kFloat));
  if (wqbmm_mxfp4_moe(x->data_ptr(), code, ld, T, H, I, E, k, renormalize, router->data_ptr(), gate_up->data_ptr(),
                      down->data_ptr(), y.data_ptr(), ids.data_ptr<int32_t>(), weights.data_ptr<float>(),
                      stream_of(*x)) != WQBMM_OK)
    return other_way();
  PyObject* all = PyTuple_New(3);
  if (!all) return nullptr;
  PyTuple_SET_ITEM(all, 0, THPVariable_Wrap(std::move(y)));
  PyTuple_SET_ITEM(all, 1, THPVariable_Wrap(std::move(ids)));
  PyTuple_SET_ITEM(all, 2, THPVariable_Wrap(std::move(weights)));
  return all;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize)), METH_FASTCALL, nullptr},
    {"dequantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(dequantize)), METH_FASTCALL, nullptr},
    {"matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(matmul)), METH_FASTCALL, nullptr},
    {"moe", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(moe)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_mx_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mx_calls() { return PyModule_Create(&module_def); }
