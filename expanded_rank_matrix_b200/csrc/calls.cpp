// Marshalling of the 8-bit inference calls between torch tensors and the C ABI:
// checks, output allocation, the call.  These calls are made once or more for
// every projection of a token, and their kernels take a few microseconds; the
// same steps in Python with ctypes took 5 to 9 us of the host on top of the
// launches' 2.5 us each, which is what a call then cost.  Nothing is computed
// here, and nothing is kept between calls.

#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/externd.h"

namespace {

// the library's entry points, as the binding loaded them
decltype(&externd_quantize_rows) g_quantize = nullptr;
decltype(&externd_matmul_i8) g_matmul = nullptr;
decltype(&externd_ternary_apply_i8) g_apply = nullptr;

struct Refused : std::runtime_error {  // becomes a ValueError
  using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int type_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return EXTERND_F32;
    case at::kHalf: return EXTERND_F16;
    case at::kBFloat16: return EXTERND_BF16;
    default: return -1;
  }
}

int64_t pad16(int64_t v) { return (v + 15) / 16 * 16; }

// Distance between the rows of 8-bit values laid out as Quantized lays them out.
int64_t row_bytes(const at::Tensor& q) { return q.size(0) > 1 ? q.stride(0) : pad16(q.size(1)); }

// A tensor [..., n] as rows at one distance with their elements side by side:
// itself, or a copy.  (Views that stand for the negatives of what they hold are
// copied too.)
struct Rows {
  at::Tensor held;  // keeps a copy alive
  const void* at = nullptr;
  int64_t rows = 0, n = 0, ld = 0;
};
Rows rows_of(const at::Tensor& X) {
  Rows r;
  if (X.dim() == 0 || X.size(-1) == 0) refuse("X must have at least one column");
  r.n = X.size(-1);
  if (X.is_contiguous() && !X.is_neg()) {
    r.rows = X.numel() / r.n;
    r.ld = r.n;
    r.at = X.const_data_ptr();
    return r;
  }
  r.held = X.dim() == 2 ? X : X.reshape({-1, r.n});
  if (r.held.is_neg()) r.held = r.held.resolve_neg();
  r.rows = r.held.size(0);
  if ((r.n > 1 && r.held.stride(1) != 1) || (r.rows > 1 && r.held.stride(0) < r.n))
    r.held = r.held.contiguous();
  r.ld = r.rows > 1 ? r.held.stride(0) : r.n;  // (the stride of a single row means nothing)
  r.at = r.held.const_data_ptr();
  return r;
}

// Activations of a product: X alone, or 8-bit rows with their scales.
struct Activations {
  Rows x;
  int type;
  const float* scale = nullptr;
  c10::SmallVector<int64_t, 6> out;  // the output's sizes
  at::ScalarType out_type;
};
Activations activations(PyObject* x_, PyObject* scale_, PyObject* dtype_, int64_t n, int64_t m,
                        c10::DeviceIndex device) {
  Activations a;
  const at::Tensor& X = tensor(x_, "X");
  if (!X.is_cuda() || X.get_device() != device) refuse("expected tensors on one CUDA device");
  if (scale_ != Py_None) {
    a.type = EXTERND_I8;
    a.scale = tensor(scale_, "scale").const_data_ptr<float>();
    a.x.at = X.const_data_ptr();
    a.x.rows = X.size(0);
    a.x.n = X.size(1);
    a.x.ld = row_bytes(X);
    a.out = {a.x.rows, m};
    a.out_type = at::kFloat;
  } else {
    a.type = type_of(X.scalar_type());
    if (a.type < 0) refuse("X must be Quantized, or an fp32, fp16 or bf16 tensor");
    a.x = rows_of(X);
    a.out.append(X.sizes().begin(), X.sizes().end());
    a.out.back() = m;
    a.out_type = X.scalar_type();
  }
  if (a.x.n != n) refuse("X must have " + std::to_string(n) + " columns");
  if (dtype_ != Py_None) {
    if (!THPDtype_Check(dtype_)) refuse("out_dtype must be a torch.dtype");
    a.out_type = reinterpret_cast<THPDtype*>(dtype_)->scalar_type;
  }
  if (type_of(a.out_type) < 0) refuse("out_dtype must be fp32, fp16 or bf16");
  return a;
}

at::Tensor allocate(at::IntArrayRef sizes, at::ScalarType type, c10::DeviceIndex device) {
  return at::detail::empty_cuda(sizes, type, c10::Device(c10::DeviceType::CUDA, device),
                                std::nullopt);
}

externd_stream_t stream_of(c10::DeviceIndex device) {
  return (externd_stream_t)c10::cuda::getCurrentCUDAStream(device).stream();
}

// The call without the interpreter's lock (a full launch queue blocks).
template <typename F>
int unlocked(F f) {
  PyThreadState* s = PyEval_SaveThread();
  const int rc = f();
  PyEval_RestoreThread(s);
  return rc;
}

template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

bool count_ok(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// bind(quantize, matmul, apply): the entry points' addresses
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_ok(n, 3)) return nullptr;
  void* p[3];
  for (int i = 0; i < 3; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_quantize = reinterpret_cast<decltype(g_quantize)>(p[0]);
  g_matmul = reinterpret_cast<decltype(g_matmul)>(p[1]);
  g_apply = reinterpret_cast<decltype(g_apply)>(p[2]);
  Py_RETURN_NONE;
}

// quantize_rows(X) -> (q, scale), or the C status
PyObject* quantize_rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_ok(n, 1)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& X = tensor(args[0], "X");
    const int type = type_of(X.scalar_type());
    if (type < 0) refuse("X must be an fp32, fp16 or bf16 tensor");
    if (!X.is_cuda()) refuse("expected a CUDA tensor");
    const c10::cuda::OptionalCUDAGuard guard(X.device());
    const Rows r = rows_of(X);
    const int64_t ldq = pad16(r.n);
    at::Tensor q = allocate({r.rows, ldq}, at::kChar, X.get_device());
    at::Tensor scale = allocate({r.rows}, at::kFloat, X.get_device());
    int8_t* qp = q.mutable_data_ptr<int8_t>();
    float* sp = scale.mutable_data_ptr<float>();
    const externd_stream_t st = stream_of(X.get_device());
    const int rc =
        unlocked([&] { return g_quantize(r.at, type, r.ld, r.rows, r.n, qp, ldq, sp, st); });
    if (rc != EXTERND_OK) return PyLong_FromLong(rc);
    if (ldq != r.n) q = q.narrow(1, 0, r.n);
    PyObject* a = THPVariable_Wrap(std::move(q));
    PyObject* b = a ? THPVariable_Wrap(std::move(scale)) : nullptr;
    PyObject* out = b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return out;
  });
}

// matmul_i8(x, xscale or None, wq, wscale, bias or None, out_dtype or None) -> y,
// or the C status; 8-bit matrices as Quantized holds them
PyObject* matmul_i8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_ok(n, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &W = tensor(args[2], "W"), &ws = tensor(args[3], "scale");
    const c10::DeviceIndex device = W.get_device();
    const c10::cuda::OptionalCUDAGuard guard(W.device());
    const int64_t m = W.size(0), inner = W.size(1);
    const Activations a = activations(args[0], args[1], args[5], inner, m, device);
    at::Tensor bias;
    if (args[4] != Py_None) {
      bias = tensor(args[4], "bias");
      if (bias.scalar_type() != at::kFloat || bias.dim() != 1 || bias.size(0) != m)
        refuse("bias must be fp32 [" + std::to_string(m) + "]");
      if (!bias.is_cuda() || bias.get_device() != device)
        refuse("expected tensors on one CUDA device");
      bias = bias.contiguous().resolve_neg();
    }
    at::Tensor Y = allocate(a.out, a.out_type, device);
    void* yp = Y.mutable_data_ptr();
    const int8_t* wp = W.const_data_ptr<int8_t>();
    const float *wsp = ws.const_data_ptr<float>(),
                *bp = bias.defined() ? bias.const_data_ptr<float>() : nullptr;
    const externd_stream_t st = stream_of(device);
    const int rc = unlocked([&] {
      return g_matmul(a.x.at, a.type, a.x.ld, a.scale, wp, row_bytes(W), wsp, bp, a.x.rows, inner, m,
                      yp, type_of(a.out_type), m, st);
    });
    if (rc != EXTERND_OK) return PyLong_FromLong(rc);
    return THPVariable_Wrap(std::move(Y));
  });
}

// apply_i8(codes_B, codes_C, D, bound, n, x, xscale or None, out_dtype or None)
// -> y, or the C status; codes as FactorCodes holds them
PyObject* apply_i8(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (!count_ok(count, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &B = tensor(args[0], "codes_B"), &C = tensor(args[1], "codes_C"),
                     &D = tensor(args[2], "D"), &bound = tensor(args[3], "bound");
    const int64_t n = PyLong_AsLongLong(args[4]);
    if (PyErr_Occurred()) return nullptr;
    const c10::DeviceIndex device = D.get_device();
    const c10::cuda::OptionalCUDAGuard guard(D.device());
    const int64_t m = B.size(0), k = D.size(0);
    const Activations a = activations(args[5], args[6], args[7], n, m, device);
    at::Tensor Y = allocate(a.out, a.out_type, device);
    void* yp = Y.mutable_data_ptr();
    const uint32_t *cb = (const uint32_t*)B.const_data_ptr<int32_t>(),
                   *cc = (const uint32_t*)C.const_data_ptr<int32_t>();
    const float *d = D.const_data_ptr<float>(), *bp = bound.const_data_ptr<float>();
    const externd_stream_t st = stream_of(device);
    const int rc = unlocked([&] {
      return g_apply(cb, cc, d, bp, m, n, k, a.x.at, a.type, a.x.ld, a.scale, a.x.rows, yp,
                     type_of(a.out_type), m, st);
    });
    if (rc != EXTERND_OK) return PyLong_FromLong(rc);
    return THPVariable_Wrap(std::move(Y));
  });
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
    {"quantize_rows", (PyCFunction)(void*)quantize_rows, METH_FASTCALL, nullptr},
    {"matmul_i8", (PyCFunction)(void*)matmul_i8, METH_FASTCALL, nullptr},
    {"apply_i8", (PyCFunction)(void*)apply_i8, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
