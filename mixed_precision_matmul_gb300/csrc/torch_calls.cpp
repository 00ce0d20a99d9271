// The torch forms' plain calls (CPython extension `_torch_calls`): reading a
// tensor's pointer, sizes and strides and allocating results takes the host
// 8 us of the 14 us of a call from Python, and 1 us from here; a product for
// one token takes the GPU 5 to 12 us.  Only marshalling: the work is the C
// ABI's, whose functions' addresses init() receives.
//
// Each function takes what the Python form has resolved (no defaults, no
// names) and returns None for anything that is not a plain call on the current
// device; the Python form then checks the arguments one by one and says what
// is wrong.  A status other than MPG_OK is returned as a number.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mpgemm.h"

namespace {

decltype(&mpg_gemm_fp8) g_gemm = nullptr;
decltype(&mpg_gemm_fp8_workspace_size) g_gemm_workspace = nullptr;
decltype(&mpg_fp8_quantize) g_quantize = nullptr;
mpg_options g_options[3];

constexpr int64_t kBlock = 128;
constexpr at::ScalarType kTypes[3] = {at::kFloat, at::kHalf, at::kBFloat16};   // by mpg_dtype

int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

bool tensor(PyObject* o, at::Tensor* t) {
  if (!THPVariable_Check(o)) return false;
  *t = THPVariable_Unpack(o);
  return t->is_cuda() && t->dim() == 2 && t->layout() == at::kStrided;
}

// An 8-bit matrix and its scales; false unless a plain one on device `dev`.
bool operand(PyObject* po, PyObject* ps, c10::DeviceIndex dev, at::Tensor* t, at::Tensor* s, mpg_fp8_operand* x) {
  if (!tensor(po, t) || !tensor(ps, s) || t->get_device() != dev || s->get_device() != dev) return false;
  const int64_t rows = t->size(0), k = t->size(1);
  if (rows < 1 || k < 1 || t->stride(1) != 1 || (rows > 1 && t->stride(0) < k)) return false;
  if (s->scalar_type() != at::kFloat || s->size(1) != blocks(k)) return false;
  if (t->scalar_type() == at::kFloat8_e4m3fn) x->format = MPG_E4M3;
  else if (t->scalar_type() == at::kFloat8_e5m2) x->format = MPG_E5M2;
  else return false;
  if (s->size(0) == rows) x->scale_rows = 1;
  else if (s->size(0) == blocks(rows)) x->scale_rows = kBlock;
  else return false;
  x->data = t->data_ptr();
  x->ld = rows > 1 ? t->stride(0) : k;
  x->scale = static_cast<const float*>(s->data_ptr());
  x->scale_row_stride = s->stride(0);
  x->scale_k_stride = s->stride(1);
  return true;
}

PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3) return PyErr_Format(PyExc_TypeError, "three addresses are expected");
  g_gemm = reinterpret_cast<decltype(g_gemm)>(PyLong_AsVoidPtr(args[0]));
  g_gemm_workspace = reinterpret_cast<decltype(g_gemm_workspace)>(PyLong_AsVoidPtr(args[1]));
  g_quantize = reinterpret_cast<decltype(g_quantize)>(PyLong_AsVoidPtr(args[2]));
  if (PyErr_Occurred()) return nullptr;
  for (int i = 0; i < 3; ++i) {
    g_options[i] = mpg_options{};
    g_options[i].c_dtype = i;
  }
  Py_RETURN_NONE;
}

// (A, a_scale, B, b_scale, alpha, mpg_dtype of C) -> C
PyObject* gemm_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 6 || !g_gemm) return PyErr_Format(PyExc_TypeError, "six arguments are expected");
  try {
    at::Tensor a, sa, b, sb;
    mpg_fp8_operand xa, xb;
    if (!tensor(args[0], &a)) Py_RETURN_NONE;
    const c10::DeviceIndex dev = c10::cuda::current_device();
    if (!operand(args[0], args[1], dev, &a, &sa, &xa) || !operand(args[2], args[3], dev, &b, &sb, &xb) ||
        a.size(1) != b.size(1))
      Py_RETURN_NONE;
    const double alpha = PyFloat_AsDouble(args[4]);
    const long type = PyLong_AsLong(args[5]);
    if (PyErr_Occurred()) return nullptr;
    if (type < 0 || type > 2) Py_RETURN_NONE;
    const int64_t rows = a.size(0), cols = b.size(0), k = a.size(1);
    at::Tensor c = at::empty({rows, cols}, a.options().dtype(kTypes[type]));
    at::Tensor ws;
    const size_t bytes = g_gemm_workspace(rows, cols, k, &xa, &xb);
    if (bytes) ws = at::empty({(int64_t)bytes}, a.options().dtype(at::kByte));
    const mpg_status st = g_gemm(rows, cols, k, &xa, &xb, c.data_ptr(), cols, (float)alpha, 0.0f,
                                 bytes ? ws.data_ptr() : nullptr, bytes,
                                 c10::cuda::getCurrentCUDAStream(dev).stream(), &g_options[type]);
    return st == MPG_OK ? THPVariable_Wrap(std::move(c)) : PyLong_FromLong(st);
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}

struct Form {
  at::Tensor q, s;
  int64_t ld, row, k;
};

// Codes on 16-byte lines and scales of a rows x cols matrix, as the Python form lays them.
Form form(int64_t rows, int64_t cols, at::ScalarType code, bool by_row, const at::TensorOptions& o) {
  Form f;
  f.ld = (cols + 15) / 16 * 16;
  f.q = at::empty_strided({rows, cols}, {f.ld, 1}, o.dtype(code));
  const int64_t kb = blocks(cols);
  f.row = by_row ? 1 : kb;
  f.k = by_row ? rows : 1;
  f.s = at::empty_strided({by_row ? rows : blocks(rows), kb}, {f.row, f.k}, o.dtype(at::kFloat));
  return f;
}

// (x, format, scale_rows, transpose) -> (q, s) or (q, s, qt, st)
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4 || !g_quantize) return PyErr_Format(PyExc_TypeError, "four arguments are expected");
  try {
    at::Tensor x;
    if (!tensor(args[0], &x)) Py_RETURN_NONE;
    const c10::DeviceIndex dev = c10::cuda::current_device();
    if (x.get_device() != dev) Py_RETURN_NONE;
    const long format = PyLong_AsLong(args[1]), scale_rows = PyLong_AsLong(args[2]);
    const int transpose = PyObject_IsTrue(args[3]);
    if (PyErr_Occurred()) return nullptr;
    int type = 0;
    while (type < 3 && x.scalar_type() != kTypes[type]) ++type;
    const int64_t rows = x.size(0), cols = x.size(1);
    if (type == 3 || rows < 1 || cols < 1 || x.stride(1) != 1 || (rows > 1 && x.stride(0) < cols)) Py_RETURN_NONE;
    const at::ScalarType code = format == MPG_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2;
    const at::TensorOptions o = at::TensorOptions().device(x.device());
    Form f = form(rows, cols, code, scale_rows == 1, o), t{};
    if (transpose) t = form(cols, rows, code, scale_rows == 1, o);
    const mpg_status st = g_quantize(
        rows, cols, x.data_ptr(), rows > 1 ? x.stride(0) : cols, (mpg_dtype)type, (mpg_fp8_format)format,
        (int32_t)scale_rows, f.q.data_ptr(), f.ld, static_cast<float*>(f.s.data_ptr()), f.row, f.k,
        transpose ? t.q.data_ptr() : nullptr, t.ld, transpose ? static_cast<float*>(t.s.data_ptr()) : nullptr, t.row, t.k,
        c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != MPG_OK) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(transpose ? 4 : 2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(f.q)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(f.s)));
    if (transpose) {
      PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(t.q)));
      PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(std::move(t.s)));
    }
    return r;
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}

PyMethodDef g_methods[] = {
    {"init", reinterpret_cast<PyCFunction>(init), METH_FASTCALL, "addresses of the C ABI's functions"},
    {"gemm_fp8", reinterpret_cast<PyCFunction>(gemm_fp8), METH_FASTCALL, "mpg_gemm_fp8 on torch tensors"},
    {"quantize", reinterpret_cast<PyCFunction>(quantize), METH_FASTCALL, "mpg_fp8_quantize on torch tensors"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&g_module); }
