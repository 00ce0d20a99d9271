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

#include <vector>

#include "mpgemm.h"

namespace {

decltype(&mpg_gemm_fp8) g_gemm = nullptr;
decltype(&mpg_gemm_fp8_workspace_size) g_gemm_workspace = nullptr;
decltype(&mpg_fp8_quantize) g_quantize = nullptr;
decltype(&mpg_gated_gemm) g_gated = nullptr;
decltype(&mpg_gated_gemm_workspace_size) g_gated_workspace = nullptr;
decltype(&mpg_gated_gemm_backward) g_gated_back = nullptr;
decltype(&mpg_gated_gemm_backward_workspace_size) g_gated_back_workspace = nullptr;
decltype(&mpg_linear_cross_entropy) g_loss = nullptr;
decltype(&mpg_linear_cross_entropy_workspace_size) g_loss_workspace = nullptr;
decltype(&mpg_linear_cross_entropy_backward) g_loss_back = nullptr;
decltype(&mpg_linear_cross_entropy_backward_workspace_size) g_loss_back_workspace = nullptr;
decltype(&mpg_clip_grad_norm) g_clip = nullptr;
decltype(&mpg_clip_grad_norm_workspace_size) g_clip_workspace = nullptr;
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
  if (n != 13) return PyErr_Format(PyExc_TypeError, "thirteen addresses are expected");
  int i = 0;
  auto take = [&](auto& f) { f = reinterpret_cast<std::decay_t<decltype(f)>>(PyLong_AsVoidPtr(args[i++])); };
  take(g_gemm);
  take(g_gemm_workspace);
  take(g_quantize);
  take(g_gated);
  take(g_gated_workspace);
  take(g_gated_back);
  take(g_gated_back_workspace);
  take(g_loss);
  take(g_loss_workspace);
  take(g_loss_back);
  take(g_loss_back_workspace);
  take(g_clip);
  take(g_clip_workspace);
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

// A 16-bit matrix of the given type on device `dev` (rows, cols: -1 for any).
bool matrix16(PyObject* o, c10::DeviceIndex dev, at::ScalarType type, int64_t rows, int64_t cols, at::Tensor* t, int64_t* ld) {
  if (!tensor(o, t) || t->get_device() != dev || t->scalar_type() != type) return false;
  const int64_t r = t->size(0), c = t->size(1);
  if (r < 1 || c < 1 || (rows >= 0 && r != rows) || (cols >= 0 && c != cols)) return false;
  if ((c > 1 && t->stride(1) != 1) || (r > 1 && t->stride(0) < c)) return false;
  *ld = r > 1 ? t->stride(0) : c;
  return true;
}
at::Tensor scratch(size_t bytes, const at::Tensor& like) { return at::empty({(int64_t)bytes}, like.options().dtype(at::kByte)); }
void* address(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The first `n` of a call's results (None for one that is not there).
PyObject* results(at::Tensor* t, int n) {
  PyObject* r = PyTuple_New(n);
  if (!r) return nullptr;
  for (int i = 0; i < n; ++i) {
    if (t[i].defined()) {
      PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(t[i])));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, i, Py_None);
    }
  }
  return r;
}

// X, Wg and Wu of a layer; false unless plain ones on the current device.
bool layer_of(PyObject* px, PyObject* pg, PyObject* pu, long act, at::Tensor* x, at::Tensor* wg, at::Tensor* wu,
              c10::DeviceIndex* dev, mpg_gated_layer* l) {
  if (!tensor(px, x)) return false;
  *dev = c10::cuda::current_device();
  const at::ScalarType type = x->scalar_type();
  if (type != at::kHalf && type != at::kBFloat16) return false;
  if (!matrix16(px, *dev, type, -1, -1, x, &l->ldx) || !matrix16(pg, *dev, type, -1, x->size(1), wg, &l->ldwg) ||
      !matrix16(pu, *dev, type, wg->size(0), x->size(1), wu, &l->ldwu))
    return false;
  l->tokens = x->size(0);
  l->hidden = x->size(1);
  l->inner = wg->size(0);
  l->dtype = type == at::kHalf ? MPG_F16 : MPG_BF16;
  l->act = (mpg_activation)act;
  l->x = x->data_ptr();
  l->wg = wg->data_ptr();
  l->wu = wu->data_ptr();
  return true;
}

// Of what a layer keeps for its gradients: fp16, or codes in a bf16 layer.
at::ScalarType kept_type(const at::Tensor& x) { return x.scalar_type() == at::kHalf ? at::kHalf : at::kShort; }

// (x, wg, wu, activation, keep) -> y or (y, a, b)
PyObject* gated_gemm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5 || !g_gated) return PyErr_Format(PyExc_TypeError, "five arguments are expected");
  try {
    const long act = PyLong_AsLong(args[3]);
    const int keep = PyObject_IsTrue(args[4]);
    if (PyErr_Occurred()) return nullptr;
    at::Tensor x, wg, wu, out[3];
    c10::DeviceIndex dev;
    mpg_gated_layer l;
    if (!layer_of(args[0], args[1], args[2], act, &x, &wg, &wu, &dev, &l)) Py_RETURN_NONE;
    for (int i = 0; i < (keep ? 3 : 1); ++i)
      out[i] = at::empty({l.tokens, l.inner}, x.options().dtype(i ? kept_type(x) : x.scalar_type()));
    const size_t bytes = g_gated_workspace(&l);
    const at::Tensor ws = bytes ? scratch(bytes, x) : at::Tensor();
    const mpg_status st = g_gated(&l, address(out[0]), l.inner, address(out[1]), l.inner, address(out[2]), l.inner,
                                  address(ws), bytes, c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != MPG_OK) return PyLong_FromLong(st);
    return keep ? results(out, 3) : THPVariable_Wrap(std::move(out[0]));
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}

// (dy, x, wg, wu, activation, a, b, need_dx, need_dw) -> (dx, dwg, dwu)
PyObject* gated_gemm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 9 || !g_gated_back) return PyErr_Format(PyExc_TypeError, "nine arguments are expected");
  try {
    const long act = PyLong_AsLong(args[4]);
    const int need_dx = PyObject_IsTrue(args[7]), need_dw = PyObject_IsTrue(args[8]);
    if (PyErr_Occurred()) return nullptr;
    at::Tensor dy, x, wg, wu, a, b, out[3];
    c10::DeviceIndex dev;
    mpg_gated_layer l;
    int64_t lddy = 0, lda = 0, ldb = 0;
    if (!layer_of(args[1], args[2], args[3], act, &x, &wg, &wu, &dev, &l)) Py_RETURN_NONE;
    if (!matrix16(args[0], dev, x.scalar_type(), l.tokens, l.inner, &dy, &lddy)) Py_RETURN_NONE;
    if (args[5] != Py_None || args[6] != Py_None)
      if (!matrix16(args[5], dev, kept_type(x), l.tokens, l.inner, &a, &lda) ||
          !matrix16(args[6], dev, kept_type(x), l.tokens, l.inner, &b, &ldb))
        Py_RETURN_NONE;
    if (need_dx) out[0] = at::empty({l.tokens, l.hidden}, x.options());
    for (int i = 1; i < 3 && need_dw; ++i) out[i] = at::empty({l.inner, l.hidden}, x.options());
    const size_t bytes = g_gated_back_workspace(&l);
    const at::Tensor ws = bytes ? scratch(bytes, x) : at::Tensor();
    const mpg_status st = g_gated_back(&l, address(dy), lddy, address(a), lda, address(b), ldb, address(out[0]), l.hidden,
                                       address(out[1]), l.hidden, address(out[2]), l.hidden, address(ws), bytes,
                                       c10::cuda::getCurrentCUDAStream(dev).stream());
    return st == MPG_OK ? results(out, 3) : PyLong_FromLong(st);
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}

// X, W and the targets; false unless plain ones on the current device.
bool loss_of(PyObject* px, PyObject* pw, PyObject* pt, PyObject* ignore, at::Tensor* x, at::Tensor* w, at::Tensor* t,
             c10::DeviceIndex* dev, mpg_vocab_loss* l) {
  if (!tensor(px, x) || !THPVariable_Check(pt)) return false;
  *dev = c10::cuda::current_device();
  const at::ScalarType type = x->scalar_type();
  if (type != at::kHalf && type != at::kBFloat16) return false;
  if (!matrix16(px, *dev, type, -1, -1, x, &l->ldx) || !matrix16(pw, *dev, type, -1, x->size(1), w, &l->ldw)) return false;
  *t = THPVariable_Unpack(pt);
  if (!t->is_cuda() || t->layout() != at::kStrided || t->get_device() != *dev || t->dim() != 1 || t->size(0) != x->size(0)) return false;
  if (t->scalar_type() != at::kLong && t->scalar_type() != at::kInt) return false;
  l->tokens = x->size(0);
  l->hidden = x->size(1);
  l->vocab = w->size(0);
  l->dtype = type == at::kHalf ? MPG_F16 : MPG_BF16;
  l->x = x->data_ptr();
  l->w = w->data_ptr();
  l->target = t->data_ptr();
  l->target_bytes = t->scalar_type() == at::kLong ? 8 : 4;
  l->target_stride = t->stride(0);
  l->ignore_index = PyLong_AsLongLong(ignore);
  return true;
}

// (x, w, target, ignore_index) -> (loss, lse)
PyObject* linear_cross_entropy(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4 || !g_loss) return PyErr_Format(PyExc_TypeError, "four arguments are expected");
  try {
    at::Tensor x, w, t, out[2];
    c10::DeviceIndex dev;
    mpg_vocab_loss l;
    if (!loss_of(args[0], args[1], args[2], args[3], &x, &w, &t, &dev, &l)) Py_RETURN_NONE;
    if (PyErr_Occurred()) return nullptr;
    for (at::Tensor& o : out) o = at::empty({l.tokens}, x.options().dtype(at::kFloat));
    const size_t bytes = g_loss_workspace(&l);
    const at::Tensor ws = bytes ? scratch(bytes, x) : at::Tensor();
    const mpg_status st = g_loss(&l, static_cast<float*>(out[0].data_ptr()), static_cast<float*>(out[1].data_ptr()),
                                 address(ws), bytes, c10::cuda::getCurrentCUDAStream(dev).stream());
    return st == MPG_OK ? results(out, 2) : PyLong_FromLong(st);
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}

// One fp32 number for each of `tokens` on device `dev`.
bool vector32(PyObject* o, c10::DeviceIndex dev, int64_t tokens, at::Tensor* t) {
  if (!THPVariable_Check(o)) return false;
  *t = THPVariable_Unpack(o);
  return t->is_cuda() && t->layout() == at::kStrided && t->get_device() == dev && t->dim() == 1 && t->size(0) == tokens &&
         t->scalar_type() == at::kFloat;
}

// (x, w, target, lse, dloss, ignore_index, need_dx, need_dw) -> (dx, dw)
PyObject* linear_cross_entropy_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 8 || !g_loss_back) return PyErr_Format(PyExc_TypeError, "eight arguments are expected");
  try {
    const int need_dx = PyObject_IsTrue(args[6]), need_dw = PyObject_IsTrue(args[7]);
    if (PyErr_Occurred()) return nullptr;
    at::Tensor x, w, t, lse, dloss, out[2];
    c10::DeviceIndex dev;
    mpg_vocab_loss l;
    if (!loss_of(args[0], args[1], args[2], args[5], &x, &w, &t, &dev, &l)) Py_RETURN_NONE;
    if (PyErr_Occurred()) return nullptr;
    if (!vector32(args[3], dev, l.tokens, &lse) || !vector32(args[4], dev, l.tokens, &dloss) ||
        (l.tokens > 1 && lse.stride(0) != 1))
      Py_RETURN_NONE;
    if (need_dx) out[0] = at::empty({l.tokens, l.hidden}, x.options());
    if (need_dw) out[1] = at::empty({l.vocab, l.hidden}, x.options());
    const size_t bytes = g_loss_back_workspace(&l);
    const at::Tensor ws = bytes ? scratch(bytes, x) : at::Tensor();
    const mpg_status st = g_loss_back(&l, static_cast<const float*>(lse.data_ptr()), static_cast<const float*>(dloss.data_ptr()),
                                      dloss.stride(0), address(out[0]), l.hidden, address(out[1]), l.hidden, address(ws),
                                      bytes, c10::cuda::getCurrentCUDAStream(dev).stream());
    return st == MPG_OK ? results(out, 2) : PyLong_FromLong(st);
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}

// A gradient and its result, packed alike; false for anything else.
bool grad_of(PyObject* pg, PyObject* po, c10::DeviceIndex dev, mpg_grad* x) {
  if (!THPVariable_Check(pg) || !THPVariable_Check(po)) return false;
  const at::Tensor &g = THPVariable_Unpack(pg), &o = THPVariable_Unpack(po);
  for (const at::Tensor* t : {&g, &o})
    if (!t->is_cuda() || t->layout() != at::kStrided || t->get_device() != dev || !t->is_contiguous()) return false;
  if (g.sizes() != o.sizes()) return false;
  int tg = 0, to = 0;
  while (tg < 3 && g.scalar_type() != kTypes[tg]) ++tg;
  while (to < 3 && o.scalar_type() != kTypes[to]) ++to;
  if (tg == 3 || to == 3) return false;
  *x = mpg_grad{g.data_ptr(), o.data_ptr(), g.numel(), (mpg_dtype)tg, (mpg_dtype)to};
  return true;
}

// (gradients, results, max_norm, eps) -> norm; both lists or tuples of one length
PyObject* clip_grad_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4 || !g_clip) return PyErr_Format(PyExc_TypeError, "four arguments are expected");
  try {
    const double max_norm = PyFloat_AsDouble(args[2]), eps = PyFloat_AsDouble(args[3]);
    if (PyErr_Occurred()) return nullptr;
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(args[0]);
    if (count < 1 || PySequence_Fast_GET_SIZE(args[1]) != count) Py_RETURN_NONE;
    PyObject* first = PySequence_Fast_GET_ITEM(args[0], 0);
    if (!THPVariable_Check(first) || !THPVariable_Unpack(first).is_cuda()) Py_RETURN_NONE;
    const c10::DeviceIndex dev = c10::cuda::current_device();
    std::vector<mpg_grad> table((size_t)count);
    for (Py_ssize_t i = 0; i < count; ++i)
      if (!grad_of(PySequence_Fast_GET_ITEM(args[0], i), PySequence_Fast_GET_ITEM(args[1], i), dev, &table[(size_t)i]))
        Py_RETURN_NONE;
    const at::TensorOptions o = at::TensorOptions().device(at::kCUDA, dev);
    at::Tensor norm = at::empty({}, o.dtype(at::kFloat));
    const size_t bytes = g_clip_workspace(count, table.data());
    const at::Tensor ws = at::empty({(int64_t)bytes}, o.dtype(at::kByte));
    const mpg_status st = g_clip(count, table.data(), (float)max_norm, (float)eps, static_cast<float*>(norm.data_ptr()),
                                 ws.data_ptr(), bytes, c10::cuda::getCurrentCUDAStream(dev).stream());
    return st == MPG_OK ? THPVariable_Wrap(std::move(norm)) : PyLong_FromLong(st);
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}

PyMethodDef g_methods[] = {
    {"init", reinterpret_cast<PyCFunction>(init), METH_FASTCALL, "addresses of the C ABI's functions"},
    {"gemm_fp8", reinterpret_cast<PyCFunction>(gemm_fp8), METH_FASTCALL, "mpg_gemm_fp8 on torch tensors"},
    {"quantize", reinterpret_cast<PyCFunction>(quantize), METH_FASTCALL, "mpg_fp8_quantize on torch tensors"},
    {"gated_gemm", reinterpret_cast<PyCFunction>(gated_gemm), METH_FASTCALL, "mpg_gated_gemm on torch tensors"},
    {"gated_gemm_backward", reinterpret_cast<PyCFunction>(gated_gemm_backward), METH_FASTCALL,
     "mpg_gated_gemm_backward on torch tensors"},
    {"linear_cross_entropy", reinterpret_cast<PyCFunction>(linear_cross_entropy), METH_FASTCALL,
     "mpg_linear_cross_entropy on torch tensors"},
    {"linear_cross_entropy_backward", reinterpret_cast<PyCFunction>(linear_cross_entropy_backward), METH_FASTCALL,
     "mpg_linear_cross_entropy_backward on torch tensors"},
    {"clip_grad_norm", reinterpret_cast<PyCFunction>(clip_grad_norm), METH_FASTCALL, "mpg_clip_grad_norm on torch tensors"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&g_module); }
