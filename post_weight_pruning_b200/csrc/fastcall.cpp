// The forward operators' usual calls, marshalled without the interpreter: CUDA tensors of one
// type on the current device, no stream, output or gradient asked for.  Each function checks
// what the Python operator of its name checks, allocates the output and calls the C entry
// point; whatever it does not take (errors among them) it leaves to that operator by returning
// None.  A small operator's time is mostly its host side: a row's norm takes 3.6 us
// this way and 10.0 through the Python checks (the launch alone 3.5), a short rotation 4.4 and
// 14.6.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cmath>
#include <cstdint>

#include "pwp.h"

namespace {

// The tensors of one call: each is taken when it is a plain CUDA tensor like the first.
struct Call {
  int device = -1;
  at::ScalarType type = at::ScalarType::Undefined;
  bool recording = c10::GradMode::is_enabled();

  // nullptr: not one of this call's kind
  const at::Tensor* any(PyObject* o, int64_t dims, at::ScalarType want) const {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || !t.has_storage() || t.layout() != at::kStrided || t.is_neg() || t.dim() != dims ||
        t.get_device() != device || t.scalar_type() != want || (recording && t.requires_grad()) ||
        t._fw_grad(/*level=*/0).defined() || t._is_zerotensor())
      return nullptr;
    return t.size(-1) > 1 && t.stride(-1) != 1 ? nullptr : &t;
  }
  const at::Tensor* first(PyObject* o, int64_t dims) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda()) return nullptr;
    device = t.get_device();
    type = t.scalar_type();
    if (device != c10::cuda::current_device() || (type != at::kBFloat16 && type != at::kFloat)) return nullptr;
    return any(o, dims, type);
  }
  // None, or a vector of n elements; false: neither
  bool vector(PyObject* o, int64_t n, const void*& p) const {
    p = nullptr;
    if (o == Py_None) return true;
    const at::Tensor* t = any(o, 1, type);
    if (!t || t->size(0) != n) return false;
    p = t->const_data_ptr();
    return true;
  }
  // None, or a status record
  bool record(PyObject* o, pwp_stats*& p) const {
    p = nullptr;
    if (o == Py_None) return true;
    const at::Tensor* t = any(o, 1, at::kByte);
    if (!t || t->size(0) != (int64_t)sizeof(pwp_stats)) return false;
    p = (pwp_stats*)t->data_ptr();
    return ((uintptr_t)p & 7) == 0;
  }
  int32_t code() const { return type == at::kBFloat16 ? PWP_BF16 : PWP_FP32; }
  at::Tensor empty(at::IntArrayRef size) const {
    return at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)device), c10::nullopt);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
};

// A finite Python float (or int) in fp32.
bool number(PyObject* o, float& x) {
  if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o)) return false;
  const double d = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  x = (float)d;
  return std::isfinite(x);
}

PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {      // x, weight, eps
  HANDLE_TH_ERRORS
  Call c;
  const at::Tensor* x = n == 3 ? c.first(a[0], 2) : nullptr;
  const void* w;
  float eps;
  if (!x || !number(a[2], eps) || eps < 0.f || !c.vector(a[1], x->size(1), w)) Py_RETURN_NONE;
  const int64_t rows = x->size(0), width = x->size(1);
  if (rows < 1 || width < 1 || width > 65536) Py_RETURN_NONE;
  at::Tensor out = c.empty({rows, width});
  if (pwp_rms_norm(x->const_data_ptr(), c.code(), rows, (int32_t)width, x->stride(0), w, eps, out.data_ptr(), width,
                   c.stream()) != PWP_OK)
    Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// q, k, positions, freqs, q_weight, k_weight, eps, layout, factor
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  const at::Tensor* q = n == 9 ? c.first(a[0], 3) : nullptr;
  const at::Tensor *k = q ? c.any(a[1], 3, c.type) : nullptr, *p = k ? c.any(a[2], 1, at::kLong) : nullptr,
                   *f = p ? c.any(a[3], 1, at::kDouble) : nullptr;
  if (!f || !PyLong_CheckExact(a[7])) Py_RETURN_NONE;
  const int64_t tokens = q->size(0), d = q->size(2), rot = 2 * f->size(0);
  pwp_rope_args r = {};
  if (tokens < 1 || q->size(1) < 1 || k->size(1) < 1 || q->size(1) > 65536 || k->size(1) > 65536 || d < 1 || d > 1024 ||
      rot > d || k->size(0) != tokens || k->size(2) != d || p->size(0) != tokens || !number(a[6], r.eps) ||
      r.eps < 0.f || !number(a[8], r.factor) || !c.vector(a[4], d, r.q_weight_dev) || !c.vector(a[5], d, r.k_weight_dev))
    Py_RETURN_NONE;
  r.n = tokens;
  r.type = c.code();
  r.hq = (int32_t)q->size(1);
  r.hk = (int32_t)k->size(1);
  r.d = (int32_t)d;
  r.rot = (int32_t)rot;
  r.layout = (int32_t)PyLong_AsLong(a[7]);
  at::Tensor qo = c.empty({tokens, r.hq, d}), ko = c.empty({tokens, r.hk, d});
  r.q_dev = q->const_data_ptr();
  r.k_dev = k->const_data_ptr();
  r.q_out_dev = qo.data_ptr();
  r.k_out_dev = ko.data_ptr();
  r.positions_dev = (const int64_t*)p->const_data_ptr();
  r.freqs_dev = (const double*)f->const_data_ptr();
  for (int i = 0; i < 2; ++i) {
    r.q_stride[i] = q->stride(i);
    r.k_stride[i] = k->stride(i);
    r.q_out_stride[i] = qo.stride(i);
    r.k_out_stride[i] = ko.stride(i);
  }
  if (pwp_qk_norm_rope(&r, c.stream()) != PWP_OK) Py_RETURN_NONE;
  PyObject* out[2] = {THPVariable_Wrap(std::move(qo)), THPVariable_Wrap(std::move(ko))};
  PyObject* both = out[0] && out[1] ? PyTuple_Pack(2, out[0], out[1]) : nullptr;
  Py_XDECREF(out[0]);
  Py_XDECREF(out[1]);
  return both;
  END_HANDLE_TH_ERRORS
}

// q, k, v, cu_seqlens, causal, scale (or None), stats
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  const at::Tensor* q = n == 7 ? c.first(a[0], 3) : nullptr;
  const at::Tensor *k = q ? c.any(a[1], 3, c.type) : nullptr, *v = k ? c.any(a[2], 3, c.type) : nullptr,
                   *cu = v ? c.any(a[3], 1, at::kInt) : nullptr;
  if (!cu || !PyBool_Check(a[4])) Py_RETURN_NONE;
  const int64_t tokens = q->size(0), hq = q->size(1), d = q->size(2), hk = k->size(1);
  pwp_attention_args r = {};
  if (tokens < 1 || hk < 1 || hq < 1 || hq % hk || d < 1 || d > 256 || tokens * hq >= (1LL << 31) || hq > (1 << 24) ||
      k->size(0) != tokens || k->size(2) != d || !v->sizes().equals(k->sizes()) || cu->size(0) < 2 ||
      cu->size(0) > (1 << 24) || !c.record(a[6], r.stats_dev))
    Py_RETURN_NONE;
  if (a[5] == Py_None)
    r.scale = (float)std::pow((double)d, -0.5);
  else if (!number(a[5], r.scale))
    Py_RETURN_NONE;
  at::Tensor out = c.empty(q->sizes());
  r.q_dev = q->const_data_ptr();
  r.k_dev = k->const_data_ptr();
  r.v_dev = v->const_data_ptr();
  r.out_dev = out.data_ptr();
  for (int i = 0; i < 2; ++i) {
    r.q_stride[i] = q->stride(i);
    r.k_stride[i] = k->stride(i);
    r.v_stride[i] = v->stride(i);
    r.out_stride[i] = out.stride(i);
  }
  r.cu_seqlens_dev = (const int32_t*)cu->const_data_ptr();
  r.n = tokens;
  r.nseq = (int32_t)cu->size(0) - 1;
  r.type = c.code();
  r.hq = (int32_t)hq;
  r.hk = (int32_t)hk;
  r.d = (int32_t)d;
  r.causal = a[4] == Py_True;
  at::Tensor scratch;
  const size_t need = pwp_attention_workspace_bytes(&r);
  if (need) {
    scratch = at::detail::empty_cuda({(int64_t)need}, at::kByte, q->device(), c10::nullopt);
    r.ws_dev = scratch.data_ptr();
    r.ws_bytes = need;
  }
  if (pwp_attention(&r, c.stream()) != PWP_OK) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// x, w, w_up (or None), bias, bias_up, activation, residual, stats
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  const at::Tensor* x = n == 8 ? c.first(a[0], 2) : nullptr;
  const at::Tensor *w = x ? c.any(a[1], 2, c.type) : nullptr, *up = nullptr, *res = nullptr;
  if (!w || !PyLong_CheckExact(a[5])) Py_RETURN_NONE;
  const int64_t rows = x->size(0), k = x->size(1), cols = w->size(0);
  pwp_linear_args r = {};
  if (rows < 1 || rows >= (1LL << 31) || k < 1 || k >= (1 << 24) || cols < 1 || cols >= (1 << 24) || w->size(1) != k ||
      !c.vector(a[3], cols, r.bias_dev) || !c.vector(a[4], cols, r.bias_up_dev) || !c.record(a[7], r.stats_dev))
    Py_RETURN_NONE;
  if (a[2] != Py_None && !((up = c.any(a[2], 2, c.type)) && up->sizes().equals(w->sizes()))) Py_RETURN_NONE;
  if (a[6] != Py_None && !((res = c.any(a[6], 2, c.type)) && res->size(0) == rows && res->size(1) == cols))
    Py_RETURN_NONE;
  r.x_dev = x->const_data_ptr();
  r.w_dev = w->const_data_ptr();
  r.w_up_dev = up ? up->const_data_ptr() : nullptr;
  r.residual_dev = res ? res->const_data_ptr() : nullptr;
  r.x_stride = x->stride(0);
  r.w_stride = w->stride(0);
  r.w_up_stride = up ? up->stride(0) : 0;
  r.residual_stride = res ? res->stride(0) : 0;
  r.out_stride = cols;
  r.rows = rows;
  r.k = (int32_t)k;
  r.n = (int32_t)cols;
  r.type = c.code();
  r.activation = (int32_t)PyLong_AsLong(a[5]);
  at::Tensor out = c.empty({rows, cols}), scratch;
  r.out_dev = out.data_ptr();
  const size_t need = pwp_linear_workspace_bytes(&r);
  if (need) {
    scratch = at::detail::empty_cuda({(int64_t)need}, at::kByte, x->device(), c10::nullopt);
    r.ws_dev = scratch.data_ptr();
    r.ws_bytes = need;
  }
  if (pwp_linear(&r, c.stream()) != PWP_OK) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rms_norm", (PyCFunction)(void (*)(void))rms_norm, METH_FASTCALL, nullptr},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
    {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
  PyObject* m = PyModule_Create(&module);
  // the PyTorch whose tensors it knows
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
