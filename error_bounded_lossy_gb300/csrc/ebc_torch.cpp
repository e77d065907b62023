// ebc_torch.cpp -- the expert-parallel and 4-bit calls on torch tensors: checks
// of the tensors, outputs from torch's allocator on the current stream, and the
// C calls of include/ebc.h.  A module of plain functions, called from
// experts.py.
//
// It is compiled because a decode step is a handful of calls of a few
// microseconds each: the same marshalling in Python and ctypes took 11 to 22 us
// a call on the Grace host (12.6 us for ebc_moe_dispatch, of which the launch
// itself was 2), more than the kernels.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ebc.h"

namespace {

PyObject* g_raise = nullptr;   // raises EbcError(code, name)

// Thrown with the Python error set.
struct Raised {};

[[noreturn]] void bad(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  throw Raised{};
}

void checked(int rc, const char* name) {
  if (rc == EBC_OK) return;
  PyObject* r = PyObject_CallFunction(g_raise, "is", rc, name);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) bad(what);
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

int type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return EBC_F32;
    case at::kBFloat16: return EBC_BF16;
    case at::kHalf: return EBC_F16;
    default: return -1;
  }
}

at::ScalarType scalar_of(int64_t type) {
  if (type == EBC_F32) return at::kFloat;
  if (type == EBC_BF16) return at::kBFloat16;
  if (type == EBC_F16) return at::kHalf;
  bad("the type must be float32, bfloat16 or float16");
}

// Several outputs of one call in one allocation, each on a 16-byte boundary:
// an allocation costs as much as half a launch.  (So one of them keeps the
// memory of all.)
struct Parts {
  at::Tensor whole;
  at::Tensor take(int64_t at, at::IntArrayRef shape, at::ScalarType type) const {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                     c10::scalarTypeToTypeMeta(type));
    impl->set_storage_offset(at / (int64_t)c10::elementSize(type));
    impl->set_sizes_contiguous(shape);
    return at::Tensor(std::move(impl));
  }
};
int64_t pad16(int64_t n) { return (n + 15) & ~(int64_t)15; }

// The context's handle and device: the first two arguments of every call.
struct Where {
  ebc_ctx* ctx;
  c10::DeviceIndex device;
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
  void here(const at::Tensor& t) const {
    if (!t.is_cuda() || t.device().index() != device) bad("a tensor is not on the operators' CUDA device");
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, device), std::nullopt));
  }
};

Where where(PyObject* const* a) {
  void* p = PyLong_AsVoidPtr(a[0]);
  if (!p && PyErr_Occurred()) throw Raised{};
  if (!p) bad("the operators were closed");
  return Where{(ebc_ctx*)p, (c10::DeviceIndex)integer(a[1])};
}

struct Rows {
  const at::Tensor& t;
  int type;
  int64_t n, width, ld;
};

// The gradients are for the reverse mode (experts.py).
void no_tangent(const at::Tensor& t) {
  if (t._fw_grad(0).defined()) bad("forward-mode derivatives of these calls are not defined");
}

// A float tensor [rows, width] with contiguous rows; a single row, or none,
// has no stride of its own.
Rows rows(const Where& w, PyObject* o) {
  const char* what = "rows must be a float32, bfloat16 or float16 CUDA tensor [rows, width] with contiguous rows";
  const at::Tensor& t = tensor(o, what);
  const int type = type_of(t);
  if (type < 0 || !t.is_cuda() || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1)) bad(what);
  w.here(t);
  const int64_t n = t.size(0), width = t.size(1);
  return Rows{t, type, n, width, n > 1 ? t.stride(0) : width};
}

void plan_tensor(const at::Tensor& t) {
  if (t.scalar_type() != at::kInt || !t.is_cuda() || !t.is_contiguous())
    bad("a plan's tensors are contiguous int32 CUDA tensors");
}

struct PlanRef {
  const at::Tensor &rows, &place, &offsets;
  int64_t tokens, top, n, experts;
  const int32_t* place_ptr() const { return (const int32_t*)place.data_ptr(); }
  const int32_t* offsets_ptr() const { return (const int32_t*)offsets.data_ptr(); }
};

// rows, place and offsets of a plan.
PlanRef plan_of(PyObject* const* a) {
  const char* what = "a plan has rows [n], place [tokens, top] and offsets [n_experts + 1]";
  const at::Tensor &r = tensor(a[0], what), &p = tensor(a[1], what), &o = tensor(a[2], what);
  if (r.dim() != 1 || p.dim() != 2 || o.dim() != 1 || o.numel() < 2 || r.numel() != p.numel()) bad(what);
  plan_tensor(r);
  plan_tensor(p);
  plan_tensor(o);
  return PlanRef{r, p, o, p.size(0), p.size(1), r.numel(), o.numel() - 1};
}

PlanRef plan_here(const Where& w, PyObject* const* a) {
  const PlanRef p = plan_of(a);
  w.here(p.place);
  w.here(p.offsets);
  return p;
}

const float* weights_of(const Where& w, PyObject* o, const PlanRef& p) {
  const char* what = "weights must be a contiguous float32 CUDA tensor [tokens, top]";
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kFloat || !t.is_contiguous() || t.sizes() != p.place.sizes()) bad(what);
  w.here(t);
  no_tangent(t);
  return (const float*)t.data_ptr();
}

struct Mx4Ref {
  const at::Tensor &codes, &scales;
  int64_t width;
  const uint8_t* codes_ptr() const { return (const uint8_t*)codes.data_ptr(); }
  const uint8_t* scales_ptr() const { return (const uint8_t*)scales.data_ptr(); }
};

// codes, scales and width of rows in 4 bits.
Mx4Ref mx4_of(PyObject* const* a) {
  const char* what = "codes and scales must be contiguous uint8 CUDA tensors";
  const at::Tensor &c = tensor(a[0], what), &s = tensor(a[1], what);
  const int64_t width = integer(a[2]), d = c.dim();
  if (width < 1 || d < 1 || s.dim() != d || c.size(-1) != EBC_MX4_CODE_BYTES(width) ||
      s.size(-1) != EBC_MX4_SCALE_BYTES(width) || c.sizes().slice(0, d - 1) != s.sizes().slice(0, d - 1))
    bad("codes and scales do not hold rows of that width");
  for (const at::Tensor* t : {&c, &s})
    if (t->scalar_type() != at::kByte || !t->is_cuda() || !t->is_contiguous()) bad(what);
  return Mx4Ref{c, s, width};
}

Mx4Ref mx4_here(const Where& w, PyObject* const* a) {
  const Mx4Ref m = mx4_of(a);
  w.here(m.codes);
  w.here(m.scales);
  return m;
}

// codes and scales of n rows, one allocation
std::pair<at::Tensor, at::Tensor> mx4_rows(const Where& w, int64_t n, int64_t width) {
  const int64_t cb = EBC_MX4_CODE_BYTES(width), sb = EBC_MX4_SCALE_BYTES(width);
  const Parts all{w.empty({n * (cb + sb)}, at::kByte)};
  return {all.take(0, {n, cb}, at::kByte), all.take(n * cb, {n, sb}, at::kByte)};
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}

template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F&& f) {
  HANDLE_TH_ERRORS
  if (have != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* py_set_raise(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_raise, f);
  Py_RETURN_NONE;
}

PyObject* py_check_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    plan_of(a);
    Py_RETURN_NONE;
  });
}

PyObject* py_check_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    mx4_of(a);
    Py_RETURN_NONE;
  });
}

// ctx, device, ids, n_experts -> rows, place, offsets
PyObject* py_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    const Where w = where(a);
    const char* what = "ids must be a contiguous int32 or int64 CUDA tensor [tokens, top]";
    const at::Tensor& ids = tensor(a[2], what);
    const int64_t experts = integer(a[3]);
    if (ids.dim() != 2 || (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong) || !ids.is_contiguous())
      bad(what);
    w.here(ids);
    if (experts < 1 || experts > EBC_MAX_EXPERTS) checked(EBC_ERR_INVALID_ARG, "ebc_moe_plan");
    const int64_t tokens = ids.size(0), top = ids.size(1);
    const int64_t each = pad16(4 * tokens * top);
    const Parts all{w.empty({2 * each + 4 * (experts + 1)}, at::kByte)};
    at::Tensor r = all.take(0, {tokens * top}, at::kInt), p = all.take(each, {tokens, top}, at::kInt),
               o = all.take(2 * each, {experts + 1}, at::kInt);
    checked(ebc_moe_plan(w.ctx, ids.data_ptr(), (int)ids.element_size(), tokens, (int)std::min<int64_t>(top, INT32_MAX),
                         (int)experts, (int32_t*)r.data_ptr(), (int32_t*)p.data_ptr(), (int32_t*)o.data_ptr(),
                         w.stream()),
            "ebc_moe_plan");
    return tuple({r, p, o});
  });
}

// Whether any of the objects is a tensor whose operations are to be recorded for gradients.
PyObject* py_recorded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (c10::GradMode::is_enabled())
    for (Py_ssize_t i = 0; i < n; ++i)
      if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i]).requires_grad()) Py_RETURN_TRUE;
  Py_RETURN_FALSE;
}

// ctx, device, x, plan (3) -> xs
PyObject* py_dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const Where w = where(a);
    const Rows x = rows(w, a[2]);
    no_tangent(x.t);
    const PlanRef p = plan_here(w, a + 3);
    if (x.n != p.tokens) bad("x has not as many rows as the plan has tokens");
    at::Tensor xs = w.empty({p.n, x.width}, x.t.scalar_type());
    checked(ebc_moe_dispatch(w.ctx, x.t.data_ptr(), x.ld, x.type, p.tokens, (int)p.top, x.width, p.place_ptr(),
                             p.offsets_ptr(), (int)p.experts, xs.data_ptr(), w.stream()),
            "ebc_moe_dispatch");
    return wrap(xs);
  });
}

// ctx, device, x, plan (3) -> codes, scales
PyObject* py_dispatch_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const Where w = where(a);
    const Rows x = rows(w, a[2]);
    const PlanRef p = plan_here(w, a + 3);
    if (x.n != p.tokens) bad("x has not as many rows as the plan has tokens");
    auto [c, s] = mx4_rows(w, p.n, x.width);
    checked(ebc_moe_dispatch_mx4(w.ctx, x.t.data_ptr(), x.ld, x.type, p.tokens, (int)p.top, x.width, p.place_ptr(),
                                 p.offsets_ptr(), (int)p.experts, (uint8_t*)c.data_ptr(), (uint8_t*)s.data_ptr(),
                                 w.stream()),
            "ebc_moe_dispatch_mx4");
    return tuple({c, s});
  });
}

// ctx, device, ys, weights or None, plan (3) -> y
PyObject* py_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Where w = where(a);
    const Rows ys = rows(w, a[2]);
    const PlanRef p = plan_here(w, a + 4);
    if (ys.n != p.n) bad("ys has not as many rows as the plan");
    const float* weights = a[3] == Py_None ? nullptr : weights_of(w, a[3], p);
    no_tangent(ys.t);
    at::Tensor y = w.empty({p.tokens, ys.width}, ys.t.scalar_type());
    checked(ebc_moe_combine(w.ctx, ys.t.data_ptr(), ys.ld, ys.type, p.tokens, (int)p.top, ys.width, p.place_ptr(),
                            weights, y.data_ptr(), w.stream()),
            "ebc_moe_combine");
    return wrap(y);
  });
}

// ctx, device, dy, ys, weights, plan (3) -> dys, dweights
PyObject* py_combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Where w = where(a);
    const Rows dy = rows(w, a[2]), ys = rows(w, a[3]);
    const PlanRef p = plan_here(w, a + 5);
    if (dy.type != ys.type || dy.n != p.tokens || ys.n != p.n || dy.width != ys.width)
      bad("dy [tokens, width] and ys [n, width] of one type do not fit the plan");
    const float* weights = weights_of(w, a[4], p);
    no_tangent(dy.t);
    no_tangent(ys.t);
    at::Tensor dys = w.empty({p.n, ys.width}, ys.t.scalar_type()), dw = w.empty({p.tokens, p.top}, at::kFloat);
    checked(ebc_moe_combine_grad(w.ctx, dy.t.data_ptr(), dy.ld, ys.t.data_ptr(), ys.ld, ys.type, p.tokens, (int)p.top,
                                 ys.width, p.place_ptr(), p.offsets_ptr(), (int)p.experts, weights, dys.data_ptr(),
                                 (float*)dw.data_ptr(), w.stream()),
            "ebc_moe_combine_grad");
    return tuple({dys, dw});
  });
}

// ctx, device, x [rows, width] -> codes, scales
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&] {
    const Where w = where(a);
    const Rows x = rows(w, a[2]);
    auto [c, s] = mx4_rows(w, x.n, x.width);
    checked(ebc_mx4_quantize(w.ctx, x.t.data_ptr(), x.ld, x.type, x.n, x.width, (uint8_t*)c.data_ptr(),
                             (uint8_t*)s.data_ptr(), w.stream()),
            "ebc_mx4_quantize");
    return tuple({c, s});
  });
}

// ctx, device, codes, scales, width, type -> values
PyObject* py_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const Where w = where(a);
    const Mx4Ref m = mx4_here(w, a + 2);
    const int64_t type = integer(a[5]);
    at::DimVector shape(m.codes.sizes().begin(), m.codes.sizes().end());
    shape.back() = m.width;
    at::Tensor x = w.empty(shape, scalar_of(type));
    checked(ebc_mx4_dequantize(w.ctx, m.codes_ptr(), m.scales_ptr(), x.numel() / m.width, m.width, (int)type,
                               x.data_ptr(), w.stream()),
            "ebc_mx4_dequantize");
    return wrap(x);
  });
}

// ctx, device, x (3), w (3), offsets or None, type -> ys
PyObject* py_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Where at = where(a);
    const Mx4Ref x = mx4_here(at, a + 2), w = mx4_here(at, a + 5);
    const bool one = a[8] == Py_None;
    if (x.codes.dim() != 2 || w.codes.dim() != (one ? 2 : 3) || x.width != w.width)
      bad("x [rows, width] and w [n_experts, outs, width] (or [outs, width] without offsets) do not multiply");
    const int64_t experts = one ? 1 : w.codes.size(0), outs = w.codes.size(-2), type = integer(a[9]);
    const int32_t* offsets = nullptr;
    if (!one) {
      const char* what = "offsets must be a contiguous int32 CUDA tensor [n_experts + 1]";
      const at::Tensor& o = tensor(a[8], what);
      if (o.scalar_type() != at::kInt || o.dim() != 1 || o.numel() != experts + 1 || !o.is_contiguous()) bad(what);
      at.here(o);
      offsets = (const int32_t*)o.data_ptr();
    }
    at::Tensor ys = at.empty({x.codes.size(0), outs}, scalar_of(type));
    checked(ebc_mx4_product(at.ctx, x.codes_ptr(), x.scales_ptr(), x.codes.size(0), x.width, w.codes_ptr(),
                            w.scales_ptr(), outs, (int)std::min<int64_t>(experts, INT32_MAX), offsets, (int)type,
                            ys.data_ptr(), at.stream()),
            "ebc_mx4_product");
    return wrap(ys);
  });
}

#define CALL(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {{"set_raise", py_set_raise, METH_O, nullptr},
                           CALL(check_plan),
                           CALL(check_mx4),
                           CALL(recorded),
                           CALL(plan),
                           CALL(dispatch),
                           CALL(dispatch_mx4),
                           CALL(combine),
                           CALL(combine_grad),
                           CALL(quantize),
                           CALL(dequantize),
                           CALL(product),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&g_module); }
