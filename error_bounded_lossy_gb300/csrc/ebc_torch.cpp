// ebc_torch.cpp -- the expert-parallel, 4- and 8-bit, router and norm calls on torch tensors: checks
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

// Rows in 4 or 8 bits.
struct MxRef {
  const at::Tensor &codes, &scales;
  int64_t width;
  const uint8_t* codes_ptr() const { return (const uint8_t*)codes.data_ptr(); }
  const uint8_t* scales_ptr() const { return (const uint8_t*)scales.data_ptr(); }
};

int64_t code_bytes(int bits, int64_t width) {
  return bits == 4 ? EBC_MX4_CODE_BYTES(width) : EBC_MX8_CODE_BYTES(width);
}

// codes, scales and width of such rows.
template <int kBits>
MxRef mx_of(PyObject* const* a) {
  const char* what = "codes and scales must be contiguous uint8 CUDA tensors";
  const at::Tensor &c = tensor(a[0], what), &s = tensor(a[1], what);
  const int64_t width = integer(a[2]), d = c.dim();
  if (width < 1 || d < 1 || s.dim() != d || c.size(-1) != code_bytes(kBits, width) ||
      s.size(-1) != EBC_MX4_SCALE_BYTES(width) || c.sizes().slice(0, d - 1) != s.sizes().slice(0, d - 1))
    bad("codes and scales do not hold rows of that width");
  for (const at::Tensor* t : {&c, &s})
    if (t->scalar_type() != at::kByte || !t->is_cuda() || !t->is_contiguous()) bad(what);
  return MxRef{c, s, width};
}

template <int kBits>
MxRef mx_here(const Where& w, PyObject* const* a) {
  const MxRef m = mx_of<kBits>(a);
  w.here(m.codes);
  w.here(m.scales);
  return m;
}

// codes and scales of n rows, one allocation
std::pair<at::Tensor, at::Tensor> mx_rows(const Where& w, int bits, int64_t n, int64_t width) {
  const int64_t cb = code_bytes(bits, width), sb = EBC_MX4_SCALE_BYTES(width);
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

template <int kBits>
PyObject* check_mx(PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    mx_of<kBits>(a);
    Py_RETURN_NONE;
  });
}
PyObject* py_check_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) { return check_mx<4>(a, n); }
PyObject* py_check_mx8(PyObject*, PyObject* const* a, Py_ssize_t n) { return check_mx<8>(a, n); }

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
    auto [c, s] = mx_rows(w, 4, p.n, x.width);
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
template <int kBits>
PyObject* quantize(PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&] {
    const Where w = where(a);
    const Rows x = rows(w, a[2]);
    auto [c, s] = mx_rows(w, kBits, x.n, x.width);
    checked((kBits == 4 ? ebc_mx4_quantize : ebc_mx8_quantize)(w.ctx, x.t.data_ptr(), x.ld, x.type, x.n, x.width,
                                                               (uint8_t*)c.data_ptr(), (uint8_t*)s.data_ptr(),
                                                               w.stream()),
            kBits == 4 ? "ebc_mx4_quantize" : "ebc_mx8_quantize");
    return tuple({c, s});
  });
}
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) { return quantize<4>(a, n); }
PyObject* py_quantize_mx8(PyObject*, PyObject* const* a, Py_ssize_t n) { return quantize<8>(a, n); }

// ctx, device, codes, scales, width, type -> values
template <int kBits>
PyObject* dequantize(PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const Where w = where(a);
    const MxRef m = mx_here<kBits>(w, a + 2);
    const int64_t type = integer(a[5]);
    at::DimVector shape(m.codes.sizes().begin(), m.codes.sizes().end());
    shape.back() = m.width;
    at::Tensor x = w.empty(shape, scalar_of(type));
    checked((kBits == 4 ? ebc_mx4_dequantize : ebc_mx8_dequantize)(w.ctx, m.codes_ptr(), m.scales_ptr(),
                                                                   x.numel() / m.width, m.width, (int)type,
                                                                   x.data_ptr(), w.stream()),
            kBits == 4 ? "ebc_mx4_dequantize" : "ebc_mx8_dequantize");
    return wrap(x);
  });
}
PyObject* py_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) { return dequantize<4>(a, n); }
PyObject* py_dequantize_mx8(PyObject*, PyObject* const* a, Py_ssize_t n) { return dequantize<8>(a, n); }

// ctx, device, x (3), w (3), offsets or None, type -> ys
template <int kBits>
PyObject* product(PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Where at = where(a);
    const MxRef x = mx_here<kBits>(at, a + 2), w = mx_here<kBits>(at, a + 5);
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
    checked((kBits == 4 ? ebc_mx4_product : ebc_mx8_product)(
                at.ctx, x.codes_ptr(), x.scales_ptr(), x.codes.size(0), x.width, w.codes_ptr(), w.scales_ptr(), outs,
                (int)std::min<int64_t>(experts, INT32_MAX), offsets, (int)type, ys.data_ptr(), at.stream()),
            kBits == 4 ? "ebc_mx4_product" : "ebc_mx8_product");
    return wrap(ys);
  });
}
PyObject* py_product(PyObject*, PyObject* const* a, Py_ssize_t n) { return product<4>(a, n); }
PyObject* py_product_mx8(PyObject*, PyObject* const* a, Py_ssize_t n) { return product<8>(a, n); }

// ctx, device, codes, scales, plan (3) -> codes, scales of the sorted rows
PyObject* py_dispatch_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Where w = where(a);
    const char* what = "rows in 4 or 8 bits must be codes and scales [tokens, bytes], contiguous uint8 CUDA tensors";
    const at::Tensor &c = tensor(a[2], what), &s = tensor(a[3], what);
    for (const at::Tensor* t : {&c, &s}) {
      if (t->scalar_type() != at::kByte || !t->is_cuda() || !t->is_contiguous() || t->dim() != 2) bad(what);
      w.here(*t);
    }
    const PlanRef p = plan_here(w, a + 4);
    if (c.size(0) != p.tokens || s.size(0) != p.tokens) bad("x has not as many rows as the plan has tokens");
    const int64_t cb = c.size(1), sb = s.size(1);
    const Parts all{w.empty({p.n * (cb + sb)}, at::kByte)};
    at::Tensor xc = all.take(0, {p.n, cb}, at::kByte), xs = all.take(p.n * cb, {p.n, sb}, at::kByte);
    checked(ebc_moe_dispatch_mx(w.ctx, (const uint8_t*)c.data_ptr(), cb, (const uint8_t*)s.data_ptr(), sb, p.tokens,
                                (int)p.top, p.place_ptr(), p.offsets_ptr(), (int)p.experts, (uint8_t*)xc.data_ptr(),
                                (uint8_t*)xs.data_ptr(), w.stream()),
            "ebc_moe_dispatch_mx");
    return tuple({xc, xs});
  });
}

// Whether a call has to be recorded for gradients.
bool recorded(std::initializer_list<PyObject*> os) {
  if (c10::GradMode::is_enabled())
    for (PyObject* o : os)
      if (THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad()) return true;
  return false;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}

int small(PyObject* o) {   // an int argument of the C call, which refuses what is out of its range
  const int64_t v = integer(o);
  return (int)std::max<int64_t>(INT32_MIN, std::min<int64_t>(v, INT32_MAX));
}

// ctx, device, logits, top, score, bias or None, groups, keep_groups, group_top, renormalize, scale -> ids, weights;
// None where the call has to be recorded for gradients
PyObject* py_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Where w = where(a);
    if (recorded({a[2]})) Py_RETURN_NONE;
    const Rows l = rows(w, a[2]);
    no_tangent(l.t);
    const int top = small(a[3]);
    const float* bias = nullptr;
    if (a[5] != Py_None) {
      const char* what = "bias must be a contiguous float32 CUDA tensor [n_experts]";
      const at::Tensor& b = tensor(a[5], what);
      if (b.scalar_type() != at::kFloat || b.dim() != 1 || b.numel() != l.width || !b.is_contiguous()) bad(what);
      w.here(b);
      bias = (const float*)b.data_ptr();
    }
    if (top < 1 || top > EBC_MAX_TOP) checked(EBC_ERR_INVALID_ARG, "ebc_moe_route");
    const Parts all{w.empty({2 * pad16(4 * l.n * top)}, at::kByte)};
    at::Tensor ids = all.take(0, {l.n, top}, at::kInt), weights = all.take(pad16(4 * l.n * top), {l.n, top}, at::kFloat);
    checked(ebc_moe_route(w.ctx, l.t.data_ptr(), l.ld, l.type, l.n, (int)std::min<int64_t>(l.width, INT32_MAX), top,
                          small(a[4]), bias, small(a[6]), small(a[7]), small(a[8]), truth(a[9]),
                          (float)real(a[10]), (int32_t*)ids.data_ptr(), (float*)weights.data_ptr(), w.stream()),
            "ebc_moe_route");
    return tuple({ids, weights});
  });
}

// ctx, device, dweights, logits, ids, score, renormalize, scale -> dlogits
PyObject* py_route_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Where w = where(a);
    const Rows l = rows(w, a[3]);
    no_tangent(l.t);
    const char* what = "dweights and ids must be contiguous float32 and int32 CUDA tensors [tokens, top]";
    const at::Tensor &g = tensor(a[2], what), &ids = tensor(a[4], what);
    if (g.scalar_type() != at::kFloat || ids.scalar_type() != at::kInt || g.dim() != 2 || g.size(0) != l.n ||
        g.sizes() != ids.sizes() || !g.is_contiguous() || !ids.is_contiguous())
      bad(what);
    w.here(g);
    w.here(ids);
    no_tangent(g);
    at::Tensor d = w.empty({l.n, l.width}, l.t.scalar_type());
    checked(ebc_moe_route_grad(w.ctx, (const float*)g.data_ptr(), l.t.data_ptr(), l.ld, l.type, l.n,
                               (int)std::min<int64_t>(l.width, INT32_MAX),
                               (int)std::min<int64_t>(g.size(1), INT32_MAX), (const int32_t*)ids.data_ptr(),
                               small(a[5]), truth(a[6]), (float)real(a[7]), d.data_ptr(), w.stream()),
            "ebc_moe_route_grad");
    return wrap(d);
  });
}

// The norm's weight [width].
const at::Tensor& gain(const Where& w, PyObject* o, int64_t width) {
  const char* what = "weight must be a contiguous float32, bfloat16 or float16 CUDA tensor [width]";
  const at::Tensor& t = tensor(o, what);
  if (type_of(t) < 0 || t.dim() != 1 || t.numel() != width || !t.is_contiguous()) bad(what);
  w.here(t);
  no_tangent(t);
  return t;
}

// Rows of the same shape and type as others.
Rows rows_like(const Where& w, PyObject* o, const Rows& like) {
  const Rows r = rows(w, o);
  if (r.type != like.type || r.n != like.n || r.width != like.width) bad("rows of one shape and type are needed");
  no_tangent(r.t);
  return r;
}

// The norm's outputs: of few bytes in one allocation, which is most of a small
// call's time; of more in their own, each as long-lived as its user.
constexpr int64_t kFewBytes = 64 << 10;
// (on 32-byte boundaries, where fp32 rows are read eight values at a time)
int64_t pad32(int64_t n) { return (n + 31) & ~(int64_t)31; }

// ctx, device, x, weight, residual or None, eps -> y, h (x without a residual); None where x is not rows, or where the
// call has to be recorded for gradients
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const Where w = where(a);
    if (recorded({a[2], a[3], a[4]}) || (THPVariable_Check(a[2]) && THPVariable_Unpack(a[2]).dim() != 2)) Py_RETURN_NONE;
    const Rows x = rows(w, a[2]);
    no_tangent(x.t);
    const at::Tensor& g = gain(w, a[3], x.width);
    const bool more = a[4] != Py_None;
    const Rows r = more ? rows_like(w, a[4], x) : x;
    at::Tensor y, h;
    const int64_t each = pad32(x.n * x.width * (int64_t)x.t.element_size());
    if (more && each <= kFewBytes) {
      const Parts all{w.empty({2 * each}, at::kByte)};
      y = all.take(0, {x.n, x.width}, x.t.scalar_type());
      h = all.take(each, {x.n, x.width}, x.t.scalar_type());
    } else {
      y = w.empty({x.n, x.width}, x.t.scalar_type());
      if (more) h = w.empty({x.n, x.width}, x.t.scalar_type());
    }
    checked(ebc_norm(w.ctx, x.t.data_ptr(), x.ld, more ? r.t.data_ptr() : nullptr, r.ld, x.type, g.data_ptr(),
                     type_of(g), x.n, x.width, (float)real(a[5]), y.data_ptr(), more ? h.data_ptr() : nullptr, nullptr,
                     nullptr, w.stream()),
            "ebc_norm");
    return tuple({y, more ? h : x.t});
  });
}

// ctx, device, x, weight, residual or None, eps, wide -> codes, scales, y (None unless wide), h; or None, as py_norm
PyObject* py_norm_mx8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const Where w = where(a);
    if (recorded({a[2], a[3], a[4]}) || (THPVariable_Check(a[2]) && THPVariable_Unpack(a[2]).dim() != 2)) Py_RETURN_NONE;
    const Rows x = rows(w, a[2]);
    no_tangent(x.t);
    const at::Tensor& g = gain(w, a[3], x.width);
    const bool more = a[4] != Py_None, wide = truth(a[6]);
    const Rows r = more ? rows_like(w, a[4], x) : x;
    const int64_t each = pad32(x.n * x.width * (int64_t)x.t.element_size()), cb = x.n * code_bytes(8, x.width),
                  sb = pad32(x.n * EBC_MX8_SCALE_BYTES(x.width));
    at::Tensor y, h, c, s;
    if ((more || wide) && cb + sb + 2 * each <= kFewBytes) {
      const Parts all{w.empty({cb + sb + (more + wide) * each}, at::kByte)};
      c = all.take(0, {x.n, code_bytes(8, x.width)}, at::kByte);
      s = all.take(cb, {x.n, EBC_MX8_SCALE_BYTES(x.width)}, at::kByte);
      if (wide) y = all.take(cb + sb, {x.n, x.width}, x.t.scalar_type());
      if (more) h = all.take(cb + sb + wide * each, {x.n, x.width}, x.t.scalar_type());
    } else {
      std::tie(c, s) = mx_rows(w, 8, x.n, x.width);
      if (wide) y = w.empty({x.n, x.width}, x.t.scalar_type());
      if (more) h = w.empty({x.n, x.width}, x.t.scalar_type());
    }
    checked(ebc_norm(w.ctx, x.t.data_ptr(), x.ld, more ? r.t.data_ptr() : nullptr, r.ld, x.type, g.data_ptr(),
                     type_of(g), x.n, x.width, (float)real(a[5]), wide ? y.data_ptr() : nullptr,
                     more ? h.data_ptr() : nullptr, (uint8_t*)c.data_ptr(), (uint8_t*)s.data_ptr(), w.stream()),
            "ebc_norm");
    return tuple({c, s, y, more ? h : x.t});   // (an undefined tensor is None)
  });
}

// ctx, device, dy, h, weight, dh or None, eps -> dx, dweight
PyObject* py_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Where w = where(a);
    const Rows dy = rows(w, a[2]);
    no_tangent(dy.t);
    const Rows h = rows_like(w, a[3], dy);
    const at::Tensor& g = gain(w, a[4], dy.width);
    const bool more = a[5] != Py_None;
    const Rows dh = more ? rows_like(w, a[5], dy) : dy;
    const int64_t xb = pad32(dy.n * dy.width * (int64_t)dy.t.element_size()), gb = pad32(dy.width * (int64_t)g.element_size()),
                  sb = pad32(EBC_NORM_GRAD_SCRATCH(dy.n, dy.width));
    at::Tensor dx, dg, scratch;
    if (xb + gb + sb <= kFewBytes) {
      const Parts all{w.empty({xb + gb + sb}, at::kByte)};
      scratch = all.take(0, {sb}, at::kByte);
      dx = all.take(sb, {dy.n, dy.width}, dy.t.scalar_type());
      dg = all.take(sb + xb, {dy.width}, g.scalar_type());
    } else {
      dx = w.empty({dy.n, dy.width}, dy.t.scalar_type());
      dg = w.empty({dy.width}, g.scalar_type());
      scratch = w.empty({sb}, at::kByte);
    }
    checked(ebc_norm_grad(w.ctx, dy.t.data_ptr(), dy.ld, h.t.data_ptr(), h.ld, more ? dh.t.data_ptr() : nullptr,
                          dh.ld, dy.type, g.data_ptr(), type_of(g), dy.n, dy.width, (float)real(a[6]),
                          dx.data_ptr(), dg.data_ptr(), (float*)scratch.data_ptr(), w.stream()),
            "ebc_norm_grad");
    return tuple({dx, dg});
  });
}

#define CALL(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {{"set_raise", py_set_raise, METH_O, nullptr},
                           CALL(check_plan),
                           CALL(check_mx4),
                           CALL(check_mx8),
                           CALL(recorded),
                           CALL(plan),
                           CALL(dispatch),
                           CALL(dispatch_mx4),
                           CALL(combine),
                           CALL(combine_grad),
                           CALL(quantize),
                           CALL(dequantize),
                           CALL(product),
                           CALL(quantize_mx8),
                           CALL(dequantize_mx8),
                           CALL(product_mx8),
                           CALL(dispatch_mx),
                           CALL(route),
                           CALL(route_grad),
                           CALL(norm),
                           CALL(norm_mx8),
                           CALL(norm_grad),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&g_module); }
