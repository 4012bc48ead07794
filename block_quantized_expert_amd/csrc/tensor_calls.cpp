// The calls of moe_rows.h, moe_int8.h, moe_norm.h and moe_mxfp4.h on torch
// tensors: argument checks, outputs, the current stream, the C entry.  Their
// kernels take a few microseconds at the size of one token, where the same steps
// in Python took three times that (one token's combine, submission: 14 us through
// ctypes); binding.py holds the signatures and the documentation.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "moe_int8.h"
#include "moe_mxfp4.h"
#include "moe_norm.h"
#include "moe_rows.h"

namespace {

PyObject* error_class = nullptr;  // binding.MoeError

struct Failed {};  // a Python exception is set

void check(moe_status s, const char* where) {
  if (s == MOE_OK) return;
  if (PyObject* e = PyObject_CallFunction(error_class, "is", (int)s, where)) {
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
  }
  throw Failed();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

int integer(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed();
  TORCH_CHECK_VALUE(v == (int)v, name, " is out of range");
  return (int)v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed();
  return (float)v;
}

at::ScalarType dtype(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPDtype_Check(o), name, " must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int act_type(at::ScalarType t, const char* name) {
  TORCH_CHECK_VALUE(t == at::kFloat || t == at::kBFloat16, name, " must be float32 or bfloat16");
  return t == at::kFloat ? MOE_ACT_F32 : MOE_ACT_BF16;
}

// A size that the library's int arguments can hold; its own limits follow.
int size(int64_t v, const char* name) {
  TORCH_CHECK_VALUE(v <= INT32_MAX, name, " is too large");
  return (int)v;
}

// The row stride of a matrix [n][c] whose rows may be strided.
int64_t rows_arg(const at::Tensor& t, const char* name, int64_t n, int64_t c, c10::Device dev) {
  TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == n && t.size(1) == c, name,
                    " must have shape (", n, ", ", c, "), has ", t.sizes());
  TORCH_CHECK_VALUE(t.device() == dev, name, " is on ", t.device(), ", expected ", dev);
  TORCH_CHECK_VALUE((c <= 1 || t.stride(1) == 1) && (n <= 1 || t.stride(0) >= c), name,
                    ": rows must be contiguous and must not overlap");
  return n > 1 ? t.stride(0) : c;
}

const at::Tensor& dense_arg(const at::Tensor& t, const char* name, at::ScalarType type, int64_t numel,
                            c10::Device dev) {
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.numel() == numel && t.is_contiguous() &&
                        t.device() == dev,
                    name, " must be a contiguous ", type, " tensor of ", numel, " elements on ",
                    dev);
  return t;
}

struct Grouping {
  int n_experts;
  const int32_t *offsets, *perm, *inv_perm;
};

Grouping grouping_arg(PyObject* o, int64_t n_slots, c10::Device dev) {
  TORCH_CHECK_VALUE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4,
                    "grouping must be (counts, offsets, perm, inv_perm)");
  const at::Tensor& off = tensor(PyTuple_GET_ITEM(o, 1), "offsets");
  const at::Tensor& perm = tensor(PyTuple_GET_ITEM(o, 2), "perm");
  const at::Tensor& inv = tensor(PyTuple_GET_ITEM(o, 3), "inv_perm");
  const int64_t e = off.numel() - 1;
  dense_arg(off, "offsets", at::kInt, off.numel(), dev);
  // without slots the arrays may hold anything
  dense_arg(perm, "perm", at::kInt, n_slots == 0 ? perm.numel() : n_slots, dev);
  dense_arg(inv, "inv_perm", at::kInt, n_slots == 0 ? inv.numel() : n_slots, dev);
  return {size(e, "offsets"), off.const_data_ptr<int32_t>(), perm.const_data_ptr<int32_t>(),
          inv.const_data_ptr<int32_t>()};
}

void on_gpu(c10::Device dev) {
  TORCH_CHECK_VALUE(dev.is_cuda(), "tensors must be on the GPU, got ", dev);
}

// The call's device and its current stream.
struct On {
  c10::hip::HIPGuard guard;
  hipStream_t stream;
  explicit On(c10::Device dev)
      : guard(dev.index()), stream(c10::hip::getCurrentHIPStream(dev.index()).stream()) {}
};

// From torch's caching allocator, on the current stream, past the dispatcher.
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  return at::Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}

// The given output, of the dtype, or a new one.
at::Tensor output(PyObject* o, const char* name, const char* like, at::IntArrayRef shape,
                  at::ScalarType type, c10::Device dev) {
  if (o == Py_None) return empty(shape, type, dev);
  const at::Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must have ", like, "'s dtype");
  return t;
}

template <typename T = void>
const T* in(const at::Tensor& t) {
  return static_cast<const T*>(t.const_data_ptr());
}
template <typename T = void>
T* out(const at::Tensor& t) {
  return static_cast<T*>(t.mutable_data_ptr());
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* const pa = THPVariable_Wrap(a);
  PyObject* const pb = THPVariable_Wrap(b);
  PyObject* const r = pa != nullptr && pb != nullptr ? PyTuple_Pack(2, pa, pb) : nullptr;
  Py_XDECREF(pa);
  Py_XDECREF(pb);
  return r;
}

using Args = PyObject* const*;

PyObject* set_error(Args a) {
  Py_INCREF(a[0]);
  error_class = a[0];
  Py_RETURN_NONE;
}

// x, grouping, top_k, rows
PyObject* dispatch(Args a) {
  const at::Tensor& x = tensor(a[0], "x");
  const c10::Device dev = x.device();
  TORCH_CHECK_VALUE(x.dim() == 2, "x must be a matrix");
  const int64_t n = x.size(0), h = x.size(1);
  const int type = act_type(x.scalar_type(), "x");
  const int64_t xs = rows_arg(x, "x", n, h, dev);
  const int k = integer(a[2], "top_k");
  const Grouping g = grouping_arg(a[1], n * k, dev);
  on_gpu(dev);
  const On on(dev);
  const at::Tensor rows = output(a[3], "rows", "x", {n * k, h}, x.scalar_type(), dev);
  const int64_t rs = rows_arg(rows, "rows", n * k, h, dev);
  check(moe_dispatch(in(x), type, xs, size(n, "x"), k, size(h, "hidden"), g.n_experts, g.offsets,
                     g.inv_perm, out(rows), rs, on.stream),
        "moe_dispatch");
  return THPVariable_Wrap(rows);
}

// drows, grouping, top_k, dx
PyObject* dispatch_backward(Args a) {
  const at::Tensor& drows = tensor(a[0], "drows");
  const c10::Device dev = drows.device();
  const int k = integer(a[2], "top_k");
  TORCH_CHECK_VALUE(drows.dim() == 2 && k > 0 && drows.size(0) % k == 0,
                    "drows must be a matrix of n*top_k rows");
  const int64_t slots = drows.size(0), n = slots / k, h = drows.size(1);
  const int type = act_type(drows.scalar_type(), "drows");
  const int64_t rs = rows_arg(drows, "drows", slots, h, dev);
  const Grouping g = grouping_arg(a[1], slots, dev);
  on_gpu(dev);
  const On on(dev);
  const at::Tensor dx = output(a[3], "dx", "drows", {n, h}, drows.scalar_type(), dev);
  const int64_t ds = rows_arg(dx, "dx", n, h, dev);
  check(moe_dispatch_backward(in(drows), type, rs, size(n, "drows"), k, size(h, "hidden"),
                              g.inv_perm, out(dx), ds, on.stream),
        "moe_dispatch_backward");
  return THPVariable_Wrap(dx);
}

// rows, w, grouping, base, y, y_dtype
PyObject* combine(Args a) {
  const at::Tensor& rows = tensor(a[0], "rows");
  const at::Tensor& w = tensor(a[1], "w");
  const c10::Device dev = rows.device();
  TORCH_CHECK_VALUE(rows.dim() == 2 && w.dim() == 2 && rows.size(0) == w.numel(),
                    "rows must be [n*top_k][hidden] and w [n][top_k]");
  const int64_t n = w.size(0), k = w.size(1), h = rows.size(1);
  const int type = act_type(rows.scalar_type(), "rows");
  const int64_t rs = rows_arg(rows, "rows", n * k, h, dev);
  dense_arg(w, "w", at::kFloat, n * k, dev);
  const Grouping g = grouping_arg(a[2], n * k, dev);
  on_gpu(dev);
  const On on(dev);
  const bool based = a[3] != Py_None;
  at::Tensor y;
  if (a[4] != Py_None)
    y = tensor(a[4], "y");
  else
    y = empty({n, h},
              based                ? tensor(a[3], "base").scalar_type()
              : a[5] != Py_None ? dtype(a[5], "y_dtype")
                                : rows.scalar_type(),
              dev);
  const int y_type = act_type(y.scalar_type(), "y");
  const int64_t ys = rows_arg(y, "y", n, h, dev);
  const void* base = nullptr;
  int64_t bs = 0;
  if (based) {
    const at::Tensor& b = tensor(a[3], "base");
    TORCH_CHECK_VALUE(b.scalar_type() == y.scalar_type(), "base must have y's dtype");
    bs = rows_arg(b, "base", n, h, dev);
    base = in(b);
  }
  check(moe_combine(in(rows), type, rs, size(n, "w"), size(k, "top_k"), size(h, "hidden"),
                    in<float>(w), g.inv_perm, base, bs, out(y), y_type, ys, on.stream),
        "moe_combine");
  return THPVariable_Wrap(y);
}

// dy, rows, w, grouping, drows, dw
PyObject* combine_backward(Args a) {
  const at::Tensor& dy = tensor(a[0], "dy");
  const at::Tensor& rows = tensor(a[1], "rows");
  const at::Tensor& w = tensor(a[2], "w");
  const c10::Device dev = rows.device();
  TORCH_CHECK_VALUE(rows.dim() == 2 && w.dim() == 2 && rows.size(0) == w.numel(),
                    "rows must be [n*top_k][hidden] and w [n][top_k]");
  const int64_t n = w.size(0), k = w.size(1), h = rows.size(1);
  const int type = act_type(rows.scalar_type(), "rows");
  const int y_type = act_type(dy.scalar_type(), "dy");
  const int64_t rs = rows_arg(rows, "rows", n * k, h, dev);
  const int64_t ys = rows_arg(dy, "dy", n, h, dev);
  dense_arg(w, "w", at::kFloat, n * k, dev);
  const Grouping g = grouping_arg(a[3], n * k, dev);
  on_gpu(dev);
  const On on(dev);
  const at::Tensor drows = output(a[4], "drows", "rows", {n * k, h}, rows.scalar_type(), dev);
  const at::Tensor dw = a[5] != Py_None ? tensor(a[5], "dw") : empty({n, k}, at::kFloat, dev);
  dense_arg(dw, "dw", at::kFloat, n * k, dev);
  const int64_t ds = rows_arg(drows, "drows", n * k, h, dev);
  check(moe_combine_backward(in(dy), y_type, ys, in(rows), type, rs, size(n, "w"),
                             size(k, "top_k"), size(h, "hidden"), g.n_experts, in<float>(w),
                             g.offsets, g.inv_perm, out(drows), ds, out<float>(dw), on.stream),
        "moe_combine_backward");
  return pair(drows, dw);
}

// logits, ids, dw, routed_scale, dlogits, dev_error
PyObject* route_backward(Args a) {
  const at::Tensor& logits = tensor(a[0], "logits");
  const at::Tensor& ids = tensor(a[1], "ids");
  const at::Tensor& dw = tensor(a[2], "dw");
  const c10::Device dev = logits.device();
  TORCH_CHECK_VALUE(logits.dim() == 2 && ids.dim() == 2 && ids.size(0) == logits.size(0),
                    "logits must be [n][n_experts] and ids [n][top_k]");
  const int64_t n = logits.size(0), e = logits.size(1), k = ids.size(1);
  dense_arg(logits, "logits", at::kFloat, n * e, dev);
  dense_arg(ids, "ids", at::kInt, n * k, dev);
  dense_arg(dw, "dw", at::kFloat, n * k, dev);
  on_gpu(dev);
  const On on(dev);
  const at::Tensor dl =
      a[4] != Py_None ? tensor(a[4], "dlogits") : empty({n, e}, at::kFloat, dev);
  dense_arg(dl, "dlogits", at::kFloat, n * e, dev);
  int32_t* err = nullptr;
  if (a[5] != Py_None)
    err = out<int32_t>(dense_arg(tensor(a[5], "dev_error"), "dev_error", at::kInt, 1, dev));
  check(moe_route_backward(in<float>(logits), in<int32_t>(ids), in<float>(dw), size(n, "logits"),
                           size(e, "n_experts"), size(k, "top_k"), number(a[3]), out<float>(dl),
                           err, on.stream),
        "moe_route_backward");
  return THPVariable_Wrap(dl);
}

// x, q, scale
PyObject* quantize_int8(Args a) {
  const at::Tensor& x = tensor(a[0], "x");
  const c10::Device dev = x.device();
  TORCH_CHECK_VALUE(x.dim() == 2, "x must be a matrix");
  const int64_t n = x.size(0), c = x.size(1);
  const int type = act_type(x.scalar_type(), "x");
  const int64_t xs = rows_arg(x, "x", n, c, dev);
  on_gpu(dev);
  const On on(dev);
  const at::Tensor q = a[1] != Py_None ? tensor(a[1], "q") : empty({n, c}, at::kChar, dev);
  const at::Tensor scale = a[2] != Py_None ? tensor(a[2], "scale") : empty({n}, at::kFloat, dev);
  dense_arg(q, "q", at::kChar, n * c, dev);
  dense_arg(scale, "scale", at::kFloat, n, dev);
  check(moe_quantize_int8(in(x), type, xs, size(n, "x"), size(c, "cols"), out<int8_t>(q),
                          out<float>(scale), on.stream),
        "moe_quantize_int8");
  return pair(q, scale);
}

// address of the moe_int8_weight and its q, address of the up one or 0 and
// its q or None, then q, scale, grouping, top_k, out_dtype, out
PyObject* product_int8(Args a) {
  const auto* w = static_cast<const moe_int8_weight*>(PyLong_AsVoidPtr(a[0]));
  const auto* up = static_cast<const moe_int8_weight*>(PyLong_AsVoidPtr(a[2]));
  if (PyErr_Occurred()) throw Failed();
  const at::Tensor& wq = tensor(a[1], "the weight");
  const at::Tensor& q = tensor(a[4], "q");
  const at::Tensor& scale = tensor(a[5], "scale");
  const c10::Device dev = q.device();
  TORCH_CHECK_VALUE(q.dim() == 2 && q.size(1) == w->cols, "q must be [rows][", w->cols, "]");
  dense_arg(q, "q", at::kChar, q.numel(), dev);
  dense_arg(scale, "scale", at::kFloat, q.size(0), dev);
  TORCH_CHECK_VALUE(wq.device() == dev, "the weights are on ", wq.device(), ", q is on ", dev);
  if (up != nullptr) {
    const c10::Device ud = tensor(a[3], "the up weight").device();
    TORCH_CHECK_VALUE(ud == dev, "the up weights are on ", ud, ", q is on ", dev);
  }
  const int k = integer(a[7], "top_k");
  const int64_t n = q.size(0) * (k != 0 ? k : 1), rows = w->rows;
  Grouping g{};
  if (a[6] != Py_None) {
    g = grouping_arg(a[6], n, dev);
    TORCH_CHECK_VALUE(g.n_experts == w->n_experts, "the grouping has ", g.n_experts,
                      " experts, the weights ", w->n_experts);
  }
  on_gpu(dev);
  const On on(dev);
  const at::Tensor o =
      a[9] != Py_None ? tensor(a[9], "out") : empty({n, rows}, dtype(a[8], "out_dtype"), dev);
  const int type = act_type(o.scalar_type(), "out");
  const int64_t os = rows_arg(o, "out", n, rows, dev);
  if (up != nullptr)
    check(moe_swiglu_int8(w, up, in<int8_t>(q), in<float>(scale), size(n, "q"), g.offsets, g.perm,
                          k, out(o), type, os, on.stream),
          "moe_swiglu_int8");
  else
    check(moe_product_int8(w, in<int8_t>(q), in<float>(scale), size(n, "q"), g.offsets, g.perm, k,
                           out(o), type, os, on.stream),
          "moe_product_int8");
  return THPVariable_Wrap(o);
}

// The rows of a norm: x, weight, eps, residual, total (arguments 0 to 4); the
// total's tensor is kept in `total`.
struct NormArgs {
  moe_norm_rows r{};
  const at::Tensor &x, &w;
  at::Tensor total;
  NormArgs(Args a) : x(tensor(a[0], "x")), w(tensor(a[1], "weight")) {
    const c10::Device dev = x.device();
    TORCH_CHECK_VALUE(x.dim() == 2, "x must be a matrix");
    const int64_t n = x.size(0), h = x.size(1);
    r.n_rows = size(n, "x");
    r.hidden = size(h, "hidden");
    r.eps = number(a[2]);
    r.x_type = act_type(x.scalar_type(), "x");
    r.x_stride = rows_arg(x, "x", n, h, dev);
    r.w_type = act_type(w.scalar_type(), "weight");
    dense_arg(w, "weight", w.scalar_type(), h, dev);
    on_gpu(dev);
    TORCH_CHECK_VALUE(a[4] == Py_None || a[3] != Py_None, "total needs a residual");
    if (a[3] != Py_None) {
      const at::Tensor& res = tensor(a[3], "residual");
      r.res_type = act_type(res.scalar_type(), "residual");
      r.res_stride = rows_arg(res, "residual", n, h, dev);
      r.residual = in(res);
    }
    r.x = in(x);
    r.weight = in(w);
  }
  // with the device set
  void open(Args a) {
    if (a[3] == Py_None) return;
    const int64_t n = x.size(0), h = x.size(1);
    const at::Tensor& res = tensor(a[3], "residual");
    total = output(a[4], "total", "the residual", {n, h}, res.scalar_type(), x.device());
    r.total_stride = rows_arg(total, "total", n, h, x.device());
    r.total = out(total);
  }
};

// The outputs that there are, alone or as a tuple.
PyObject* results(std::initializer_list<const at::Tensor*> list) {
  PyObject* made[3];
  Py_ssize_t n = 0;
  bool whole = true;
  for (const at::Tensor* t : list)
    if (t->defined() && whole) {
      made[n] = THPVariable_Wrap(*t);
      whole = made[n] != nullptr;
      n += whole;
    }
  if (whole && n == 1) return made[0];
  PyObject* const r = whole ? PyTuple_New(n) : nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (r != nullptr)
      PyTuple_SET_ITEM(r, i, made[i]);
    else
      Py_DECREF(made[i]);
  }
  return r;
}

// x, weight, eps, residual, total, y, y_dtype
PyObject* rmsnorm(Args a) {
  NormArgs v(a);
  const c10::Device dev = v.x.device();
  const int64_t n = v.x.size(0), h = v.x.size(1);
  const On on(dev);
  v.open(a);
  const at::Tensor y =
      a[5] != Py_None
          ? tensor(a[5], "y")
          : empty({n, h}, a[6] != Py_None ? dtype(a[6], "y_dtype") : v.x.scalar_type(), dev);
  const int type = act_type(y.scalar_type(), "y");
  const int64_t ys = rows_arg(y, "y", n, h, dev);
  check(moe_rmsnorm(&v.r, out(y), type, ys, on.stream), "moe_rmsnorm");
  return results({&y, &v.total});
}

// x, weight, eps, residual, total, q, scale
PyObject* rmsnorm_int8(Args a) {
  NormArgs v(a);
  const c10::Device dev = v.x.device();
  const int64_t n = v.x.size(0), h = v.x.size(1);
  const On on(dev);
  v.open(a);
  const at::Tensor q = a[5] != Py_None ? tensor(a[5], "q") : empty({n, h}, at::kChar, dev);
  const at::Tensor scale = a[6] != Py_None ? tensor(a[6], "scale") : empty({n}, at::kFloat, dev);
  dense_arg(q, "q", at::kChar, n * h, dev);
  dense_arg(scale, "scale", at::kFloat, n, dev);
  check(moe_rmsnorm_int8(&v.r, out<int8_t>(q), out<float>(scale), on.stream), "moe_rmsnorm_int8");
  return results({&q, &scale, &v.total});
}

// Scale words of n rows of c columns.  The shape is looked at, not the size
// alone: scale bytes by rows [n][c / 32] are as many where c is a multiple of 512.
void scale_words_arg(const at::Tensor& t, int64_t n, int64_t c, c10::Device dev) {
  const int64_t words = MOE_MXFP4_WORDS(c);
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == words && t.size(1) == n && t.size(2) == 16,
                    "scales must be words of shape (", words, ", ", n, ", 16), have ", t.sizes());
  dense_arg(t, "scales", at::kByte, words * n * 16, dev);
}

// Codes and scale words of n rows of c columns, given or new.
struct Mxfp4Out {
  at::Tensor codes, scales;
  Mxfp4Out(PyObject* given, PyObject* given_scales, int64_t n, int64_t c, c10::Device dev) {
    const int64_t words = MOE_MXFP4_WORDS(c);
    codes = given != Py_None ? tensor(given, "codes") : empty({n, c / 2}, at::kByte, dev);
    scales = given_scales != Py_None ? tensor(given_scales, "scales")
                                     : empty({words, n, 16}, at::kByte, dev);
    dense_arg(codes, "codes", at::kByte, n * (c / 2), dev);
    scale_words_arg(scales, n, c, dev);
  }
};

// x, weight, eps, residual, total, codes, scales
PyObject* rmsnorm_mxfp4(Args a) {
  NormArgs v(a);
  const c10::Device dev = v.x.device();
  const On on(dev);
  v.open(a);
  const Mxfp4Out o(a[5], a[6], v.x.size(0), v.x.size(1), dev);
  check(moe_rmsnorm_mxfp4(&v.r, out<uint8_t>(o.codes), out<uint8_t>(o.scales), on.stream),
        "moe_rmsnorm_mxfp4");
  return results({&o.codes, &o.scales, &v.total});
}

// dy, s, weight, eps, dtotal, dx, dweight, need_dweight
PyObject* rmsnorm_backward(Args a) {
  const at::Tensor& dy = tensor(a[0], "dy");
  const at::Tensor& s = tensor(a[1], "s");
  const at::Tensor& w = tensor(a[2], "weight");
  const c10::Device dev = s.device();
  TORCH_CHECK_VALUE(s.dim() == 2, "s must be a matrix");
  const int64_t n = s.size(0), h = s.size(1);
  const int dy_type = act_type(dy.scalar_type(), "dy"), s_type = act_type(s.scalar_type(), "s");
  const int w_type = act_type(w.scalar_type(), "weight");
  const int64_t ys = rows_arg(dy, "dy", n, h, dev), ss = rows_arg(s, "s", n, h, dev);
  dense_arg(w, "weight", w.scalar_type(), h, dev);
  const int rows = size(n, "s"), hidden = size(h, "hidden");
  const float eps = number(a[3]);
  const int need = PyObject_IsTrue(a[7]);
  if (need < 0) throw Failed();
  on_gpu(dev);
  const void* dtotal = nullptr;
  int64_t ts = 0;
  if (a[4] != Py_None) {
    const at::Tensor& t = tensor(a[4], "dtotal");
    TORCH_CHECK_VALUE(t.scalar_type() == s.scalar_type(), "dtotal must have s's dtype");
    ts = rows_arg(t, "dtotal", n, h, dev);
    dtotal = in(t);
  }
  const On on(dev);
  const at::Tensor dx = output(a[5], "dx", "s", {n, h}, s.scalar_type(), dev);
  const int64_t ds = rows_arg(dx, "dx", n, h, dev);
  at::Tensor dw, workspace;
  size_t bytes = 0;
  if (a[6] != Py_None || need) {
    dw = a[6] != Py_None ? tensor(a[6], "dweight") : empty({h}, at::kFloat, dev);
    dense_arg(dw, "dweight", at::kFloat, h, dev);
    bytes = moe_rmsnorm_backward_workspace_bytes(rows, hidden);
    // freed to the stream's pool when the call returns, behind its kernels
    workspace = empty({(int64_t)bytes}, at::kByte, dev);
  }
  check(moe_rmsnorm_backward(in(dy), dy_type, ys, in(s), s_type, ss, in(w), w_type, dtotal, ts, rows,
                             hidden, eps, out(dx), ds, dw.defined() ? out<float>(dw) : nullptr,
                             workspace.defined() ? out(workspace) : nullptr, bytes, on.stream),
        "moe_rmsnorm_backward");
  return results({&dx, &dw});
}

// x, codes, scales
PyObject* quantize_mxfp4(Args a) {
  const at::Tensor& x = tensor(a[0], "x");
  const c10::Device dev = x.device();
  TORCH_CHECK_VALUE(x.dim() == 2, "x must be a matrix");
  const int64_t n = x.size(0), c = x.size(1);
  const int type = act_type(x.scalar_type(), "x");
  const int64_t xs = rows_arg(x, "x", n, c, dev);
  on_gpu(dev);
  const On on(dev);
  const Mxfp4Out o(a[1], a[2], n, c, dev);
  check(moe_quantize_mxfp4(in(x), type, xs, size(n, "x"), size(c, "cols"), out<uint8_t>(o.codes),
                           out<uint8_t>(o.scales), on.stream),
        "moe_quantize_mxfp4");
  return pair(o.codes, o.scales);
}

// Codes [n][cols/2] and scale words [words][n][16] of a product's left operand.
struct Mxfp4In {
  const at::Tensor &codes, &scales;
  int64_t n, cols;
  c10::Device dev;
  Mxfp4In(PyObject* c, PyObject* s)
      : codes(tensor(c, "codes")), scales(tensor(s, "scales")), n(0), cols(0), dev(codes.device()) {
    TORCH_CHECK_VALUE(codes.dim() == 2, "codes must be [rows][cols / 2]");
    n = codes.size(0);
    cols = 2 * codes.size(1);
    dense_arg(codes, "codes", at::kByte, n * (cols / 2), dev);
    scale_words_arg(scales, n, cols, dev);
  }
};

// codes, scales, dtype, x
PyObject* dequantize_mxfp4(Args a) {
  const Mxfp4In v(a[0], a[1]);
  on_gpu(v.dev);
  const On on(v.dev);
  const at::Tensor x =
      a[3] != Py_None ? tensor(a[3], "x") : empty({v.n, v.cols}, dtype(a[2], "dtype"), v.dev);
  const int type = act_type(x.scalar_type(), "x");
  const int64_t xs = rows_arg(x, "x", v.n, v.cols, v.dev);
  check(moe_dequantize_mxfp4(in<uint8_t>(v.codes), in<uint8_t>(v.scales), size(v.n, "codes"),
                             size(v.cols, "cols"), out(x), type, xs, on.stream),
        "moe_dequantize_mxfp4");
  return THPVariable_Wrap(x);
}

// address of the moe_mxfp4_weight and its codes, address of the up one or 0
// and its codes or None, then codes, scales, grouping, top_k, out_dtype, out
PyObject* product_mxfp4(Args a) {
  const auto* w = static_cast<const moe_mxfp4_weight*>(PyLong_AsVoidPtr(a[0]));
  const auto* up = static_cast<const moe_mxfp4_weight*>(PyLong_AsVoidPtr(a[2]));
  if (PyErr_Occurred()) throw Failed();
  const c10::Device wd = tensor(a[1], "the weight").device();
  const Mxfp4In x(a[4], a[5]);
  TORCH_CHECK_VALUE(x.cols == w->cols, "codes must be [rows][", w->cols / 2, "]");
  TORCH_CHECK_VALUE(wd == x.dev, "the weights are on ", wd, ", codes are on ", x.dev);
  if (up != nullptr) {
    const c10::Device ud = tensor(a[3], "the up weight").device();
    TORCH_CHECK_VALUE(ud == x.dev, "the up weights are on ", ud, ", codes are on ", x.dev);
  }
  const int k = integer(a[7], "top_k");
  const int64_t n = x.n * (k != 0 ? k : 1), rows = w->rows;
  Grouping g{};
  if (a[6] != Py_None) {
    g = grouping_arg(a[6], n, x.dev);
    TORCH_CHECK_VALUE(g.n_experts == w->n_experts, "the grouping has ", g.n_experts,
                      " experts, the weights ", w->n_experts);
  }
  on_gpu(x.dev);
  const On on(x.dev);
  const at::Tensor o =
      a[9] != Py_None ? tensor(a[9], "out") : empty({n, rows}, dtype(a[8], "out_dtype"), x.dev);
  const int type = act_type(o.scalar_type(), "out");
  const int64_t os = rows_arg(o, "out", n, rows, x.dev);
  const auto *codes = in<uint8_t>(x.codes), *scales = in<uint8_t>(x.scales);
  if (up != nullptr)
    check(moe_swiglu_mxfp4(w, up, codes, scales, size(n, "codes"), g.offsets, g.perm, k, out(o),
                           type, os, on.stream),
          "moe_swiglu_mxfp4");
  else
    check(moe_product_mxfp4(w, codes, scales, size(n, "codes"), g.offsets, g.perm, k, out(o), type,
                            os, on.stream),
          "moe_product_mxfp4");
  return THPVariable_Wrap(o);
}

template <PyObject* (*F)(Args), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Failed&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(Args), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<set_error, 1>("set_error"),
                         method<dispatch, 4>("dispatch"),
                         method<dispatch_backward, 4>("dispatch_backward"),
                         method<combine, 6>("combine"),
                         method<combine_backward, 6>("combine_backward"),
                         method<route_backward, 6>("route_backward"),
                         method<quantize_int8, 3>("quantize_int8"),
                         method<product_int8, 10>("product_int8"),
                         method<rmsnorm, 7>("rmsnorm"),
                         method<rmsnorm_int8, 7>("rmsnorm_int8"),
                         method<rmsnorm_mxfp4, 7>("rmsnorm_mxfp4"),
                         method<rmsnorm_backward, 8>("rmsnorm_backward"),
                         method<quantize_mxfp4, 3>("quantize_mxfp4"),
                         method<dequantize_mxfp4, 4>("dequantize_mxfp4"),
                         method<product_mxfp4, 10>("product_mxfp4"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "tensor_calls", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tensor_calls() { return PyModule_Create(&module); }
