// The calls of moe_rows.h and moe_int8.h on torch tensors: argument checks,
// outputs, the current stream, the C entry.  Their kernels take a few
// microseconds at the size of one token, where the same steps in Python took
// three times that (one token's combine, submission: 14 us through ctypes);
// binding.py holds the signatures and the documentation.
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
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "tensor_calls", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tensor_calls() { return PyModule_Create(&module); }
