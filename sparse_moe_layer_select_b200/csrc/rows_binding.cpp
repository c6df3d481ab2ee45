// rows_binding.cpp -- argument marshalling of the row and 8-bit integer calls of
// include/moe_rows.h (module _rows_binding, used by moe.py).
//
// These calls take few microseconds on the device at decode sizes, less than Python
// needs to ask five tensors for their shapes, strides and addresses and to convert a
// dozen arguments (8 to 16 us a call).  Here types, sizes and strides are read and
// checked in C++ and the C ABI function is called directly.  Every function takes its
// arguments in the order of its Python namesake and returns the call's status code, or
// a string that says which argument does not fit (nothing has been launched then).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/moe_rows.h"

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const char *name, const std::string &why) {
  throw Refused(std::string(name) + ": " + why);
}

std::string shape_of(const at::Tensor &t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

// The arguments of one call, and the one device that its tensors are on.
struct Args {
  PyObject *const *a;
  Py_ssize_t n;
  int device = -1;

  Args(PyObject *const *args, Py_ssize_t nargs, Py_ssize_t expected) : a(args), n(nargs) {
    if (n != expected) throw Refused("wrong number of arguments");
  }
  bool none(int i) const { return a[i] == Py_None; }

  // Tensor i; its device becomes the call's, or has to be it.
  const at::Tensor &tensor(int i, const char *name) {
    if (!THPVariable_Check(a[i])) refuse(name, "not a tensor");
    const at::Tensor &t = THPVariable_Unpack(a[i]);
    const int dev = t.is_cuda() ? static_cast<int>(t.get_device()) : -1;
    if (dev < 0) refuse(name, "not on a CUDA device");
    if (device >= 0 && dev != device) refuse(name, "on another device than the arguments before it");
    device = dev;
    return t;
  }
  // The raw stream of the call: the given one, or the current one of the tensors' device,
  // which has to be the current device.
  void *stream(int i) {
    if (device >= 0 && c10::cuda::current_device() != device)
      throw Refused("the tensors are not on the current device");
    if (none(i)) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    PyObject *v = PyObject_GetAttrString(a[i], "cuda_stream");
    void *s = v != nullptr ? PyLong_AsVoidPtr(v) : nullptr;
    Py_XDECREF(v);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse("stream", "not a CUDA stream");
    }
    // (torch's streams name their device; others are taken as they are)
    PyObject *d = PyObject_GetAttrString(a[i], "device_index");
    const long on = d != nullptr ? PyLong_AsLong(d) : device;
    Py_XDECREF(d);
    PyErr_Clear();
    if (device >= 0 && on != device) refuse("stream", "of another device than the tensors");
    return s;
  }
};

moe_dims_t dims_of(PyObject *o) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    refuse("dims", "not a moe_dims_t");
  }
  const bool ok = b.len == static_cast<Py_ssize_t>(sizeof(moe_dims_t));
  moe_dims_t d{};
  if (ok) d = *static_cast<const moe_dims_t *>(b.buf);
  PyBuffer_Release(&b);
  if (!ok) refuse("dims", "not a moe_dims_t");
  return d;
}

int dtype_of(const at::Tensor &t, const char *name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_DTYPE_BF16;
    case at::kHalf: return MOE_DTYPE_F16;
    case at::kFloat: return MOE_DTYPE_F32;
    default: refuse(name, std::string("type ") + c10::toString(t.scalar_type()));
  }
}

// A [rows, cols] matrix whose rows are contiguous: its address and row stride (a single
// row has none: one that is a multiple of 16).
struct Rows {
  void *p = nullptr;
  int64_t stride = 0;
  int dtype = MOE_DTYPE_BF16;
};

Rows matrix(const at::Tensor &t, int64_t rows, int64_t cols, const char *name) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(name, "shape " + shape_of(t) + ", expected (" + std::to_string(rows) + ", " +
                     std::to_string(cols) + ")");
  if (cols > 1 && t.stride(1) != 1) refuse(name, "elements of a row are not adjacent");
  Rows r;
  r.p = t.data_ptr();
  r.stride = rows > 1 ? t.stride(0) : (cols + 15) / 16 * 16;
  return r;
}

Rows rows_of(const at::Tensor &t, int64_t rows, int64_t cols, const char *name) {
  const int dtype = dtype_of(t, name);
  Rows r = matrix(t, rows, cols, name);
  r.dtype = dtype;
  return r;
}

// The same of a given type.
Rows rows_like(const at::Tensor &t, int64_t rows, int64_t cols, int dtype, const char *name) {
  Rows r = rows_of(t, rows, cols, name);
  if (r.dtype != dtype) refuse(name, "another type than the rows it goes with");
  return r;
}

Rows codes_of(const at::Tensor &t, int64_t rows, int64_t cols, const char *name) {
  if (t.scalar_type() != at::kChar) refuse(name, "not int8");
  return matrix(t, rows, cols, name);
}

void *flat(const at::Tensor &t, int64_t n, at::ScalarType type, const char *name) {
  if (t.numel() != n || t.scalar_type() != type || !t.is_contiguous())
    refuse(name, std::to_string(t.numel()) + " elements of " + c10::toString(t.scalar_type()) +
                     ", expected " + std::to_string(n) + " of " + c10::toString(type) +
                     ", contiguous");
  return t.data_ptr();
}

int32_t *ints(const at::Tensor &t, int64_t n, const char *name) {
  return static_cast<int32_t *>(flat(t, n, at::kInt, name));
}
float *floats(const at::Tensor &t, int64_t n, const char *name) {
  return static_cast<float *>(flat(t, n, at::kFloat, name));
}

// A workspace: its address and bytes; null where it may be left out.
void *workspace(Args &g, int i, size_t *bytes) {
  if (g.none(i)) return nullptr;
  const at::Tensor &t = g.tensor(i, "ws");
  *bytes = static_cast<size_t>(t.numel()) * t.element_size();
  if (*bytes < 256 || !t.is_contiguous()) refuse("ws", "fewer than 256 bytes, or not contiguous");
  return t.data_ptr();
}

int64_t slots(const moe_dims_t &d) { return static_cast<int64_t>(d.T) * d.num_experts_per_tok; }

// sort(dims, topk_idx, counts, offsets, perm, inv, ws, x, x_perm, stream)
int sort(Args g) {
  const moe_dims_t d = dims_of(g.a[0]);
  const int64_t n = slots(d);
  const int32_t *idx = ints(g.tensor(1, "topk_idx"), n, "topk_idx");
  int32_t *counts = ints(g.tensor(2, "counts"), d.num_experts, "counts");
  int32_t *offsets = ints(g.tensor(3, "offsets"), d.num_experts + int64_t(1), "offsets");
  int32_t *perm = ints(g.tensor(4, "perm"), n, "perm");
  int32_t *inv = ints(g.tensor(5, "inv"), n, "inv");
  size_t bytes = 0;
  void *ws = workspace(g, 6, &bytes);
  Rows x, p;
  if (g.none(7) != g.none(8)) throw Refused("x without x_perm, or x_perm without x");
  if (!g.none(7)) {
    x = rows_of(g.tensor(7, "x"), d.T, d.d_model, "x");
    p = rows_like(g.tensor(8, "x_perm"), n, d.d_model, x.dtype, "x_perm");
  }
  return moe_sort(&d, idx, counts, offsets, perm, inv, x.dtype, x.p, x.stride, p.p, p.stride, ws,
                  bytes, g.stream(9));
}

// dispatch(dims, x, inv, x_perm, ws, stream)
int dispatch(Args g) {
  const moe_dims_t d = dims_of(g.a[0]);
  const int64_t n = slots(d);
  const Rows x = rows_of(g.tensor(1, "x"), d.T, d.d_model, "x");
  const int32_t *inv = ints(g.tensor(2, "inv"), n, "inv");
  const Rows p = rows_like(g.tensor(3, "x_perm"), n, d.d_model, x.dtype, "x_perm");
  size_t bytes = 0;
  void *ws = workspace(g, 4, &bytes);
  return moe_dispatch(&d, x.dtype, x.p, x.stride, inv, p.p, p.stride, ws, g.stream(5));
}

// dispatch_backward(dims, d_x_perm, inv, d_x, ws, add, stream)
int dispatch_backward(Args g) {
  const moe_dims_t d = dims_of(g.a[0]);
  const int64_t n = slots(d);
  const Rows p = rows_of(g.tensor(1, "d_x_perm"), n, d.d_model, "d_x_perm");
  const int32_t *inv = ints(g.tensor(2, "inv"), n, "inv");
  const Rows x = rows_of(g.tensor(3, "d_x"), d.T, d.d_model, "d_x");
  size_t bytes = 0;
  void *ws = workspace(g, 4, &bytes);
  Rows add;
  if (!g.none(5)) add = rows_like(g.tensor(5, "add"), d.T, d.d_model, p.dtype, "add");
  return moe_dispatch_backward(&d, p.dtype, p.p, p.stride, inv, add.p, add.stride, x.dtype, x.p,
                               x.stride, ws, g.stream(6));
}

// combine(dims, o, inv, topk_w, y, ws, shared, stream)
int combine(Args g) {
  const moe_dims_t d = dims_of(g.a[0]);
  const int64_t n = slots(d);
  const Rows o = rows_of(g.tensor(1, "o"), n, d.d_model, "o");
  const int32_t *inv = ints(g.tensor(2, "inv"), n, "inv");
  const float *w = floats(g.tensor(3, "topk_w"), n, "topk_w");
  const Rows y = rows_of(g.tensor(4, "y"), d.T, d.d_model, "y");
  size_t bytes = 0;
  void *ws = workspace(g, 5, &bytes);
  Rows sh;
  if (!g.none(6)) sh = rows_like(g.tensor(6, "shared"), d.T, d.d_model, o.dtype, "shared");
  return moe_combine(&d, o.dtype, o.p, o.stride, inv, w, sh.p, sh.stride, y.dtype, y.p, y.stride,
                     ws, g.stream(7));
}

// combine_backward(dims, d_y, o, inv, topk_w, d_o, d_topk_w, ws, stream)
int combine_backward(Args g) {
  const moe_dims_t d = dims_of(g.a[0]);
  const int64_t n = slots(d);
  const Rows y = rows_of(g.tensor(1, "d_y"), d.T, d.d_model, "d_y");
  const Rows o = rows_like(g.tensor(2, "o"), n, d.d_model, y.dtype, "o");
  const int32_t *inv = ints(g.tensor(3, "inv"), n, "inv");
  const float *w = floats(g.tensor(4, "topk_w"), n, "topk_w");
  const Rows go = rows_like(g.tensor(5, "d_o"), n, d.d_model, y.dtype, "d_o");
  float *gw = floats(g.tensor(6, "d_topk_w"), n, "d_topk_w");
  size_t bytes = 0;
  void *ws = workspace(g, 7, &bytes);
  return moe_combine_backward(&d, y.dtype, y.p, y.stride, o.p, o.stride, inv, w, go.p, go.stride,
                              gw, ws, g.stream(8));
}

// route_backward(dims, logits, topk_idx, d_topk_w, d_logits, ws, stream)
int route_backward(Args g) {
  const moe_dims_t d = dims_of(g.a[0]);
  const int64_t n = slots(d), all = static_cast<int64_t>(d.T) * d.num_experts;
  const float *l = floats(g.tensor(1, "logits"), all, "logits");
  const int32_t *idx = ints(g.tensor(2, "topk_idx"), n, "topk_idx");
  const float *w = floats(g.tensor(3, "d_topk_w"), n, "d_topk_w");
  float *out = floats(g.tensor(4, "d_logits"), all, "d_logits");
  size_t bytes = 0;
  void *ws = workspace(g, 5, &bytes);
  return moe_route_backward(&d, l, idx, w, out, ws, g.stream(6));
}

// quantize_int8(x, codes, scales, n_rows, stream)
int quantize_int8(Args g) {
  const at::Tensor &t = g.tensor(0, "x");
  if (t.dim() != 2) refuse("x", "shape " + shape_of(t) + ", expected a matrix");
  const int64_t rows = t.size(0), cols = t.size(1);
  if (rows > INT32_MAX || cols > INT32_MAX) refuse("x", "more than 2^31 - 1 rows or columns");
  const Rows x = rows_of(t, rows, cols, "x");
  const Rows q = codes_of(g.tensor(1, "codes"), rows, cols, "codes");
  float *s = floats(g.tensor(2, "scales"), rows, "scales");
  const int32_t *valid = g.none(3) ? nullptr : ints(g.tensor(3, "n_rows"), 1, "n_rows");
  return moe_quantize_int8(static_cast<int32_t>(rows), static_cast<int32_t>(cols), x.dtype, x.p,
                           x.stride, valid, static_cast<int8_t *>(q.p), q.stride, s, g.stream(4));
}

// dispatch_int8(dims, x, inv, codes, scales, ws, stream)
int dispatch_int8(Args g) {
  const moe_dims_t d = dims_of(g.a[0]);
  const int64_t n = slots(d);
  const Rows x = rows_of(g.tensor(1, "x"), d.T, d.d_model, "x");
  const int32_t *inv = ints(g.tensor(2, "inv"), n, "inv");
  const Rows q = codes_of(g.tensor(3, "codes"), n, d.d_model, "codes");
  float *s = floats(g.tensor(4, "scales"), n, "scales");
  size_t bytes = 0;
  void *ws = workspace(g, 5, &bytes);
  return moe_dispatch_int8(&d, x.dtype, x.p, x.stride, inv, static_cast<int8_t *>(q.p), q.stride,
                           s, ws, g.stream(6));
}

// matmul_int8(a, a_scale, b, b_scale, out, ws, offsets, swiglu, stream)
int matmul_int8(Args g) {
  const at::Tensor &ta = g.tensor(0, "a");
  if (ta.dim() != 2) refuse("a", "shape " + shape_of(ta) + ", expected a matrix");
  const int64_t M = ta.size(0), K = ta.size(1);
  const bool grouped = !g.none(6);
  const int sw = PyObject_IsTrue(g.a[7]);
  if (sw < 0) {
    PyErr_Clear();
    refuse("swiglu", "not a truth value");
  }
  const at::Tensor &tb = g.tensor(2, "b");
  if (tb.dim() != (grouped ? 3 : 2) || tb.size(-1) != K)
    refuse("b", "shape " + shape_of(tb) + " for a of " + shape_of(ta));
  if (tb.scalar_type() != at::kChar) refuse("b", "not int8");
  const int64_t G = grouped ? tb.size(0) : 1, b_rows = tb.size(-2);
  if (sw == 1 && b_rows % 2 != 0) refuse("b", "an odd number of rows for gate and up");
  const int64_t N = sw == 1 ? b_rows / 2 : b_rows;
  if (M > INT32_MAX || K > INT32_MAX || N > INT32_MAX || G > INT32_MAX)
    refuse("a, b", "more than 2^31 - 1 rows or columns");
  if (K > 1 && tb.stride(-1) != 1) refuse("b", "elements of a row are not adjacent");
  // rows of all groups, one stride apart
  int64_t b_stride = (K + 15) / 16 * 16;
  if (b_rows > 1) b_stride = tb.stride(-2);
  else if (G > 1) b_stride = tb.stride(0);
  if (G > 1 && b_rows > 1 && tb.stride(0) != b_rows * b_stride)
    refuse("b", "the groups' rows are not evenly spaced");
  moe_int8_matmul_t m{};
  m.struct_size = sizeof(m);
  m.M = static_cast<int32_t>(M);
  m.N = static_cast<int32_t>(N);
  m.K = static_cast<int32_t>(K);
  m.G = static_cast<int32_t>(G);
  m.flags = sw == 1 ? MOE_INT8_SWIGLU : 0;
  const Rows a = codes_of(ta, M, K, "a");
  m.a = static_cast<const int8_t *>(a.p);
  m.a_stride = a.stride;
  m.a_scale = floats(g.tensor(1, "a_scale"), M, "a_scale");
  m.b = static_cast<const int8_t *>(tb.data_ptr());
  m.b_stride = b_stride;
  m.b_scale = floats(g.tensor(3, "b_scale"), G * b_rows, "b_scale");
  const Rows out = rows_of(g.tensor(4, "out"), M, N, "out");
  m.out_dtype = out.dtype;
  m.out = out.p;
  m.out_stride = out.stride;
  size_t bytes = 0;
  void *ws = workspace(g, 5, &bytes);
  if (grouped) m.offsets = ints(g.tensor(6, "offsets"), G + 1, "offsets");
  return moe_matmul_int8(&m, ws, bytes, g.stream(8));
}

template <int (*F)(Args), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
  try {
    return PyLong_FromLong(F(Args(args, nargs, N)));
  } catch (const Refused &e) {
    return PyUnicode_FromString(e.what());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    return nullptr;
  }
}

#define MOE_METHOD(f, n) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOE_METHOD(sort, 10),           MOE_METHOD(dispatch, 6),
                         MOE_METHOD(dispatch_backward, 7), MOE_METHOD(combine, 8),
                         MOE_METHOD(combine_backward, 9),  MOE_METHOD(route_backward, 7),
                         MOE_METHOD(quantize_int8, 5),     MOE_METHOD(dispatch_int8, 7),
                         MOE_METHOD(matmul_int8, 9),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rows_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__rows_binding() { return PyModule_Create(&module); }
