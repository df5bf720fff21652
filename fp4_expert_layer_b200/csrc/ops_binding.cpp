// ops_binding.cpp -- the operators of moe_ops.h on torch tensors.
//
// A small call is bound by the host: its launch takes some 2.6 us, and checking and
// marshalling a call through ctypes took another 4 to 5.  Here they take about one.
// Nothing is computed: each function checks its arguments, allocates what the caller
// gave no place for, and calls the C entry point (by the address that ops.py passes,
// so that the checked library is reached the same way).
//
// A function returns None, having done nothing, when its first tensor is not on the
// current CUDA device; ops.py then makes that device current (or refuses).  What it
// refuses raises MoEError with MOE_ERR_INVALID_ARG, what the entry point refuses
// MoEError with its status and text.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>

#include "moe_ops.h"

namespace {

// ---------------------------------------------------------- what ops.py passes
PyObject *g_error = nullptr;      // MoEError(status, text)
PyTypeObject *g_fp4 = nullptr;    // FP4Tensor, a tuple (codes, scales, global_scale, fmt)
decltype(&moe_fp4_quantize) c_quantize = nullptr;
decltype(&moe_fp4_dequantize) c_dequantize = nullptr;
decltype(&moe_fp4_matmul) c_matmul = nullptr;
decltype(&moe_sort_tokens) c_sort = nullptr;
decltype(&moe_dispatch) c_dispatch = nullptr;
decltype(&moe_dispatch_backward) c_dispatch_backward = nullptr;
decltype(&moe_combine) c_combine = nullptr;
decltype(&moe_combine_backward) c_combine_backward = nullptr;
decltype(&moe_last_error) c_last_error = nullptr;

// A refusal on its way up: the Python error is set.
struct Refused {};

[[noreturn]] void raise(int status, const char *text) {
  if (PyObject *e = PyObject_CallFunction(g_error, "is", status, text)) {
    PyErr_SetObject(reinterpret_cast<PyObject *>(Py_TYPE(e)), e);
    Py_DECREF(e);
  }
  throw Refused{};
}
[[noreturn]] void bad(const char *fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  raise(MOE_ERR_INVALID_ARG, text);
}
void done(moe_status_t st) {
  if (st != MOE_OK) raise(st, c_last_error());
}

// -------------------------------------------------------------------- arguments
using at::Tensor;

const Tensor &tensor(PyObject *o, const char *fn, const char *name) {
  if (!THPVariable_Check(o)) bad("%s: %s must be a tensor, not %s", fn, name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
// Whether the call can run as things are: its first tensor on the current device.
bool here(const Tensor &t) { return t.is_cuda() && t.get_device() == c10::cuda::current_device(); }

void same(const char *fn, const Tensor &first, const char *name, const Tensor &t) {
  if (t.device() != first.device())
    bad("%s: %s is on %s, not on %s", fn, name, t.device().str().c_str(), first.device().str().c_str());
}
int32_t any_type(const char *fn, const char *name, const Tensor &t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MOE_DT_F32;
    case at::kBFloat16: return MOE_DT_BF16;
    case at::kHalf: return MOE_DT_F16;
    case at::kByte: return MOE_DT_U8;
    default: bad("%s: %s cannot be %s", fn, name, c10::toString(t.scalar_type()));
  }
}
int32_t float_type(const char *fn, const char *name, const Tensor &t) {
  const int32_t d = any_type(fn, name, t);
  if (d == MOE_DT_U8) bad("%s: %s must be float32, bfloat16 or float16", fn, name);
  return d;
}
// Row stride of a 2-D tensor with contiguous rows.
int64_t row_stride(const char *fn, const char *name, const Tensor &t) {
  if (t.size(1) > 1 && t.stride(1) != 1) bad("%s: the rows of %s must be contiguous", fn, name);
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}
void two_axes(const char *fn, const char *name, const Tensor &t) {
  if (t.dim() != 2) bad("%s: %s must have two axes, not %d", fn, name, (int)t.dim());
}
// The entry points take sizes as int32.
int32_t size32(const char *fn, const char *what, int64_t n) {
  if (n < 0 || n > 0x7FFFFFFF) bad("%s: %s = %lld must be 0 to 2^31 - 1", fn, what, (long long)n);
  return (int32_t)n;
}
void contiguous(const char *fn, const char *name, const Tensor &t, at::ScalarType type, at::IntArrayRef shape) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) {
    std::string want;
    for (int64_t n : shape) want += (want.empty() ? "" : ", ") + std::to_string(n);
    bad("%s: %s must be contiguous %s [%s]", fn, name, c10::toString(type), want.c_str());
  }
}
Tensor make(at::IntArrayRef shape, at::ScalarType type, const Tensor &like) {
  int64_t strides[4], s = 1;
  for (int i = (int)shape.size() - 1; i >= 0; --i) {
    strides[i] = s;
    s *= std::max<int64_t>(shape[i], 1);
  }
  return at::detail::empty_strided_cuda(shape, at::IntArrayRef(strides, shape.size()), type, like.device());
}
void *stream_of(const Tensor &t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }
template <typename T>
T *ptr(const Tensor &t) { return static_cast<T *>(t.data_ptr()); }

PyObject *wrap(const Tensor &t) {
  PyObject *o = THPVariable_Wrap(t);
  if (!o) throw Refused{};
  return o;
}
PyObject *given(PyObject *o) { Py_INCREF(o); return o; }

// What autograd has to know of a caller's tensor that is written past the dispatcher.  A
// graph that records it would keep the old value's gradient: refused, as torch's own out=
// is.  A graph that has saved it goes by its version.
const Tensor &writable(const char *fn, const Tensor &out) {
  if (c10::GradMode::is_enabled() && out.requires_grad())
    bad("%s: out requires grad, and the write would not be in its graph (detach it, or call under torch.no_grad())", fn);
  return out;
}
// An input whose gradient the caller may expect: the result is detached all the same.
void detached(const char *fn, const char *name, const Tensor &t) {
  if (!t.requires_grad() || !c10::GradMode::is_enabled()) return;
  char text[256];
  snprintf(text, sizeof text,
           "%s: %s requires grad, but no graph is recorded: the gradients are calls of their own (detach it, or call "
           "under torch.no_grad() or within a torch.autograd.Function)", fn, name);
  if (PyErr_WarnEx(PyExc_UserWarning, text, 2) < 0) throw Refused{};
}
void written(const Tensor &out) {
  if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
}
// The call's result: a new tensor, or the one that the caller gave.
PyObject *handed(PyObject *out_o, const Tensor &out) {
  if (out_o == Py_None) return wrap(out);
  written(out);
  return given(out_o);
}

int block_of(PyObject *fmt) {       // elements of a block, 0 if the format is unknown
  if (!PyUnicode_Check(fmt)) return 0;
  if (PyUnicode_CompareWithASCIIString(fmt, "mxfp4") == 0) return 32;
  return PyUnicode_CompareWithASCIIString(fmt, "nvfp4") == 0 ? 16 : 0;
}
int64_t whole(const char *fn, const char *name, PyObject *o) {
  const int64_t n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad("%s: %s must be a whole number", fn, name);
  }
  return n;
}
at::ScalarType dtype_of(const char *fn, PyObject *o) {
  if (!THPDtype_Check(o)) bad("%s: a dtype was expected, not %s", fn, Py_TYPE(o)->tp_name);
  return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// An FP4Tensor whose parts fit together and are on one device.
struct Fp4 {
  const Tensor *codes, *scales, *G;   // G: NULL for mxfp4
  PyObject *fmt_name;
  int32_t fmt;
  int64_t K, rows;
  const uint8_t *c() const { return ptr<const uint8_t>(*codes); }
  const uint8_t *s() const { return ptr<const uint8_t>(*scales); }
  float *g() const { return G ? ptr<float>(*G) : nullptr; }
};
const Tensor &codes_of(PyObject *o, const char *fn, const char *name) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4)
    bad("%s: %s must be an FP4Tensor (codes, scales, global_scale, fmt)", fn, name);
  return tensor(PyTuple_GET_ITEM(o, 0), fn, "codes");
}
Fp4 fp4(PyObject *o, const char *fn, const char *name, const Tensor &first) {
  Fp4 q;
  q.codes = &codes_of(o, fn, name);
  q.scales = &tensor(PyTuple_GET_ITEM(o, 1), fn, "scales");
  q.fmt_name = PyTuple_GET_ITEM(o, 3);
  const int block = block_of(q.fmt_name);
  if (!block) bad("%s: the format of %s is not 'mxfp4' or 'nvfp4'", fn, name);
  q.fmt = block == 16 ? MOE_FMT_NVFP4 : MOE_FMT_MXFP4;
  PyObject *g = PyTuple_GET_ITEM(o, 2);
  if ((g == Py_None) != (block == 32)) bad("%s: %s.global_scale belongs to nvfp4, and to it alone", fn, name);
  q.G = g == Py_None ? nullptr : &tensor(g, fn, "global_scale");
  const Tensor &c = *q.codes;
  if (c.dim() < 1 || c.scalar_type() != at::kByte || !c.is_contiguous()) bad("%s: %s.codes must be contiguous uint8", fn, name);
  q.K = 2 * c.size(-1);
  if (q.K % 32) bad("%s: K = %lld of %s is not a multiple of 32", fn, (long long)q.K, name);
  q.rows = 1;
  for (int64_t n : c.sizes().slice(0, c.dim() - 1)) q.rows *= n;
  const Tensor &s = *q.scales;
  bool fits = s.scalar_type() == at::kByte && s.is_contiguous() && s.dim() == c.dim() && s.size(-1) == q.K / block;
  for (int i = 0; fits && i + 1 < c.dim(); ++i) fits = s.size(i) == c.size(i);
  if (!fits) bad("%s: %s.scales must be contiguous uint8, one for each %d elements of the codes", fn, name, block);
  same(fn, first, "codes", c);
  same(fn, first, "scales", s);
  if (q.G) {
    if (q.G->scalar_type() != at::kFloat || !q.G->is_contiguous()) bad("%s: %s.global_scale must be contiguous float32", fn, name);
    same(fn, first, "global_scale", *q.G);
  }
  return q;
}
PyObject *make_fp4(const Tensor &codes, const Tensor &scales, const Tensor *G, PyObject *fmt) {
  PyObject *items = PyTuple_New(4), *args = PyTuple_New(1);
  PyTuple_SET_ITEM(items, 0, wrap(codes));
  PyTuple_SET_ITEM(items, 1, wrap(scales));
  PyTuple_SET_ITEM(items, 2, G ? wrap(*G) : given(Py_None));
  PyTuple_SET_ITEM(items, 3, given(fmt));
  PyTuple_SET_ITEM(args, 0, items);
  PyObject *q = PyTuple_Type.tp_new(g_fp4, args, nullptr);   // as the named tuple's own constructor does
  Py_DECREF(args);
  if (!q) throw Refused{};
  return q;
}

// ------------------------------------------------------------------------- FP4
// (x, fmt, rows_per_scale | None, out | None)
PyObject *quantize(PyObject *const *a) {
  static const char fn[] = "fp4_quantize";
  const Tensor &x = tensor(a[0], fn, "x");
  if (!here(x)) Py_RETURN_NONE;
  const int block = block_of(a[1]);
  if (!block) bad("%s: the format is not 'mxfp4' or 'nvfp4'", fn);
  const bool nv = block == 16;
  const int dim = (int)x.dim();
  if (dim != 2 && dim != 3) bad("%s: x must have two or three axes, not %d", fn, dim);
  const int64_t K = x.size(-1), n = dim == 2 ? x.size(0) : x.size(0) * x.size(1);
  int64_t per = dim == 3 ? std::max<int64_t>(1, x.size(1)) : 1;
  if (a[2] != Py_None) per = whole(fn, "rows_per_scale", a[2]);
  if (per < 1 || n % per) bad("%s: %lld rows are not a multiple of rows_per_scale = %lld", fn, (long long)n, (long long)per);
  if (K < 32 || K % 32) bad("%s: K = %lld is not a multiple of 32", fn, (long long)K);
  const int32_t type = float_type(fn, "x", x);
  if (x.stride(-1) != 1) bad("%s: the rows of x must be contiguous", fn);
  // one row stride for all rows: that of the axis that has more than one entry
  int64_t ld = K;
  if (dim == 2) {
    if (n > 1) ld = x.stride(0);
  } else if (n > 1) {
    ld = x.size(1) > 1 ? x.stride(1) : x.stride(0);
    if (x.size(0) > 1 && x.size(1) > 1 && x.stride(0) != x.size(1) * ld)
      bad("%s: the matrices of x must follow one another at one row stride", fn);
  }
  int64_t cs[3], ss[3];
  for (int i = 0; i < dim; ++i) cs[i] = ss[i] = x.size(i);
  cs[dim - 1] = K / 2;
  ss[dim - 1] = K / block;
  Tensor codes, scales, G;
  if (a[3] == Py_None) {
    codes = make(at::IntArrayRef(cs, dim), at::kByte, x);
    scales = make(at::IntArrayRef(ss, dim), at::kByte, x);
    if (nv) G = make({n / per}, at::kFloat, x);
  } else {
    const Fp4 q = fp4(a[3], fn, "out", x);
    if ((q.fmt == MOE_FMT_NVFP4) != nv || q.codes->sizes() != at::IntArrayRef(cs, dim))
      bad("%s: out is of another format or shape", fn);
    codes = *q.codes;
    scales = *q.scales;
    if (nv) {
      G = writable(fn, *q.G);
      contiguous(fn, "out.global_scale", G, at::kFloat, {n / per});
    }
  }
  done(c_quantize(x.data_ptr(), type, n, K, ld, nv ? MOE_FMT_NVFP4 : MOE_FMT_MXFP4, per, ptr<uint8_t>(codes),
                  ptr<uint8_t>(scales), nv ? ptr<float>(G) : nullptr, stream_of(x)));
  if (a[3] == Py_None) return make_fp4(codes, scales, nv ? &G : nullptr, a[1]);
  written(codes);
  written(scales);
  if (nv) written(G);
  return given(a[3]);
}

// (q, dtype, out | None)
PyObject *dequantize(PyObject *const *a) {
  static const char fn[] = "fp4_dequantize";
  const Tensor &c = codes_of(a[0], fn, "q");
  if (!here(c)) Py_RETURN_NONE;
  const Fp4 q = fp4(a[0], fn, "q", c);
  const int dim = (int)c.dim();
  if (dim > 4) bad("%s: q has more than four axes", fn);
  int64_t per = 1;
  if (q.G) {
    const int64_t groups = q.G->numel();
    if (q.rows && (!groups || q.rows % groups))
      bad("%s: %lld global scales do not divide %lld rows", fn, (long long)groups, (long long)q.rows);
    per = std::max<int64_t>(1, q.rows / std::max<int64_t>(1, groups));
    detached(fn, "q.global_scale", *q.G);
  }
  int64_t shape[4];
  for (int i = 0; i < dim; ++i) shape[i] = c.size(i);
  shape[dim - 1] = q.K;
  Tensor out;
  int64_t ld = q.K;
  if (a[2] == Py_None) {
    out = make(at::IntArrayRef(shape, dim), dtype_of(fn, a[1]), c);
  } else {
    out = writable(fn, tensor(a[2], fn, "out"));
    same(fn, c, "out", out);
    if (out.sizes() != at::IntArrayRef(shape, dim)) bad("%s: out is of another shape", fn);
    if (dim == 2) ld = row_stride(fn, "out", out);
    else if (!out.is_contiguous()) bad("%s: out must be contiguous", fn);
  }
  done(c_dequantize(q.c(), q.s(), q.g(), q.fmt, q.rows, q.K, per, out.data_ptr(), float_type(fn, "out", out), ld,
                    stream_of(c)));
  return handed(a[2], out);
}

// (x, w, offsets | None, out_dtype, out | None)
PyObject *matmul(PyObject *const *a) {
  static const char fn[] = "fp4_matmul";
  const Tensor &xc = codes_of(a[0], fn, "x");
  if (!here(xc)) Py_RETURN_NONE;
  const Fp4 x = fp4(a[0], fn, "x", xc), w = fp4(a[1], fn, "w", xc);
  const int wd = (int)w.codes->dim();
  if (xc.dim() != 2 || (wd != 2 && wd != 3) || w.K != x.K || w.fmt != x.fmt)
    bad("%s: x (%lld rows of %lld) and w (%d axes, rows of %lld) do not multiply, or differ in format", fn,
        (long long)x.rows, (long long)x.K, wd, (long long)w.K);
  const int32_t n = size32(fn, "rows", x.rows), N = size32(fn, "N", w.codes->size(wd - 2)),
                groups = wd == 3 ? size32(fn, "groups", w.codes->size(0)) : 1, K = size32(fn, "K", x.K);
  if (x.G) {
    contiguous(fn, "x.global_scale", *x.G, at::kFloat, {n});
    contiguous(fn, "w.global_scale", *w.G, at::kFloat, {groups});
    detached(fn, "x.global_scale", *x.G);
    detached(fn, "w.global_scale", *w.G);
  }
  const int32_t *offsets = nullptr;
  if (a[2] != Py_None) {
    const Tensor &o = tensor(a[2], fn, "offsets");
    contiguous(fn, "offsets", o, at::kInt, {(int64_t)groups + 1});
    same(fn, xc, "offsets", o);
    offsets = ptr<const int32_t>(o);
  } else if (groups != 1) {
    bad("%s: %d groups need offsets", fn, groups);
  }
  Tensor out;
  if (a[4] == Py_None) {
    out = make({n, N}, dtype_of(fn, a[3]), xc);
  } else {
    out = writable(fn, tensor(a[4], fn, "out"));
    same(fn, xc, "out", out);
    if (out.dim() != 2 || out.size(0) != n || out.size(1) != N) bad("%s: out must be [%d, %d]", fn, n, N);
  }
  done(c_matmul(x.c(), x.s(), x.g(), n, w.c(), w.s(), w.g(), groups, N, K, x.fmt, offsets, out.data_ptr(),
                float_type(fn, "out", out), row_stride(fn, "out", out), stream_of(xc)));
  return handed(a[4], out);
}

// ------------------------------------------------------------------ expert rows
// (ids, n_experts)
PyObject *sort_tokens(PyObject *const *a) {
  static const char fn[] = "sort_tokens";
  static PyObject *names[4] = {PyUnicode_InternFromString("counts"), PyUnicode_InternFromString("offsets"),
                               PyUnicode_InternFromString("perm"), PyUnicode_InternFromString("inv")};
  const Tensor &ids = tensor(a[0], fn, "ids");
  if (!here(ids)) Py_RETURN_NONE;
  if (ids.dim() != 2 || ids.scalar_type() != at::kInt || !ids.is_contiguous())
    bad("%s: ids must be contiguous int32 [T, k]", fn);
  const int64_t T = ids.size(0), k = ids.size(1), E = whole(fn, "n_experts", a[1]);
  size32(fn, "T * k", T * k);
  if (E < 1 || E > 1024) bad("%s: %lld experts: 1 to 1024 are supported", fn, (long long)E);
  const Tensor got[4] = {make({E}, at::kInt, ids), make({E + 1}, at::kInt, ids), make({T * k}, at::kInt, ids),
                         make({T, k}, at::kInt, ids)};
  done(c_sort(ptr<const int32_t>(ids), size32(fn, "T", T), (int32_t)k, (int32_t)E, ptr<int32_t>(got[0]),
              ptr<int32_t>(got[1]), ptr<int32_t>(got[2]), ptr<int32_t>(got[3]), stream_of(ids)));
  PyObject *d = PyDict_New();
  for (int i = 0; i < 4; ++i) {
    PyObject *t = wrap(got[i]);
    PyDict_SetItem(d, names[i], t);
    Py_DECREF(t);
  }
  return d;
}

struct Pairs {
  const int32_t *inv;
  const float *gates;
  int32_t T, k;
};
// inv int32 [T, k] (T: -1 for any) and gates fp32 of its shape, or None.
Pairs pairs(const char *fn, const Tensor &first, PyObject *inv_o, PyObject *gates_o, int64_t T) {
  const Tensor &inv = tensor(inv_o, fn, "inv");
  if (inv.dim() != 2 || inv.scalar_type() != at::kInt || !inv.is_contiguous() || (T >= 0 && inv.size(0) != T))
    bad("%s: inv must be contiguous int32 [T, k]%s", fn, T >= 0 ? ", a row for each token" : "");
  same(fn, first, "inv", inv);
  size32(fn, "T * k", inv.size(0) * inv.size(1));
  Pairs p{ptr<const int32_t>(inv), nullptr, size32(fn, "T", inv.size(0)), size32(fn, "k", inv.size(1))};
  if (gates_o && gates_o != Py_None) {
    const Tensor &g = tensor(gates_o, fn, "gates");
    contiguous(fn, "gates", g, at::kFloat, inv.sizes());
    same(fn, first, "gates", g);
    detached(fn, "gates", g);
    p.gates = ptr<const float>(g);
  }
  return p;
}
// The result: `out_o` if it is [n, cols] (and of this type, if one is asked for), else a new tensor.
Tensor result(const char *fn, const Tensor &first, PyObject *out_o, int64_t n, int64_t cols, at::ScalarType type,
              bool typed) {
  if (out_o == Py_None) return make({n, cols}, type, first);
  const Tensor &out = writable(fn, tensor(out_o, fn, "out"));
  same(fn, first, "out", out);
  if (out.dim() != 2 || out.size(0) != n || out.size(1) != cols || (typed && out.scalar_type() != type))
    bad("%s: out must be %s [%lld, %lld]", fn, typed ? c10::toString(type) : "of a float type", (long long)n, (long long)cols);
  return out;
}

// (x, inv, rows | None, out | None)
PyObject *dispatch(PyObject *const *a) {
  static const char fn[] = "dispatch";
  const Tensor &x = tensor(a[0], fn, "x");
  if (!here(x)) Py_RETURN_NONE;
  two_axes(fn, "x", x);
  detached(fn, "x", x);
  const int64_t H = x.size(1);
  const Pairs p = pairs(fn, x, a[1], nullptr, x.size(0));
  int64_t rows = (int64_t)p.T * p.k;
  if (a[2] != Py_None) rows = whole(fn, "rows", a[2]);
  else if (a[3] != Py_None && THPVariable_Check(a[3]) && THPVariable_Unpack(a[3]).dim() == 2) rows = THPVariable_Unpack(a[3]).size(0);
  size32(fn, "rows", rows);
  const int32_t type = any_type(fn, "x", x);
  const Tensor out = result(fn, x, a[3], rows, H, x.scalar_type(), true);
  done(c_dispatch(x.data_ptr(), type, p.T, p.k, size32(fn, "H", H), row_stride(fn, "x", x), p.inv, (int32_t)rows,
                  out.data_ptr(), row_stride(fn, "out", out), stream_of(x)));
  return handed(a[3], out);
}

// (dxs, inv, out | None)
PyObject *dispatch_backward(PyObject *const *a) {
  static const char fn[] = "dispatch_backward";
  const Tensor &d = tensor(a[0], fn, "dxs");
  if (!here(d)) Py_RETURN_NONE;
  two_axes(fn, "dxs", d);
  detached(fn, "dxs", d);
  const int32_t rows = size32(fn, "rows", d.size(0)), H = size32(fn, "H", d.size(1)), type = float_type(fn, "dxs", d);
  const Pairs p = pairs(fn, d, a[1], nullptr, -1);
  const Tensor out = result(fn, d, a[2], p.T, H, d.scalar_type(), true);
  done(c_dispatch_backward(d.data_ptr(), type, rows, p.T, p.k, H, row_stride(fn, "dxs", d), p.inv, out.data_ptr(),
                           row_stride(fn, "out", out), stream_of(d)));
  return handed(a[2], out);
}

// (ys, inv, gates | None, out_dtype | None, out | None)
PyObject *combine(PyObject *const *a) {
  static const char fn[] = "combine";
  const Tensor &ys = tensor(a[0], fn, "ys");
  if (!here(ys)) Py_RETURN_NONE;
  two_axes(fn, "ys", ys);
  detached(fn, "ys", ys);
  const int32_t rows = size32(fn, "rows", ys.size(0)), H = size32(fn, "H", ys.size(1)), type = float_type(fn, "ys", ys);
  const Pairs p = pairs(fn, ys, a[1], a[2], -1);
  const at::ScalarType want = a[3] == Py_None ? ys.scalar_type() : dtype_of(fn, a[3]);
  const Tensor out = result(fn, ys, a[4], p.T, H, want, a[3] != Py_None);
  done(c_combine(ys.data_ptr(), type, rows, p.T, p.k, H, row_stride(fn, "ys", ys), p.inv, p.gates, out.data_ptr(),
                 float_type(fn, "out", out), row_stride(fn, "out", out), stream_of(ys)));
  return handed(a[4], out);
}

// (dy, ys, inv, gates | None, out | None)
PyObject *combine_backward(PyObject *const *a) {
  static const char fn[] = "combine_backward";
  const Tensor &dy = tensor(a[0], fn, "dy");
  if (!here(dy)) Py_RETURN_NONE;
  const Tensor &ys = tensor(a[1], fn, "ys");
  two_axes(fn, "dy", dy);
  two_axes(fn, "ys", ys);
  same(fn, dy, "ys", ys);
  detached(fn, "dy", dy);
  detached(fn, "ys", ys);
  if (ys.size(1) != dy.size(1)) bad("%s: dy and ys have rows of %lld and %lld", fn, (long long)dy.size(1), (long long)ys.size(1));
  const int32_t rows = size32(fn, "rows", ys.size(0)), H = size32(fn, "H", ys.size(1));
  const int32_t td = float_type(fn, "dy", dy), ts = float_type(fn, "ys", ys);
  const Pairs p = pairs(fn, dy, a[2], a[3], dy.size(0));
  const Tensor out = result(fn, dy, a[4], rows, H, ys.scalar_type(), true);
  const Tensor dgates = make({p.T, p.k}, at::kFloat, dy);
  done(c_combine_backward(dy.data_ptr(), td, row_stride(fn, "dy", dy), ys.data_ptr(), ts, row_stride(fn, "ys", ys), rows,
                          p.T, p.k, H, p.inv, p.gates, out.data_ptr(), row_stride(fn, "out", out), ptr<float>(dgates),
                          stream_of(dy)));
  PyObject *both = PyTuple_New(2);
  PyTuple_SET_ITEM(both, 0, handed(a[4], out));
  PyTuple_SET_ITEM(both, 1, wrap(dgates));
  return both;
}

// ----------------------------------------------------------------------- module
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// setup(MoEError, FP4Tensor, addresses of the nine entry points in the order below)
PyObject *setup(PyObject *, PyObject *args) {
  PyObject *error, *fp4;
  unsigned long long p[9];
  if (!PyArg_ParseTuple(args, "OOKKKKKKKKK", &error, &fp4, p, p + 1, p + 2, p + 3, p + 4, p + 5, p + 6, p + 7, p + 8))
    return nullptr;
  if (!PyType_Check(fp4) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject *>(fp4), &PyTuple_Type)) {
    PyErr_SetString(PyExc_TypeError, "FP4Tensor must be a tuple type");
    return nullptr;
  }
  Py_INCREF(error);
  Py_INCREF(fp4);
  g_error = error;
  g_fp4 = reinterpret_cast<PyTypeObject *>(fp4);
  c_quantize = reinterpret_cast<decltype(c_quantize)>(p[0]);
  c_dequantize = reinterpret_cast<decltype(c_dequantize)>(p[1]);
  c_matmul = reinterpret_cast<decltype(c_matmul)>(p[2]);
  c_sort = reinterpret_cast<decltype(c_sort)>(p[3]);
  c_dispatch = reinterpret_cast<decltype(c_dispatch)>(p[4]);
  c_dispatch_backward = reinterpret_cast<decltype(c_dispatch_backward)>(p[5]);
  c_combine = reinterpret_cast<decltype(c_combine)>(p[6]);
  c_combine_backward = reinterpret_cast<decltype(c_combine_backward)>(p[7]);
  c_last_error = reinterpret_cast<decltype(c_last_error)>(p[8]);
  Py_RETURN_NONE;
}

#define MOE_FAST(name, f, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, nullptr},
    MOE_FAST("fp4_quantize", quantize, 4),
    MOE_FAST("fp4_dequantize", dequantize, 3),
    MOE_FAST("fp4_matmul", matmul, 5),
    MOE_FAST("sort_tokens", sort_tokens, 2),
    MOE_FAST("dispatch", dispatch, 4),
    MOE_FAST("dispatch_backward", dispatch_backward, 3),
    MOE_FAST("combine", combine, 5),
    MOE_FAST("combine_backward", combine_backward, 5),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", "operators on torch tensors (see ops.py)", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__ops() {
  PyObject *m = PyModule_Create(&module);
  if (m) PyModule_AddStringConstant(m, "built_for", MOE_TORCH_VERSION);
  return m;
}
