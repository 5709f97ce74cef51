// torch_binding.cpp -- the operators' tensor calls: shape and
// type checks, pointers, leading dimensions, the current stream, outputs and
// workspaces, one call into the C ABI (include/dgemm.h).  No arithmetic.
//
// The functions take their arguments by position from ops.py, which documents
// them.  They are C++ rather than Python because a small call is over in a few
// microseconds on the GPU: on a GB300's host layer_norm of one row with its
// statistics costs 6.6 us here and 14 us through ctypes, most of it
// allocations and attribute reads that are several times cheaper from C++.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>
#include <vector>

#include "../../include/dgemm.h"

namespace {

using at::Tensor;

// A refusal: becomes the Python exception `type`.
struct Refused {
  PyObject *type;
  std::string text;
};
[[noreturn]] void value_error(const std::string &s) { throw Refused{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string &s) { throw Refused{PyExc_TypeError, s}; }
struct PythonError {};  // the Python error is already set

PyObject *g_raise = nullptr;  // ops._raise(status, what)

void check(int status, const char *what) {
  if (status == DGEMM_OK) return;
  PyObject *r = PyObject_CallFunction(g_raise, "is", status, what);
  Py_XDECREF(r);
  if (r != nullptr) PyErr_SetString(PyExc_RuntimeError, what);  // not reached: _raise raises
  throw PythonError{};
}

std::string name_of(at::ScalarType t) { return std::string("torch.") + c10::toString(t); }

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}
bool given(PyObject *o) { return o != Py_None; }

int type_code(const Tensor &x, const char *what, bool f32) {
  switch (x.scalar_type()) {
    case at::kBFloat16: return DGEMM_DTYPE_BF16;
    case at::kHalf: return DGEMM_DTYPE_F16;
    case at::kFloat:
      if (f32) return DGEMM_DTYPE_F32;
      break;
    default: break;
  }
  type_error(std::string(what) + " takes torch.bfloat16, torch.float16" +
             (f32 ? ", torch.float32" : "") + ", got " + name_of(x.scalar_type()));
}

int as_int(int64_t n, const char *name) {
  if (n > INT_MAX) value_error(std::string(name) + ": " + std::to_string(n) + " is too large");
  return (int)n;
}

void want_type(const Tensor &t, const char *name, at::ScalarType type) {
  if (t.scalar_type() != type)
    type_error(std::string(name) + ": expected " + name_of(type) + ", got " +
               name_of(t.scalar_type()));
}

// A tensor's leading dimensions flattened into rows.
struct Mat {
  void *p;
  int rows, cols, ld;
};
Mat rows_of(const Tensor &t, const char *name, at::ScalarType type) {
  want_type(t, name, type);
  if (t.dim() == 0) value_error(std::string(name) + ": expected at least one dimension");
  const int64_t cols = t.size(-1);
  int64_t rows = 1, ld, inner;
  if (t.dim() == 2) {
    rows = t.size(0), ld = t.stride(0), inner = t.stride(1);
  } else {
    for (int64_t i = 0; i + 1 < t.dim(); ++i) rows *= t.size(i);
    // every leading stride has to be the one the dimension after it gives
    ld = t.dim() > 1 ? t.stride(-2) : cols, inner = t.stride(-1);
    int64_t want = 0;
    bool first = true;
    for (int64_t i = t.dim() - 2; i >= 0 && rows > 1; --i) {
      if (t.size(i) == 1) continue;
      if (first) {
        ld = t.stride(i);
        first = false;
      } else if (t.stride(i) != want) {
        value_error(std::string(name) + ": the leading dimensions do not flatten into rows");
      }
      want = t.stride(i) * t.size(i);
    }
  }
  if (inner != 1 && cols > 1 && rows > 0)
    value_error(std::string(name) + ": the last dimension must be contiguous");
  if (rows <= 1) ld = cols > 0 ? cols : 1;
  return {t.data_ptr(), as_int(rows, name), as_int(cols, name), as_int(ld, name)};
}
Mat like(const Tensor &t, const char *name, at::ScalarType type, int rows, int cols) {
  const Mat m = rows_of(t, name, type);
  if (m.cols != cols)
    value_error(std::string(name) + ": the last dimension is " + std::to_string(m.cols) +
                ", expected " + std::to_string(cols));
  if (m.rows != rows)
    value_error(std::string(name) + ": " + std::to_string(m.rows) + " rows, expected " +
                std::to_string(rows));
  return m;
}
Mat like_or_none(PyObject *o, const char *name, at::ScalarType type, int rows, int cols) {
  if (!given(o)) return {nullptr, rows, cols, cols > 0 ? cols : 1};
  return like(tensor(o, name), name, type, rows, cols);
}

void *vector_or_none(PyObject *o, const char *name, at::ScalarType type, int n) {
  if (!given(o)) return nullptr;
  const Tensor &t = tensor(o, name);
  want_type(t, name, type);
  if (t.dim() != 1 || t.size(0) != n)
    value_error(std::string(name) + ": expected " + std::to_string(n) + " elements");
  if (n > 1 && t.stride(0) != 1) value_error(std::string(name) + ": must be contiguous");
  return t.data_ptr();
}

// The statistics of n rows, contiguous in any shape.
void *stats(PyObject *o, const char *name, int n) {
  const Tensor &t = tensor(o, name);
  want_type(t, name, at::kFloat);
  if (t.numel() != n) value_error(std::string(name) + ": expected " + std::to_string(n) + " elements");
  if (!t.is_contiguous()) value_error(std::string(name) + ": must be contiguous");
  return t.data_ptr();
}

// A weight: inner x outer, or outer x inner when transposed.
Mat weight(const Tensor &w, const char *name, at::ScalarType type, int inner, int outer, bool t) {
  want_type(w, name, type);
  const int rows = t ? outer : inner, cols = t ? inner : outer;
  if (w.dim() != 2 || w.size(0) != rows || w.size(1) != cols)
    value_error(std::string(name) + ": expected " + std::to_string(rows) + "x" +
                std::to_string(cols));
  return rows_of(w, name, type);
}

int outer_of(const Tensor &w, const char *name, bool t) {
  if (w.dim() != 2) value_error(std::string(name) + ": expected a 2-D matrix");
  return as_int(t ? w.size(0) : w.size(1), name);
}

cudaStream_t current_stream(const Tensor &x) {
  if (!x.is_cuda()) value_error("expected CUDA tensors");
  return c10::cuda::getCurrentCUDAStream(x.device().index()).stream();
}

Tensor make(at::IntArrayRef sizes, const Tensor &like) { return at::empty(sizes, like.options()); }
// x's shape with `cols` for its last dimension.
Tensor make_rows(const Tensor &x, int64_t cols) {
  if (x.dim() == 2) return make({x.size(0), cols}, x);
  auto sizes = x.sizes().vec();
  sizes.back() = cols;
  return make(sizes, x);
}
// A rows x cols workspace whose rows start on 16-byte boundaries.
Tensor pitched(int64_t rows, int64_t cols, const Tensor &like, int *ld) {
  const int64_t pitch = (cols + 7) / 8 * 8;
  *ld = as_int(pitch > 0 ? pitch : 1, "a workspace's rows");
  return make({rows, pitch}, like);
}
// `out`, which has to have x's leading dimensions and `cols` columns of `type`, or a
// new tensor like that.
Tensor out_or_new(PyObject *out, const Tensor &x, int rows, int cols, Mat *m, at::ScalarType type) {
  Tensor t;
  if (given(out)) {
    t = tensor(out, "out");
  } else if (type == x.scalar_type()) {
    t = make_rows(x, cols);
  } else {
    auto sizes = x.sizes().vec();
    sizes.back() = cols;
    t = at::empty(sizes, x.options().dtype(type));
  }
  if (given(out)) {
    bool same = t.dim() == x.dim();
    for (int64_t i = 0; same && i < x.dim(); ++i)
      same = t.size(i) == (i + 1 < x.dim() ? x.size(i) : cols);
    if (!same) value_error("out: has another shape than the result");
  }
  *m = like(t, "out", type, rows, cols);
  return t;
}
Tensor out_or_new(PyObject *out, const Tensor &x, int rows, int cols, Mat *m) {
  return out_or_new(out, x, rows, cols, m, x.scalar_type());
}

int pos(int n) { return n > 0 ? n : 1; }

PyObject *tuple(std::initializer_list<const Tensor *> ts) {
  PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
  if (r == nullptr) throw PythonError{};
  Py_ssize_t i = 0;
  for (const Tensor *t : ts) {
    PyObject *o = t != nullptr ? THPVariable_Wrap(*t) : (Py_INCREF(Py_None), Py_None);
    if (o == nullptr) {
      Py_DECREF(r);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

bool flag(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}
int integer(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return (int)v;
}

// A forward call's results have no gradient function, so an argument that requires
// gradients is refused where autograd would record.
void refuse_recording(const char *what, PyObject *const *args, int n, bool backward = true) {
  if (!c10::GradMode::is_enabled()) return;
  for (int i = 0; i < n; ++i)
    if (THPVariable_Check(args[i]) && THPVariable_Unpack(args[i]).requires_grad())
      throw Refused{PyExc_RuntimeError,
                    std::string(what) + " does not record gradients, and an argument requires them: call "
                    "it under torch.no_grad()" +
                        (backward ? std::string(", and ") + what + "_backward for the gradients" : "")};
}

// (x, weight, bias, eps, return_stats, out)
PyObject *layer_norm(PyObject *const *a) {
  refuse_recording("layer_norm", a, 6);
  const Tensor &x = tensor(a[0], "x");
  const int dt = type_code(x, "layer_norm", true);
  const auto type = x.scalar_type();
  const Mat m = rows_of(x, "x", type);
  void *w = vector_or_none(a[1], "weight", type, m.cols), *b = vector_or_none(a[2], "bias", type, m.cols);
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw PythonError{};
  const cudaStream_t stream = current_stream(x);
  Mat y;
  const Tensor out = out_or_new(a[5], x, m.rows, m.cols, &y);
  if (!flag(a[4])) {
    check(dgemm_layer_norm(dt, m.rows, m.cols, (float)eps, m.p, m.ld, w, b, y.p, y.ld, nullptr,
                           nullptr, stream),
          "layer_norm");
    return THPVariable_Wrap(out);
  }
  const auto sizes = x.sizes().slice(0, x.dim() - 1);
  const auto options = x.options().dtype(at::kFloat);
  // rows without columns have no statistics, and the library writes none
  auto stat = [&] { return m.cols > 0 ? at::empty(sizes, options) : at::full(sizes, NAN, options); };
  const Tensor mean = stat(), rstd = stat();
  check(dgemm_layer_norm(dt, m.rows, m.cols, (float)eps, m.p, m.ld, w, b, y.p, y.ld,
                         static_cast<float *>(mean.data_ptr()),
                         static_cast<float *>(rstd.data_ptr()), stream),
        "layer_norm");
  return tuple({&out, &mean, &rstd});
}

// (dy, x, weight, mean, rstd, dresidual)
PyObject *layer_norm_backward(PyObject *const *a) {
  const Tensor &x = tensor(a[1], "x");
  const int dt = type_code(x, "layer_norm_backward", true);
  const auto type = x.scalar_type();
  const Mat m = rows_of(x, "x", type);
  const Mat dy = like(tensor(a[0], "dy"), "dy", type, m.rows, m.cols);
  const Mat dr = like_or_none(a[5], "dresidual", type, m.rows, m.cols);
  void *w = vector_or_none(a[2], "weight", type, m.cols);
  const float *mean = static_cast<float *>(stats(a[3], "mean", m.rows));
  const float *rstd = static_cast<float *>(stats(a[4], "rstd", m.rows));
  const cudaStream_t stream = current_stream(x);
  const Tensor dx = make(x.sizes(), x), dw = make({m.cols}, x), db = make({m.cols}, x);
  check(dgemm_layer_norm_backward(dt, m.rows, m.cols, dy.p, dy.ld, m.p, m.ld, w, mean, rstd, dr.p,
                                  dr.ld, dx.data_ptr(), pos(m.cols), dw.data_ptr(), db.data_ptr(),
                                  stream),
        "layer_norm_backward");
  return tuple({&dx, &dw, &db});
}

// (x, w, bias, activation, residual, trans_w, return_preact, out)
PyObject *linear(PyObject *const *a) {
  refuse_recording("linear", a, 8);
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
  const int dt = type_code(x, "linear", false), act = integer(a[3]);
  const bool t = flag(a[5]), keep = flag(a[6]);
  const auto type = x.scalar_type();
  const Mat m = rows_of(x, "x", type);
  const int N = outer_of(w, "w", t);
  const Mat mw = weight(w, "w", type, m.cols, N, t);
  void *b = vector_or_none(a[2], "bias", type, N);
  const Mat r = like_or_none(a[4], "residual", type, m.rows, N);
  if (given(a[7])) (void)like(tensor(a[7], "out"), "out", type, m.rows, N);
  const cudaStream_t stream = current_stream(x);
  Mat d;
  const Tensor out = out_or_new(a[7], x, m.rows, N, &d);
  Tensor z;
  if (keep) z = make_rows(x, N);
  check(dgemm_linear(dt, act, t ? DGEMM_OP_T : DGEMM_OP_N, m.rows, N, m.cols, m.p, m.ld, mw.p,
                     mw.ld, b, r.p, r.ld, d.p, d.ld, keep ? z.data_ptr() : nullptr, pos(N), stream),
        "linear");
  return keep ? tuple({&out, &z}) : THPVariable_Wrap(out);
}

// (dd, x, w, activation, preact, trans_w, with_bias)
PyObject *linear_backward(PyObject *const *a) {
  const Tensor &x = tensor(a[1], "x"), &w = tensor(a[2], "w");
  const int dt = type_code(x, "linear_backward", false), act = integer(a[3]);
  const bool t = flag(a[5]), bias = flag(a[6]);
  const auto type = x.scalar_type();
  const Mat m = rows_of(x, "x", type);
  const int N = outer_of(w, "w", t);
  const Mat mw = weight(w, "w", type, m.cols, N, t);
  const Mat dd = like(tensor(a[0], "dd"), "dd", type, m.rows, N);
  Mat z = {nullptr, m.rows, N, pos(N)};
  Tensor dz;
  int lddz = pos(N);
  if (act != DGEMM_ACT_NONE) {
    if (!given(a[4])) value_error("preact is needed for this activation");
    z = like(tensor(a[4], "preact"), "preact", type, m.rows, N);
  }
  const cudaStream_t stream = current_stream(x);
  if (act != DGEMM_ACT_NONE) dz = pitched(m.rows, N, x, &lddz);
  const Tensor dx = make(x.sizes(), x), dw = make(w.sizes(), w);
  Tensor db;
  if (bias) db = make({N}, x);
  check(dgemm_linear_backward(dt, act, t ? DGEMM_OP_T : DGEMM_OP_N, m.rows, N, m.cols, dd.p, dd.ld,
                              m.p, m.ld, mw.p, mw.ld, z.p, z.ld, dz.defined() ? dz.data_ptr() : nullptr,
                              lddz, dx.data_ptr(), pos(m.cols), dw.data_ptr(), pos(mw.cols),
                              bias ? db.data_ptr() : nullptr, stream),
        "linear_backward");
  return tuple({&dx, &dw, bias ? &db : nullptr});
}

// A gated block's input and weights.
struct Block {
  int dt, F;
  at::ScalarType type;
  Mat x, wg, wu, wd;
};
Block block(const char *what, const Tensor &x, const Tensor &wg, const Tensor &wu,
            const Tensor &wd, bool t) {
  Block b;
  b.dt = type_code(x, what, false);
  b.type = x.scalar_type();
  b.x = rows_of(x, "x", b.type);
  b.F = outer_of(wg, "w_gate", t);
  b.wg = weight(wg, "w_gate", b.type, b.x.cols, b.F, t);
  b.wu = weight(wu, "w_up", b.type, b.x.cols, b.F, t);
  b.wd = weight(wd, "w_down", b.type, b.F, b.x.cols, t);
  return b;
}

// (x, w_gate, w_up, w_down, activation, residual, trans_w, return_saved, out)
PyObject *gated_ffn(PyObject *const *a) {
  refuse_recording("gated_ffn", a, 9);
  const Tensor &x = tensor(a[0], "x");
  const bool t = flag(a[6]), keep = flag(a[7]);
  const int act = integer(a[4]);
  const Block b = block("gated_ffn", x, tensor(a[1], "w_gate"), tensor(a[2], "w_up"),
                        tensor(a[3], "w_down"), t);
  const Mat r = like_or_none(a[5], "residual", b.type, b.x.rows, b.x.cols);
  if (given(a[8])) (void)like(tensor(a[8], "out"), "out", b.type, b.x.rows, b.x.cols);
  const cudaStream_t stream = current_stream(x);
  Mat y;
  const Tensor out = out_or_new(a[8], x, b.x.rows, b.x.cols, &y);
  Tensor g, u;
  if (keep) g = make_rows(x, b.F), u = make_rows(x, b.F);
  int ldh = 1;
  const Tensor h = pitched(b.x.rows, b.F, x, &ldh);
  check(dgemm_gated_ffn(b.dt, act, t ? DGEMM_OP_T : DGEMM_OP_N, b.x.rows, b.x.cols, b.F, b.x.p,
                        b.x.ld, b.wg.p, b.wg.ld, b.wu.p, b.wu.ld, b.wd.p, b.wd.ld, r.p, r.ld,
                        h.data_ptr(), ldh, keep ? g.data_ptr() : nullptr, pos(b.F),
                        keep ? u.data_ptr() : nullptr, pos(b.F), y.p, y.ld, stream),
        "gated_ffn");
  return keep ? tuple({&out, &g, &u}) : THPVariable_Wrap(out);
}

// (dy, x, w_gate, w_up, w_down, g, u, activation, trans_w)
PyObject *gated_ffn_backward(PyObject *const *a) {
  const Tensor &x = tensor(a[1], "x"), &wg = tensor(a[2], "w_gate"), &wu = tensor(a[3], "w_up");
  const Tensor &wd = tensor(a[4], "w_down");
  const bool t = flag(a[8]);
  const int act = integer(a[7]);
  const Block b = block("gated_ffn_backward", x, wg, wu, wd, t);
  const Mat dy = like(tensor(a[0], "dy"), "dy", b.type, b.x.rows, b.x.cols);
  const Mat g = like(tensor(a[5], "g"), "g", b.type, b.x.rows, b.F);
  const Mat u = like(tensor(a[6], "u"), "u", b.type, b.x.rows, b.F);
  const cudaStream_t stream = current_stream(x);
  const Tensor dx = make(x.sizes(), x), dwg = make(wg.sizes(), x), dwu = make(wu.sizes(), x);
  const Tensor dwd = make(wd.sizes(), x);
  int ld = 1;
  // H, dG and dU in one workspace of three times the rows
  const Tensor work = pitched(3 * (int64_t)b.x.rows, b.F, x, &ld);
  char *h = static_cast<char *>(work.data_ptr());
  const int64_t part = (int64_t)b.x.rows * work.size(1) * 2;
  check(dgemm_gated_ffn_backward(b.dt, act, t ? DGEMM_OP_T : DGEMM_OP_N, b.x.rows, b.x.cols, b.F,
                                 dy.p, dy.ld, b.x.p, b.x.ld, b.wg.p, b.wg.ld, b.wu.p, b.wu.ld,
                                 b.wd.p, b.wd.ld, g.p, g.ld, u.p, u.ld, h, ld, h + part, ld,
                                 h + 2 * part, ld, dx.data_ptr(), pos(b.x.cols), dwg.data_ptr(),
                                 pos(b.wg.cols), dwu.data_ptr(), pos(b.wg.cols), dwd.data_ptr(),
                                 pos(b.wd.cols), stream),
        "gated_ffn_backward");
  return tuple({&dx, &dwg, &dwu, &dwd});
}

// A scale for each of n rows, contiguous in any shape.
const float *scales(PyObject *o, const char *name, int n) {
  return static_cast<const float *>(stats(o, name, n));
}
Tensor bytes_like(size_t n, const Tensor &x) {
  return at::empty({(int64_t)n}, x.options().dtype(at::kByte));
}

// A tensor of the given sizes whose rows start on 16-byte boundaries, in 8 bits.
Tensor rows_of_bytes(at::IntArrayRef sizes, const Tensor &like) {
  const int64_t cols = sizes.back(), pitch = (cols + 15) / 16 * 16;
  int64_t rows = 1;
  std::vector<int64_t> strides(sizes.size(), 1);
  for (int64_t i = (int64_t)sizes.size() - 2; i >= 0; --i) {
    strides[i] = pitch * rows;
    rows *= sizes[i];
  }
  return at::empty({rows * pitch}, like.options().dtype(at::kChar)).as_strided(sizes, strides);
}

// (x, transpose)
PyObject *quantize_int8(PyObject *const *a) {
  refuse_recording("quantize_int8", a, 2, false);
  const Tensor &x = tensor(a[0], "x");
  const int dt = type_code(x, "quantize_int8", true);
  const bool t = flag(a[1]);
  const Mat m = rows_of(x, "x", x.scalar_type());
  if (t && x.dim() != 2) value_error("x: expected a 2-D matrix");
  const cudaStream_t stream = current_stream(x);
  const auto floats = x.options().dtype(at::kFloat);
  // (longer rows than the library takes are refused by it)
  const int pitch = (int)std::min<int64_t>(((int64_t)(t ? m.rows : m.cols) + 15) / 16 * 16, INT_MAX);
  const Tensor q = t ? rows_of_bytes({m.cols, m.rows}, x) : rows_of_bytes(x.sizes(), x);
  const Tensor s = t ? at::empty({m.cols}, floats) : at::empty(x.sizes().slice(0, x.dim() - 1), floats);
  check(dgemm_quantize_int8(dt, t ? DGEMM_OP_T : DGEMM_OP_N, m.rows, m.cols, m.p, m.ld,
                            static_cast<signed char *>(q.data_ptr()), pos(pitch),
                            static_cast<float *>(s.data_ptr()), stream),
        "quantize_int8");
  return tuple({&q, &s});
}

// A weight in 8 bits, outer x inner.
Mat weight_int8(const Tensor &w, const char *name, int outer, int inner) {
  return weight(w, name, at::kChar, inner, outer, true);
}

// (x, w, w_scale, bias, activation, residual, x_scale, dtype, out)
PyObject *linear_int8(PyObject *const *a) {
  refuse_recording("linear_int8", a, 9, false);
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
  const bool ints = x.scalar_type() == at::kChar;
  at::ScalarType type = ints ? at::kBFloat16 : x.scalar_type();
  if (given(a[7])) {
    if (!THPDtype_Check(a[7])) type_error("dtype: expected a torch.dtype");
    const auto want = reinterpret_cast<THPDtype *>(a[7])->scalar_type;
    if (!ints && want != type) type_error("dtype: the result has x's type, " + name_of(type));
    type = want;
  }
  if (ints != given(a[6])) type_error("x_scale comes with an int8 x, and with no other");
  if (!ints && type != at::kBFloat16 && type != at::kHalf)
    type_error("linear_int8 takes torch.bfloat16, torch.float16, torch.int8, got " + name_of(type));
  if (type != at::kBFloat16 && type != at::kHalf)
    type_error("dtype: torch.bfloat16 or torch.float16, got " + name_of(type));
  const int dt = type == at::kHalf ? DGEMM_DTYPE_F16 : DGEMM_DTYPE_BF16, act = integer(a[4]);
  const Mat m = rows_of(x, "x", x.scalar_type());
  const int N = outer_of(w, "w", true);
  const Mat mw = weight_int8(w, "w", N, m.cols);
  const float *ws = scales(a[2], "w_scale", N);
  const float *xs = ints ? scales(a[6], "x_scale", m.rows) : nullptr;
  void *b = vector_or_none(a[3], "bias", type, N);
  const Mat r = like_or_none(a[5], "residual", type, m.rows, N);
  if (given(a[8])) (void)like(tensor(a[8], "out"), "out", type, m.rows, N);
  const cudaStream_t stream = current_stream(x);
  Mat d;
  const Tensor out = out_or_new(a[8], x, m.rows, N, &d, type);
  const Tensor work = bytes_like(dgemm_linear_int8_workspace(m.rows, m.cols), x);
  check(dgemm_linear_int8(dt, act, m.rows, N, m.cols, m.p, m.ld, xs,
                          static_cast<const signed char *>(mw.p), mw.ld, ws, b, r.p, r.ld, d.p, d.ld,
                          work.data_ptr(), stream),
        "linear_int8");
  return THPVariable_Wrap(out);
}

// (x, w_gate, gate_scale, w_up, up_scale, w_down, down_scale, activation, residual, out)
PyObject *gated_ffn_int8(PyObject *const *a) {
  refuse_recording("gated_ffn_int8", a, 10, false);
  const Tensor &x = tensor(a[0], "x"), &wg = tensor(a[1], "w_gate");
  const int dt = type_code(x, "gated_ffn_int8", false), act = integer(a[7]);
  const auto type = x.scalar_type();
  const Mat m = rows_of(x, "x", type);
  const int F = outer_of(wg, "w_gate", true);
  const Mat mg = weight_int8(wg, "w_gate", F, m.cols);
  const Mat mu = weight_int8(tensor(a[3], "w_up"), "w_up", F, m.cols);
  const Mat md = weight_int8(tensor(a[5], "w_down"), "w_down", m.cols, F);
  const float *sg = scales(a[2], "gate_scale", F), *su = scales(a[4], "up_scale", F);
  const float *sd = scales(a[6], "down_scale", m.cols);
  const Mat r = like_or_none(a[8], "residual", type, m.rows, m.cols);
  if (given(a[9])) (void)like(tensor(a[9], "out"), "out", type, m.rows, m.cols);
  const cudaStream_t stream = current_stream(x);
  Mat y;
  const Tensor out = out_or_new(a[9], x, m.rows, m.cols, &y);
  const Tensor work = bytes_like(dgemm_gated_ffn_int8_workspace(m.rows, m.cols, F), x);
  auto bytes = [](const Mat &w) { return static_cast<const signed char *>(w.p); };
  check(dgemm_gated_ffn_int8(dt, act, m.rows, m.cols, F, m.p, m.ld, bytes(mg), mg.ld, sg, bytes(mu),
                             mu.ld, su, bytes(md), md.ld, sd, r.p, r.ld, y.p, y.ld, work.data_ptr(),
                             stream),
        "gated_ffn_int8");
  return THPVariable_Wrap(out);
}

double number(PyObject *o, const char *name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    if (!PyErr_ExceptionMatches(PyExc_TypeError)) throw PythonError{};
    PyErr_Clear();
    type_error(std::string(name) + ": expected a number");
  }
  return v;
}

// A new reference to a list or tuple of `o`'s items, released with the object.
struct Items {
  PyObject *seq;
  Items(PyObject *o, const char *name) : seq(PySequence_Fast(o, "")) {
    if (seq == nullptr) {
      PyErr_Clear();
      type_error(std::string(name) + ": expected a sequence of numbers");
    }
  }
  ~Items() { Py_XDECREF(seq); }
  Items(const Items &) = delete;
  Items &operator=(const Items &) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject *operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

// (x, steps, coefficients, eps, scale, residual, residual_scale, out)
PyObject *orthogonalize(PyObject *const *a) {
  refuse_recording("orthogonalize", a, 8, false);
  const Tensor &x = tensor(a[0], "x");
  const int dx = type_code(x, "orthogonalize", true);
  if (x.dim() != 2) value_error("x: expected a 2-D matrix");
  const long steps = PyLong_AsLong(a[1]);
  if (steps == -1 && PyErr_Occurred()) throw PythonError{};
  if (steps < 1 || steps > DGEMM_NEWTON_MAX_STEPS)
    value_error("steps: 1 to " + std::to_string(DGEMM_NEWTON_MAX_STEPS));
  float c[3 * DGEMM_NEWTON_MAX_STEPS];
  {
    const Items items(a[2], "coefficients");
    const bool each = items.size() > 0 && !PyNumber_Check(items[0]);
    if (items.size() != (each ? steps : 3))
      value_error("coefficients: three numbers, or three for each step");
    for (long k = 0; k < steps; ++k) {
      auto fill = [&](const Items &t) {
        if (t.size() != 3) value_error("coefficients: three numbers, or three for each step");
        for (int j = 0; j < 3; ++j) {
          const double v = number(t[j], "coefficients");
          if (!(std::fabs(v) <= 64.0)) value_error("coefficients: at most 64 in size");
          c[3 * k + j] = (float)v;
        }
      };
      if (each)
        fill(Items(items[k], "coefficients"));
      else
        fill(items);
    }
  }
  const double eps = number(a[3], "eps"), scale = number(a[4], "scale"), keep = number(a[6], "residual_scale");
  const Mat m = rows_of(x, "x", x.scalar_type());
  const auto type = given(a[5])   ? tensor(a[5], "residual").scalar_type()
                    : given(a[7]) ? tensor(a[7], "out").scalar_type()
                                  : x.scalar_type();
  const int dt = given(a[5])   ? type_code(tensor(a[5], "residual"), "residual", true)
                 : given(a[7]) ? type_code(tensor(a[7], "out"), "out", true)
                               : dx;
  const Mat r = like_or_none(a[5], "residual", type, m.rows, m.cols);
  if (given(a[7])) (void)like(tensor(a[7], "out"), "out", type, m.rows, m.cols);
  const cudaStream_t stream = current_stream(x);
  Mat d;
  const Tensor out = out_or_new(a[7], x, m.rows, m.cols, &d, type);
  const Tensor work = bytes_like(dgemm_orthogonalize_workspace(m.rows, m.cols), x);
  check(dgemm_orthogonalize(dx, dt, (int)steps, c, (float)eps, (float)scale, (float)keep, m.rows, m.cols,
                            m.p, m.ld, r.p, r.ld, d.p, d.ld, work.data_ptr(), stream),
        "orthogonalize");
  return THPVariable_Wrap(out);
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != N) type_error("wrong number of arguments");
    return F(args);
  } catch (const Refused &r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  } catch (const PythonError &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject *on_error(PyObject *, PyObject *f) {
  Py_INCREF(f);
  Py_XDECREF(g_raise);
  g_raise = f;
  Py_RETURN_NONE;
}

#define DG_FAST(f, n) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&call<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {DG_FAST(layer_norm, 6),       DG_FAST(layer_norm_backward, 6),
                           DG_FAST(linear, 8),           DG_FAST(linear_backward, 7),
                           DG_FAST(gated_ffn, 9),        DG_FAST(gated_ffn_backward, 9),
                           DG_FAST(quantize_int8, 2),    DG_FAST(linear_int8, 9),
                           DG_FAST(gated_ffn_int8, 10),  DG_FAST(orthogonalize, 8),
                           {"on_error", &on_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&g_module); }
