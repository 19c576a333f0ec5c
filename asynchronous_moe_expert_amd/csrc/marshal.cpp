// _marshal: the binding's checks of the home rank's operators' tensors, and the filling of their
// argument structs.  A decode step's calls take the GPU 3-4 us each and the launch itself takes the
// host 3.0 us, so what stands between a Python call and the launch counts: the checks of
// moe_residual_norm's nine tensors and its struct took 4.6 us in Python, where each look at a tensor
// costs 0.05-0.1 us, and take 0.3 us here (a call of 64 rows 8.4 and 4.1 us).
//
// Every function takes its operator's tensors (None where one is left out) and numbers in order, and
// last the stream's handle; the current device is the tensors' own.  A view that the kernels cannot
// address, or a size that the struct cannot hold, raises MoeError and enqueues nothing.  The
// library's entry points are handed over by setup(), which refuses a library that was built from
// another moe_step.h (other sizes of the argument structs, or another version).
#include <Python.h>

#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <exception>

#include <torch/csrc/autograd/python_variable.h>

#include "moe_step.h"

namespace {

PyObject* g_error = nullptr;  // MoeError

enum Entry { kRoute, kRouteBack, kSort, kMerge, kMergeBack, kNorm, kNormBack, kEntries };
void* g_entry[kEntries] = {};
const char* (*g_strerror)(int) = nullptr;

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const char* format, ...) {
  va_list ap;
  va_start(ap, format);
  PyErr_FormatV(g_error, format, ap);
  va_end(ap);
  throw Refused{};
}

constexpr unsigned F32 = 1, BF16 = 2, U8 = 4, I32 = 8, FP8 = U8;

unsigned kind(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return F32;
    case at::kBFloat16: return BF16;
    case at::kByte:
    case at::kFloat8_e4m3fn: return U8;
    case at::kInt: return I32;
    default: return 0;
  }
}
int code(const at::Tensor& t) { return kind(t) == F32 ? MOE_F32 : kind(t) == BF16 ? MOE_BF16 : MOE_FP8_E4M3; }
unsigned same(const at::Tensor& t) { return kind(t); }

// The call's arguments in order, and the device that its tensors share.
class Call {
 public:
  Call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : a_(args) {
    if (n != want) refuse("%zd arguments, %zd expected", n, want);
  }

  // the next argument as a tensor, nullptr for None
  const at::Tensor* opt(const char* what) {
    PyObject* o = a_[i_++];
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse("%s: a tensor is expected", what);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) refuse("%s: must be a strided tensor", what);
    if (!first_) first_ = &t;
    else if (t.device() != first_->device() && !other_) other_ = &t;
    return &t;
  }
  const at::Tensor& tensor(const char* what) {
    const at::Tensor* t = opt(what);
    if (!t) refuse("%s: required", what);
    return *t;
  }
  int64_t whole() {
    const long long v = PyLong_AsLongLong(a_[i_++]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("a whole number within the documented limits is expected");
    }
    return v;
  }
  int truth() {
    const int v = PyObject_IsTrue(a_[i_++]);
    if (v < 0) throw Refused{};
    return v;
  }
  float real() {
    const double v = PyFloat_AsDouble(a_[i_++]);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    if (std::isfinite(v) && std::fabs(v) > FLT_MAX) refuse("a number that fp32 cannot hold");
    return (float)v;
  }

  // Once every tensor is there: runs the entry point on the stream given as the last argument.
  PyObject* run(Entry e, const void* args) {
    const unsigned long long stream = PyLong_AsUnsignedLongLong(a_[i_++]);
    if (stream == (unsigned long long)-1 && PyErr_Occurred()) throw Refused{};
    if (other_)
      refuse("tensors on %s and %s", first_->device().str().c_str(), other_->device().str().c_str());
    if (!first_->is_cuda()) refuse("tensors must be on a GPU, got %s", first_->device().str().c_str());
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = ((int (*)(const void*, hipStream_t))g_entry[e])(args, (hipStream_t)stream);
    Py_END_ALLOW_THREADS
    if (rc != MOE_OK) refuse("%s (%d)", g_strerror(rc), rc);
    Py_RETURN_NONE;
  }

 private:
  PyObject* const* a_;
  Py_ssize_t i_ = 0;
  const at::Tensor* first_ = nullptr;
  const at::Tensor* other_ = nullptr;
};

int32_t i32(int64_t v) {
  if (v < INT32_MIN || v > INT32_MAX) refuse("a size of %lld is over the documented limits", (long long)v);
  return (int32_t)v;
}

void type(const char* what, const at::Tensor& t, unsigned types) {
  if (!(kind(t) & types)) refuse("%s: unsupported dtype %s", what, c10::toString(t.scalar_type()));
}

struct Shape {
  int64_t rows, cols;
};
Shape shape(const char* what, const at::Tensor& t) {
  if (t.dim() != 2) refuse("%s: %lld dimensions, 2 expected", what, (long long)t.dim());
  return {t.size(0), t.size(1)};
}

// A [rows][cols] tensor of one of `types` whose rows are contiguous; its pitch.
int64_t mat(const char* what, const at::Tensor& t, int64_t rows, int64_t cols, unsigned types) {
  type(what, t, types);
  const Shape s = shape(what, t);
  if (s.rows != rows || s.cols != cols)
    refuse("%s: shape (%lld, %lld), expected (%lld, %lld)", what, (long long)s.rows, (long long)s.cols, (long long)rows,
           (long long)cols);
  if (t.stride(1) != 1 && cols > 1) refuse("%s: the elements of a row must be contiguous", what);
  if (rows <= 1) return cols;
  if (t.stride(0) < cols)
    refuse("%s: rows overlap (stride %lld for %lld elements)", what, (long long)t.stride(0), (long long)cols);
  return t.stride(0);
}

// A contiguous tensor of one of `types` with at least n elements; its address.
void* vec(const char* what, const at::Tensor* t, int64_t n, unsigned types) {
  if (!t) return nullptr;
  type(what, *t, types);
  if (t->numel() < n)
    refuse("%s: %lld elements, at least %lld expected", what, (long long)t->numel(), (long long)n);
  if (!t->is_contiguous()) refuse("%s: must be contiguous", what);
  return t->data_ptr();
}

// What vec() takes as the first rows of a [][cols] array: flat, or with as many columns.
void* table(const char* what, const at::Tensor* t, int64_t rows, int64_t cols, unsigned types) {
  void* p = vec(what, t, rows * cols, types);
  if (t && rows && t->dim() != 1 && (t->dim() != 2 || t->size(1) != cols))
    refuse("%s: %lld dimensions, the last of %lld; %lld columns expected", what, (long long)t->dim(),
           (long long)(t->dim() ? t->size(-1) : 0), (long long)cols);
  return p;
}

// A contiguous [T][K] tensor of type `k`; its address.
void* each(const char* what, const at::Tensor& t, int64_t T, int64_t K, unsigned k) {
  mat(what, t, T, K, k);
  return vec(what, &t, T * K, k);
}

int64_t groups(int64_t H, int64_t group) {
  if (group != 0 && group != 32 && group != 64 && group != 128)
    refuse("group must be 0, 32, 64 or 128, got %lld", (long long)group);
  return group ? (H + group - 1) / group : 1;
}

size_t room(const at::Tensor* t) {
  if (!t) return 0;
  if (!t->is_contiguous()) refuse("workspace: must be contiguous");
  return (size_t)t->numel() * t->element_size();
}
void* address(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

int32_t score_of(int64_t v) {
  const int64_t gate = v & ~(int64_t)MOE_BIAS_ON_SCORE;
  if (gate != MOE_SOFTMAX && gate != MOE_SIGMOID)
    refuse("score must be MOE_SOFTMAX or MOE_SIGMOID, with MOE_BIAS_ON_SCORE or without, got %lld", (long long)v);
  return (int32_t)v;
}

// pos: T x K whole numbers in token order ([T][K] or flat), w like it or nothing; K
int64_t positions(const at::Tensor& pos, const at::Tensor* w, int64_t T) {
  const int64_t n = pos.numel(), K = T ? n / T : pos.dim() > 1 ? pos.size(-1) : 1;
  if (pos.dim() > 1 && pos.size(0) != T)
    refuse("pos: %lld rows for %lld tokens", (long long)pos.size(0), (long long)T);
  if (n != T * K) refuse("pos: %lld elements are not a whole number for each of %lld tokens", (long long)n, (long long)T);
  if (w && w->numel() != n) refuse("w: %lld elements, %lld expected", (long long)w->numel(), (long long)n);
  return K;
}

PyObject* route(Call& c) {
  const at::Tensor &logits = c.tensor("logits"), &expert = c.tensor("expert"), &w = c.tensor("w");
  const at::Tensor* bias = c.opt("bias");
  const Shape s = shape("logits", logits);
  const int64_t K = shape("expert", expert).cols;
  moe_route_args a{};
  a.T = i32(s.rows); a.E = i32(s.cols); a.K = i32(K);
  a.pitch = mat("logits", logits, s.rows, s.cols, F32 | BF16);
  a.logits = logits.data_ptr();
  a.dtype = code(logits);
  a.bias = (const float*)vec("bias", bias, s.cols, F32);
  a.score = score_of(c.whole());
  a.renorm = c.truth();
  a.scale = c.real();
  a.expert = (int32_t*)each("expert", expert, s.rows, K, I32);
  a.w = (float*)each("w", w, s.rows, K, F32);
  return c.run(kRoute, &a);
}

PyObject* route_backward(Call& c) {
  const at::Tensor &logits = c.tensor("logits"), &expert = c.tensor("expert"), &dw = c.tensor("dw"),
                   &dlogits = c.tensor("dlogits"), &err = c.tensor("err");
  const Shape s = shape("logits", logits);
  const int64_t K = shape("expert", expert).cols;
  moe_route_backward_args a{};
  a.T = i32(s.rows); a.E = i32(s.cols); a.K = i32(K);
  a.pitch = mat("logits", logits, s.rows, s.cols, F32 | BF16);
  a.logits = logits.data_ptr();
  a.dtype = code(logits);
  a.dlogits_pitch = mat("dlogits", dlogits, s.rows, s.cols, same(logits));
  a.dlogits = dlogits.data_ptr();
  a.score = score_of(c.whole());
  a.renorm = c.truth();
  a.scale = c.real();
  a.expert = (const int32_t*)each("expert", expert, s.rows, K, I32);
  a.dw = (const float*)each("dw", dw, s.rows, K, F32);
  a.err = (uint32_t*)vec("err", &err, 1, I32);
  return c.run(kRouteBack, &a);
}

PyObject* sort_rows(Call& c) {
  const at::Tensor& expert = c.tensor("expert");
  const int64_t E_loc = c.whole();
  const at::Tensor *x = c.opt("x"), *xs = c.opt("xs"), *perm = c.opt("perm");
  const at::Tensor &pos = c.tensor("pos"), &counts = c.tensor("counts"), &offsets = c.tensor("offsets"),
                   &err = c.tensor("err");
  const at::Tensor* workspace = c.opt("workspace");
  const int64_t base = c.whole();
  const at::Tensor *row_slot = c.opt("row_slot"), *x_scale = c.opt("x_scale");
  const int64_t group = c.whole();
  const Shape s = shape("expert", expert);
  const int64_t n = s.rows * s.cols;
  moe_sort_rows_args a{};
  a.T = i32(s.rows); a.K = i32(s.cols); a.E_loc = i32(E_loc); a.expert_base = i32(base); i32(n);
  a.expert = (const int32_t*)each("expert", expert, s.rows, s.cols, I32);
  a.H = 8; a.x_dtype = MOE_BF16; a.x_pitch = a.xs_pitch = 8;
  if (xs) {
    if (!x) refuse("x: required with xs");
    const int64_t H = shape("xs", *xs).cols;
    a.H = i32(H);
    a.x_pitch = mat("x", *x, s.rows, H, F32 | BF16 | FP8);
    a.x = x->data_ptr();
    a.x_dtype = code(*x);
    a.xs_pitch = mat("xs", *xs, n, H, a.x_dtype == MOE_FP8_E4M3 ? BF16 : same(*x));
    a.xs = xs->data_ptr();
    if (a.x_dtype == MOE_FP8_E4M3) {
      if (!x_scale) refuse("x_scale: required for fp8 rows");
      a.x_scale = (const float*)table("x_scale", x_scale, s.rows, groups(H, group), F32);
      a.group = (int32_t)group;
    }
  }
  a.perm = (int32_t*)vec("perm", perm, n, I32);
  a.pos = (int32_t*)table("pos", &pos, s.rows, s.cols, I32);
  a.counts = (int32_t*)vec("counts", &counts, E_loc, I32);
  a.offsets = (int32_t*)vec("offsets", &offsets, E_loc + 1, I32);
  a.row_slot = (int32_t*)vec("row_slot", row_slot, n, I32);
  a.err = (uint32_t*)vec("err", &err, 1, I32);
  a.workspace_bytes = room(workspace);
  a.workspace = address(workspace);
  return c.run(kSort, &a);
}

PyObject* merge_rows(Call& c) {
  const at::Tensor &rows = c.tensor("rows"), &pos = c.tensor("pos");
  const at::Tensor* w = c.opt("w");
  const at::Tensor &out = c.tensor("out"), &err = c.tensor("err");
  const Shape s = shape("out", out);
  const int64_t K = positions(pos, w, s.rows);
  moe_merge_rows_args a{};
  a.T = i32(s.rows); a.K = i32(K); a.H = i32(s.cols);
  a.n_rows = shape("rows", rows).rows;
  a.row_pitch = mat("rows", rows, a.n_rows, s.cols, F32 | BF16);
  a.rows = rows.data_ptr();
  a.row_dtype = code(rows);
  a.pos = (const int32_t*)table("pos", &pos, s.rows, K, I32);
  a.w = (const float*)table("w", w, s.rows, K, F32);
  a.out_pitch = mat("out", out, s.rows, s.cols, F32 | BF16);
  a.out = out.data_ptr();
  a.out_dtype = code(out);
  a.err = (uint32_t*)vec("err", &err, 1, I32);
  return c.run(kMerge, &a);
}

PyObject* merge_rows_backward(Call& c) {
  const at::Tensor& dout = c.tensor("dout");
  const at::Tensor* rows = c.opt("rows");
  const at::Tensor& pos = c.tensor("pos");
  const at::Tensor *w = c.opt("w"), *drows = c.opt("drows"), *dw = c.opt("dw");
  const at::Tensor& err = c.tensor("err");
  const Shape s = shape("dout", dout);
  const int64_t K = positions(pos, w, s.rows);
  const at::Tensor* one = rows ? rows : drows;
  if (!one || (!drows && !dw) || (dw && !rows)) refuse("drows, or dw with rows, must be given");
  moe_merge_rows_backward_args a{};
  a.T = i32(s.rows); a.K = i32(K); a.H = i32(s.cols);
  a.dout_pitch = mat("dout", dout, s.rows, s.cols, F32 | BF16);
  a.dout = dout.data_ptr();
  a.dout_dtype = code(dout);
  a.n_rows = shape("rows", *one).rows;
  a.row_pitch = a.drows_pitch = s.cols;
  if (rows) {
    a.row_pitch = mat("rows", *rows, a.n_rows, s.cols, F32 | BF16);
    a.rows = rows->data_ptr();
  }
  if (drows) {
    a.drows_pitch = mat("drows", *drows, a.n_rows, s.cols, rows ? same(*rows) : F32 | BF16);
    a.drows = drows->data_ptr();
  }
  a.row_dtype = code(*one);
  a.pos = (const int32_t*)table("pos", &pos, s.rows, K, I32);
  a.w = (const float*)table("w", w, s.rows, K, F32);
  a.dw = (float*)table("dw", dw, s.rows, K, F32);
  a.err = (uint32_t*)vec("err", &err, 1, I32);
  return c.run(kMergeBack, &a);
}

PyObject* residual_norm(Call& c) {
  const at::Tensor& x = c.tensor("x");
  const at::Tensor* residual = c.opt("residual");
  const at::Tensor& gamma = c.tensor("gamma");
  const float eps = c.real();
  const at::Tensor& out = c.tensor("out");
  const at::Tensor *residual_out = c.opt("residual_out"), *rstd = c.opt("rstd"), *out_scale = c.opt("out_scale");
  const int64_t group = c.whole();
  const at::Tensor *row_list = c.opt("row_list"), *row_count = c.opt("row_count"), *err = c.opt("err");
  const Shape s = shape("x", x);
  moe_residual_norm_args a{};
  a.T = i32(s.rows); a.H = i32(s.cols);
  a.x_pitch = mat("x", x, s.rows, s.cols, F32 | BF16);
  a.x = x.data_ptr();
  a.x_dtype = a.res_dtype = code(x);
  a.res_pitch = a.res_out_pitch = s.cols;
  if (residual) {
    a.res_pitch = mat("residual", *residual, s.rows, s.cols, F32 | BF16);
    a.residual = residual->data_ptr();
    a.res_dtype = code(*residual);
  }
  if (residual_out) {
    a.res_out_pitch = mat("residual_out", *residual_out, s.rows, s.cols, residual ? same(*residual) : F32 | BF16);
    a.residual_out = residual_out->data_ptr();
    a.res_dtype = code(*residual_out);
  }
  a.gamma = vec("gamma", &gamma, s.cols, F32 | BF16);
  a.gamma_dtype = code(gamma);
  a.eps = eps;
  a.out_pitch = mat("out", out, s.rows, s.cols, F32 | BF16 | FP8);
  a.out = out.data_ptr();
  a.out_dtype = code(out);
  if (a.out_dtype == MOE_FP8_E4M3) {
    if (!out_scale) refuse("out_scale: required for fp8 output");
    a.out_scale = (float*)table("out_scale", out_scale, s.rows, groups(s.cols, group), F32);
    a.group = (int32_t)group;
  }
  a.rstd = (float*)vec("rstd", rstd, s.rows, F32);
  a.row_list = (const int32_t*)vec("row_list", row_list, s.rows, I32);
  a.row_count = (const int32_t*)vec("row_count", row_count, 1, I32);
  a.err = (uint32_t*)vec("err", err, 1, I32);
  return c.run(kNorm, &a);
}

PyObject* residual_norm_backward(Call& c) {
  const at::Tensor &dout = c.tensor("dout"), &h = c.tensor("h"), &gamma = c.tensor("gamma"), &rstd = c.tensor("rstd");
  const at::Tensor *dx = c.opt("dx"), *dgamma = c.opt("dgamma"), *workspace = c.opt("workspace"),
                   *dres = c.opt("dres"), *dresidual = c.opt("dresidual");
  const Shape s = shape("dout", dout);
  moe_residual_norm_backward_args a{};
  a.T = i32(s.rows); a.H = i32(s.cols);
  a.dout_pitch = mat("dout", dout, s.rows, s.cols, F32 | BF16);
  a.dout = dout.data_ptr();
  a.dtype = code(dout);
  a.h_pitch = mat("h", h, s.rows, s.cols, F32 | BF16);
  a.h = h.data_ptr();
  a.h_dtype = code(h);
  a.gamma = vec("gamma", &gamma, s.cols, F32 | BF16);
  a.gamma_dtype = code(gamma);
  a.rstd = (const float*)vec("rstd", &rstd, s.rows, F32);
  a.dres_pitch = a.dx_pitch = a.dresidual_pitch = s.cols;
  if (dres) a.dres_pitch = mat("dres", *dres, s.rows, s.cols, same(h));
  if (dx) a.dx_pitch = mat("dx", *dx, s.rows, s.cols, same(dout));
  if (dresidual) a.dresidual_pitch = mat("dresidual", *dresidual, s.rows, s.cols, same(h));
  a.dres = address(dres);
  a.dx = address(dx);
  a.dresidual = address(dresidual);
  a.dgamma = (float*)vec("dgamma", dgamma, s.cols, F32);
  a.workspace_bytes = room(workspace);
  a.workspace = address(workspace);
  return c.run(kNormBack, &a);
}

// No C++ exception leaves a function that Python calls.
template <PyObject* (*F)(Call&), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!g_error || !g_entry[kRoute]) {
    PyErr_SetString(PyExc_RuntimeError, "_marshal.setup() has not been called");
    return nullptr;
  }
  try {
    Call c(args, n, N);
    return F(c);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(g_error, e.what());
    return nullptr;
  }
}

// sizeof of each entry's argument struct as compiled here; moe_struct_size's ids begin at 5 for kRoute
constexpr int kFirstStruct = 5;
constexpr size_t kStructSize[kEntries] = {
    sizeof(moe_route_args),        sizeof(moe_route_backward_args),      sizeof(moe_sort_rows_args),
    sizeof(moe_merge_rows_args),   sizeof(moe_merge_rows_backward_args), sizeof(moe_residual_norm_args),
    sizeof(moe_residual_norm_backward_args)};

// setup(MoeError, addresses of moe_strerror, moe_version and moe_struct_size, addresses of the entry
// points in Entry's order); what was set up before stays if it raises
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr int kHelpers = 3;
  if (n != 1 + kHelpers + kEntries) {
    PyErr_SetString(PyExc_TypeError, "setup: wrong number of arguments");
    return nullptr;
  }
  void* p[kHelpers + kEntries];
  for (int i = 0; i < kHelpers + kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(args[1 + i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "setup: an address of 0");
      return nullptr;
    }
  }
  const int version = ((int (*)(void))p[1])();
  if (version != MOE_STEP_VERSION)
    return PyErr_Format(args[0], "the library has version %d, _marshal was built for %d: build both again", version,
                        MOE_STEP_VERSION);
  for (int i = 0; i < kEntries; ++i) {
    const size_t size = ((size_t(*)(int))p[2])(kFirstStruct + i);
    if (size != kStructSize[i])
      return PyErr_Format(args[0], "struct layout mismatch (id %d): library %zu vs _marshal %zu: build both again",
                          kFirstStruct + i, size, kStructSize[i]);
  }
  Py_INCREF(args[0]);
  Py_XDECREF(g_error);
  g_error = args[0];
  g_strerror = (const char* (*)(int))p[0];
  for (int i = 0; i < kEntries; ++i) g_entry[i] = p[kHelpers + i];
  Py_RETURN_NONE;
}

#define FAST(f) (PyCFunction)(void*)(f), METH_FASTCALL
PyMethodDef g_methods[] = {
    {"setup", FAST(setup), "hands over the library's entry points"},
    {"moe_route", FAST((entry<route, 8>)), nullptr},
    {"moe_route_backward", FAST((entry<route_backward, 9>)), nullptr},
    {"moe_sort_rows", FAST((entry<sort_rows, 15>)), nullptr},
    {"moe_merge_rows", FAST((entry<merge_rows, 6>)), nullptr},
    {"moe_merge_rows_backward", FAST((entry<merge_rows_backward, 8>)), nullptr},
    {"moe_residual_norm", FAST((entry<residual_norm, 13>)), nullptr},
    {"moe_residual_norm_backward", FAST((entry<residual_norm_backward, 10>)), nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&g_module); }
