// Argument marshalling of the layer operators for Python: checks of torch
// tensors, their outputs, and the packed call into librsq's C ABI. Nothing is
// computed here. A token's kernels take a few microseconds, and the same checks
// written in Python took longer than the kernels.
//
// Each function takes the stream (an integer) and its operands by position,
// with None for one that is left out, and raises ValueError for operands that
// do not fit and rsq's Error (made by the package) for what the library refuses.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "rsq.h"

namespace {

struct Library {
  rsq_status (*causal_conv)(const rsq_conv*, void*);
  rsq_status (*scan_workspace)(const rsq_ssm*, size_t*);
  rsq_status (*scan)(const rsq_ssm*, void*);
  rsq_status (*step)(const rsq_ssm*, void*);
  rsq_status (*state_workspace)(const rsq_state*, size_t*);
  rsq_status (*state_step)(rsq_state*, const rsq_ssm*, void*);
  rsq_status (*norm)(const rsq_norm*, void*);
  rsq_status (*w4)(const rsq_w4*, void*);
} lib;
PyObject* raise_status = nullptr;   // the package's check(): raises for a status

struct Status {   // a refusal of the library
  rsq_status code;
};

typedef at::IntArrayRef Dims;

std::string text(Dims d) {
  std::ostringstream s;
  s << "(";
  for (size_t i = 0; i < d.size(); ++i) s << (i ? ", " : "") << d[i];
  s << ")";
  return s.str();
}

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

inline void need(bool ok, const char* what) {
  if (!ok) refuse(what);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The operand that sets device and type.
struct Like {
  int device;
  at::ScalarType type;
  explicit Like(const at::Tensor& x) : device(x.is_cuda() ? (int)x.get_device() : -1), type(x.scalar_type()) {
    need(device >= 0, "the tensors must be on a GPU");
  }
};

int act_type(at::ScalarType t) {
  if (t == at::kFloat) return RSQ_F32;
  if (t == at::kBFloat16) return RSQ_BF16;
  refuse("x must be float32 or bfloat16, got " + std::string(c10::toString(t)));
}

void check_tensor(const at::Tensor& t, const Like& like, at::ScalarType type, Dims shape, const char* name) {
  if (t.is_cuda() && t.get_device() == like.device && t.scalar_type() == type && t.sizes() == shape) return;
  refuse(std::string(name) + " must be a " + c10::toString(type) + " tensor of shape " + text(shape) +
         " on the device of the others, got " + c10::toString(t.scalar_type()) + " " + text(t.sizes()) + " on " + t.device().str());
}

// Address of a contiguous tensor, nullptr for None.
void* param(PyObject* o, const Like& like, at::ScalarType type, Dims shape, const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  check_tensor(t, like, type, shape, name);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

// Step between the rows of a tensor [*lead, *row] whose rows are contiguous;
// `inner` dimensions make a row, the one or two before them step alike.
int64_t row_step(const at::Tensor& t, int inner, const char* name) {
  const Dims n = t.sizes(), st = t.strides();
  const int d = (int)n.size(), lead = d - inner;
  bool ok = st[d - 1] == 1 || n[d - 1] == 1;
  if (inner == 2) ok = ok && (st[d - 2] == n[d - 1] || n[d - 2] == 1);
  if (!ok) refuse(std::string(name) + " must have contiguous rows");
  int64_t rows = n[0], step = st[0];
  if (lead == 2) {
    rows = n[0] * n[1];
    step = n[1] > 1 ? st[1] : st[0];
    if (n[0] > 1 && n[1] > 1 && st[0] != n[1] * st[1]) refuse(std::string(name) + " must have rows at one common step");
  }
  if (rows <= 1) {
    // no row follows: any step will do, in the 16 bytes that the library asks of steps
    const int64_t width = n[d - 1] * (inner == 2 ? n[d - 2] : 1);
    step = (width + 7) / 8 * 8;
  }
  return step;
}

// The output: `o`, or a new tensor. Owns a reference.
at::Tensor output(PyObject* o, const at::Tensor& x, const Like& like, at::ScalarType type, Dims shape) {
  if (o == Py_None) return at::empty(shape, x.options().dtype(type).requires_grad(false));
  const at::Tensor& t = tensor(o, "out");
  check_tensor(t, like, type, shape, "out");
  return t;
}

long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::runtime_error("");   // the error is set
  return v;
}

void* stream_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw std::runtime_error("");
  return p;
}

template <typename F>
void call(F f) {
  rsq_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f();
  Py_END_ALLOW_THREADS
  if (s != RSQ_OK) throw Status{s};
}

// Sequences of x: [seqs, T, ...], or packed [tokens, ...] with offsets.
template <typename P>
void sequences(P& p, const at::Tensor& x, int inner, PyObject* offsets, PyObject* max_len, const Like& like) {
  const Dims n = x.sizes();
  const int lead = (int)n.size() - inner;
  const bool given = max_len != Py_None;
  const int64_t longest = given ? (int64_t)integer(max_len) : 0;
  int64_t seqs;
  if (offsets == Py_None) {
    if (lead != 2) refuse("x must have shape [sequences, tokens, ...] without offsets, got " + text(n));
    if (given && longest != n[1]) refuse("max_len is not the number of tokens a sequence of x has");
    seqs = n[0];
    p.tokens = n[0] * n[1];
    p.max_len = n[1];
    p.offsets = nullptr;
  } else {
    if (lead != 1) refuse("x must have shape [tokens, ...] with offsets, got " + text(n));
    const at::Tensor& o = tensor(offsets, "offsets");
    if (!(o.is_cuda() && o.get_device() == like.device && o.scalar_type() == at::kInt && o.dim() == 1 && o.size(0) > 1 &&
          o.is_contiguous()))
      refuse("offsets must be a contiguous int32 tensor [sequences + 1] on the device of x");
    need(given && longest >= 0 && longest <= n[0],
         "max_len, the longest sequence, must be given with offsets, at most the rows of x");
    seqs = o.size(0) - 1;
    p.tokens = n[0];
    p.max_len = longest;
    p.offsets = o.data_ptr<int32_t>();
  }
  need(seqs <= 0x7fffffff, "too many sequences");
  p.seqs = (int32_t)seqs;
}

int32_t small(int64_t v, const char* what) {
  if (v > 0x7fffffff || v < -0x7fffffff) refuse(std::string(what) + " is out of range");
  return (int32_t)v;
}

// Runs a function and turns what it throws into a Python error.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Status& s) {
    if (PyObject* r = PyObject_CallFunction(raise_status, "i", (int)s.code)) Py_DECREF(r);
    return nullptr;
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

inline bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd operands, got %zd", want, n);
  return false;
}

// conv(stream, x, weight, bias, state, offsets, max_len, activation, token, out)
PyObject* conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor(a[1], "x");
    const at::Tensor& w = tensor(a[2], "weight");
    const Like like(x);
    rsq_conv p{};
    p.dtype = act_type(like.type);
    if (a[8] == Py_True) {
      if (x.dim() != 2) refuse("x must have shape [sequences, channels], got " + text(x.sizes()));
      p.seqs = small(x.size(0), "sequences");
      p.tokens = x.size(0), p.max_len = 1;
    } else {
      sequences(p, x, 1, a[5], a[6], like);
    }
    if (w.dim() != 2) refuse("weight must have shape [channels, width], got " + text(w.sizes()));
    const int64_t C = w.size(0), W = w.size(1);
    if (x.size(-1) != C) refuse("x must have as many channels as weight, got " + text(x.sizes()));
    p.channels = small(C, "channels"), p.width = small(W, "width");
    p.activation = (int32_t)integer(a[7]);
    p.x = x.data_ptr(), p.x_stride = row_step(x, 1, "x");
    p.weight = static_cast<const float*>(param(a[2], like, at::kFloat, {C, W}, "weight"));
    p.bias = static_cast<const float*>(param(a[3], like, at::kFloat, {C}, "bias"));
    p.state = param(a[4], like, like.type, {p.seqs, C, W - 1}, "state");
    at::Tensor out = output(a[9], x, like, like.type, x.sizes());
    p.y = out.data_ptr(), p.y_stride = row_step(out, 1, "out");
    void* s = stream_of(a[0]);
    call([&] { return lib.causal_conv(&p, s); });
    return THPVariable_Wrap(std::move(out));
  });
}

// x, dt, A, B, C, D, dt_bias, softplus from a[0] on; seqs, tokens, max_len and offsets are set
void ssm_operands(rsq_ssm& p, const at::Tensor& x, const Like& like, PyObject* const* a) {
  const at::Tensor& dt = tensor(a[1], "dt");
  const at::Tensor& B = tensor(a[3], "B");
  const at::Tensor& C = tensor(a[4], "C");
  p.dtype = act_type(like.type);
  const Dims n = x.sizes();
  const int lead = (int)n.size() - 2;
  if (B.dim() != x.dim()) refuse("B must have shape [..., groups, d_k], got " + text(B.sizes()));
  const int64_t H = n[lead], dv = n[lead + 1], G = B.size(lead), dk = B.size(lead + 1);
  p.heads = small(H, "heads"), p.d_v = small(dv, "d_v"), p.groups = small(G, "groups"), p.d_k = small(dk, "d_k");
  int64_t keys[4], steps[3];
  for (int i = 0; i < lead; ++i) keys[i] = steps[i] = n[i];
  keys[lead] = G, keys[lead + 1] = dk, steps[lead] = H;
  const Dims keyed(keys, lead + 2), stepped(steps, lead + 1);
  check_tensor(B, like, like.type, keyed, "B");
  check_tensor(C, like, like.type, keyed, "C");
  check_tensor(dt, like, like.type, stepped, "dt");
  p.x = x.data_ptr(), p.x_stride = row_step(x, 2, "x");
  p.B = B.data_ptr(), p.b_stride = row_step(B, 2, "B");
  p.C = C.data_ptr(), p.c_stride = row_step(C, 2, "C");
  p.dt = dt.data_ptr(), p.dt_stride = row_step(dt, 1, "dt");
  need(a[2] != Py_None, "A is required");
  p.A = static_cast<const float*>(param(a[2], like, at::kFloat, {H}, "A"));
  p.D = static_cast<const float*>(param(a[5], like, at::kFloat, {H}, "D"));
  p.dt_bias = static_cast<const float*>(param(a[6], like, at::kFloat, {H}, "dt_bias"));
  const int soft = PyObject_IsTrue(a[7]);
  if (soft < 0) throw std::runtime_error("");
  p.softplus = soft;
}

void ssm_out(rsq_ssm& p, const at::Tensor& out) { p.y = out.data_ptr(), p.y_stride = row_step(out, 2, "out"); }

// scan(stream, x, dt, A, B, C, D, dt_bias, softplus, state, offsets, max_len, out) -> (y, state)
PyObject* scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor(a[1], "x");
    const Like like(x);
    if (x.dim() != 3 && x.dim() != 4) refuse("x must have shape [..., heads, d_v], got " + text(x.sizes()));
    rsq_ssm p{};
    sequences(p, x, 2, a[10], a[11], like);
    ssm_operands(p, x, like, a + 1);
    const int64_t shape[4] = {p.seqs, p.heads, p.d_k, p.d_v};
    p.state_in = a[9] != Py_None;
    at::Tensor state;
    if (p.state_in) {
      p.state = static_cast<float*>(param(a[9], like, at::kFloat, shape, "state"));
      state = THPVariable_Unpack(a[9]);
    } else {
      state = at::empty(shape, x.options().dtype(at::kFloat).requires_grad(false));
      p.state = state.data_ptr<float>();
    }
    at::Tensor out = output(a[12], x, like, like.type, x.sizes());
    ssm_out(p, out);
    size_t bytes = 0;
    call([&] { return lib.scan_workspace(&p, &bytes); });
    at::Tensor work;
    if (bytes) {
      // the call's stream owns it: it is reused there only
      work = at::empty({(int64_t)bytes}, x.options().dtype(at::kByte).requires_grad(false));
      p.workspace = work.data_ptr(), p.workspace_bytes = bytes;
    }
    void* s = stream_of(a[0]);
    call([&] { return lib.scan(&p, s); });
    PyObject* y = THPVariable_Wrap(std::move(out));
    if (!y) return nullptr;
    PyObject* st = a[9];
    if (p.state_in) Py_INCREF(st);
    else st = THPVariable_Wrap(std::move(state));
    PyObject* r = st ? PyTuple_Pack(2, y, st) : nullptr;
    Py_DECREF(y);
    Py_XDECREF(st);
    return r;
  });
}

// step(stream, state, x, dt, A, B, C, D, dt_bias, softplus, out): state a dense tensor
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor(a[2], "x");
    const Like like(x);
    if (x.dim() != 3) refuse("x must have shape [sequences, heads, d_v], got " + text(x.sizes()));
    rsq_ssm p{};
    p.seqs = small(x.size(0), "sequences");
    p.tokens = x.size(0), p.max_len = 1;
    ssm_operands(p, x, like, a + 2);
    need(a[1] != Py_None, "state is required");
    p.state = static_cast<float*>(param(a[1], like, at::kFloat, {p.seqs, p.heads, p.d_k, p.d_v}, "state"));
    p.state_in = 1;
    at::Tensor out = output(a[10], x, like, like.type, x.sizes());
    ssm_out(p, out);
    void* s = stream_of(a[0]);
    call([&] { return lib.step(&p, s); });
    return THPVariable_Wrap(std::move(out));
  });
}

// state_step(stream, handle, x, dt, A, B, C, D, dt_bias, softplus, out): state an rsq_state
PyObject* state_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor(a[2], "x");
    const Like like(x);
    if (x.dim() != 3) refuse("x must have shape [batch, heads, d_v], got " + text(x.sizes()));
    rsq_ssm p{};
    p.seqs = small(x.size(0), "sequences");
    p.tokens = x.size(0), p.max_len = 1;
    ssm_operands(p, x, like, a + 2);
    p.state_in = 1;
    rsq_state* h = static_cast<rsq_state*>(stream_of(a[1]));
    at::Tensor out = output(a[10], x, like, like.type, x.sizes());
    ssm_out(p, out);
    size_t bytes = 0;
    call([&] { return lib.state_workspace(h, &bytes); });
    // torch's allocations are 512-byte aligned; the call's stream owns this one
    at::Tensor work = at::empty({(int64_t)bytes}, x.options().dtype(at::kByte).requires_grad(false));
    p.workspace = work.data_ptr(), p.workspace_bytes = bytes;
    void* s = stream_of(a[0]);
    call([&] { return lib.state_step(h, &p, s); });
    return THPVariable_Wrap(std::move(out));
  });
}

at::ScalarType out_type(long t) {
  switch (t) {
    case RSQ_F32: return at::kFloat;
    case RSQ_BF16: return at::kBFloat16;
    case RSQ_INT8: return at::kChar;
    case RSQ_E4M3: return at::kFloat8_e4m3fn;
    default: refuse("out_dtype is not a type of an output");
  }
}

// norm(stream, x, weight, eps, residual, out_type (-1: x's), group, out, scales) -> y or (codes, scales)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor(a[1], "x");
    const Like like(x);
    rsq_norm p{};
    p.dtype = act_type(like.type);
    const Dims dims = x.sizes();
    if (dims.size() != 2 && dims.size() != 3)
      refuse("x must have shape [rows, cols] or [sequences, tokens, cols], got " + text(dims));
    const int64_t cols = dims.back();
    const long t = integer(a[5]);
    const at::ScalarType type = t < 0 ? like.type : out_type(t);
    p.out_dtype = t < 0 ? p.dtype : (int32_t)t;
    const bool codes = p.out_dtype == RSQ_INT8 || p.out_dtype == RSQ_E4M3;
    p.cols = small(cols, "cols");
    const long group = integer(a[6]);
    p.group = small(group, "group");
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw std::runtime_error("");
    p.eps = (float)eps;
    p.rows = dims.size() == 2 ? dims[0] : dims[0] * dims[1];
    p.x = x.data_ptr(), p.x_stride = row_step(x, 1, "x");
    need(a[2] != Py_None, "weight is required");
    p.weight = static_cast<const float*>(param(a[2], like, at::kFloat, {cols}, "weight"));
    if (a[4] != Py_None) {
      const at::Tensor& r = tensor(a[4], "residual");
      check_tensor(r, like, like.type, dims, "residual");
      p.residual = r.data_ptr(), p.residual_stride = row_step(r, 1, "residual");
    }
    at::Tensor out = output(a[7], x, like, type, dims);
    p.y = out.data_ptr(), p.y_stride = row_step(out, 1, "out");
    PyObject* sc = nullptr;
    if (codes) {
      int64_t shape[3];
      const size_t lead = dims.size() - 1;
      for (size_t i = 0; i < lead; ++i) shape[i] = dims[i];
      shape[lead] = group > 0 ? cols / group : 1;
      const Dims sdims(shape, lead + 1);
      if (a[8] == Py_None) {
        at::Tensor s = at::empty(sdims, x.options().dtype(at::kFloat).requires_grad(false));
        p.scales = s.data_ptr<float>();
        sc = THPVariable_Wrap(std::move(s));
        if (!sc) return nullptr;
      } else {
        p.scales = static_cast<float*>(param(a[8], like, at::kFloat, sdims, "scales"));
        Py_INCREF(sc = a[8]);
      }
    } else {
      need(a[8] == Py_None, "scales go with an 8-bit output");
    }
    try {
      void* s = stream_of(a[0]);
      call([&] { return lib.norm(&p, s); });
    } catch (...) {
      Py_XDECREF(sc);
      throw;
    }
    PyObject* y = THPVariable_Wrap(std::move(out));
    if (!codes) return y;
    PyObject* r = y ? PyTuple_Pack(2, y, sc) : nullptr;
    Py_XDECREF(y);
    Py_DECREF(sc);
    return r;
  });
}

// w4(stream, x, packed, n, k, group, scale_dtype, x_scale, out_type (-1: by x), out)
PyObject* w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor(a[1], "x");
    const at::Tensor& packed = tensor(a[2], "weight");
    const Like like(x);
    rsq_w4 p{};
    switch (like.type) {
      case at::kFloat: p.x_dtype = RSQ_F32; break;
      case at::kBFloat16: p.x_dtype = RSQ_BF16; break;
      case at::kChar: p.x_dtype = RSQ_INT8; break;
      case at::kFloat8_e4m3fn: p.x_dtype = RSQ_E4M3; break;
      default: refuse("x must be float32, bfloat16, int8 or float8_e4m3fn, got " + std::string(c10::toString(like.type)));
    }
    const Dims dims = x.sizes();
    if (dims.size() != 2 && dims.size() != 3)
      refuse("x must have shape [rows, k] or [sequences, tokens, k], got " + text(dims));
    p.n = (int32_t)integer(a[3]), p.k = (int32_t)integer(a[4]);
    p.group = (int32_t)integer(a[5]), p.scale_dtype = (int32_t)integer(a[6]);
    if (dims.back() != p.k) refuse("x must have as many columns as weight, got " + text(dims));
    if (!(packed.is_cuda() && packed.get_device() == like.device)) refuse("weight and x must be on one device");
    const size_t lead = dims.size() - 1;
    p.m = small(lead == 1 ? dims[0] : dims[0] * dims[1], "rows");
    p.x = x.data_ptr(), p.x_stride = row_step(x, 1, "x");
    if (a[7] != Py_None) {
      const at::Tensor& s = tensor(a[7], "x_scale");
      const Dims sd = s.sizes();
      const int64_t groups = p.group > 0 ? p.k / p.group : 0;
      bool ok = sd.size() >= lead;
      for (size_t i = 0; ok && i < lead; ++i) ok = sd[i] == dims[i];
      const bool grouped = ok && sd.size() == lead + 1 && groups > 1 && sd[lead] == groups;
      if (!ok || !(sd.size() == lead || (sd.size() == lead + 1 && (sd[lead] == 1 || grouped))))
        refuse("x_scale must have one value a row of x, or one a group of it, got shape " + text(sd));
      p.x_group = grouped ? p.group : 0;
      p.x_scale = static_cast<const float*>(param(a[7], like, at::kFloat, sd, "x_scale"));
    }
    const long t = integer(a[8]);
    p.out_dtype = t >= 0 ? (int32_t)t : like.type == at::kFloat ? RSQ_F32 : RSQ_BF16;
    need(p.out_dtype == RSQ_F32 || p.out_dtype == RSQ_BF16, "out_dtype must be 'f32' or 'bf16'");
    int64_t shape[3];
    for (size_t i = 0; i < lead; ++i) shape[i] = dims[i];
    shape[lead] = p.n;
    at::Tensor out = output(a[9], x, like, out_type(p.out_dtype), Dims(shape, lead + 1));
    p.y = out.data_ptr(), p.y_stride = row_step(out, 1, "out");
    p.packed = packed.data_ptr(), p.packed_bytes = (size_t)packed.numel();
    void* s = stream_of(a[0]);
    call([&] { return lib.w4(&p, s); });
    return THPVariable_Wrap(std::move(out));
  });
}

// bind(check, addresses of the library's functions in Library's order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t kFunctions = sizeof(Library) / sizeof(void*);
  if (!arity(n, 1 + kFunctions)) return nullptr;
  void** f = reinterpret_cast<void**>(&lib);
  for (Py_ssize_t i = 0; i < kFunctions; ++i) {
    f[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function of the library is missing");
      return nullptr;
    }
  }
  Py_INCREF(a[0]);
  Py_XDECREF(raise_status);
  raise_status = a[0];
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(conv), FAST(scan), FAST(step), FAST(state_step), FAST(norm), FAST(w4),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
