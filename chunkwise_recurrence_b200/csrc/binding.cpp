// Marshalling of the linear recurrence and of layer normalisation from
// PyTorch tensors into the C ABI of include/gdr.h, as a CPython extension.
//
// A decoding step runs these calls once per layer and token on a few
// kilobytes, where the checks and allocations around a launch decide how long
// a call takes: through ctypes and checks in Python a step took 10 us, of
// which the launch was 3.  Arguments arrive by position, as the functions of
// chunkwise_recurrence_b200/__init__.py pass them; wrong ones raise ValueError
// before anything is allocated, and what the library returns is handed on as
// an int if it is not GDR_OK.  Launches go to the current stream of x's
// device, where the results are allocated too.

#include <Python.h>

#include <array>
#include <cstdint>
#include <initializer_list>
#include <utility>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gdr.h"

namespace {

using at::IntArrayRef;
using at::Tensor;

struct Refused {};   // a Python error is set

template <typename... A>
[[noreturn]] void refuse(const char *fmt, A... a) {
  PyErr_Format(PyExc_ValueError, fmt, a...);
  throw Refused();
}

bool given(PyObject *o) { return o != Py_None; }

const Tensor &tensor(const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// The activations of a call.
struct Input {
  const Tensor *t;
  IntArrayRef shape;
  long long ld;          // elements from one token to the next
  at::Device device;
  gdr_dtype dtype;
};

// x [.., inner dimensions]: the inner ones contiguous, tokens evenly spaced.
Input input(PyObject *o, int inner) {
  const Tensor &t = tensor("x", o);
  Input x{&t, t.sizes(), 1, t.device(), GDR_BF16};
  const int n = (int)x.shape.size(), outer = n - inner;
  if (outer < 0)
    refuse("x has too few dimensions");
  if (!t.is_cuda()) refuse("x must be a CUDA tensor");
  if (t.scalar_type() == at::kFloat)
    x.dtype = GDR_FP32;
  else if (t.scalar_type() != at::kBFloat16)
    refuse("x must be bfloat16 or float32");
  for (int i = outer; i < n; ++i) x.ld *= x.shape[i];
  if (t.is_contiguous()) return x;
  const IntArrayRef strides = t.strides();
  long long step = 1;
  for (int i = n - 1; i >= outer; --i) {
    if (x.shape[i] != 1 && strides[i] != step)
      refuse("x: a token's dimensions must be contiguous");
    step *= x.shape[i];
  }
  long long ld = 0, rows = 1;
  for (int i = outer - 1; i >= 0; --i) {
    if (x.shape[i] == 1) continue;
    if (!ld) {
      ld = strides[i];
      if (ld < step)
        refuse("x: tokens must not overlap");
    } else if (strides[i] != ld * rows) {
      refuse("x: tokens must be evenly spaced");
    }
    rows *= x.shape[i];
  }
  if (ld) x.ld = ld;
  return x;
}

// Another tensor of the call: its address, or nullptr for None.
void *check(const char *name, PyObject *o, IntArrayRef shape,
            at::ScalarType type, const Input &x) {
  if (!given(o)) return nullptr;
  const Tensor &t = tensor(name, o);
  if (t.sizes() != shape)
    refuse("%s has the wrong shape", name);
  if (t.scalar_type() != type)
    refuse("%s must be %s", name, at::toString(type));
  if (t.device() != x.device)
    refuse("%s must be on the device of x", name);
  if (!t.is_contiguous())
    refuse("%s must be contiguous", name);
  return t.data_ptr();
}
void *check_like(const char *name, PyObject *o, const Input &x) {
  return check(name, o, x.shape, x.t->scalar_type(), x);
}

Tensor like(const Input &x) {
  if (x.t->is_contiguous()) return at::empty_like(*x.t);
  return at::empty(x.shape, x.t->options());
}
Tensor floats(IntArrayRef shape, const Input &x) {
  return at::empty(shape, x.t->options().dtype(at::kFloat));
}

// A result: the caller's tensor, or a new one.
struct Result {
  PyObject *o = nullptr;   // owned
  void *p = nullptr;
  Result() = default;
  Result(const Result &) = delete;
  ~Result() { Py_XDECREF(o); }
  void set(PyObject *theirs, void *at) {
    Py_INCREF(theirs);
    o = theirs;
    p = at;
  }
  void set(Tensor t) {
    p = t.data_ptr();
    o = THPVariable_Wrap(std::move(t));
    if (!o) throw Refused();
  }
  PyObject *get() const { return o ? o : Py_None; }
};

PyObject *tuple(std::initializer_list<const Result *> rs) {
  PyObject *t = PyTuple_New((Py_ssize_t)rs.size());
  if (!t) throw Refused();
  Py_ssize_t i = 0;
  for (const Result *r : rs) {
    Py_INCREF(r->get());
    PyTuple_SET_ITEM(t, i++, r->get());
  }
  return t;
}
PyObject *dict(
    std::initializer_list<std::pair<const char *, const Result *>> rs) {
  PyObject *d = PyDict_New();
  if (!d) throw Refused();
  for (const auto &r : rs)
    if (PyDict_SetItemString(d, r.first, r.second->get()) < 0) {
      Py_DECREF(d);
      throw Refused();
    }
  return d;
}

cudaStream_t stream_of(const Input &x) {
  return c10::cuda::getCurrentCUDAStream(x.device.index()).stream();
}

bool flag(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v;
}

// gate (a name or None), its log-decays and options for x [.., H, d]
struct Gate {
  gdr_opts opts;
  const float *la;
};
Gate gate_of(PyObject *name, PyObject *log_alpha, const Input &x) {
  Gate g{};
  g.opts.dtype = x.dtype;
  g.opts.algo = GDR_ALGO_AUTO;
  int kind = -1;
  if (given(name)) {
    static const char *const names[] = {"none", "scalar", "channel"};
    for (int i = 0; i < 3; ++i)
      if (PyUnicode_Check(name) &&
          PyUnicode_CompareWithASCIIString(name, names[i]) == 0)
        kind = i;
    if (kind < 0)
      refuse("gate must be 'none', 'scalar' or 'channel'");
  }
  if (!given(log_alpha)) {
    if (kind > 0) refuse("a gate needs log_alpha");
    g.opts.gate = GDR_GATE_NONE;
    return g;
  }
  if (kind == 0) refuse("log_alpha needs a gate");
  const Tensor &t = tensor("log_alpha", log_alpha);
  if (kind < 0) kind = t.dim() == (int64_t)x.shape.size() - 1 ? 1 : 2;
  g.opts.gate = kind == 1 ? GDR_GATE_SCALAR : GDR_GATE_CHANNEL;
  g.la = static_cast<const float *>(
      check("log_alpha", log_alpha,
            kind == 1 ? x.shape.slice(0, x.shape.size() - 1) : x.shape,
            at::kFloat, x));
  return g;
}

// What the two sequence entries have in common: x [B, T, H, d], packed or not.
struct Sequences {
  Input x;
  Gate g;
  int B, T, H, d;
  std::array<int64_t, 3> states, chunks;
  float *s0;
};
int size_of(int64_t n) {
  if (n > INT32_MAX)
    refuse("x has a dimension of 2^31 or more");
  return (int)n;
}
Sequences sequences(PyObject *xo, PyObject *la, PyObject *s0, PyObject *gate,
                    PyObject *cu) {
  if (tensor("x", xo).dim() != 4)
    refuse("x must be [B, T, H, d]");
  Sequences s{input(xo, 2), {}, 0, 0, 0, 0, {}, {}, nullptr};
  s.B = size_of(s.x.shape[0]);
  s.T = size_of(s.x.shape[1]);
  s.H = size_of(s.x.shape[2]);
  s.d = size_of(s.x.shape[3]);
  s.g = gate_of(gate, la, s.x);
  int64_t n = s.B;
  if (given(cu)) {
    if (s.B != 1)
      refuse("packed sequences (cu_seqlens) need B = 1");
    const Tensor &t = tensor("cu_seqlens", cu);
    if (t.dim() != 1 || t.numel() < 1)
      refuse("cu_seqlens must be [num_seqs + 1]");
    n = t.numel() - 1;
    s.g.opts.cu_seqlens = static_cast<const int32_t *>(
        check("cu_seqlens", cu, t.sizes(), at::kInt, s.x));
    s.g.opts.num_seqs = size_of(n);
  }
  s.states = {n, s.H, s.d};
  s.chunks = {(int64_t)s.B * s.T / GDR_LINEAR_CHUNK + n, s.H, s.d};
  s.s0 = static_cast<float *>(
      check("initial_state", s0, s.states, at::kFloat, s.x));
  return s;
}

// Without the interpreter's lock while it lives: a launch may wait for room in
// the driver's queue, and what empties the queue may be another Python thread.
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
int call(F &&f) {
  const Unlocked u;
  return f();
}

template <typename F>
PyObject *guarded(Py_ssize_t have, Py_ssize_t want, F &&f) {
  HANDLE_TH_ERRORS
  if (have != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// x, log_alpha, initial_state, gate, cu_seqlens, out, final_state,
// output_final_state, output_chunk_states
PyObject *linear_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject * {
    const Sequences s = sequences(a[0], a[1], a[2], a[3], a[4]);
    void *o = check_like("out", a[5], s.x);
    void *f = check("final_state", a[6], s.states, at::kFloat, s.x);
    const bool want_f = flag(a[7]), want_c = flag(a[8]);
    const c10::cuda::CUDAGuard guard(s.x.device);
    Result out, fin, cs;
    given(a[5]) ? out.set(a[5], o) : out.set(like(s.x));
    if (given(a[6]))
      fin.set(a[6], f);
    else if (want_f)
      fin.set(floats(s.states, s.x));
    if (want_c) cs.set(floats(s.chunks, s.x));
    const int rc = call([&] {
      return gdr_linear_fwd(s.x.t->data_ptr(), s.x.ld, s.g.la, s.s0, out.p,
                            static_cast<float *>(fin.p),
                            static_cast<float *>(cs.p), s.B, s.T, s.H, s.d,
                            stream_of(s.x), &s.g.opts);
    });
    if (rc != GDR_OK) return PyLong_FromLong(rc);
    return want_c ? tuple({&out, &fin, &cs}) : tuple({&out, &fin});
  });
}

// x, log_alpha, state, out, state_out, gate
PyObject *linear_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject * {
    if (tensor("x", a[0]).dim() != 3)
      refuse("x must be [N, H, d]");
    const Input x = input(a[0], 2);
    const int N = size_of(x.shape[0]), H = size_of(x.shape[1]);
    const int d = size_of(x.shape[2]);
    const Gate g = gate_of(a[5], a[1], x);
    void *s = check("state", a[2], x.shape, at::kFloat, x);
    void *o = check_like("out", a[3], x);
    void *so = check("state_out", a[4], x.shape, at::kFloat, x);
    const c10::cuda::CUDAGuard guard(x.device);
    Result out, state;
    given(a[3]) ? out.set(a[3], o) : out.set(like(x));
    if (given(a[4]))
      state.set(a[4], so);
    else if (given(a[2]))
      state.set(a[2], s);
    else
      state.set(floats(x.shape, x));
    const int rc = call([&] {
      return gdr_linear_step(x.t->data_ptr(), x.ld, g.la,
                             static_cast<float *>(s),
                             static_cast<float *>(state.p), out.p, N, H, d,
                             stream_of(x), &g.opts);
    });
    if (rc != GDR_OK) return PyLong_FromLong(rc);
    return tuple({&out, &state});
  });
}

// x, log_alpha, initial_state, d_out, d_final_state, chunk_states, gate,
// cu_seqlens, need_initial_state_grad
PyObject *linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject * {
    const Sequences s = sequences(a[0], a[1], a[2], a[6], a[7]);
    if (!given(a[3])) refuse("d_out must be given");
    void *dout = check_like("d_out", a[3], s.x);
    void *ds = check("d_final_state", a[4], s.states, at::kFloat, s.x);
    void *cs = check("chunk_states", a[5], s.chunks, at::kFloat, s.x);
    const bool want = flag(a[8]);
    const c10::cuda::CUDAGuard guard(s.x.device);
    Result dx, dla, ds0;
    dx.set(like(s.x));
    if (given(a[1])) dla.set(at::empty_like(THPVariable_Unpack(a[1])));
    if (want) ds0.set(floats(s.states, s.x));
    const int rc = call([&] {
      return gdr_linear_backward(
          s.x.t->data_ptr(), s.x.ld, s.g.la, s.s0, static_cast<float *>(cs),
          dout, static_cast<float *>(ds), dx.p, static_cast<float *>(dla.p),
          static_cast<float *>(ds0.p), s.B, s.T, s.H, s.d, stream_of(s.x),
          &s.g.opts);
    });
    if (rc != GDR_OK) return PyLong_FromLong(rc);
    return dict({{"dx", &dx},
                 {"dlog_alpha", &dla},
                 {"dinitial_state", &ds0}});
  });
}

// x [.., d] or, with a weight [H, d], [.., H, d]
struct Normed {
  Input x;
  int ntok, H, d;
  IntArrayRef params;
  float *w;
};
Normed normed(PyObject *xo, PyObject *weight) {
  int inner = 1;
  if (given(weight)) {
    inner = (int)tensor("weight", weight).dim();
    if (inner != 1 && inner != 2)
      refuse("weight must be [d] or [H, d]");
  }
  Normed r{input(xo, inner), 0, 1, 0, {}, nullptr};
  r.params = r.x.shape.slice(r.x.shape.size() - inner);
  r.d = size_of(r.params[inner - 1]);
  if (inner == 2) r.H = size_of(r.params[0]);
  const int64_t n = r.x.t->numel();
  r.ntok = n ? size_of(n / ((int64_t)r.H * r.d)) : 0;
  r.w = static_cast<float *>(
      check("weight", weight, r.params, at::kFloat, r.x));
  return r;
}
float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)v;
}

// x, weight, bias, eps, out
PyObject *layer_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    if (given(a[2]) && !given(a[1]))
      refuse("a bias needs a weight");
    const Normed r = normed(a[0], a[1]);
    void *b = check("bias", a[2], r.params, at::kFloat, r.x);
    const float eps = number(a[3]);
    void *o = check_like("out", a[4], r.x);
    const c10::cuda::CUDAGuard guard(r.x.device);
    Result out;
    given(a[4]) ? out.set(a[4], o) : out.set(like(r.x));
    const int rc = call([&] {
      return gdr_layer_norm(r.x.t->data_ptr(), r.x.ld, r.w,
                            static_cast<float *>(b), out.p, r.ntok, r.H, r.d,
                            eps, r.x.dtype, stream_of(r.x));
    });
    if (rc != GDR_OK) return PyLong_FromLong(rc);
    Py_INCREF(out.o);
    return out.o;
  });
}

// x, weight, d_out, eps, need_param_grads
PyObject *layer_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    const Normed r = normed(a[0], a[1]);
    if (!given(a[2])) refuse("d_out must be given");
    void *dy = check_like("d_out", a[2], r.x);
    const float eps = number(a[3]);
    const bool params = flag(a[4]) && given(a[1]);
    const c10::cuda::CUDAGuard guard(r.x.device);
    Result dx, dw, db;
    dx.set(like(r.x));
    if (params) {
      dw.set(floats(r.params, r.x));
      db.set(floats(r.params, r.x));
    }
    const int rc = call([&] {
      return gdr_layer_norm_backward(
          r.x.t->data_ptr(), r.x.ld, r.w, dy, dx.p,
          static_cast<float *>(dw.p), static_cast<float *>(db.p), r.ntok, r.H,
          r.d, eps, r.x.dtype, stream_of(r.x));
    });
    if (rc != GDR_OK) return PyLong_FromLong(rc);
    return dict({{"dx", &dx}, {"dweight", &dw}, {"dbias", &db}});
  });
}

using Fast = PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t);
PyCFunction fast(Fast f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"linear_fwd", fast(linear_fwd), METH_FASTCALL, nullptr},
    {"linear_step", fast(linear_step), METH_FASTCALL, nullptr},
    {"linear_backward", fast(linear_backward), METH_FASTCALL, nullptr},
    {"layer_norm", fast(layer_norm), METH_FASTCALL, nullptr},
    {"layer_norm_backward", fast(layer_norm_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
