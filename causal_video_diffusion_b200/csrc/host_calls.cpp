// host_calls.cpp -- the Python side of the 8-bit cache's and the block norms' calls: tensors and
// arguments checked, outputs made, the stream found, the C ABI called.
//
// These calls are made several times for every layer of every forward, and for small chunks their
// kernels take 4 microseconds; marshalling them through Python objects took 6 to 15 (checks of nine
// tensors, a structure for each norm, eighteen converted arguments), here it is about one.  Argument
// errors become ValueError, the ABI's status codes the UnstepError that bind() was given.  Nothing
// but what bind() was given is kept between calls, and that by each module object for itself: a second
// instance of the binding, on another build of the library, does not reach the first one's calls.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <climits>
#include <string>

#include "../../include/unstep.h"

namespace {

// A module object's own: the library's entry points and the exception of its status codes, from bind().
struct Library {
  decltype(&unstep_norm_modulate) norm_modulate;
  decltype(&unstep_gate_residual_norm) gate_residual_norm;
  decltype(&unstep_q8_rope_kv_append) append;
  decltype(&unstep_q8_window_attn) attn;
  decltype(&unstep_q8_cache_read) read;
  PyObject *error;
};

struct BadArgument {
  std::string what;
};
struct PythonError {};  // already set

[[noreturn]] void refuse(const std::string &what) { throw BadArgument{what}; }

const Library &library(PyObject *module) {
  const Library *l = static_cast<const Library *>(PyModule_GetState(module));
  if (!l->error) refuse("bind() comes before any call");
  return *l;
}

// Other Python threads run while this lives: an allocation or a launch may wait for the device, and
// what the device waits for may be a host function that needs the interpreter.
class Unlocked {
  PyThreadState *state = PyEval_SaveThread();

 public:
  Unlocked() = default;
  Unlocked(const Unlocked &) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

bool is_none(PyObject *o) { return o == nullptr || o == Py_None; }

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

long long integer(PyObject *o, const char *name) {
  PyObject *i = PyNumber_Index(o);
  if (!i) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(i, &over);
  Py_DECREF(i);
  if (over || v < INT_MIN || v > INT_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return v;
}

double number(PyObject *o, const char *name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return v;
}

long long attribute(PyObject *o, const char *name) {
  PyObject *a = PyObject_GetAttrString(o, name);
  if (!a) throw PythonError{};
  const unsigned long long v = PyLong_AsUnsignedLongLongMask(a);
  Py_DECREF(a);
  if (PyErr_Occurred()) throw PythonError{};
  return static_cast<long long>(v);
}

// A call's place: its device, made current for as long as this lives, and the stream.
struct Place {
  int index;
  c10::cuda::CUDAGuard guard;
  c10::cuda::CUDAStream current, stream;  // the device's current stream; the call's
  unstep_stream_t handle;

  Place(int device, PyObject *s)
      : index(device),
        guard(static_cast<c10::DeviceIndex>(device)),
        current(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device))),
        stream(is_none(s) ? current : given(device, s)),
        handle(stream.stream()) {}

  static c10::cuda::CUDAStream given(int device, PyObject *s) {
    const long long at = attribute(s, "device_index");
    if (at != device)
      refuse("stream is on cuda:" + std::to_string(at) + ", the tensors on cuda:" +
             std::to_string(device));
    return c10::cuda::CUDAStream(
        c10::Stream::unpack3(attribute(s, "stream_id"), static_cast<c10::DeviceIndex>(at),
                             static_cast<c10::DeviceType>(attribute(s, "device_type"))));
  }

  // A new output that the call writes on `stream`.  It comes from that stream's memory: a block of
  // the current stream's may have been freed behind work there that still reads it, which the call
  // would not wait for.  The caller goes on with it on the current stream, so it is recorded there.
  at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type) const {
    const auto options = at::TensorOptions(at::Device(at::kCUDA, index)).dtype(type);
    const Unlocked others;
    if (stream == current) return at::empty(shape, options);
    at::Tensor t;
    {
      const c10::cuda::CUDAStreamGuard on(stream);
      t = at::empty(shape, options);
    }
    t.record_stream(current);
    return t;
  }
};

void check(const Library &lib, int status, const char *name) {
  if (status >= 0) return;
  PyObject *e = PyObject_CallFunction(lib.error, "is", status, name);
  if (e) {
    PyErr_SetObject(lib.error, e);
    Py_DECREF(e);
  }
  throw PythonError{};
}

// torch's own errors (out of memory, a device error) become the exceptions that torch raises for them.
template <class F>
PyObject *guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const PythonError &) {
  } catch (const BadArgument &e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

// A library call's status, the interpreter unlocked meanwhile.
template <class F, class... Args>
int call(F f, Args... args) {
  const Unlocked others;
  return f(args...);
}

PyObject *same(PyObject *o) {
  Py_INCREF(o);
  return o;
}

// ---------------------------------------------------------------------------------------------
// the norms
// ---------------------------------------------------------------------------------------------
int type_code(const at::Tensor &t) {
  return t.scalar_type() == at::kBFloat16 ? UNSTEP_BF16 : t.scalar_type() == at::kFloat ? UNSTEP_F32
                                                                                       : -1;
}

struct Rows {
  long long n, ld;
};

// Rows of a tensor whose last axis is contiguous and whose leading axes walk them at one stride.
Rows rows_of(const at::Tensor &t, const char *name) {
  const auto shape = t.sizes(), strides = t.strides();
  const int axes = static_cast<int>(shape.size());
  if (axes < 2) refuse(std::string(name) + " must have a row axis and a channel axis");
  const long long C = shape[axes - 1];
  if (C > 1 && strides[axes - 1] != 1) refuse(std::string(name) + "'s channels must be contiguous");
  if (t.numel() == 0) return {0, C};
  Rows r{1, C};
  for (int a = axes - 2; a >= 0; --a) {
    if (shape[a] == 1) continue;
    if (r.n == 1)
      r.ld = strides[a];
    else if (strides[a] != r.ld * r.n)
      refuse(std::string(name) + "'s rows must lie at one stride");
    r.n *= shape[a];
  }
  if (r.ld < C) refuse(std::string(name) + "'s rows must not overlap");
  return r;
}

// What all of a call's tensors share.
struct Batch {
  int index;
  long long rows, C, groups;  // groups 0: no modulation seen yet
  long long per_group() const { return rows ? rows / (groups ? groups : 1) : 1; }
  // more than 32 bits hold: a count that the library refuses as it refuses any above its limit
  int channels() const { return static_cast<int>(C < INT_MAX ? C : INT_MAX - 7); }
};

struct Vectors {
  const void *p;
  long long stride;
};

// A [G][C] modulation tensor.
Vectors vectors(PyObject *o, Batch &b, const char *name) {
  const at::Tensor &t = tensor(o, name);
  if (t.dim() != 2 || t.size(1) != b.C || t.get_device() != b.index || type_code(t) < 0)
    refuse(std::string(name) + " must be bf16 or fp32 [groups][" + std::to_string(b.C) +
           "] on cuda:" + std::to_string(b.index));
  if (t.stride(1) != 1) refuse(std::string(name) + "'s channels must be contiguous");
  const long long G = t.size(0);
  if (G < 1 || b.rows % G || (b.groups && b.groups != G))
    refuse(std::string(name) + " has " + std::to_string(G) + " groups for " +
           std::to_string(b.rows) + " rows" +
           (b.groups ? ", other modulations " + std::to_string(b.groups) : ""));
  b.groups = G;
  return {t.data_ptr(), G > 1 ? t.stride(0) : 0};
}

// A Norm tuple (kind, eps, weight, bias, scale, shift).
unstep_norm_t norm_of(PyObject *o, Batch &b) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 6) refuse("a norm must be a Norm");
  unstep_norm_t n{};
  PyObject *kind = PyTuple_GET_ITEM(o, 0);
  if (PyUnicode_Check(kind) && !PyUnicode_CompareWithASCIIString(kind, "layer"))
    n.kind = UNSTEP_NORM_LAYER;
  else if (PyUnicode_Check(kind) && !PyUnicode_CompareWithASCIIString(kind, "rms"))
    n.kind = UNSTEP_NORM_RMS;
  else
    refuse("norm kind: 'layer' or 'rms'");
  n.eps = static_cast<float>(number(PyTuple_GET_ITEM(o, 1), "eps"));
  int type = -2;  // none yet
  auto typed = [&](const at::Tensor &t) {
    const int c = type_code(t);
    if (c < 0 || (type != -2 && c != type))
      refuse("a norm's weight, bias, scale and shift must be all bf16 or all fp32");
    type = c;
  };
  static const char *const names[4] = {"weight", "bias", "scale", "shift"};
  const void **const slots[4] = {&n.weight, &n.bias, &n.scale, &n.shift};
  for (int i = 0; i < 4; ++i) {
    PyObject *item = PyTuple_GET_ITEM(o, 2 + i);
    if (is_none(item)) continue;
    if (i < 2) {
      const at::Tensor &t = tensor(item, names[i]);
      if (t.dim() != 1 || t.size(0) != b.C || !t.is_contiguous() || t.get_device() != b.index)
        refuse(std::string(names[i]) + " must be contiguous [" + std::to_string(b.C) +
               "] on cuda:" + std::to_string(b.index));
      *slots[i] = t.data_ptr();
    } else {
      const Vectors v = vectors(item, b, names[i]);
      if (i == 3 && n.scale && v.stride != n.mod_stride)
        refuse("scale and shift must have the same row stride");
      *slots[i] = v.p;
      n.mod_stride = v.stride;
    }
    typed(tensor(item, names[i]));
  }
  n.param_type = type == -2 ? UNSTEP_F32 : type;
  return n;
}

Batch batch_of(const at::Tensor &x, Rows &rows) {
  if (!x.is_cuda() || type_code(x) < 0) refuse("x must be a bf16 or fp32 CUDA tensor");
  rows = rows_of(x, "x");
  return Batch{static_cast<int>(x.get_device()), rows.n, x.size(-1), 0};
}

// An output of x's shape: checked, or new.
struct Output {
  at::Tensor t;
  PyObject *given;
  long long ld;
  PyObject *release() const { return given ? same(given) : THPVariable_Wrap(t); }
};

Output output(PyObject *o, const at::Tensor &x, at::ScalarType type, const char *name,
              const Place &at) {
  if (is_none(o)) return {at.fresh(x.sizes(), type), nullptr, x.size(-1)};
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != type || t.sizes() != x.sizes() || t.get_device() != at.index)
    refuse(std::string(name) + " must be " + c10::toString(type) + " " + shape_text(x.sizes()) +
           " on cuda:" + std::to_string(at.index));
  return {t, o, rows_of(t, name).ld};
}

// (x, norm, out, stream) -> out
PyObject *norm_modulate(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 4) refuse("norm_modulate takes four arguments");
    const Library &lib = library(self);
    const at::Tensor &x = tensor(a[0], "x");
    Rows xr;
    Batch b = batch_of(x, xr);
    const unstep_norm_t spec = norm_of(a[1], b);
    const Place at(b.index, a[3]);
    const Output out = output(a[2], x, at::kBFloat16, "out", at);
    const int status =
        call(lib.norm_modulate, x.data_ptr(), type_code(x), xr.ld, out.t.data_ptr(), out.ld, b.rows,
             b.channels(), b.per_group(), &spec, at.handle);
    check(lib, status, "unstep_norm_modulate");
    return out.release();
  });
}

// (x, y, gate, res_scale, post, next, x_out, out, stream) -> (x_out, out)
PyObject *gate_residual_norm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 9) refuse("gate_residual_norm takes nine arguments");
    const Library &lib = library(self);
    const at::Tensor &x = tensor(a[0], "x");
    Rows xr;
    Batch b = batch_of(x, xr);
    const at::Tensor &y = tensor(a[1], "y");
    if (y.scalar_type() != at::kBFloat16 || y.sizes() != x.sizes() || y.get_device() != b.index)
      refuse("y must be bfloat16 " + shape_text(x.sizes()) + " on cuda:" + std::to_string(b.index));
    const Rows yr = rows_of(y, "y");
    Vectors gate{nullptr, 0};
    int gate_type = UNSTEP_F32;
    if (!is_none(a[2])) {
      gate = vectors(a[2], b, "gate");
      gate_type = type_code(tensor(a[2], "gate"));
    }
    const float res_scale = static_cast<float>(number(a[3], "res_scale"));
    unstep_norm_t post, next;
    if (!is_none(a[4])) post = norm_of(a[4], b);
    if (!is_none(a[5]))
      next = norm_of(a[5], b);
    else if (!is_none(a[7]))
      refuse("out without a next norm");
    const Place at(b.index, a[8]);
    const Output xo = is_none(a[6]) ? Output{x, a[0], xr.ld}
                                    : output(a[6], x, x.scalar_type(), "x_out", at);
    Output out{{}, Py_None, 0};
    if (!is_none(a[5])) out = output(a[7], x, at::kBFloat16, "out", at);
    const int status = call(
        lib.gate_residual_norm, x.data_ptr(), type_code(x), xr.ld, y.data_ptr(), yr.ld, gate.p,
        gate_type, gate.stride, res_scale, is_none(a[4]) ? nullptr : &post, is_none(a[5]) ? nullptr : &next,
        xo.t.data_ptr(), xo.ld, is_none(a[5]) ? nullptr : out.t.data_ptr(), out.ld, b.rows,
        b.channels(), b.per_group(), at.handle);
    check(lib, status, "unstep_gate_residual_norm");
    PyObject *first = xo.release(), *second = first ? out.release() : nullptr;
    if (!second) {
      Py_XDECREF(first);
      return nullptr;
    }
    PyObject *pair = PyTuple_Pack(2, first, second);
    Py_DECREF(first);
    Py_DECREF(second);
    return pair;
  });
}

// ---------------------------------------------------------------------------------------------
// the 8-bit cache: the first arguments are the address of its unstep_q8_cache_t and its device
// ---------------------------------------------------------------------------------------------
struct Cache {
  unstep_q8_cache_t *q8;
  int index;

  Cache(PyObject *address, PyObject *device)
      : q8(static_cast<unstep_q8_cache_t *>(PyLong_AsVoidPtr(address))),
        index(static_cast<int>(integer(device, "device"))) {
    if (!q8) refuse("no cache");
  }

  // Address of a chunk's activations [act_B][frames * Hg * Wg][act_H][D].
  void *activation(PyObject *o, long long frames, const char *name) const {
    const unstep_cache_t &c = q8->base;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kBFloat16) refuse(std::string(name) + " must be bfloat16");
    const int64_t want[4] = {c.act_B > 0 ? c.act_B : c.B, frames * c.Hg * c.Wg,
                             c.act_H > 0 ? c.act_H : c.H, c.D};
    if (t.sizes() != at::IntArrayRef(want, 4))
      refuse(std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " +
             shape_text(at::IntArrayRef(want, 4)));
    if (!t.is_cuda() || t.get_device() != index)
      refuse(std::string(name) + " must be on the cache's device, cuda:" + std::to_string(index));
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
  }
};

// (cache, device, q, k, v, frame_idx, frames, q_out, stream) -> q_out
PyObject *q8_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 9) refuse("q8_append takes nine arguments");
    const Library &lib = library(self);
    const Cache c(a[0], a[1]);
    const long long first = integer(a[5], "frame_idx"), frames = integer(a[6], "frames");
    const void *q = c.activation(a[2], frames, "q");
    const void *k = c.activation(a[3], frames, "k"), *v = c.activation(a[4], frames, "v");
    PyObject *out = is_none(a[7]) ? a[2] : a[7];
    void *q_out = c.activation(out, frames, "q_out");
    const Place at(c.index, a[8]);
    const unstep_grid_t grid{static_cast<int>(frames), c.q8->base.Hg, c.q8->base.Wg};
    const int status =
        call(lib.append, q, q_out, k, v, c.q8, static_cast<int>(first), grid, at.handle);
    check(lib, status, "unstep_q8_rope_kv_append");
    return same(out);
  });
}

// (cache, device, q, window, out, stream) -> out
PyObject *q8_attn(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 6) refuse("q8_attn takes six arguments");
    const Library &lib = library(self);
    const Cache c(a[0], a[1]);
    const int frames = c.q8->base.last_chunk_frames;
    const void *q = c.activation(a[2], frames, "q");
    const long long window = integer(a[3], "window");
    const Place at(c.index, a[5]);
    at::Tensor fresh;
    void *out;
    if (is_none(a[4])) {
      fresh = at.fresh(tensor(a[2], "q").sizes(), at::kBFloat16);
      out = fresh.data_ptr();
    } else {
      out = c.activation(a[4], frames, "out");
    }
    const int status = call(lib.attn, q, c.q8, static_cast<int>(window), out, at.handle);
    check(lib, status, "unstep_q8_window_attn");
    return is_none(a[4]) ? THPVariable_Wrap(fresh) : same(a[4]);
  });
}

// (cache, device, first_frame, frames, k_out, v_out, stream) -> (k, v)
PyObject *q8_read(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 7) refuse("q8_read takes seven arguments");
    const Library &lib = library(self);
    const Cache c(a[0], a[1]);
    const unstep_cache_t &base = c.q8->base;
    const long long first = integer(a[2], "first_frame"), frames = integer(a[3], "frames");
    // before any output is made
    if (frames < 1 || frames > base.cap_frames)
      check(lib, frames < 1 ? UNSTEP_ERR_ARG : UNSTEP_ERR_WINDOW, "unstep_q8_cache_read");
    const int64_t want[4] = {base.B, base.H, frames * base.Hg * base.Wg, base.D};
    const Place at(c.index, a[6]);
    at::Tensor outs[2];
    static const char *const names[2] = {"k_out", "v_out"};
    for (int i = 0; i < 2; ++i) {
      if (is_none(a[4 + i])) {
        outs[i] = at.fresh(at::IntArrayRef(want, 4), at::kBFloat16);
        continue;
      }
      const at::Tensor &t = tensor(a[4 + i], names[i]);
      if (t.scalar_type() != at::kBFloat16 || t.sizes() != at::IntArrayRef(want, 4) ||
          t.get_device() != c.index || !t.is_contiguous())
        refuse(std::string(names[i]) + " must be contiguous bfloat16 " +
               shape_text(at::IntArrayRef(want, 4)) + " on cuda:" + std::to_string(c.index));
      outs[i] = t;
    }
    const int status = call(lib.read, c.q8, static_cast<int>(first), static_cast<int>(frames),
                            outs[0].data_ptr(), outs[1].data_ptr(), at.handle);
    check(lib, status, "unstep_q8_cache_read");
    PyObject *k = is_none(a[4]) ? THPVariable_Wrap(outs[0]) : same(a[4]);
    PyObject *v = !k ? nullptr : is_none(a[5]) ? THPVariable_Wrap(outs[1]) : same(a[5]);
    PyObject *pair = v ? PyTuple_Pack(2, k, v) : nullptr;
    Py_XDECREF(k);
    Py_XDECREF(v);
    return pair;
  });
}

// (UnstepError, addresses of the five entry points)
PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six arguments");
    return nullptr;
  }
  void *p[5];
  for (int i = 0; i < 5; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(a[1 + i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null entry point");
      return nullptr;
    }
  Library *l = static_cast<Library *>(PyModule_GetState(self));
  Py_INCREF(a[0]);
  PyObject *old = l->error;
  *l = {reinterpret_cast<decltype(l->norm_modulate)>(p[0]),
        reinterpret_cast<decltype(l->gate_residual_norm)>(p[1]),
        reinterpret_cast<decltype(l->append)>(p[2]), reinterpret_cast<decltype(l->attn)>(p[3]),
        reinterpret_cast<decltype(l->read)>(p[4]), a[0]};
  Py_XDECREF(old);
  Py_RETURN_NONE;
}

#define UNSTEP_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {UNSTEP_METHOD(bind),      UNSTEP_METHOD(norm_modulate),
                         UNSTEP_METHOD(gate_residual_norm), UNSTEP_METHOD(q8_append),
                         UNSTEP_METHOD(q8_attn),   UNSTEP_METHOD(q8_read),
                         {nullptr, nullptr, 0, nullptr}};
int traverse(PyObject *m, visitproc visit, void *arg) {
  if (const Library *l = static_cast<const Library *>(PyModule_GetState(m))) Py_VISIT(l->error);
  return 0;
}

int clear(PyObject *m) {
  if (Library *l = static_cast<Library *>(PyModule_GetState(m))) Py_CLEAR(l->error);
  return 0;
}

PyModuleDef_Slot slots[] = {{0, nullptr}};  // multi-phase: a state for every module object
// the docstring names the torch and Python that this was compiled for; the build looks for it
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host_calls", UNSTEP_MADE_FOR, sizeof(Library), methods, slots,
                      traverse, clear, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host_calls() { return PyModuleDef_Init(&module); }
