// Argument marshalling of the 8-bit token path's calls for Python, as an extension module: each takes a few
// microseconds on the GPU, about what ctypes needs to convert sixteen arguments (5.8 us a call of
// wr_gemm_i8 through ctypes). The functions forward to the C entry points of the same names in
// libwr.so. Device operands are torch CUDA tensors on the current device, addresses (int) or None; torch
// supplies the current device and stream, nothing else.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "wr.h"

namespace {

PyObject* g_error = nullptr;                        // WrError(function, status)
PyObject *g_get_device, *g_data_ptr, *g_cuda_stream;   // method names
PyObject *g_current_device = nullptr, *g_raw_stream = nullptr;   // torch's, looked up at the first need

bool torch_calls() {
  if (g_raw_stream) return true;
  PyObject* torch = PyImport_ImportModule("torch");
  if (!torch) return false;
  PyObject* cuda = PyObject_GetAttrString(torch, "cuda");
  PyObject* init = cuda ? PyObject_CallMethod(cuda, "init", nullptr) : nullptr;
  PyObject* c = init ? PyObject_GetAttrString(torch, "_C") : nullptr;
  PyObject* dev = c ? PyObject_GetAttrString(c, "_cuda_getDevice") : nullptr;
  PyObject* raw = dev ? PyObject_GetAttrString(c, "_cuda_getCurrentRawStream") : nullptr;
  Py_XDECREF(c);
  Py_XDECREF(init);
  Py_XDECREF(cuda);
  Py_DECREF(torch);
  if (!raw) {
    Py_XDECREF(dev);
    return false;
  }
  g_current_device = dev;
  g_raw_stream = raw;
  return true;
}

bool as_int(PyObject* o, long long* v) {
  *v = PyLong_AsLongLong(o);
  return !(*v == -1 && PyErr_Occurred());
}
bool as_int32(PyObject* o, int32_t* v) {
  long long x;
  if (!as_int(o, &x)) return false;
  if (x < INT32_MIN || x > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "int32 argument out of range");
    return false;
  }
  *v = (int32_t)x;
  return true;
}
bool as_float(PyObject* o, float* v) {
  const double x = PyFloat_AsDouble(o);
  *v = (float)x;
  return !(x == -1.0 && PyErr_Occurred());
}

// The device of a call: that of torch's current context, asked for once a call and only if needed.
struct Call {
  long device = -1;
  bool know_device() {
    if (device >= 0) return true;
    if (!torch_calls()) return false;
    PyObject* d = PyObject_CallNoArgs(g_current_device);
    if (!d) return false;
    device = PyLong_AsLong(d);
    Py_DECREF(d);
    return !(device == -1 && PyErr_Occurred());
  }
  bool pointer(PyObject* o, const void** p) {
    if (!o || o == Py_None) {
      *p = nullptr;
      return true;
    }
    if (PyLong_Check(o)) {
      *p = PyLong_AsVoidPtr(o);
      return !(*p == nullptr && PyErr_Occurred());
    }
    PyObject* d = PyObject_CallMethodNoArgs(o, g_get_device);
    if (!d) return false;
    const long dev = PyLong_AsLong(d);
    Py_DECREF(d);
    if (dev == -1 && PyErr_Occurred()) return false;
    if (dev < 0) {
      PyErr_SetString(PyExc_ValueError, "expected a CUDA tensor, got one on the host");
      return false;
    }
    if (!know_device()) return false;
    if (dev != device) {
      PyErr_Format(PyExc_ValueError, "tensor on cuda:%ld, but the current device is cuda:%ld", dev, device);
      return false;
    }
    PyObject* a = PyObject_CallMethodNoArgs(o, g_data_ptr);
    if (!a) return false;
    *p = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    return !(*p == nullptr && PyErr_Occurred());
  }
  template <typename T>
  bool pointer(PyObject* o, T** p) {
    const void* v;
    if (!pointer(o, &v)) return false;
    *p = const_cast<T*>(static_cast<const T*>(v));
    return true;
  }
  bool stream(PyObject* o, void** s) {
    PyObject* v = nullptr;
    if (!o || o == Py_None) {
      if (!know_device()) return false;
      PyObject* d = PyLong_FromLong(device);
      v = d ? PyObject_CallOneArg(g_raw_stream, d) : nullptr;
      Py_XDECREF(d);
    } else if (PyLong_Check(o)) {
      v = Py_NewRef(o);
    } else {
      v = PyObject_GetAttr(o, g_cuda_stream);
    }
    if (!v) return false;
    *s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !(*s == nullptr && PyErr_Occurred());
  }
};

// Names of a function's parameters; the first `required` have to be given, the first `positional` may be
// given without their names.
struct Signature {
  const char* function;
  int count, required, positional;
  const char* const* names;
  PyObject** interned;

  bool parse(PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames, PyObject** out) const {
    if (nargs > positional) {
      PyErr_Format(PyExc_TypeError, "%s() takes %d positional arguments but %zd were given", function, positional, nargs);
      return false;
    }
    for (int i = 0; i < count; ++i) out[i] = i < nargs ? args[i] : nullptr;
    const Py_ssize_t nkw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    int at = 0;   // callers mostly keep the order: search from the last hit on
    for (Py_ssize_t k = 0; k < nkw; ++k) {
      PyObject* name = PyTuple_GET_ITEM(kwnames, k);
      int found = -1;
      for (int i = 0; i < count && found < 0; ++i) {
        const int j = at + i < count ? at + i : at + i - count;
        if (interned[j] == name) found = j;
      }
      for (int j = 0; j < count && found < 0; ++j) {
        if (PyUnicode_Compare(interned[j], name) == 0) found = j;
        if (PyErr_Occurred()) return false;
      }
      if (found < 0) {
        PyErr_Format(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", function, name);
        return false;
      }
      if (out[found]) {
        PyErr_Format(PyExc_TypeError, "%s() got multiple values for argument '%s'", function, names[found]);
        return false;
      }
      out[found] = args[nargs + k];
      at = found;
    }
    for (int i = 0; i < required; ++i) {
      if (!out[i]) {
        PyErr_Format(PyExc_TypeError, "%s() missing required argument '%s'", function, names[i]);
        return false;
      }
    }
    return true;
  }
};

PyObject* finish(const char* function, wr_status st) {
  if (st == WR_OK) Py_RETURN_NONE;
  PyObject* e = PyObject_CallFunction(g_error, "si", function, (int)st);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// ---------------------------------------------------------------- wr_quantize_rows

const char* const kQuantNames[] = {"type", "M", "K", "x", "ldx", "q", "ldq", "scale", "gate", "ldg", "stream"};
PyObject* quant_interned[11];
const Signature kQuant = {"wr_quantize_rows", 11, 8, 11, kQuantNames, quant_interned};

PyObject* quantize_rows(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  PyObject* v[11];
  if (!kQuant.parse(args, nargs, kwnames, v)) return nullptr;
  Call c;
  int32_t type;
  long long M, K, ldx, ldq, ldg = 0;
  const void *x, *gate;
  int8_t* q;
  float* scale;
  void* stream;
  if (!as_int32(v[0], &type) || !as_int(v[1], &M) || !as_int(v[2], &K) || !c.pointer(v[3], &x) || !as_int(v[4], &ldx) ||
      !c.pointer(v[5], &q) || !as_int(v[6], &ldq) || !c.pointer(v[7], &scale) || !c.pointer(v[8], &gate) ||
      (v[9] && !as_int(v[9], &ldg)) || !c.stream(v[10], &stream))
    return nullptr;
  wr_status st;
  Py_BEGIN_ALLOW_THREADS
  st = wr_quantize_rows(type, M, K, x, ldx, gate, ldg, q, ldq, scale, stream);
  Py_END_ALLOW_THREADS
  return finish("wr_quantize_rows", st);
}

// ---------------------------------------------------------------- wr_gemm_i8

const char* const kGemmNames[] = {"M", "N", "K", "x", "ldx", "x_scale", "w", "ldw", "w_scale", "y_type", "y", "ldy", "workspace",
                                  "workspace_bytes", "bias", "stream"};
PyObject* gemm_interned[16];
const Signature kGemm = {"wr_gemm_i8", 16, 14, 16, kGemmNames, gemm_interned};

PyObject* gemm_i8(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  PyObject* v[16];
  if (!kGemm.parse(args, nargs, kwnames, v)) return nullptr;
  Call c;
  long long M, N, K, ldx, ldw, ldy, bytes;
  int32_t y_type;
  const int8_t *x, *w;
  const float *xs, *ws, *bias;
  void *y, *workspace, *stream;
  if (!as_int(v[0], &M) || !as_int(v[1], &N) || !as_int(v[2], &K) || !c.pointer(v[3], &x) || !as_int(v[4], &ldx) ||
      !c.pointer(v[5], &xs) || !c.pointer(v[6], &w) || !as_int(v[7], &ldw) || !c.pointer(v[8], &ws) || !as_int32(v[9], &y_type) ||
      !c.pointer(v[10], &y) || !as_int(v[11], &ldy) || !c.pointer(v[12], &workspace) || !as_int(v[13], &bytes) ||
      !c.pointer(v[14], &bias) || !c.stream(v[15], &stream))
    return nullptr;
  if (bytes < 0) bytes = 0;
  wr_status st;
  Py_BEGIN_ALLOW_THREADS
  st = wr_gemm_i8(M, N, K, x, ldx, xs, w, ldw, ws, bias, y_type, y, ldy, workspace, (size_t)bytes, stream);
  Py_END_ALLOW_THREADS
  return finish("wr_gemm_i8", st);
}

// ---------------------------------------------------------------- wr_residual_norm

enum NormArg { M_, D_, BLOCK, LD_BLOCK, BLOCK_TYPE, RESIDUAL, LD_RESIDUAL, RESIDUAL_OUT, LD_RESIDUAL_OUT, RESIDUAL_TYPE, GATE,
               LD_GATE, GATE_TYPE, POST_WEIGHT, NORM_WEIGHT, WEIGHT_TYPE, WEIGHT_OFFSET, POST_NORM, Y, LD_Y, Y_TYPE, Y_SCALE,
               RESIDUAL_SCALE, EPS, STREAM, NORM_ARGS };
const char* const kNormNames[] = {"M", "D", "block", "ld_block", "block_type", "residual", "ld_residual", "residual_out",
                                  "ld_residual_out", "residual_type", "gate", "ld_gate", "gate_type", "post_weight",
                                  "norm_weight", "weight_type", "weight_offset", "post_norm", "y", "ld_y", "y_type", "y_scale",
                                  "residual_scale", "eps", "stream"};
PyObject* norm_interned[NORM_ARGS];
const Signature kNorm = {"wr_residual_norm", NORM_ARGS, 2, 2, kNormNames, norm_interned};

PyObject* residual_norm(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  PyObject* v[NORM_ARGS];
  if (!kNorm.parse(args, nargs, kwnames, v)) return nullptr;
  Call c;
  wr_residual_norm_args a = {};
  a.eps = 1e-6f;
  a.residual_scale = 1.f;
  void* stream;
  auto integer = [&](int i, int64_t* o) {
    long long x;
    if (!v[i]) return true;
    if (!as_int(v[i], &x)) return false;
    *o = x;
    return true;
  };
  auto type = [&](int i, int32_t* o) { return !v[i] || as_int32(v[i], o); };
  auto real = [&](int i, float* o) { return !v[i] || as_float(v[i], o); };
  if (!integer(M_, &a.M) || !integer(D_, &a.D) || !c.pointer(v[BLOCK], &a.block) || !integer(LD_BLOCK, &a.ld_block) ||
      !type(BLOCK_TYPE, &a.block_type) || !c.pointer(v[RESIDUAL], &a.residual) || !integer(LD_RESIDUAL, &a.ld_residual) ||
      !c.pointer(v[RESIDUAL_OUT], &a.residual_out) || !integer(LD_RESIDUAL_OUT, &a.ld_residual_out) ||
      !type(RESIDUAL_TYPE, &a.residual_type) || !c.pointer(v[GATE], &a.gate) || !integer(LD_GATE, &a.ld_gate) ||
      !type(GATE_TYPE, &a.gate_type) || !c.pointer(v[POST_WEIGHT], &a.post_weight) ||
      !c.pointer(v[NORM_WEIGHT], &a.norm_weight) || !type(WEIGHT_TYPE, &a.weight_type) || !real(WEIGHT_OFFSET, &a.weight_offset) ||
      !c.pointer(v[Y], &a.y) || !integer(LD_Y, &a.ld_y) || !type(Y_TYPE, &a.y_type) || !c.pointer(v[Y_SCALE], &a.y_scale) ||
      !real(RESIDUAL_SCALE, &a.residual_scale) || !real(EPS, &a.eps) || !c.stream(v[STREAM], &stream))
    return nullptr;
  if (!v[POST_NORM] || v[POST_NORM] == Py_None) {
    a.post_norm = a.post_weight != nullptr;
  } else {
    a.post_norm = PyObject_IsTrue(v[POST_NORM]);
    if (a.post_norm < 0) return nullptr;
  }
  wr_status st;
  Py_BEGIN_ALLOW_THREADS
  st = wr_residual_norm(&a, stream);
  Py_END_ALLOW_THREADS
  return finish("wr_residual_norm", st);
}

// ---------------------------------------------------------------- the module

PyObject* set_error(PyObject*, PyObject* e) {
  Py_XSETREF(g_error, Py_NewRef(e));
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"set_error", set_error, METH_O, "The exception class of refused calls."},
    {"wr_quantize_rows", (PyCFunction)(void (*)(void))quantize_rows, METH_FASTCALL | METH_KEYWORDS,
     "wr_quantize_rows(type, M, K, x, ldx, q, ldq, scale, gate=None, ldg=0, stream=None)\n--\n\n"
     "Rows of x (or of silu(gate) * x) -> int8 codes q and one fp32 scale per row (device)."},
    {"wr_gemm_i8", (PyCFunction)(void (*)(void))gemm_i8, METH_FASTCALL | METH_KEYWORDS,
     "wr_gemm_i8(M, N, K, x, ldx, x_scale, w, ldw, w_scale, y_type, y, ldy, workspace, workspace_bytes, bias=None, stream=None)\n--\n\n"
     "y = (x w^T) * x_scale[:, None] * w_scale (+ bias) from int8 tokens and int8 output channels (device)."},
    {"wr_residual_norm", (PyCFunction)(void (*)(void))residual_norm, METH_FASTCALL | METH_KEYWORDS,
     "wr_residual_norm(M, D, *, block=None, ld_block=0, block_type=0, residual=None, ld_residual=0, residual_out=None, "
     "ld_residual_out=0, residual_type=0, gate=None, ld_gate=0, gate_type=0, post_weight=None, norm_weight=None, weight_type=0, "
     "weight_offset=0.0, post_norm=None, y=None, ld_y=0, y_type=0, y_scale=None, residual_scale=1.0, eps=1e-06, stream=None)\n--\n\n"
     "h' = residual_scale * residual + gate * post(block) and y = norm(h'), in one pass (wr_residual_norm of\n"
     "include/wr.h; types default to WR_F32). post_norm: whether the block's output is normed first; by default,\n"
     "whether post_weight is given."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", "Argument marshalling of libwr's 8-bit token path.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

bool intern(const Signature& s) {
  for (int i = 0; i < s.count; ++i)
    if (!(s.interned[i] = PyUnicode_InternFromString(s.names[i]))) return false;
  return true;
}

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  g_get_device = PyUnicode_InternFromString("get_device");
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!g_get_device || !g_data_ptr || !g_cuda_stream || !intern(kQuant) || !intern(kGemm) || !intern(kNorm)) return nullptr;
  g_error = Py_NewRef(PyExc_RuntimeError);
  return PyModule_Create(&kModule);
}
