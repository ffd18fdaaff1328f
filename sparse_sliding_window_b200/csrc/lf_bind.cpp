// lf_bind.cpp -- the Python entry of include/lf_paged.h (module _lf_bind).
//
// A decode step is a few microseconds of GPU work per call, and checking ten
// tensors' shapes, types, devices and strides from Python costs more than
// that.  These functions make the same checks on the tensors themselves and
// call the library; each takes about half a microsecond of its own.  They
// return None, an LF_* code of the library, or the text of a refused argument.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <stdarg.h>
#include <stdio.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "lf_paged.h"

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const char *fmt, ...) {
  char text[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  throw Refused(text);
}

std::string dims(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); i++) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse("%s is no tensor", name);
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse("%s is not on a GPU", name);
  return t;
}

// t has this shape and dtype and is on CUDA device dev; packed: contiguous,
// else only its last dimension.
const at::Tensor &want(PyObject *o, const char *name, c10::IntArrayRef shape, at::ScalarType dtype, int dev,
                       bool packed = true) {
  const at::Tensor &t = tensor(o, name);
  if (t.sizes() != shape)
    refuse("%s has shape %s, %s is wanted", name, dims(t.sizes()).c_str(), dims(shape).c_str());
  if (t.scalar_type() != dtype) refuse("%s is %s, %s is wanted", name, c10::toString(t.scalar_type()), c10::toString(dtype));
  if (t.get_device() != dev) refuse("%s is on cuda:%d, the call on cuda:%d", name, (int)t.get_device(), dev);
  if (packed ? !t.is_contiguous() : shape.back() > 1 && t.stride(-1) != 1)
    refuse("%s is not contiguous%s", name, packed ? "" : " in its last dimension");
  return t;
}

int code_of(const at::Tensor &t, const char *name) {
  switch (t.scalar_type()) {
    case at::kFloat: return LF_F32;
    case at::kBFloat16: return LF_BF16;
    case at::kHalf: return LF_F16;
    default: refuse("%s is %s: float32, bfloat16 or float16 is wanted", name, c10::toString(t.scalar_type()));
  }
}

at::ScalarType type_of(int code) {
  if (code < LF_F32 || code > LF_F16) refuse("bad dtype %d", code);
  return code == LF_F32 ? at::kFloat : code == LF_BF16 ? at::kBFloat16 : at::kHalf;
}

// A ctypes structure of the library's, read in place.
struct Params {
  Py_buffer b;
  Params(PyObject *o, size_t bytes, const char *name) {
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) {
      PyErr_Clear();
      refuse("%s are no parameters", name);
    }
    if ((size_t)b.len != bytes) {
      PyBuffer_Release(&b);
      refuse("%s are no parameters", name);
    }
  }
  ~Params() { PyBuffer_Release(&b); }
  template <typename T> const T *as() const { return (const T *)b.buf; }
};

// The stream: None for dev's current one, else (device, handle).
struct Target {
  c10::cuda::OptionalCUDAGuard guard;
  void *stream;
  Target(int dev, PyObject *o) {
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    } else {
      const long on = PyLong_AsLong(PyTuple_GetItem(o, 0));
      if (on != dev) refuse("the stream is on cuda:%ld, the tensors on cuda:%d", on, dev);
      stream = PyLong_AsVoidPtr(PyTuple_GetItem(o, 1));
    }
    if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
  }
};

// Other Python threads may run while the library launches.
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename F> PyObject *call(F f) {
  int code;
  try {
    code = f();
  } catch (const Refused &e) {
    return PyUnicode_FromString(e.what());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  if (code != LF_OK) return PyLong_FromLong(code);
  Py_RETURN_NONE;
}

bool args(Py_ssize_t n, Py_ssize_t wanted) {
  if (n == wanted) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are wanted", n, wanted);
  return false;
}

// rope(backward, params, xs, outs, positions, stream)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t na) {
  if (!args(na, 6)) return nullptr;
  return call([&] {
    const Params r(a[1], sizeof(lf_rope_params), "rope");
    const bool backward = a[0] == Py_True;
    PyObject *xs = a[2], *outs = a[3];
    if (!PyList_Check(xs) || !PyList_Check(outs)) refuse("lists of tensors are wanted");
    const Py_ssize_t nt = PyList_GET_SIZE(xs);
    if (nt < 1 || nt > 8 || PyList_GET_SIZE(outs) != nt) refuse("1 to 8 tensors are wanted, and an output for each");
    const at::Tensor &first = tensor(PyList_GET_ITEM(xs, 0), "x");
    const int code = code_of(first, "x"), dev = first.get_device();
    if (first.dim() != 4) refuse("x has shape %s, [B, heads, n, 64] is wanted", dims(first.sizes()).c_str());
    const int64_t B = first.size(0), n = first.size(2);
    if (B > INT32_MAX || n > INT32_MAX) refuse("x is too large");
    lf_rope_tensor t[8];
    for (Py_ssize_t i = 0; i < nt; i++) {
      const at::Tensor &shape_of = tensor(PyList_GET_ITEM(xs, i), "x");
      if (shape_of.dim() != 4) refuse("x has shape %s, [B, heads, n, 64] is wanted", dims(shape_of.sizes()).c_str());
      const int64_t heads = shape_of.size(1), shape[4] = {B, heads, n, 64};
      if (heads > 128) refuse("x has %lld heads, at most 128 are supported", (long long)heads);
      const at::Tensor &x = want(PyList_GET_ITEM(xs, i), "x", shape, first.scalar_type(), dev, false);
      const at::Tensor &out = want(PyList_GET_ITEM(outs, i), "out", shape, first.scalar_type(), dev, false);
      t[i].x = x.const_data_ptr();
      t[i].out = out.mutable_data_ptr();
      t[i].heads = (int)heads;
      for (int k = 0; k < 3; k++) {
        t[i].x_stride[k] = x.stride(k);
        t[i].out_stride[k] = out.stride(k);
      }
    }
    const lf_rope_params *p = r.as<lf_rope_params>();
    const int32_t *positions = nullptr;
    if (a[4] != Py_None) positions = want(a[4], "positions", {p->n_axes, B, n}, at::kInt, dev).const_data_ptr<int32_t>();
    const Target to(dev, a[5]);
    const Unlocked unlocked;
    return (backward ? lf_rope_bwd : lf_rope_fwd)(p, (int)B, (int)n, code, (int)nt, t, positions, to.stream);
  });
}

// What append and decode have in common.
struct Cache {
  const lf_paged_params *p;
  at::ScalarType type;
  int dev;
  void *k, *v, *ws;
  const int32_t *table, *lengths;
  size_t ws_bytes;
  Cache(const Params &params, PyObject *kp, PyObject *vp, PyObject *tab, PyObject *len, PyObject *work)
      : p(params.as<lf_paged_params>()), type(type_of(p->dtype)), dev(tensor(kp, "k_pages").get_device()) {
    const int64_t pool[4] = {p->num_pages, p->Hkv, p->page_size, 64};
    k = want(kp, "k_pages", pool, type, dev).mutable_data_ptr();
    v = want(vp, "v_pages", pool, type, dev).mutable_data_ptr();
    table = want(tab, "block_table", {p->B, p->max_pages}, at::kInt, dev).const_data_ptr<int32_t>();
    lengths = want(len, "lengths", {p->B}, at::kInt, dev).const_data_ptr<int32_t>();
    const at::Tensor &w = tensor(work, "the workspace");
    if (w.scalar_type() != at::kByte || w.get_device() != dev || !w.is_contiguous())
      refuse("the workspace is a contiguous uint8 tensor on cuda:%d", dev);
    ws = w.mutable_data_ptr();
    ws_bytes = (size_t)w.numel();
  }
};

// append(params, rope, q, k, v, lengths, table, q_out, k_pages, v_pages, ws, cu_new, positions, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t na) {
  if (!args(na, 14)) return nullptr;
  return call([&] {
    const Params params(a[0], sizeof(lf_paged_params), "params");
    const Cache c(params, a[8], a[9], a[6], a[5], a[10]);
    const at::Tensor &kt = tensor(a[3], "k");
    if (kt.dim() != 3 || kt.size(0) > INT32_MAX) refuse("k has shape %s, [T, Hkv, 64] is wanted", dims(kt.sizes()).c_str());
    const int64_t T = kt.size(0), kv[3] = {T, c.p->Hkv, 64}, qs[3] = {T, c.p->H, 64};
    const at::Tensor &k = want(a[3], "k", kv, c.type, c.dev, false), &v = want(a[4], "v", kv, c.type, c.dev, false);
    int64_t strides[6] = {0, 0, k.stride(0), k.stride(1), v.stride(0), v.stride(1)};
    const void *q = nullptr;
    void *q_out = nullptr;
    if ((a[2] == Py_None) != (a[7] == Py_None)) refuse("q and q_out go together");
    if (a[2] != Py_None) {
      const at::Tensor &t = want(a[2], "q", qs, c.type, c.dev, false);
      q = t.const_data_ptr();
      strides[0] = t.stride(0);
      strides[1] = t.stride(1);
      q_out = want(a[7], "q_out", qs, c.type, c.dev).mutable_data_ptr();
    }
    const int32_t *cu = nullptr, *positions = nullptr;
    if (a[11] != Py_None) cu = want(a[11], "cu_new", {c.p->B + 1}, at::kInt, c.dev).const_data_ptr<int32_t>();
    const bool turns = a[1] != Py_None;
    const Params r(turns ? a[1] : a[0], turns ? sizeof(lf_rope_params) : sizeof(lf_paged_params), "rope");
    const lf_rope_params *rope = turns ? r.as<lf_rope_params>() : nullptr;
    if (a[12] != Py_None)
      positions = want(a[12], "positions", {turns ? rope->n_axes : 1, T}, at::kInt, c.dev).const_data_ptr<int32_t>();
    const Target to(c.dev, a[13]);
    const Unlocked unlocked;
    return lf_cache_append(c.p, rope, (int)T, q, k.const_data_ptr(), v.const_data_ptr(), strides, cu, c.lengths,
                           positions, c.table, q_out, c.k, c.v, c.ws, c.ws_bytes, to.stream);
  });
}

// decode(params, q, k_pages, v_pages, table, lengths, o, lse, ws, prefix_table, stream)
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t na) {
  if (!args(na, 11)) return nullptr;
  return call([&] {
    const Params params(a[0], sizeof(lf_paged_params), "params");
    const Cache c(params, a[2], a[3], a[4], a[5], a[8]);
    const int64_t rows[3] = {c.p->B, c.p->H, 64};
    const at::Tensor &q = want(a[1], "q", rows, c.type, c.dev, false);
    void *o = want(a[6], "o", rows, c.type, c.dev).mutable_data_ptr();
    float *lse = nullptr;
    if (a[7] != Py_None) lse = want(a[7], "lse", {c.p->B, c.p->H}, at::kFloat, c.dev).mutable_data_ptr<float>();
    const int prefix = c.p->prefix_len;
    const int32_t *prefix_table = nullptr;
    if ((a[9] == Py_None) != (prefix <= 0)) refuse("prefix_table goes with prefix_len > 0");
    if (prefix > 0) {
      if (c.p->page_size < 1) refuse("page_size must be a power of two, 16..1024 (got %d)", c.p->page_size);
      prefix_table = want(a[9], "prefix_table", {((int64_t)prefix + c.p->page_size - 1) / c.p->page_size}, at::kInt, c.dev)
                         .const_data_ptr<int32_t>();
    }
    const int64_t strides[2] = {q.stride(0), q.stride(1)};
    const Target to(c.dev, a[10]);
    const Unlocked unlocked;
    return lf_paged_decode(c.p, q.const_data_ptr(), strides, c.k, c.v, c.table, c.lengths, prefix_table, o, lse, c.ws,
                           c.ws_bytes, to.stream);
  });
}

PyMethodDef methods[] = {{"rope", (PyCFunction)(void *)rope, METH_FASTCALL, nullptr},
                         {"append", (PyCFunction)(void *)append, METH_FASTCALL, nullptr},
                         {"decode", (PyCFunction)(void *)decode, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
// the module's docstring names the torch it was built against
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lf_bind", LF_BIND_TAG, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lf_bind() { return PyModule_Create(&module); }
