// Native half of the Python binding of the row operators (rows.cu, norm.cu): takes the tensors'
// pointers, sizes, types and row strides, checks them against each other, and calls the C ABI on
// the tensors' device. A call of this kind takes a few microseconds on the GPU for one decoded
// token; marshalled in Python (17 to 35 arguments through ctypes, the checks, the stream lookup) it
// cost the host 15 to 25 microseconds, here 2 to 3 with the launch.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <stdexcept>
#include <string>

#include "moe_w4a16.h"

namespace {

PyObject* g_error = nullptr;      // the package's MoeError

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};            // a Python exception is already set

struct Rows {
  void* p = nullptr;
  int64_t ld = 0, n = 0, width = 0;
  int dtype = -1;
};
struct Gate {
  const void* p = nullptr;
  int64_t ld = 0;
  int mode = MOE_GATE_NONE;
};

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return MOE_DTYPE_BF16;
    case at::kHalf: return MOE_DTYPE_F16;
    case at::kFloat: return MOE_DTYPE_F32;
    default: return -1;
  }
}

// One call: its positional arguments and the device that its tensors share.
class Call {
 public:
  Call(const char* name, PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : name_(name), args_(args) {
    if (n != want) refuse("wrong number of arguments");
  }

  [[noreturn]] void refuse(const std::string& what) const { throw Refused(std::string(name_) + ": " + what); }

  bool none(int i) const { return args_[i] == Py_None; }
  double number(int i) const {
    const double v = PyFloat_AsDouble(args_[i]);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return v;
  }
  bool truth(int i) const {
    const int v = PyObject_IsTrue(args_[i]);
    if (v < 0) throw PythonError();
    return v != 0;
  }
  int whole(int i) const {
    const long v = PyLong_AsLong(args_[i]);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    if (v < INT32_MIN || v > INT32_MAX) refuse("a size does not fit 32 bits");
    return (int)v;
  }

  // A matrix of rows [n][width] (either -1: any) with neighbouring values, of type code dtype (-1: any
  // of the three).
  Rows rows(int i, const char* what, int64_t n = -1, int64_t width = -1, int dtype = -1) {
    const at::Tensor& t = tensor(i, what);
    if (t.dim() != 2) refuse(std::string(what) + " is not a matrix of rows");
    Rows r;
    r.n = t.size(0);
    r.width = t.size(1);
    if ((n >= 0 && r.n != n) || (width >= 0 && r.width != width))
      refuse(std::string(what) + " is [" + std::to_string(r.n) + "][" + std::to_string(r.width) + "], expected [" +
             (n >= 0 ? std::to_string(n) : "rows") + "][" + (width >= 0 ? std::to_string(width) : "values") + "]");
    if (r.n > INT32_MAX || r.width > INT32_MAX) refuse(std::string(what) + " has a size that does not fit 32 bits");
    r.dtype = dtype_code(t.scalar_type());
    if (r.dtype < 0 || (dtype >= 0 && r.dtype != dtype))
      refuse(std::string(what) + " is " + c10::toString(t.scalar_type()));
    if (r.n > 0 && r.width > 1 && t.stride(1) != 1)
      refuse("the values of a row of " + std::string(what) + " are not neighbours");
    r.ld = r.n > 1 ? t.stride(0) : r.width;
    r.p = t.data_ptr();
    return r;
  }

  // A contiguous tensor of this type and of `dims` sizes (a -1 fits any).
  void* dense(int i, const char* what, at::ScalarType type, std::initializer_list<int64_t> sizes) {
    const at::Tensor& t = tensor(i, what);
    bool fits = t.dim() == (int64_t)sizes.size();
    int d = 0;
    for (int64_t s : sizes) {
      if (!fits) break;
      fits = s < 0 || t.size(d) == s;
      ++d;
    }
    if (!fits) {
      std::string want;
      for (int64_t s : sizes) want += "[" + (s < 0 ? std::string("any") : std::to_string(s)) + "]";
      refuse(std::string(what) + " is not of shape " + want);
    }
    if (t.scalar_type() != type)
      refuse(std::string(what) + " is " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(type));
    if (!t.is_contiguous()) refuse(std::string(what) + " is not contiguous");
    return t.data_ptr();
  }
  void* maybe_dense(int i, const char* what, at::ScalarType type, std::initializer_list<int64_t> sizes) {
    return none(i) ? nullptr : dense(i, what, type, sizes);
  }
  Rows maybe_rows(int i, const char* what, int64_t n, int64_t width, int dtype) {
    return none(i) ? Rows{} : rows(i, what, n, width, dtype);
  }

  // int32 [T][k]
  int32_t* pairs(int i, const char* what, int* T, int* k) {
    void* p = dense(i, what, at::kInt, {-1, -1});
    const at::Tensor& t = THPVariable_Unpack(args_[i]);
    if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX || t.size(0) * t.size(1) > INT32_MAX)
      refuse(std::string(what) + " has more than 2^31-1 pairs");
    *T = (int)t.size(0);
    *k = (int)t.size(1);
    return static_cast<int32_t*>(p);
  }

  // What broadcasts over the rows: [H] per channel (`channel`: its type), fp32 [T][1] or [T] per token,
  // [T][H] of type dtype per value. A single dimension that fits both ways (fp32 channels, T = H) is per
  // channel, unless the call's gate, of mode `as`, says otherwise.
  Gate gate(int i, const char* what, int64_t T, int64_t H, int dtype, at::ScalarType channel, int as = -1) {
    Gate g;
    if (none(i)) return g;
    const at::Tensor& t = tensor(i, what);
    if (t.dim() == 1) {
      const bool fits = t.scalar_type() == channel && t.size(0) == H;
      if (as == MOE_GATE_TOKEN || (as < 0 && !fits && t.scalar_type() == at::kFloat && t.size(0) == T)) {
        g.p = dense(i, what, at::kFloat, {T});
        g.mode = MOE_GATE_TOKEN;
      } else {
        g.p = dense(i, what, channel, {H});
        g.mode = MOE_GATE_CHANNEL;
      }
    } else if (t.dim() == 2 && t.size(0) == T && t.size(1) == 1 && t.scalar_type() == at::kFloat &&
               !(H == 1 && dtype == MOE_DTYPE_F32)) {         // fp32 rows of one value: per value, any stride
      g.p = dense(i, what, at::kFloat, {T, 1});
      g.mode = MOE_GATE_TOKEN;
    } else {
      const Rows r = rows(i, what, T, H, dtype);
      g.p = r.p;
      g.ld = r.ld;
      g.mode = MOE_GATE_FULL;
    }
    return g;
  }

  void* workspace(int i, size_t* bytes) {
    *bytes = 0;
    if (none(i)) return nullptr;
    const at::Tensor& t = tensor(i, "ws");
    if (!t.is_contiguous()) refuse("ws is not contiguous");
    *bytes = t.nbytes();
    return t.data_ptr();
  }

  // Runs f(stream) on the tensors' device: argument i is None (that device's current stream) or a
  // torch.cuda.Stream of that device.
  template <typename F>
  PyObject* run(int i, F f) {
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device_);
    moe_stream_t s;
    if (none(i)) {
      s = reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device_).stream());
    } else {
      if (attribute(i, "device_index") != device_) refuse("the stream is on another device than the tensors");
      s = reinterpret_cast<moe_stream_t>(static_cast<intptr_t>(attribute(i, "cuda_stream")));
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f(s);
    Py_END_ALLOW_THREADS
    if (rc != MOE_OK) return raise(rc, moe_last_error_string());
    Py_RETURN_NONE;
  }

  static PyObject* raise(int code, const char* text) {
    PyObject* e = PyObject_CallFunction(g_error, "is", code, text);
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    return nullptr;
  }

 private:
  const at::Tensor& tensor(int i, const char* what) {
    if (!THPVariable_Check(args_[i])) refuse(std::string(what) + " is not a tensor");
    const at::Tensor& t = THPVariable_Unpack(args_[i]);
    if (!t.is_cuda()) refuse(std::string(what) + " is not on a CUDA device");
    if (t.layout() != at::kStrided) refuse(std::string(what) + " is not a dense tensor");
    if (device_ < 0) device_ = t.get_device();
    else if (t.get_device() != device_) refuse(std::string(what) + " is on another device than the tensors before it");
    return t;
  }
  long long attribute(int i, const char* name) const {
    PyObject* v = PyObject_GetAttrString(args_[i], name);
    if (!v) throw PythonError();
    const long long n = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (n == -1 && PyErr_Occurred()) throw PythonError();
    return n;
  }

  const char* name_;
  PyObject* const* args_;
  int64_t device_ = -1;
};

// Turns what a call throws into a Python exception: no C++ exception leaves an entry.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const Refused& e) {
    return Call::raise(MOE_ERR_ARG, e.what());
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// x, idx, E, counts, offsets, perm, inv, xp, stream
PyObject* dispatch(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_dispatch", args, n, 9);
  int T, k;
  const int32_t* idx = c.pairs(1, "idx", &T, &k);
  const Rows x = c.rows(0, "x", T);
  const int E = c.whole(2), H = (int)x.width;
  auto ints = [&](int i, const char* what, std::initializer_list<int64_t> s) {
    return static_cast<int32_t*>(c.dense(i, what, at::kInt, s));
  };
  int32_t *counts = ints(3, "counts", {E}), *offsets = ints(4, "offsets", {(int64_t)E + 1});
  int32_t *perm = ints(5, "perm", {(int64_t)T * k}), *inv = ints(6, "inv", {T, k});
  const Rows xp = c.rows(7, "xp", (int64_t)T * k, H, x.dtype);
  return c.run(8, [&](moe_stream_t s) {
    return moe_dispatch(x.p, x.ld, x.dtype, idx, T, H, E, k, counts, offsets, perm, inv, xp.p, xp.ld, s);
  });
}

// dxp, inv, dx, stream
PyObject* dispatch_backward(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_dispatch_backward", args, n, 4);
  int T, k;
  const int32_t* inv = c.pairs(1, "inv", &T, &k);
  const Rows dx = c.rows(2, "dx", T);
  const Rows dxp = c.rows(0, "dxp", (int64_t)T * k, dx.width, dx.dtype);
  return c.run(3, [&](moe_stream_t s) {
    return moe_dispatch_backward(dxp.p, dxp.ld, dxp.dtype, inv, T, (int)dx.width, k, dx.p, dx.ld, s);
  });
}

// yp, inv, wts, out, stream
PyObject* combine(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_combine", args, n, 5);
  int T, k;
  const int32_t* inv = c.pairs(1, "inv", &T, &k);
  const Rows out = c.rows(3, "out", T);
  const Rows yp = c.rows(0, "yp", (int64_t)T * k, out.width);
  const float* wts = static_cast<float*>(c.dense(2, "wts", at::kFloat, {T, k}));
  return c.run(4, [&](moe_stream_t s) {
    return moe_combine(yp.p, yp.ld, yp.dtype, inv, wts, T, (int)out.width, k, out.p, out.ld, out.dtype, s);
  });
}

// dout, yp, inv, wts, dyp, dwts, stream
PyObject* combine_backward(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_combine_backward", args, n, 7);
  int T, k;
  const int32_t* inv = c.pairs(2, "inv", &T, &k);
  const Rows dout = c.rows(0, "dout", T);
  const int64_t P = (int64_t)T * k;
  const Rows yp = c.maybe_rows(1, "yp", P, dout.width, -1);
  const Rows dyp = c.maybe_rows(4, "dyp", P, dout.width, yp.dtype);
  const float* wts = static_cast<float*>(c.dense(3, "wts", at::kFloat, {T, k}));
  float* dwts = static_cast<float*>(c.maybe_dense(5, "dwts", at::kFloat, {T, k}));
  const int type = yp.dtype >= 0 ? yp.dtype : dyp.dtype >= 0 ? dyp.dtype : dout.dtype;
  return c.run(6, [&](moe_stream_t s) {
    return moe_combine_backward(dout.p, dout.ld, dout.dtype, yp.p, yp.ld, type, inv, wts, T, (int)dout.width, k, dyp.p,
                                dyp.ld, dwts, s);
  });
}

// idx, wts, dwts, dlogits, stream
PyObject* route_topk_backward(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_route_topk_backward", args, n, 5);
  int T, k;
  const int32_t* idx = c.pairs(0, "idx", &T, &k);
  const float* wts = static_cast<float*>(c.dense(1, "wts", at::kFloat, {T, k}));
  const float* dwts = static_cast<float*>(c.dense(2, "dwts", at::kFloat, {T, k}));
  const Rows dl = c.rows(3, "dlogits", T);
  return c.run(4, [&](moe_stream_t s) {
    return moe_route_topk_backward(idx, wts, dwts, T, (int)dl.width, k, dl.p, dl.ld, dl.dtype, s);
  });
}

at::ScalarType scalar_type(int dtype) {
  return dtype == MOE_DTYPE_BF16 ? at::kBFloat16 : dtype == MOE_DTYPE_F16 ? at::kHalf : at::kFloat;
}

// h, w, eps, x, stream
PyObject* norm_pre(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_norm_pre", args, n, 5);
  const Rows h = c.rows(0, "h");
  const Rows x = c.rows(3, "x", h.n, h.width, h.dtype);
  const void* w = c.maybe_dense(1, "w", scalar_type(h.dtype), {h.width});
  const float eps = (float)c.number(2);
  return c.run(4, [&](moe_stream_t s) {
    return moe_norm_pre(h.p, h.ld, h.dtype, w, eps, (int)h.n, (int)h.width, x.p, x.ld, s);
  });
}

// dx, h, w, eps, dh, dres, dw, ws, stream
PyObject* norm_pre_backward(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_norm_pre_backward", args, n, 9);
  const Rows h = c.rows(1, "h");
  const Rows dx = c.rows(0, "dx", h.n, h.width, h.dtype), dh = c.rows(4, "dh", h.n, h.width, h.dtype);
  const Rows dres = c.maybe_rows(5, "dres", h.n, h.width, h.dtype);
  const void* w = c.maybe_dense(2, "w", scalar_type(h.dtype), {h.width});
  float* dw = static_cast<float*>(c.maybe_dense(6, "dw", at::kFloat, {h.width}));
  const float eps = (float)c.number(3);
  size_t bytes;
  void* ws = c.workspace(7, &bytes);
  return c.run(8, [&](moe_stream_t s) {
    return moe_norm_pre_backward(dx.p, dx.ld, h.p, h.ld, h.dtype, w, eps, (int)h.n, (int)h.width, dres.p, dres.ld, dh.p,
                                 dh.ld, dw, ws, bytes, s);
  });
}

// What moe_norm_post and moe_combine_norm_post share, from argument i on: h, h_out, eps, alpha, norm_y,
// w, gate, w_next, x_next.
struct Post {
  Rows h, h_out, x_next;
  Gate gate;
  const void *w, *w_next;
  float eps, alpha;
  int flags;
  Post(Call& c, int i) {
    h = c.rows(i, "h");
    h_out = c.rows(i + 1, "h_out", h.n, h.width, h.dtype);
    eps = (float)c.number(i + 2);
    alpha = (float)c.number(i + 3);
    const bool norm_y = c.truth(i + 4), next = !c.none(i + 8);
    if (!norm_y && !c.none(i + 5)) c.refuse("w without norm_y");
    if (!next && !c.none(i + 7)) c.refuse("w_next without x_next");
    w = c.maybe_dense(i + 5, "w", scalar_type(h.dtype), {h.width});
    gate = c.gate(i + 6, "gate", h.n, h.width, h.dtype, scalar_type(h.dtype));
    w_next = c.maybe_dense(i + 7, "w_next", scalar_type(h.dtype), {h.width});
    x_next = c.maybe_rows(i + 8, "x_next", h.n, h.width, h.dtype);
    flags = (norm_y ? MOE_NORM_Y : 0) | (next ? MOE_NORM_NEXT : 0);
  }
};

// y, h, h_out, eps, alpha, norm_y, w, gate, w_next, x_next, stream
PyObject* norm_post(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_norm_post", args, n, 11);
  const Post a(c, 1);
  const Rows y = c.rows(0, "y", a.h.n, a.h.width, a.h.dtype);
  return c.run(10, [&](moe_stream_t s) {
    return moe_norm_post(y.p, y.ld, a.h.p, a.h.ld, a.h.dtype, a.w, a.gate.p, a.gate.ld, a.gate.mode, a.alpha, a.eps,
                         (int)a.h.n, (int)a.h.width, a.flags, a.h_out.p, a.h_out.ld, a.w_next, a.x_next.p, a.x_next.ld,
                         s);
  });
}

// yp, inv, wts, h, h_out, eps, alpha, norm_y, w, gate, w_next, x_next, y_out, stream
PyObject* combine_norm_post(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_combine_norm_post", args, n, 14);
  const Post a(c, 3);
  int T, k;
  const int32_t* inv = c.pairs(1, "inv", &T, &k);
  if (T != a.h.n) c.refuse("inv has " + std::to_string(T) + " tokens, h " + std::to_string(a.h.n));
  const Rows yp = c.rows(0, "yp", (int64_t)T * k, a.h.width);
  const float* wts = static_cast<float*>(c.dense(2, "wts", at::kFloat, {T, k}));
  const Rows yo = c.maybe_rows(12, "y_out", a.h.n, a.h.width, a.h.dtype);
  return c.run(13, [&](moe_stream_t s) {
    return moe_combine_norm_post(yp.p, yp.ld, yp.dtype, inv, wts, k, a.h.p, a.h.ld, a.h.dtype, a.w, a.gate.p, a.gate.ld,
                                 a.gate.mode, a.alpha, a.eps, T, (int)a.h.width, a.flags, a.h_out.p, a.h_out.ld,
                                 a.w_next, a.x_next.p, a.x_next.ld, yo.p, yo.ld, s);
  });
}

// dh_out, y, dh, dy, eps, alpha, norm_y, w, dw, gate, dgate, h_out, w_next, dx_next, dw_next, ws, stream
PyObject* norm_post_backward(PyObject* const* args, Py_ssize_t n) {
  Call c("moe_norm_post_backward", args, n, 17);
  const Rows d = c.rows(0, "dh_out");
  const int64_t T = d.n, H = d.width;
  const Rows y = c.rows(1, "y", T, H, d.dtype), dh = c.rows(2, "dh", T, H, d.dtype),
             dy = c.rows(3, "dy", T, H, d.dtype);
  const float eps = (float)c.number(4), alpha = (float)c.number(5);
  const bool norm_y = c.truth(6), next = !c.none(13);
  if (!next && (!c.none(11) || !c.none(12) || !c.none(14))) c.refuse("h_out, w_next or dw_next without dx_next");
  if (next && c.none(11)) c.refuse("dx_next without h_out");
  if (!norm_y && (!c.none(7) || !c.none(8))) c.refuse("w or dw without norm_y");
  const at::ScalarType type = scalar_type(d.dtype);
  const void* w = c.maybe_dense(7, "w", type, {H});
  float* dw = static_cast<float*>(c.maybe_dense(8, "dw", at::kFloat, {H}));
  const Gate g = c.gate(9, "gate", T, H, d.dtype, type);
  const Gate dg = c.gate(10, "dgate", T, H, d.dtype, at::kFloat, g.mode);
  if (dg.p && dg.mode != g.mode) c.refuse("dgate has another form than gate");
  const Rows ho = c.maybe_rows(11, "h_out", T, H, d.dtype);
  const void* wn = c.maybe_dense(12, "w_next", type, {H});
  const Rows dx = c.maybe_rows(13, "dx_next", T, H, d.dtype);
  float* dwn = static_cast<float*>(c.maybe_dense(14, "dw_next", at::kFloat, {H}));
  size_t bytes;
  void* ws = c.workspace(15, &bytes);
  const int flags = (norm_y ? MOE_NORM_Y : 0) | (next ? MOE_NORM_NEXT : 0);
  return c.run(16, [&](moe_stream_t s) {
    return moe_norm_post_backward(d.p, d.ld, y.p, y.ld, d.dtype, w, g.p, g.ld, g.mode, alpha, eps, (int)T, (int)H,
                                  flags, ho.p, ho.ld, wn, dx.p, dx.ld, dh.p, dh.ld, dy.p, dy.ld, dw,
                                  const_cast<void*>(dg.p),
                                  dg.ld, dwn, ws, bytes, s);
  });
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

#define MOE_ENTRY(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {MOE_ENTRY(dispatch),
                         MOE_ENTRY(dispatch_backward),
                         MOE_ENTRY(combine),
                         MOE_ENTRY(combine_backward),
                         MOE_ENTRY(route_topk_backward),
                         MOE_ENTRY(norm_pre),
                         MOE_ENTRY(norm_pre_backward),
                         MOE_ENTRY(norm_post),
                         MOE_ENTRY(combine_norm_post),
                         MOE_ENTRY(norm_post_backward),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rows", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch whose tensors this module reads; the package refuses it under another.
PyMODINIT_FUNC PyInit__rows(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
