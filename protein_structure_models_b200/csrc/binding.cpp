// binding.cpp -- the calls of the sequence operators from Python: checks the
// tensors, allocates what the caller did not give, and calls the C ABI of
// libfipa.so (include/fipa.h), whose entry points it is given by address.
//
// These operators are called many times a step on small tensors, where a call
// lasts as long as the host takes to make it: the same checks and allocations
// through Python and ctypes took 9 to 14 us a call, most of it more than the kernel.
//
// Every function returns a tuple of tensors (None where there is none), or the
// status of a call that was refused; tensors that do not fit raise ValueError.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "fipa.h"

namespace {

struct Entry {
  decltype(&fipa_window_attention) window;
  decltype(&fipa_window_attention_workspace_size) window_size;
  decltype(&fipa_window_attention_backward) window_backward;
  decltype(&fipa_window_attention_backward_workspace_size) window_backward_size;
  decltype(&fipa_norm_residual) norm;
  decltype(&fipa_norm_residual_backward_workspace_size) norm_size;
  decltype(&fipa_norm_residual_backward) norm_backward;
  decltype(&fipa_embedding) embedding;
  decltype(&fipa_embedding_backward_workspace_size) embedding_size;
  decltype(&fipa_embedding_backward) embedding_backward;
} entry;

struct Refused {                       // a ValueError
  std::string why;
};
struct Raised {};                      // a Python error that is set already

using at::Tensor;

void need(bool ok, const char* why) {
  if (!ok) throw Refused{why};
}
// Arguments in order.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  PyObject* next() {
    if (i >= n) {
      PyErr_SetString(PyExc_TypeError, "too few arguments");
      throw Raised{};
    }
    return a[i++];
  }
  const Tensor& tensor() {
    PyObject* o = next();
    if (!THPVariable_Check(o)) {
      PyErr_SetString(PyExc_TypeError, "a tensor was expected");
      throw Raised{};
    }
    return THPVariable_Unpack(o);
  }
  Tensor optional() {
    if (i < n && a[i] == Py_None) {
      ++i;
      return Tensor();
    }
    return tensor();
  }
  long long integer() {
    const long long x = PyLong_AsLongLong(next());
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    return x;
  }
  int i32() {
    const long long x = integer();
    return (int)(x < -0x7fffffffll ? -0x7fffffffll : (x > 0x7fffffffll ? 0x7fffffffll : x));
  }
  double real() {
    const double x = PyFloat_AsDouble(next());
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return x;
  }
  bool none() {
    const bool x = i < n && a[i] == Py_None;
    if (x) ++i;
    return x;
  }
  // the address of a stream, or None: the device's current one
  void* stream(int device) {
    if (none()) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    PyObject* o = next();
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw Raised{};
    return p;
  }
};
void* at_of(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
bool floats(const Tensor& t) { return t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16; }
fipa_dtype code(at::ScalarType t) { return t == at::kFloat ? FIPA_F32 : FIPA_BF16; }
bool bytes(const Tensor& t) { return t.scalar_type() == at::kBool || t.scalar_type() == at::kByte; }
// contiguous, of this type and shape, on device `dev`
bool fits(const Tensor& t, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.sizes() == shape && t.is_contiguous();
}
Tensor make(const Tensor& like, at::IntArrayRef shape, at::ScalarType type) { return at::empty(shape, like.options().dtype(type)); }
Tensor room(const Tensor& given, const Tensor& like, size_t bytes, int dev) {
  if (!given.defined()) return make(like, {(int64_t)bytes}, at::kByte);
  need(given.is_cuda() && given.get_device() == dev && given.is_contiguous(), "workspace: need a contiguous tensor on the inputs' device");
  return given;
}
PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <typename... T>
PyObject* answer(fipa_status st, const T&... t) {
  if (st != FIPA_OK) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New(sizeof...(t));
  if (r == nullptr) return nullptr;
  Py_ssize_t k = 0;
  for (PyObject* o : {wrap(t)...}) PyTuple_SET_ITEM(r, k++, o);
  return r;
}
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.why.c_str());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ---------------------------------------------------------------- window attention
struct Window {
  fipa_handle* h;
  int dev;
  at::ScalarType type;
  Tensor q, k, v, mask, start;
  fipa_heads hq, hk, hv;
  fipa_window w;
};
fipa_heads heads(const Tensor& t) {
  need(t.stride(3) == 1 || t.size(3) <= 1, "q, k, v: need a contiguous width");
  return fipa_heads{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}
int size32(int64_t x) {
  need(x <= 0x7fffffff, "a size beyond 2^31");
  return (int)x;
}
// handle, dtype, device, q, k, v, left, right, sinks, mask, q_start, scale
Window window_args(Args& a) {
  Window p;
  p.h = reinterpret_cast<fipa_handle*>(a.integer());
  p.type = a.integer() == FIPA_F32 ? at::kFloat : at::kBFloat16;
  p.dev = (int)a.integer();
  p.q = a.tensor();
  p.k = a.tensor();
  p.v = a.tensor();
  for (const Tensor* t : {&p.q, &p.k, &p.v})
    need(t->dim() == 4 && t->is_cuda() && t->get_device() == p.dev && t->scalar_type() == p.type,
         "q, k, v: need tensors [B, N, heads, width] of the handle's dtype on its device");
  const int64_t B = p.q.size(0), Nq = p.q.size(1), H = p.q.size(2), D = p.q.size(3), Nk = p.v.size(1), Hkv = p.v.size(2), Dv = p.v.size(3);
  need(p.k.size(0) == B && p.v.size(0) == B && p.k.size(1) == Nk && p.k.size(2) == Hkv && p.k.size(3) == D,
       "q [B,Nq,H,D], k [B,Nk,Hkv,D], v [B,Nk,Hkv,Dv] do not fit together");
  p.hq = heads(p.q);
  p.hk = heads(p.k);
  p.hv = heads(p.v);
  p.w.B = size32(B); p.w.Nq = size32(Nq); p.w.Nk = size32(Nk); p.w.H = size32(H); p.w.Hkv = size32(Hkv);
  p.w.D = size32(D); p.w.Dv = size32(Dv);
  p.w.left = a.i32();
  p.w.right = a.i32();
  p.w.sinks = a.i32();
  p.mask = a.optional();
  if (p.mask.defined()) need(bytes(p.mask) && fits(p.mask, p.mask.scalar_type(), {B, Nk}, p.dev), "mask: need a contiguous bool/uint8 tensor [B, Nk] on the inputs' device");
  p.start = a.optional();
  if (p.start.defined()) need(fits(p.start, at::kInt, {B}, p.dev), "q_start: need a contiguous int32 tensor [B] on the inputs' device");
  p.w.scale = a.none() ? (D > 0 ? 1.0 / std::sqrt((double)D) : 0.0) : a.real();
  return p;
}
// ..., want_lse, out, lse, workspace, stream -> out, lse
PyObject* window(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{argv, n};
    Window p = window_args(a);
    const fipa_window& w = p.w;
    const bool want = a.integer() != 0;
    Tensor out = a.optional(), lse = a.optional();
    if (out.defined()) {
      need(fits(out, p.type, {w.B, w.Nq, w.H, w.Dv}, p.dev), "out: need a contiguous tensor [B, Nq, H, Dv] of the handle's dtype");
      need(!lse.defined() || fits(lse, at::kFloat, {w.B, w.H, w.Nq}, p.dev), "lse: need a contiguous float32 tensor [B, H, Nq]");
    } else {
      out = make(p.q, {w.B, w.Nq, w.H, w.Dv}, p.type);
      if (want) lse = make(p.q, {w.B, w.H, w.Nq}, at::kFloat);
    }
    Tensor ws = a.optional();
    size_t size = 0;
    if (!ws.defined()) {
      const fipa_status st = entry.window_size(p.h, &p.hq, &p.hk, &p.hv, &w, &size);
      if (st != FIPA_OK) return PyLong_FromLong(st);
    }
    if (ws.defined() || size > 0) ws = room(ws, p.q, size, p.dev);
    return answer(entry.window(p.h, &p.hq, &p.hk, &p.hv, static_cast<const uint8_t*>(at_of(p.mask)), static_cast<const int32_t*>(at_of(p.start)),
                               &w, out.data_ptr(), static_cast<float*>(at_of(lse)), at_of(ws), ws.defined() ? ws.nbytes() : 0, a.stream(p.dev)),
                  out, lse);
  });
}
// ..., out, lse, d_out, d_q, d_k, d_v, workspace, stream -> d_q, d_k, d_v
PyObject* window_backward(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{argv, n};
    Window p = window_args(a);
    const fipa_window& w = p.w;
    const Tensor &out = a.tensor(), &lse = a.tensor(), &d_out = a.tensor();
    need(fits(out, p.type, {w.B, w.Nq, w.H, w.Dv}, p.dev) && fits(d_out, p.type, {w.B, w.Nq, w.H, w.Dv}, p.dev) &&
             fits(lse, at::kFloat, {w.B, w.H, w.Nq}, p.dev),
         "out, d_out [B, Nq, H, Dv] of the handle's dtype, lse [B, H, Nq] float32: need contiguous tensors on the inputs' device");
    Tensor g[3];
    const int64_t shape[3][4] = {{w.B, w.Nq, w.H, w.D}, {w.B, w.Nk, w.Hkv, w.D}, {w.B, w.Nk, w.Hkv, w.Dv}};
    for (int i = 0; i < 3; ++i) {
      g[i] = a.optional();
      if (g[i].defined()) need(fits(g[i], p.type, shape[i], p.dev), "gradients: need contiguous tensors of the shapes of q, k, v");
      else g[i] = make(p.q, shape[i], p.type);
    }
    Tensor ws = a.optional();
    size_t size = 0;
    if (!ws.defined()) {
      const fipa_status st = entry.window_backward_size(p.h, &p.hq, &p.hk, &p.hv, &w, &size);
      if (st != FIPA_OK) return PyLong_FromLong(st);
    }
    ws = room(ws, p.q, size, p.dev);
    return answer(entry.window_backward(p.h, &p.hq, &p.hk, &p.hv, static_cast<const uint8_t*>(at_of(p.mask)),
                                        static_cast<const int32_t*>(at_of(p.start)), &w, out.data_ptr(), static_cast<const float*>(lse.data_ptr()),
                                        d_out.data_ptr(), g[0].data_ptr(), g[1].data_ptr(), g[2].data_ptr(), ws.data_ptr(), ws.nbytes(),
                                        a.stream(p.dev)),
                  g[0], g[1], g[2]);
  });
}

// ---------------------------------------------------------------- junction
struct Norm {
  int dev;
  at::ScalarType branch;
  Tensor s, u, gate, mask, par[5];     // res_scale, post_w, post_b, pre_w, pre_b
  fipa_norm_dims d;
  fipa_norm_inputs in;
};
// s, u, gate, res_scale, post_w, post_b, pre_w, pre_b, mask, kind, eps, branch dtype (-1: that of u or s)
Norm norm_args(Args& a) {
  Norm p;
  p.s = a.tensor();
  p.u = a.optional();
  p.gate = a.optional();
  need(p.s.is_cuda() && p.s.dim() > 0 && floats(p.s) && p.s.is_contiguous(), "s: need a contiguous float32 or bfloat16 CUDA tensor [..., C]");
  p.dev = (int)p.s.get_device();
  const int64_t C = p.s.size(-1);
  for (Tensor& t : p.par) t = a.optional();
  p.mask = a.optional();
  const long long kind = a.integer();
  const double eps = a.real();
  const long long branch = a.integer();
  p.branch = p.u.defined() ? p.u.scalar_type() : (branch < 0 ? p.s.scalar_type() : (branch == FIPA_F32 ? at::kFloat : at::kBFloat16));
  need(!p.u.defined() || (floats(p.u) && fits(p.u, p.branch, p.s.sizes(), p.dev)), "u: need a contiguous float32 or bfloat16 tensor of the shape of s");
  need(!p.gate.defined() || fits(p.gate, p.branch, p.s.sizes(), p.dev), "gate: need a contiguous tensor of the shape of s and the type of u");
  for (const Tensor& t : p.par)
    need(!t.defined() || fits(t, at::kFloat, {C}, p.dev), "res_scale, post, pre: need contiguous float32 tensors [C] on the device of s");
  if (p.mask.defined())
    need(bytes(p.mask) && fits(p.mask, p.mask.scalar_type(), p.s.sizes().slice(0, p.s.dim() - 1), p.dev), "mask: need a contiguous bool/uint8 tensor of the leading shape of s");
  p.d = fipa_norm_dims{C > 0 ? p.s.numel() / C : 0, size32(C), code(p.s.scalar_type()), code(p.branch), kind == 0 ? FIPA_NORM_LAYER : FIPA_NORM_RMS, eps};
  auto f = [&](int i) { return static_cast<const float*>(at_of(p.par[i])); };
  p.in = fipa_norm_inputs{p.s.data_ptr(), at_of(p.u), at_of(p.gate), static_cast<const uint8_t*>(at_of(p.mask)), f(0), f(1), f(2), f(3), f(4)};
  return p;
}
// ..., want_stats, given (whether r, x, stats are the caller's), r, x, stats, stream -> r, x, stats
PyObject* norm(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{argv, n};
    Norm p = norm_args(a);
    const bool want = a.integer() != 0, given = a.integer() != 0;
    Tensor r = a.optional(), x = a.optional(), stats = a.optional();
    c10::cuda::CUDAGuard on((c10::DeviceIndex)p.dev);
    if (given) {
      need(!r.defined() || fits(r, p.s.scalar_type(), p.s.sizes(), p.dev), "r: need a contiguous tensor like s");
      need(!x.defined() || fits(x, p.branch, p.s.sizes(), p.dev), "x: need a contiguous tensor of the shape of s and the branch's type");
      need(!stats.defined() || fits(stats, at::kFloat, {p.d.rows, 4}, p.dev), "stats: need a contiguous float32 tensor [rows, 4]");
    } else {
      if (p.u.defined()) r = make(p.s, p.s.sizes(), p.s.scalar_type());
      if (p.par[3].defined()) x = make(p.s, p.s.sizes(), p.branch);
      if (want) stats = make(p.s, {p.d.rows, 4}, at::kFloat);
    }
    return answer(entry.norm(&p.d, &p.in, at_of(r), at_of(x), static_cast<float*>(at_of(stats)), a.stream(p.dev)), r, x, stats);
  });
}
// ..., stats, d_r, d_x, given, gradients of s, u, gate and the parameters (8), workspace, stream -> gradients (8)
PyObject* norm_backward(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{argv, n};
    Norm p = norm_args(a);
    const Tensor& stats = a.tensor();
    Tensor d_r = a.optional(), d_x = a.optional();
    need(fits(stats, at::kFloat, {p.d.rows, 4}, p.dev), "stats: need a contiguous float32 tensor [rows, 4]");
    need(!d_r.defined() || fits(d_r, p.s.scalar_type(), p.s.sizes(), p.dev), "d_r: need a contiguous tensor like s");
    need(!d_x.defined() || fits(d_x, p.branch, p.s.sizes(), p.dev), "d_x: need a contiguous tensor of the shape of s and the branch's type");
    const bool given = a.integer() != 0;
    const Tensor* of[8] = {&p.s, &p.u, &p.gate, &p.par[0], &p.par[1], &p.par[2], &p.par[3], &p.par[4]};
    Tensor g[8];
    c10::cuda::CUDAGuard on((c10::DeviceIndex)p.dev);
    for (int i = 0; i < 8; ++i) {
      g[i] = a.optional();
      if (given) {
        need(!g[i].defined() || (of[i]->defined() && fits(g[i], of[i]->scalar_type(), of[i]->sizes(), p.dev)),
             "gradients: need contiguous tensors like the inputs that were given");
      } else if (of[i]->defined()) {
        g[i] = make(p.s, of[i]->sizes(), of[i]->scalar_type());
      }
    }
    Tensor ws = a.optional();
    size_t size = 0;
    if (!ws.defined()) {
      const fipa_status st = entry.norm_size(&p.d, &size);
      if (st != FIPA_OK) return PyLong_FromLong(st);
    }
    ws = room(ws, p.s, size, p.dev);
    auto f = [&](int i) { return static_cast<float*>(at_of(g[i])); };
    const fipa_norm_grads gr{at_of(g[0]), at_of(g[1]), at_of(g[2]), f(3), f(4), f(5), f(6), f(7)};
    return answer(entry.norm_backward(&p.d, &p.in, static_cast<const float*>(stats.data_ptr()), at_of(d_r), at_of(d_x), &gr, ws.data_ptr(),
                                      ws.nbytes(), a.stream(p.dev)),
                  g[0], g[1], g[2], g[3], g[4], g[5], g[6], g[7]);
  });
}

// ---------------------------------------------------------------- embedding
// idx, table, scale, out, stream -> out
PyObject* embedding(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{argv, n};
    const Tensor &idx = a.tensor(), &table = a.tensor();
    need(table.is_cuda() && table.dim() == 2 && floats(table) && table.is_contiguous(), "table: need a contiguous float32 or bfloat16 CUDA tensor [V, C]");
    const int dev = (int)table.get_device();
    need(fits(idx, at::kInt, idx.sizes(), dev), "idx: need a contiguous int32 tensor on the table's device");
    const double scale = a.real();
    Tensor out = a.optional();
    at::DimVector shape(idx.sizes().begin(), idx.sizes().end());
    shape.push_back(table.size(1));
    c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
    if (out.defined()) need(fits(out, table.scalar_type(), shape, dev), "out: need a contiguous tensor [..., C] of the table's type");
    else out = make(table, shape, table.scalar_type());
    return answer(entry.embedding(code(table.scalar_type()), static_cast<const int32_t*>(idx.data_ptr()), table.data_ptr(), idx.numel(),
                                  size32(table.size(0)), size32(table.size(1)), scale, out.data_ptr(), a.stream(dev)),
                  out);
  });
}
// idx, d_out, V, scale, gradient, workspace, stream -> gradient
PyObject* embedding_backward(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{argv, n};
    const Tensor &idx = a.tensor(), &d = a.tensor();
    need(d.is_cuda() && d.dim() > 0 && floats(d) && d.is_contiguous(), "d_out: need a contiguous float32 or bfloat16 CUDA tensor [..., C]");
    const int dev = (int)d.get_device();
    need(fits(idx, at::kInt, d.sizes().slice(0, d.dim() - 1), dev), "idx: need a contiguous int32 tensor of the leading shape of d_out on its device");
    const int64_t V = a.integer(), C = d.size(-1);
    const double scale = a.real();
    Tensor g = a.optional(), ws = a.optional();
    size_t size = 0;
    const fipa_status st = entry.embedding_size(idx.numel(), size32(V), size32(C), &size);
    if (st != FIPA_OK) return PyLong_FromLong(st);
    c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
    if (g.defined()) need(fits(g, at::kFloat, {V, C}, dev), "table: need a contiguous float32 tensor [V, C]");
    else g = make(d, {V, C}, at::kFloat);
    ws = room(ws, d, size, dev);
    return answer(entry.embedding_backward(code(d.scalar_type()), static_cast<const int32_t*>(idx.data_ptr()), d.data_ptr(), idx.numel(), (int)V,
                                           (int)C, scale, static_cast<float*>(g.data_ptr()), ws.data_ptr(), ws.nbytes(), a.stream(dev)),
                  g);
  });
}

// bind(name -> address of the entry points)
PyObject* bind(PyObject*, PyObject* dict) {
  auto get = [&](const char* name) -> void* {
    PyObject* o = PyDict_GetItemString(dict, name);
    void* p = o == nullptr ? nullptr : PyLong_AsVoidPtr(o);
    if (p == nullptr && !PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "no address of %s", name);
    return p;
  };
#define FIPA_BIND(field, name)                                          \
  if ((entry.field = reinterpret_cast<decltype(entry.field)>(get(#name))) == nullptr) return nullptr;
  FIPA_BIND(window, fipa_window_attention)
  FIPA_BIND(window_size, fipa_window_attention_workspace_size)
  FIPA_BIND(window_backward, fipa_window_attention_backward)
  FIPA_BIND(window_backward_size, fipa_window_attention_backward_workspace_size)
  FIPA_BIND(norm, fipa_norm_residual)
  FIPA_BIND(norm_size, fipa_norm_residual_backward_workspace_size)
  FIPA_BIND(norm_backward, fipa_norm_residual_backward)
  FIPA_BIND(embedding, fipa_embedding)
  FIPA_BIND(embedding_size, fipa_embedding_backward_workspace_size)
  FIPA_BIND(embedding_backward, fipa_embedding_backward)
#undef FIPA_BIND
  Py_RETURN_NONE;
}

#define FIPA_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FIPA_FAST(window), FIPA_FAST(window_backward), FIPA_FAST(norm), FIPA_FAST(norm_backward), FIPA_FAST(embedding),
                         FIPA_FAST(embedding_backward), {"bind", &bind, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
// FIPA_BUILT_FOR: the Python and PyTorch that this was compiled against, for the build to find in the file.
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", FIPA_BUILT_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
