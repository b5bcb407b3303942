// calls.cpp -- the Python side of moe_route, w4a16_moe, token_logprobs and
// token_logprobs_backward as a CPython module: metadata checks, allocation of
// results and workspaces, the current stream, and the C ABI call.
//
// These kernels take 3 to 30 us at decode sizes, less than ctypes, the checks
// in Python and torch.empty took around them (11 us for the router of one
// token, 20 us for token_logprobs, 24 us for w4a16_moe).  No computation
// happens here; every call ends in the C ABI of include/nvfp4_lm_head.h.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <utility>

#include "../../include/nvfp4_lm_head.h"

namespace {

struct ValueError : std::runtime_error {
  using std::runtime_error::runtime_error;
};

// A Python exception is already set.
struct PyFailure {};

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw ValueError(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// On the GPU of `first`, the call's first tensor.
void check_device(const at::Tensor& t, const char* name, const at::Tensor& first) {
  if (!t.is_cuda()) throw ValueError(std::string(name) + " must be a CUDA tensor");
  if (t.device() != first.device())
    throw ValueError(std::string(name) + " is on " + t.device().str() + ", not on " +
                     first.device().str());
}

void check(const at::Tensor& t, at::ScalarType dtype, const char* name,
           std::initializer_list<int64_t> shape, const at::Tensor& first) {
  check_device(t, name, first);
  if (t.scalar_type() != dtype)
    throw ValueError(std::string(name) + " must be " + c10::toString(dtype) + ", got " +
                     c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) throw ValueError(std::string(name) + " must be contiguous");
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want)
    throw ValueError(std::string(name) + " must have shape " + shape_text(want) + ", got " +
                     shape_text(t.sizes()));
}

// The tensor of `o`, checked; none where it is None.
at::Tensor optional(PyObject* o, at::ScalarType dtype, const char* name,
                    std::initializer_list<int64_t> shape, const at::Tensor& first) {
  if (o == Py_None) return {};
  const at::Tensor& t = tensor(o, name);
  check(t, dtype, name, shape, first);
  return t;
}

// The results of one call, cut from one allocation at 256-byte steps: the six
// of token_logprobs, allocated one by one, took the host 10.5 us a call, more
// than the kernel takes for one row; this way a call is 5 us.
class Results {
 public:
  at::Tensor* add(at::ScalarType dtype, std::initializer_list<int64_t> shape) {
    Part& p = parts_[n_++];
    int64_t bytes = (int64_t)c10::elementSize(dtype);
    p.dtype = dtype;
    p.dims = 0;
    for (const int64_t d : shape) {
      p.shape[p.dims++] = d;
      bytes *= d;
    }
    p.at = total_;
    total_ += (bytes + 255) / 256 * 256;
    return &p.t;
  }
  void allocate(const at::Tensor& like) {
    const at::Tensor base = at::empty({total_}, like.options().dtype(at::kByte));
    for (int i = 0; i < n_; ++i) {
      Part& p = parts_[i];
      p.t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()),
                                                     c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                     c10::scalarTypeToTypeMeta(p.dtype));
      p.t.unsafeGetTensorImpl()->set_storage_offset(p.at / (int64_t)c10::elementSize(p.dtype));
      p.t.unsafeGetTensorImpl()->set_sizes_contiguous({p.shape, (size_t)p.dims});
    }
  }

 private:
  struct Part {
    at::ScalarType dtype;
    int64_t shape[2], at;
    int dims;
    at::Tensor t;
  };
  Part parts_[6];
  int n_ = 0;
  int64_t total_ = 0;
};

const void* optional_f32(PyObject* o, const char* name, int64_t n, const at::Tensor& first) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  check(t, at::kFloat, name, {n}, first);
  return t.data_ptr();
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyFailure();
  return v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyFailure();
  return (float)v;
}

// A torch stream or an integer handle.
void* stream_of(PyObject* o) {
  PyObject* h = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream")
                                                         : PyNumber_Long(o);
  if (!h) throw PyFailure();
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!s && PyErr_Occurred()) throw PyFailure();
  return s;
}

// The stream of a call: `given`, or the current one.  While this lives, memory
// is allocated in the order of that stream, so that a block whose last use is
// still queued on another stream is not given out to the call's kernels.
class OnStream {
 public:
  OnStream(PyObject* given, const at::Tensor& like)
      : caller_(c10::cuda::getCurrentCUDAStream()), handle_(caller_.stream()) {
    // the kernels run on the current device, whose streams these are
    if (like.device() != caller_.device())
      throw ValueError("the tensors are on " + like.device().str() + ", the current device is " +
                       caller_.device().str());
    if (given == Py_None) return;
    handle_ = static_cast<cudaStream_t>(stream_of(given));
    if (handle_ != caller_.stream())
      guard_.reset_stream(c10::cuda::getStreamFromExternal(handle_, like.get_device()));
  }
  void* handle() const { return handle_; }
  // A result allocated here: the caller's stream uses it next.
  void result(const at::Tensor& t) const {
    if (handle_ != caller_.stream()) t.record_stream(caller_.unwrap());
  }

 private:
  const c10::cuda::CUDAStream caller_;
  cudaStream_t handle_;
  c10::cuda::OptionalCUDAStreamGuard guard_;
};

// The package's own exception for a status that is not NVFP4_OK.
void done(nvfp4_status st, const char* where) {
  if (st == NVFP4_OK) return;
  PyObject* pkg = PyImport_ImportModule("nvfp4_weight_only_rows_gb300");
  if (pkg) {
    PyObject* r = PyObject_CallMethod(pkg, "_check", "is", (int)st, where);
    Py_XDECREF(r);
    Py_DECREF(pkg);
  }
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
  throw PyFailure();
}

int dtype_code(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kFloat) return NVFP4_OUT_F32;
  if (t.scalar_type() == at::kBFloat16) return NVFP4_OUT_BF16;
  throw ValueError(what);
}

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* t = PyTuple_New((Py_ssize_t)ts.size());
  if (!t) throw PyFailure();
  Py_ssize_t i = 0;
  for (const at::Tensor& x : ts) {
    PyObject* o = THPVariable_Wrap(x);
    if (!o) {
      Py_DECREF(t);
      throw PyFailure();
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// The exception class torch raises where its allocator has no memory left.
void set_out_of_memory(const char* what) {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
  if (type) PyErr_SetString(type, what);
  Py_XDECREF(type);
  Py_XDECREF(torch);
}

// k as results are allocated for it: one out of range is refused by the C ABI
// call, not by an allocation of its size.
int64_t within(int64_t k, int64_t n, int64_t most) {
  return std::max<int64_t>(0, std::min(k, std::min(n, most)));
}

template <int64_t kArgs, typename F>
PyObject* guarded(Py_ssize_t n, F f) {
  try {
    if (n != kArgs) {
      PyErr_Format(PyExc_TypeError, "expected %lld arguments, got %zd", (long long)kArgs, n);
      return nullptr;
    }
    return f();
  } catch (const PyFailure&) {
  } catch (const ValueError& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    set_out_of_memory(e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// router_logits, k, renormalize, scoring code, bias, scale, expert_ids, weights, stream
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<9>(n, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "router_logits");
    const int code = dtype_code(x, "router_logits must be float32 or bfloat16 [M, E]");
    if (x.dim() != 2) throw ValueError("router_logits must be float32 or bfloat16 [M, E]");
    const int64_t M = x.size(0), E = x.size(1), k = integer(a[1]), kk = std::max<int64_t>(k, 0);
    const int64_t fit = within(k, E, NVFP4_ROUTE_MAX_K);
    check(x, x.scalar_type(), "router_logits", {M, E}, x);
    const void* bias = optional_f32(a[4], "bias", E, x);
    at::Tensor ids = optional(a[6], at::kInt, "expert_ids", {M, kk}, x);
    at::Tensor w = optional(a[7], at::kFloat, "weights", {M, kk}, x);
    const OnStream on(a[8], x);
    if (!ids.defined() && !w.defined()) {
      Results r;
      at::Tensor &ri = *r.add(at::kInt, {M, fit}), &rw = *r.add(at::kFloat, {M, fit});
      r.allocate(x);
      ids = std::move(ri);
      w = std::move(rw);
    } else {
      if (!ids.defined()) ids = at::empty({M, fit}, x.options().dtype(at::kInt));
      if (!w.defined()) w = at::empty({M, fit}, x.options().dtype(at::kFloat));
    }
    done(moe_route(x.data_ptr(), code, M, E, k, (int)integer(a[3]), (int)integer(a[2]),
                   static_cast<const float*>(bias), number(a[5]),
                   static_cast<int32_t*>(ids.data_ptr()), static_cast<float*>(w.data_ptr()),
                   on.handle()),
         "moe_route");
    if (a[6] == Py_None) on.result(ids);
    if (a[7] == Py_None) on.result(w);
    return tuple({ids, w});
  });
}

// x, expert_ids, weights, w13 (3), w2 (3), out, bf16 out (if out is None), workspace, stream
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<13>(n, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &ids = tensor(a[1], "expert_ids");
    const at::Tensor &w = tensor(a[2], "weights"), &p13 = tensor(a[3], "w13_packed");
    const at::Tensor &s13 = tensor(a[4], "w13_scales"), &g13 = tensor(a[5], "w13_global");
    const at::Tensor &p2 = tensor(a[6], "w2_packed"), &s2 = tensor(a[7], "w2_scales");
    const at::Tensor& g2 = tensor(a[8], "w2_global");
    if (x.dim() != 2) throw ValueError("x must be 2-D [M, H]");
    if (ids.dim() != 2) throw ValueError("expert_ids must be 2-D [M, k]");
    if (p2.dim() != 3) throw ValueError("w2_packed must be 3-D [E, H, I/2]");
    const int64_t M = x.size(0), H = x.size(1), k = ids.size(1), E = p2.size(0), I = p2.size(2) * 2;
    check(x, at::kBFloat16, "x", {M, H}, x);
    check(ids, at::kInt, "expert_ids", {M, k}, x);
    check(w, at::kFloat, "weights", {M, k}, x);
    if (s13.element_size() != 1 || s2.element_size() != 1)
      throw ValueError("scales must be float8_e4m3fn (or uint8 bit patterns)");
    check(p13, at::kByte, "w13_packed", {E, 2 * I, H / 2}, x);
    check(s13, s13.scalar_type(), "w13_scales", {E, 2 * I, H / 16}, x);
    check(g13, at::kFloat, "w13_global", {E}, x);
    check(p2, at::kByte, "w2_packed", {E, H, I / 2}, x);
    check(s2, s2.scalar_type(), "w2_scales", {E, H, I / 16}, x);
    check(g2, at::kFloat, "w2_global", {E}, x);
    at::ScalarType dt = integer(a[10]) ? at::kBFloat16 : at::kFloat;
    if (a[9] != Py_None) dt = tensor(a[9], "out").scalar_type();
    at::Tensor out = optional(a[9], dt, "out", {M, H}, x), ws;
    if (a[11] != Py_None) {
      ws = tensor(a[11], "workspace");
      check_device(ws, "workspace", x);
      // (an expanded or strided view has more elements than bytes of its own)
      if (!ws.is_contiguous()) throw ValueError("workspace must be contiguous");
    }
    const OnStream on(a[12], x);
    if (!out.defined()) out = at::empty({M, H}, x.options().dtype(dt));
    const int code = dtype_code(out, "out must be float32 or bfloat16");
    if (!ws.defined())
      ws = at::empty({std::max<int64_t>((int64_t)w4a16_moe_workspace_bytes(M, k, H, I), 256)},
                     x.options().dtype(at::kByte));
    using u8 = const uint8_t*;
    using f32 = const float*;
    done(w4a16_moe(x.data_ptr(), M, k, H, I, E, static_cast<const int32_t*>(ids.data_ptr()),
                   f32(w.data_ptr()), u8(p13.data_ptr()), u8(s13.data_ptr()), f32(g13.data_ptr()),
                   u8(p2.data_ptr()), u8(s2.data_ptr()), f32(g2.data_ptr()), out.data_ptr(), code,
                   ws.data_ptr(), (size_t)ws.numel() * ws.element_size(), on.handle()),
         "w4a16_moe");
    if (a[9] == Py_None) on.result(out);
    return THPVariable_Wrap(out);
  });
}

struct Logits {
  int code;
  int64_t M, N, ld;
};

Logits logits_args(const at::Tensor& x, const at::Tensor& tokens) {
  const char* what = "logits must be a float32 or bfloat16 CUDA tensor [M, N]";
  const int code = dtype_code(x, what);
  if (x.dim() != 2 || !x.is_cuda()) throw ValueError(what);
  const int64_t M = x.size(0), N = x.size(1), ld = M > 1 ? x.stride(0) : N;
  if (N > 1 && x.stride(1) != 1) throw ValueError("the logits of a row must be contiguous");
  if (ld < N) throw ValueError("the rows of logits overlap");
  check(tokens, at::kLong, "token_ids", {M}, x);
  return {code, M, N, ld};
}

// logits, token_ids, k, inv_temperature, stream
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<5>(n, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "logits"), &tok = tensor(a[1], "token_ids");
    const Logits l = logits_args(x, tok);
    const int64_t k = integer(a[2]), kk = within(k, l.N, NVFP4_TOPK_MAX);
    const OnStream on(a[4], x);
    Results r;
    at::Tensor &ranks = *r.add(at::kLong, {l.M}), &ids = *r.add(at::kLong, {l.M, kk});
    at::Tensor &lp = *r.add(at::kFloat, {l.M}), &ent = *r.add(at::kFloat, {l.M});
    at::Tensor &lse = *r.add(at::kFloat, {l.M}), &top = *r.add(at::kFloat, {l.M, kk});
    r.allocate(x);
    auto pf = [](const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); };
    auto pi = [](const at::Tensor& t) { return static_cast<int64_t*>(t.data_ptr()); };
    done(token_logprobs(x.data_ptr(), l.code, l.M, l.N, l.ld, pi(tok), number(a[3]), k, pf(lp),
                        pf(ent), pf(lse), pi(ranks), pi(ids), pf(top), on.handle()),
         "token_logprobs");
    on.result(lp);  // all six: one allocation
    return tuple({lp, ent, lse, ranks, ids, top});
  });
}

// logits, token_ids, lse, entropy, grad_logprobs, grad_entropy, inv_temperature, out, stream
PyObject* logprobs_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<9>(n, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "logits"), &tok = tensor(a[1], "token_ids");
    const Logits l = logits_args(x, tok);
    const at::Tensor &lse = tensor(a[2], "lse"), &g = tensor(a[4], "grad_logprobs");
    check(lse, at::kFloat, "lse", {l.M}, x);
    check(g, at::kFloat, "grad_logprobs", {l.M}, x);
    const void* ent = optional_f32(a[3], "entropy", l.M, x);
    const void* ge = optional_f32(a[5], "grad_entropy", l.M, x);
    if (a[5] != Py_None && a[3] == Py_None) throw ValueError("grad_entropy needs the forward's entropy");
    at::Tensor out;
    if (a[7] != Py_None) {
      out = tensor(a[7], "out");
      check_device(out, "out", x);
      if (out.scalar_type() != x.scalar_type() || out.sizes() != x.sizes() ||
          (l.N > 1 && out.stride(1) != 1))
        throw ValueError("out must be a CUDA tensor of the logits' shape and dtype, rows contiguous");
    }
    const OnStream on(a[8], x);
    if (!out.defined()) out = at::empty({l.M, l.N}, x.options());
    using f32 = const float*;
    done(token_logprobs_backward(x.data_ptr(), l.code, l.M, l.N, l.ld,
                                 static_cast<const int64_t*>(tok.data_ptr()), number(a[6]),
                                 f32(lse.data_ptr()), f32(ent), f32(g.data_ptr()), f32(ge),
                                 out.data_ptr(), l.M > 1 ? out.stride(0) : l.N, on.handle()),
         "token_logprobs_backward");
    if (a[7] == Py_None) on.result(out);
    return THPVariable_Wrap(out);
  });
}

PyMethodDef kMethods[] = {
    {"moe_route", (PyCFunction)(void (*)())route, METH_FASTCALL, nullptr},
    {"w4a16_moe", (PyCFunction)(void (*)())moe, METH_FASTCALL, nullptr},
    {"token_logprobs", (PyCFunction)(void (*)())logprobs, METH_FASTCALL, nullptr},
    {"token_logprobs_backward", (PyCFunction)(void (*)())logprobs_backward, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
