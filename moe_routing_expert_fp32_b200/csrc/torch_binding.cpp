// torch_binding.cpp -- the Python calls of the 8-bit entry points, compiled.
//
// These calls take a few microseconds on the GPU at decode sizes; checking,
// allocating and marshalling them in Python took 11 (moe_linear_fp8) to 25
// (moe_dispatch_fp8).  Every function here checks its tensors (ValueError), makes
// the outputs and the workspace that the caller did not give, calls the C ABI
// (include/moe.h) on the current stream of the tensors' device, and returns the
// outputs, or the negative moe_status as an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "moe.h"

namespace {

struct Refusal {
  std::string text;
};

std::string text_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

constexpr auto kF8 = at::kFloat8_e4m3fn;

// The tensors of a call: all on the device of the first one named.
struct Tensors {
  int dev = -1;
  const char* first = nullptr;

  const at::Tensor& any(PyObject* o, const char* name, at::ScalarType type) {
    if (!THPVariable_Check(o)) throw Refusal{std::string(name) + " must be a tensor"};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous())
      throw Refusal{std::string(name) + " must be a contiguous CUDA " + c10::toString(type) +
                    " tensor"};
    const int d = t.get_device();
    if (!first) {
      first = name;
      dev = d;
    } else if (d != dev) {
      throw Refusal{std::string(name) + " is on cuda:" + std::to_string(d) + ", " + first +
                    " on cuda:" + std::to_string(dev)};
    }
    return t;
  }
  const at::Tensor& get(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor& t = any(o, name, type);
    if (t.sizes() != shape)
      throw Refusal{std::string(name) + " has shape " + text_of(t.sizes()) + ", expected " +
                    text_of(shape)};
    return t;
  }
  const at::Tensor& rank(PyObject* o, const char* name, at::ScalarType type, int64_t dims) {
    const at::Tensor& t = any(o, name, type);
    if (t.dim() != dims)
      throw Refusal{std::string(name) + " has " + std::to_string(t.dim()) +
                    " dimensions, expected " + std::to_string(dims)};
    return t;
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev),
                                  c10::nullopt);
  }
  // the caller's tensor, or a new one
  at::Tensor out(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    return o == Py_None ? make(shape, type) : get(o, name, type, shape);
  }
};

struct Workspace {
  at::Tensor t;
  void* p = nullptr;
  size_t bytes = 0;
};

Workspace given(Tensors& ts, PyObject* o) {
  Workspace w;
  w.t = ts.any(o, "ws", at::kByte);
  w.p = w.t.data_ptr();
  w.bytes = (size_t)w.t.numel();
  return w;
}

Workspace workspace(Tensors& ts, PyObject* o, size_t need) {
  if (o != Py_None) return given(ts, o);
  Workspace w;
  w.bytes = need < 256 ? 256 : need;
  w.t = ts.make({(int64_t)w.bytes}, at::kByte);
  w.p = w.t.data_ptr();
  return w;
}

// For calls that need only the status word: without a caller's workspace, one
// that the calls of a device share (nothing reads its status, so it does not
// matter that calls on several streams clear it).  It comes from cudaMalloc: a
// block of the caching allocator may still be in use by work queued on the stream
// that freed it, which a call on another stream does not wait for.
Workspace status_only(Tensors& ts, PyObject* o) {
  if (o != Py_None) return given(ts, o);
  constexpr int kDevices = 64;
  static void* kept[kDevices] = {};  // never freed
  if (ts.dev >= kDevices) return workspace(ts, Py_None, 256);
  if (!kept[ts.dev]) {
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)ts.dev);
    // an allocation is no part of a graph that this or another thread captures
    const c10::cuda::CUDAStreamCaptureModeGuard relaxed(cudaStreamCaptureModeRelaxed);
    if (cudaMalloc(&kept[ts.dev], 256) != cudaSuccess) {
      (void)cudaGetLastError();  // no memory outside the allocator: one of the call's own
      kept[ts.dev] = nullptr;
      return workspace(ts, Py_None, 256);
    }
  }
  Workspace w;
  w.p = kept[ts.dev];
  w.bytes = 256;
  return w;
}

// Runs call(stream) with the tensors' device current and the GIL released.
template <typename F>
int run(const Tensors& ts, F&& call) {
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)ts.dev));
  void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)ts.dev).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call(stream);
  Py_END_ALLOW_THREADS
  return rc;
}

template <typename... T>
PyObject* outputs(int rc, const T&... t) {
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  if constexpr (sizeof...(T) == 1) {
    return THPVariable_Wrap(t...);
  } else {
    PyObject* items[] = {THPVariable_Wrap(t)...};
    PyObject* r = PyTuple_New(sizeof...(T));
    for (PyObject* i : items)
      if (!i) Py_CLEAR(r);  // an exception is set: no tuple with a hole in it
    for (size_t i = 0; i < sizeof...(T); ++i) {
      if (r) PyTuple_SET_ITEM(r, i, items[i]);
      else Py_XDECREF(items[i]);
    }
    return r;
  }
}

int64_t int_of(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refusal{std::string(name) + " must be an int"};
  }
  return v;
}
int int32_of(PyObject* o, const char* name) {
  const int64_t v = int_of(o, name);
  if (v < INT32_MIN || v > INT32_MAX) throw Refusal{std::string(name) + " is out of range"};
  return (int)v;
}
// a size that the C ABI takes as int
int size32(int64_t v, const char* name) {
  if (v > INT32_MAX) throw Refusal{std::string(name) + " is out of range"};
  return (int)v;
}
float float_of(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refusal{std::string(name) + " must be a number"};
  }
  return (float)v;
}
bool flag_of(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Refusal{std::string(name) + " must be true or false"};
  }
  return v == 1;
}

int64_t c128(int64_t n) { return (n + 127) / 128; }
template <typename T = void>
T* ptr(const at::Tensor& t) { return reinterpret_cast<T*>(t.data_ptr()); }
moe_fp8* f8(const at::Tensor& t) { return ptr<moe_fp8>(t); }
moe_bf16* bf(const at::Tensor& t) { return ptr<moe_bf16>(t); }
float* f32(const at::Tensor& t) { return ptr<float>(t); }
int32_t* i32(const at::Tensor& t) { return ptr<int32_t>(t); }

// --------------------------------------------------------------- functions
// (x, block_rows, pow2, q or None, scale or None) -> (q, scale)
PyObject* quantize(PyObject* const* a) {
  Tensors ts;
  const at::Tensor& x = ts.any(a[0], "x", at::kBFloat16);
  const int rows = int32_of(a[1], "block_rows");
  const bool pow2 = flag_of(a[2], "pow2_scales");
  const int64_t n = x.dim();
  if (rows == 1 ? n < 1 : n != 2 && n != 3)
    throw Refusal{rows == 1 ? "x needs at least one dimension"
                            : "x must be [N, K] or [E, N, K] with block_rows = 128"};
  at::DimVector s_shape(x.sizes());
  const int64_t K = s_shape[n - 1];
  s_shape[n - 1] = c128(K);
  int64_t B = 1, M = 1;
  if (rows == 1) {
    for (int64_t i = 0; i + 1 < n; ++i) M *= s_shape[i];
  } else {
    M = s_shape[n - 2];
    B = n == 3 ? s_shape[0] : 1;
    s_shape[n - 2] = c128(M);
  }
  const int k = size32(K, "K");
  const at::Tensor q = ts.out(a[3], "q", kF8, x.sizes());
  const at::Tensor s = ts.out(a[4], "scale", at::kFloat, s_shape);
  const int rc = run(ts, [&](void* st) {
    return moe_quantize_fp8(bf(x), B, M, k, rows, pow2, f8(q), f32(s), st);
  });
  return outputs(rc, q, s);
}

// (topk_idx, x_e, E, pow2, ws or None) -> (counts, offsets, perm, pos, xq, x_scale)
PyObject* dispatch(PyObject* const* a) {
  Tensors ts;
  const at::Tensor& x = ts.rank(a[1], "x_e", at::kBFloat16, 2);
  const at::Tensor& idx = ts.rank(a[0], "topk_idx", at::kInt, 2);
  const int64_t N = idx.size(0), S = idx.numel();
  const int K = size32(idx.size(1), "top_k"), d = size32(x.size(1), "d_e");
  if (x.size(0) != N)
    throw Refusal{"x_e has shape " + text_of(x.sizes()) + ", expected " + text_of({N, d})};
  const int E = int32_of(a[2], "num_experts");
  const bool pow2 = flag_of(a[3], "pow2_scales");
  if (E < 1) throw Refusal{"num_experts must be positive"};
  if (E > 1024) return PyLong_FromLong(MOE_ERR_UNSUPPORTED);  // before allocating for it
  // the integers and, without a caller's workspace, the workspace share an
  // allocation
  const size_t need = a[4] == Py_None ? moe_dispatch_workspace_size(N, K, E) : 0;
  const int64_t at = (int64_t)((need + 255) / 256 * 64);
  const at::Tensor ints = ts.make({at + 2 * (int64_t)E + 1 + 2 * S}, at::kInt);
  Workspace w;
  if (a[4] == Py_None) {
    w.p = ints.data_ptr();
    w.bytes = 4 * (size_t)at;
  } else {
    w = given(ts, a[4]);
  }
  const at::AutoDispatchBelowADInplaceOrView no_autograd;
  auto part = [&](int64_t from, int64_t n) { return ints.as_strided({n}, {1}, from); };
  const at::Tensor counts = part(at, E), offsets = part(at + E, E + 1),
                   perm = part(at + 2 * (int64_t)E + 1, S),
                   pos = part(at + 2 * (int64_t)E + 1 + S, S);
  const at::Tensor xq = ts.make({S, d}, kF8), xs = ts.make({S, c128(d)}, at::kFloat);
  const int rc = run(ts, [&](void* st) {
    return moe_dispatch_fp8(i32(idx), N, K, E, bf(x), d, pow2, i32(counts), i32(offsets),
                            i32(perm), i32(pos), f8(xq), f32(xs), w.p, w.bytes, st);
  });
  return outputs(rc, counts, offsets, perm, pos, xq, xs);
}

// (xq, x_scale, w, w_scale, residual or None, out or None, ws or None) -> out
PyObject* linear(PyObject* const* a) {
  Tensors ts;
  const at::Tensor& xq = ts.rank(a[0], "xq", kF8, 2);
  const at::Tensor& w = ts.rank(a[2], "w", kF8, 2);
  const int64_t M = xq.size(0);
  const int K = size32(xq.size(1), "K"), N = size32(w.size(0), "N_out");
  if (w.size(1) != K)
    throw Refusal{"w has shape " + text_of(w.sizes()) + ", expected " + text_of({N, K})};
  const at::Tensor& xs = ts.get(a[1], "x_scale", at::kFloat, {M, c128(K)});
  const at::Tensor& ws = ts.get(a[3], "w_scale", at::kFloat, {c128(N), c128(K)});
  const moe_bf16* res =
      a[4] == Py_None ? nullptr : bf(ts.get(a[4], "residual", at::kBFloat16, {M, N}));
  const at::Tensor y = ts.out(a[5], "out", at::kBFloat16, {M, N});
  const Workspace wk = status_only(ts, a[6]);
  const int rc = run(ts, [&](void* st) {
    return moe_linear_fp8(f8(xq), f32(xs), M, K, f8(w), f32(ws), N, res, bf(y), wk.p, wk.bytes,
                          st);
  });
  return outputs(rc, y);
}

// (xq, x_scale, offsets, w, w_scale, out or None, ws or None) -> out
PyObject* grouped(PyObject* const* a) {
  Tensors ts;
  const at::Tensor& xq = ts.rank(a[0], "xq", kF8, 2);
  const at::Tensor& w = ts.rank(a[3], "w", kF8, 3);
  const int64_t S = xq.size(0);
  const int K = size32(xq.size(1), "K"), E = size32(w.size(0), "E"), N = size32(w.size(1), "N_out");
  if (w.size(2) != K)
    throw Refusal{"w has shape " + text_of(w.sizes()) + ", expected " + text_of({E, N, K})};
  const at::Tensor& xs = ts.get(a[1], "x_scale", at::kFloat, {S, c128(K)});
  const at::Tensor& off = ts.get(a[2], "offsets", at::kInt, {(int64_t)E + 1});
  const at::Tensor& ws = ts.get(a[4], "w_scale", at::kFloat, {E, c128(N), c128(K)});
  const at::Tensor y = ts.out(a[5], "out", at::kBFloat16, {S, N});
  const Workspace wk = status_only(ts, a[6]);
  const int rc = run(ts, [&](void* st) {
    return moe_grouped_linear_fp8(f8(xq), f32(xs), i32(off), E, S, K, f8(w), f32(ws), N, bf(y),
                                  wk.p, wk.bytes, st);
  });
  return outputs(rc, y);
}

// w1, w1_scale, w3, w3_scale, w2, w2_scale at a[0..5]
moe_fp8_experts experts_of(Tensors& ts, PyObject* const* a, int* E, int* F, int* d) {
  const at::Tensor& w1 = ts.rank(a[0], "w1", kF8, 3);
  const int64_t e = w1.size(0), f = w1.size(1), n = w1.size(2);
  *E = size32(e, "E");
  *F = size32(f, "F");
  *d = size32(n, "d_e");
  moe_fp8_experts x;
  x.w1 = f8(w1);
  x.w1_scale = f32(ts.get(a[1], "w1_scale", at::kFloat, {e, c128(f), c128(n)}));
  x.w3 = f8(ts.get(a[2], "w3", kF8, {e, f, n}));
  x.w3_scale = f32(ts.get(a[3], "w3_scale", at::kFloat, {e, c128(f), c128(n)}));
  x.w2 = f8(ts.get(a[4], "w2", kF8, {e, n, f}));
  x.w2_scale = f32(ts.get(a[5], "w2_scale", at::kFloat, {e, c128(n), c128(f)}));
  return x;
}

// kind, beta, linear_beta at a[0..2]
moe_act_cfg act_of(PyObject* const* a) {
  moe_act_cfg act;
  act.kind = int32_of(a[0], "kind");
  act.beta = float_of(a[1], "beta");
  act.linear_beta = float_of(a[2], "linear_beta");
  return act;
}

// (xq, x_scale, offsets, w1, w1_scale, w3, w3_scale, w2, w2_scale, kind, beta,
//  linear_beta, pow2, y or None, ws or None) -> y
PyObject* expert_ffn(PyObject* const* a) {
  Tensors ts;
  int E, F, d;
  const at::Tensor& xq = ts.rank(a[0], "xq", kF8, 2);
  const moe_fp8_experts x = experts_of(ts, a + 3, &E, &F, &d);
  const int64_t S = xq.size(0);
  if (xq.size(1) != d)
    throw Refusal{"xq has shape " + text_of(xq.sizes()) + ", expected " + text_of({S, d})};
  const at::Tensor& xs = ts.get(a[1], "x_scale", at::kFloat, {S, c128(d)});
  const at::Tensor& off = ts.get(a[2], "offsets", at::kInt, {(int64_t)E + 1});
  const moe_act_cfg act = act_of(a + 9);
  const bool pow2 = flag_of(a[12], "pow2_scales");
  const at::Tensor y = ts.out(a[13], "y", at::kBFloat16, {S, d});
  const Workspace wk =
      workspace(ts, a[14], a[14] == Py_None ? moe_expert_ffn_fp8_workspace_size(S, d, E, F) : 0);
  const int rc = run(ts, [&](void* st) {
    return moe_expert_ffn_fp8(f8(xq), f32(xs), i32(off), E, S, d, F, &x, &act, pow2, bf(y), wk.p,
                              wk.bytes, st);
  });
  return outputs(rc, y);
}

// (x_r, W, bias or None, route (8 numbers), w1 .. w2_scale, kind, beta, linear_beta,
//  x_e or None, pow2, ws, out, topk_idx, topk_w (None or tensors)) -> out
PyObject* forward(PyObject* const* a) {
  Tensors ts;
  const at::Tensor& x = ts.rank(a[0], "x_r", at::kBFloat16, 2);
  const int64_t N = x.size(0);
  const int d_r = size32(x.size(1), "d_r");
  moe_route_cfg c;
  PyObject* const* r = a + 3;
  c.num_experts = int32_of(r[0], "num_experts");
  c.n_group = int32_of(r[1], "n_group");
  c.topk_group = int32_of(r[2], "topk_group");
  c.top_k = int32_of(r[3], "top_k");
  c.norm_topk_prob = flag_of(r[4], "norm_topk_prob");
  c.route_scale = float_of(r[5], "route_scale");
  c.score_func = int32_of(r[6], "score_func");
  c.group_score = int32_of(r[7], "group_score");
  a += 11;
  int E, F, d;
  const moe_fp8_experts w = experts_of(ts, a, &E, &F, &d);
  if (E != c.num_experts) throw Refusal{"w1 does not hold num_experts experts"};
  const at::Tensor& W = ts.get(r[-2], "W", at::kFloat, {E, d_r});
  const float* bias = r[-1] == Py_None ? nullptr : f32(ts.get(r[-1], "bias", at::kFloat, {E}));
  const moe_act_cfg act = act_of(a + 6);
  if (a[9] == Py_None && d != d_r)
    throw Refusal{"x_e is required when the experts' width differs from the router's"};
  const moe_bf16* x_e =
      a[9] == Py_None ? nullptr : bf(ts.get(a[9], "x_e", at::kBFloat16, {N, d}));
  const bool pow2 = flag_of(a[10], "pow2_scales");
  const Workspace wk = workspace(
      ts, a[11], a[11] == Py_None ? moe_forward_fp8_workspace_size(N, d_r, d, &c, F) : 0);
  const at::Tensor out = ts.out(a[12], "out", at::kBFloat16, {N, d});
  int32_t* idx =
      a[13] == Py_None ? nullptr : i32(ts.get(a[13], "topk_idx", at::kInt, {N, c.top_k}));
  float* tw = a[14] == Py_None ? nullptr : f32(ts.get(a[14], "topk_w", at::kFloat, {N, c.top_k}));
  const int rc = run(ts, [&](void* st) {
    return moe_forward_fp8(bf(x), x_e, N, d_r, d, f32(W), bias, &c, &w, F, &act, pow2, bf(out),
                           idx, tw, wk.p, wk.bytes, st);
  });
  return outputs(rc, out);
}

template <PyObject* (*FN)(PyObject* const*), int NARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != NARGS) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments", NARGS);
    return nullptr;
  }
  try {
    return FN(args);
  } catch (const Refusal& r) {
    PyErr_SetString(PyExc_ValueError, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*FN)(PyObject* const*), int NARGS>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)(void))entry<FN, NARGS>, METH_FASTCALL, nullptr};
}

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding(void) {
  static PyMethodDef methods[] = {
      method<quantize, 5>("quantize_fp8"),    method<dispatch, 5>("dispatch_fp8"),
      method<linear, 7>("linear_fp8"),        method<grouped, 7>("grouped_linear_fp8"),
      method<expert_ffn, 15>("expert_ffn_fp8"), method<forward, 26>("forward_fp8"),
      {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods};
  return PyModule_Create(&def);
}
