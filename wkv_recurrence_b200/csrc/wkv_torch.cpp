// The calling path of the gated recurrence and the RMS norm from Python: one
// native call checks the tensors, allocates the results, finds the stream and
// the workspace and calls libwkv.so's entry point (through the addresses that
// the package hands over, so that it is the library the package loaded). A
// decode step launches a kernel of a few microseconds; the same work in Python
// took 17 us per call.
//
// Host code only. Errors are Python exceptions; no C++ exception leaves a
// function here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAException.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <map>
#include <mutex>
#include <string>

#include "../../include/wkv.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {  // becomes a Python exception
  PyObject* type;
  std::string text;
};
struct Raised {};  // a Python exception is set

[[noreturn]] void bad_value(const std::string& t) { throw Refused{PyExc_ValueError, t}; }
[[noreturn]] void bad_type(const std::string& t) { throw Refused{PyExc_TypeError, t}; }

std::string name_of(ScalarType t) {
  if (t == at::kFloat) return "torch.float32";
  if (t == at::kBFloat16) return "torch.bfloat16";
  return std::string("torch.") + c10::toString(t);
}
std::string list_of(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

// ---------------------------------------------------------------------------
// the library
// ---------------------------------------------------------------------------
struct Library {
  decltype(&wkv_gated_workspace_size) gated_workspace_size;
  decltype(&wkv_gated_forward) gated_forward;
  decltype(&wkv_gated_backward) gated_backward;
  decltype(&wkv_gated_step) gated_step;
  decltype(&wkv_rms_norm) rms_norm;
  decltype(&wkv_rms_norm_quant) rms_norm_quant;
  decltype(&wkv_rms_norm_backward_workspace_size) norm_workspace_size;
  decltype(&wkv_rms_norm_backward) rms_norm_backward;
  PyObject* check;  // check(status, name) raises for a status that is not 0
  PyObject* out_of_memory;  // torch's exception
} lib;

// Runs `call(stream)` on the current stream of `dev`, with `dev` current and
// the interpreter released.
template <typename F>
void on_stream(c10::Device dev, const char* where, F call) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != dev.index()) guard.set_device(dev);
  void* st = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  wkv_status code;
  Py_BEGIN_ALLOW_THREADS;
  code = call(st);
  Py_END_ALLOW_THREADS;
  if (code != WKV_OK) {
    PyObject* r = PyObject_CallFunction(lib.check, "is", (int)code, where);
    if (r) {
      Py_DECREF(r);
      throw Refused{PyExc_RuntimeError, where};
    }
    throw Raised{};
  }
}

// ---------------------------------------------------------------------------
// arguments
// ---------------------------------------------------------------------------
const Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad_value(std::string(name) + " must be a CUDA tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) bad_value(std::string(name) + " must be a CUDA tensor");
  return t;
}
// float32 or bfloat16, as the library numbers them
wkv_dtype value_type(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return WKV_F32;
  if (t.scalar_type() == at::kBFloat16) return WKV_BF16;
  bad_type(std::string(name) + ": dtype " + name_of(t.scalar_type()) + " is not supported (float32 or bfloat16)");
}
void same_device(const Tensor& t, const char* name, c10::Device dev) {
  if (t.device() != dev)
    bad_value(std::string(name) + " must be on " + dev.str() + ", the device of the other arguments");
}
// A contiguous tensor of this device, type and shape.
const Tensor& exact(PyObject* o, const char* name, c10::Device dev, at::IntArrayRef shape, ScalarType type) {
  const Tensor& t = cuda_tensor(o, name);
  same_device(t, name, dev);
  if (t.scalar_type() != type) bad_type(std::string(name) + " must be " + name_of(type));
  if (t.sizes() != shape) bad_value(std::string(name) + " must be " + list_of(shape));
  if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
  return t;
}
// From torch's allocator without its dispatcher (a third of the call's time
// would go into finding that a CUDA tensor is wanted).
Tensor fresh(c10::Device dev, at::IntArrayRef shape, ScalarType type) {
  return Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}
// The tensor passed, checked, or a new one.
Tensor result(PyObject* o, const char* name, c10::Device dev, at::IntArrayRef shape, ScalarType type) {
  return o == Py_None ? fresh(dev, shape, type) : exact(o, name, dev, shape, type);
}
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
Tensor optional(PyObject* o, const char* name, c10::Device dev, at::IntArrayRef shape, ScalarType type) {
  return o == Py_None ? Tensor() : exact(o, name, dev, shape, type);
}
// Tells autograd that a tensor of the caller's was written (which torch's own
// in-place operators do): a backward that saved it before raises. Inference
// tensors have no version.
void written(PyObject* given, const Tensor& t) {
  if (given != Py_None && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
// The output's type: asked for, or that of `out`, or the input's.
ScalarType out_type(PyObject* dtype, PyObject* out, const Tensor& x, wkv_dtype* code) {
  ScalarType t = x.scalar_type();
  if (dtype != Py_None) {
    if (!THPDtype_Check(dtype)) bad_type("out_dtype must be a torch.dtype");
    t = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  } else if (out != Py_None && THPVariable_Check(out)) {
    t = THPVariable_Unpack(out).scalar_type();
  }
  if ((t != at::kFloat && t != at::kBFloat16) || (x.scalar_type() == at::kFloat && t != at::kFloat))
    bad_type("output dtype " + name_of(t) + " is not supported for " + name_of(x.scalar_type()) + " inputs");
  *code = t == at::kFloat ? WKV_F32 : WKV_BF16;
  return t;
}
bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw Raised{};
  return r != 0;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
void workspace_of_caller(const Tensor& t, c10::Device dev) {
  same_device(t, "workspace", dev);
  if (!t.is_contiguous()) bad_value("workspace must be contiguous");
}

// ---------------------------------------------------------------------------
// the gated recurrence
// ---------------------------------------------------------------------------
struct Gated {
  const Tensor& x;
  const Tensor& z;
  wkv_dtype xt, zt;
  wkv_gate gate;
  c10::Device dev;
};

Gated gated_inputs(PyObject* ox, PyObject* oz, PyObject* ogate, int64_t dims, const char* what) {
  const Tensor& x = cuda_tensor(ox, "x");
  const Tensor& z = cuda_tensor(oz, "z");
  const wkv_dtype xt = value_type(x, "x"), zt = value_type(z, "z");
  if (x.dim() != dims || x.sizes() != z.sizes()) bad_value(std::string("x and z must both be ") + what);
  if (x.device() != z.device()) bad_value("x and z must be on one device");
  if (x.size(-1) > 1 && (x.stride(-1) != 1 || z.stride(-1) != 1))
    bad_value("the channel axis of x and z must be contiguous");
  if (zt != xt && zt != WKV_F32) bad_type("z must be float32 or of x's dtype");
  const char* g = PyUnicode_Check(ogate) ? PyUnicode_AsUTF8(ogate) : nullptr;
  if (!g) PyErr_Clear();
  wkv_gate gate = WKV_GATE_SIGMOID;
  if (g && std::string(g) == "decay") {
    gate = WKV_GATE_DECAY;
  } else if (!g || std::string(g) != "sigmoid") {
    bad_value("gate must be \"sigmoid\" or \"decay\"");
  }
  return Gated{x, z, xt, zt, gate, x.device()};
}

// The zero-filled workspaces that are kept, by device and stream.
struct Kept {
  std::mutex mu;
  std::map<std::pair<int, void*>, Tensor> by_stream;
};
Kept& kept() {
  static Kept* k = new Kept;  // never freed: the runtime may be gone at exit
  return *k;
}
std::pair<int, void*> kept_key(c10::Device dev) {
  return {dev.index(), c10::cuda::getCurrentCUDAStream(dev.index()).stream()};
}

// Zero bytes, by no operator of torch's: under its modes and transforms these
// may return other than plain tensors, and a workspace is kept for later calls.
Tensor zeros(c10::Device dev, int64_t bytes, cudaStream_t st) {
  const Tensor t = fresh(dev, {bytes}, at::kByte);
  C10_CUDA_CHECK(cudaMemsetAsync(t.data_ptr(), 0, (size_t)bytes, st));
  return t;
}

// The workspace of this device and stream. A call that is being captured gets
// one of its own, from the graph's memory: graphs captured on one stream may be
// replayed on several at once.
Tensor gated_workspace(c10::Device dev, int64_t bytes) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != dev.index()) guard.set_device(dev);
  cudaStream_t st = c10::cuda::getCurrentCUDAStream(dev.index());
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) return zeros(dev, bytes, st);
  Kept& k = kept();
  std::lock_guard<std::mutex> lk(k.mu);
  Tensor& t = k.by_stream[{dev.index(), st}];
  if (!t.defined() || t.numel() < bytes) {
    const Tensor more = zeros(dev, std::max<int64_t>(bytes, 1 << 20), st);
    if (t.defined())  // the status is carried on: a workspace of one tile is its header
      C10_CUDA_CHECK(cudaMemcpyAsync(more.data_ptr(), t.data_ptr(), lib.gated_workspace_size(1, 1, 1),
                                     cudaMemcpyDeviceToDevice, st));
    t = more;
  }
  return t;
}

// (device index): the workspace kept for that device's current stream, or None
PyObject* gated_kept_workspace(PyObject* const* a) {
  Tensor t;
  {
    Kept& k = kept();
    std::lock_guard<std::mutex> lk(k.mu);
    const auto at = k.by_stream.find(kept_key(c10::Device(c10::kCUDA, (c10::DeviceIndex)integer(a[0]))));
    if (at != k.by_stream.end()) t = at->second;
  }
  return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
}

Tensor gated_scratch(PyObject* o, int64_t B, int64_t T, int64_t C, c10::Device dev) {
  if (o != Py_None) {
    const Tensor& t = cuda_tensor(o, "workspace");
    workspace_of_caller(t, dev);
    return t;
  }
  if (T <= WKV_GATED_TILE) return Tensor();  // one tile: the library uses none
  const size_t need = lib.gated_workspace_size(B, T, C);
  if (need == 0) bad_value("invalid sizes");
  return gated_workspace(dev, (int64_t)need);
}
size_t bytes_of(const Tensor& t) { return t.defined() ? (size_t)t.nbytes() : 0; }

int64_t tiles_of(int64_t T) { return (T + WKV_GATED_TILE - 1) / WKV_GATED_TILE; }

// A tuple of them, None for those that are not there.
PyObject* tuple_of(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      throw Raised{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// (x)
PyObject* gated_checkpoints(PyObject* const* a) {
  const Tensor& x = cuda_tensor(a[0], "x");
  if (x.dim() != 3) bad_value("x must be [B, T, C]");
  return THPVariable_Wrap(fresh(x.device(), {x.size(0), tiles_of(x.size(1)), x.size(2)}, at::kFloat));
}

// (x, z, state, gate, out_dtype, out, state_out, checkpoints, workspace)
PyObject* gated_forward(PyObject* const* a) {
  const Gated g = gated_inputs(a[0], a[1], a[3], 3, "[B, T, C]");
  const int64_t B = g.x.size(0), T = g.x.size(1), C = g.x.size(2);
  wkv_dtype ot;
  const ScalarType os = out_type(a[4], a[5], g.x, &ot);
  const Tensor state = optional(a[2], "state", g.dev, {B, C}, at::kFloat);
  const Tensor marks = optional(a[7], "checkpoints", g.dev, {B, tiles_of(T), C}, at::kFloat);
  const Tensor ws = gated_scratch(a[8], B, T, C, g.dev);
  const Tensor out = result(a[5], "out", g.dev, {B, T, C}, os);
  const Tensor state_out = result(a[6], "state_out", g.dev, {B, C}, at::kFloat);
  on_stream(g.dev, "wkv_gated_forward", [&](void* st) {
    return lib.gated_forward(B, T, C, g.x.data_ptr(), g.xt, g.x.stride(0), g.x.stride(1), g.z.data_ptr(), g.zt,
                             g.z.stride(0), g.z.stride(1), g.gate, out.data_ptr(), ot, (const float*)ptr(state),
                             (float*)state_out.data_ptr(), (float*)ptr(marks), ptr(ws), bytes_of(ws), st);
  });
  written(a[5], out);
  written(a[6], state_out);
  written(a[7], marks);
  return tuple_of({out, state_out});
}

// (x, z, gout, state, dstate, gate, checkpoints, workspace)
PyObject* gated_backward(PyObject* const* a) {
  const Gated g = gated_inputs(a[0], a[1], a[5], 3, "[B, T, C]");
  const int64_t B = g.x.size(0), T = g.x.size(1), C = g.x.size(2);
  wkv_dtype ot;
  const ScalarType os = out_type(Py_None, a[2], g.x, &ot);
  const Tensor& gout = exact(a[2], "gout", g.dev, {B, T, C}, os);
  const Tensor state = optional(a[3], "state", g.dev, {B, C}, at::kFloat);
  const Tensor dstate = optional(a[4], "dstate", g.dev, {B, C}, at::kFloat);
  Tensor marks = optional(a[6], "checkpoints", g.dev, {B, tiles_of(T), C}, at::kFloat);
  const Tensor ws = gated_scratch(a[7], B, T, C, g.dev);
  if (!marks.defined() && T > WKV_GATED_TILE) {  // the forward again, for its states alone
    marks = fresh(g.dev, {B, tiles_of(T), C}, at::kFloat);
    on_stream(g.dev, "wkv_gated_forward", [&](void* st) {
      return lib.gated_forward(B, T, C, g.x.data_ptr(), g.xt, g.x.stride(0), g.x.stride(1), g.z.data_ptr(), g.zt,
                               g.z.stride(0), g.z.stride(1), g.gate, nullptr, ot, (const float*)ptr(state), nullptr,
                               (float*)marks.data_ptr(), ptr(ws), bytes_of(ws), st);
    });
  }
  const Tensor dx = fresh(g.dev, {B, T, C}, g.x.scalar_type()), dz = fresh(g.dev, {B, T, C}, g.z.scalar_type());
  const Tensor dstate_in = fresh(g.dev, {B, C}, at::kFloat);
  on_stream(g.dev, "wkv_gated_backward", [&](void* st) {
    return lib.gated_backward(B, T, C, g.x.data_ptr(), g.xt, g.x.stride(0), g.x.stride(1), g.z.data_ptr(), g.zt,
                              g.z.stride(0), g.z.stride(1), g.gate, gout.data_ptr(), ot, (const float*)ptr(state),
                              (const float*)ptr(dstate), (const float*)ptr(marks), dx.data_ptr(), dz.data_ptr(),
                              (float*)dstate_in.data_ptr(), ptr(ws), bytes_of(ws), st);
  });
  return tuple_of({dx, dz, dstate_in});
}

// (state, x, z, gate, out_dtype, out, state_out, inplace)
PyObject* gated_step(PyObject* const* a) {
  const Gated g = gated_inputs(a[1], a[2], a[3], 2, "[S, C]");
  const int64_t S = g.x.size(0), C = g.x.size(1);
  wkv_dtype ot;
  const ScalarType os = out_type(a[4], a[5], g.x, &ot);
  const Tensor& state = exact(a[0], "state", g.dev, {S, C}, at::kFloat);
  const Tensor out = result(a[5], "out", g.dev, {S, C}, os);
  const bool inplace = truth(a[7]);
  if (inplace && a[6] != Py_None && a[6] != a[0]) bad_value("state_out must be left out (or be state) with inplace");
  PyObject* const to = inplace ? a[0] : a[6];
  const Tensor state_out = result(to, "state_out", g.dev, {S, C}, at::kFloat);
  on_stream(g.dev, "wkv_gated_step", [&](void* st) {
    return lib.gated_step(S, C, g.x.data_ptr(), g.xt, g.x.stride(0), g.z.data_ptr(), g.zt, g.z.stride(0), g.gate,
                          out.data_ptr(), ot, (const float*)state.data_ptr(), (float*)state_out.data_ptr(), st);
  });
  written(a[5], out);
  written(to, state_out);
  return tuple_of({out, state_out});
}

// ---------------------------------------------------------------------------
// the RMS norm
// ---------------------------------------------------------------------------
// [..., C] seen as rows of one stride, without a copy.
void rows_of(const Tensor& t, const char* name, int64_t* n, int64_t* stride) {
  const int64_t C = t.size(-1);
  int64_t rows = 1;
  for (int64_t i = 0; i + 1 < t.dim(); ++i) rows *= t.size(i);
  *n = rows;
  *stride = C;
  if (rows == 0 || C == 0 || t.is_contiguous()) return;
  if (C > 1 && t.stride(-1) != 1) bad_value(std::string("the last axis of ") + name + " must be contiguous");
  int64_t st = -1, span = 0;  // of the innermost leading axis longer than one, and of the axes so far
  for (int64_t i = t.dim() - 2; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (st < 0) {
      st = t.stride(i);
    } else if (t.stride(i) != span) {
      bad_value(std::string("the leading axes of ") + name + " must be seen as rows of one stride");
    }
    span = t.stride(i) * t.size(i);
  }
  *stride = st < 0 ? C : st;
}

struct Norm {
  const Tensor& x;
  const Tensor& weight;
  Tensor residual;
  wkv_dtype xt, rt;
  int64_t N, C, xs, rs, groups;
  float eps;
  c10::Device dev;
};

void norm_scalars(double eps, int64_t groups, int64_t C) {
  if (!(eps > 0) || !std::isfinite(eps) || !((float)eps > 0)) bad_value("eps must be positive and finite");
  if (groups < 1 || C % groups) bad_value("groups must divide the columns");
}

Norm norm_inputs(PyObject* ox, PyObject* ow, PyObject* ores, PyObject* oeps, PyObject* ogroups) {
  const Tensor& x = cuda_tensor(ox, "x");
  const wkv_dtype xt = value_type(x, "x");
  if (x.dim() < 1) bad_value("x must be [..., C]");
  const int64_t C = x.size(-1), groups = integer(ogroups);
  const double eps = number(oeps);
  norm_scalars(eps, groups, C);
  const Tensor& w = exact(ow, "weight", x.device(), {C}, at::kFloat);
  Norm n{x, w, Tensor(), xt, xt, 0, C, C, C, groups, (float)eps, x.device()};
  rows_of(x, "x", &n.N, &n.xs);
  if (ores != Py_None) {
    n.residual = cuda_tensor(ores, "residual");
    n.rt = value_type(n.residual, "residual");
    same_device(n.residual, "residual", n.dev);
    if (n.residual.sizes() != x.sizes()) bad_value("residual must be " + list_of(x.sizes()));
    if (xt == WKV_F32 && n.rt != WKV_F32) bad_type("residual must be float32 beside a float32 x");
    int64_t rows;
    rows_of(n.residual, "residual", &rows, &n.rs);
  }
  return n;
}

Tensor norm_sum(const Norm& n, PyObject* o) {
  if (!n.residual.defined()) {
    if (o != Py_None) bad_value("residual_out without a residual");
    return Tensor();
  }
  return result(o, "residual_out", n.dev, n.x.sizes(), n.residual.scalar_type());
}

// (x, weight, residual, eps, groups, out_dtype, out, residual_out)
PyObject* rms_norm(PyObject* const* a) {
  const Norm n = norm_inputs(a[0], a[1], a[2], a[3], a[4]);
  wkv_dtype yt;
  const ScalarType ys = out_type(a[5], a[6], n.x, &yt);
  const Tensor y = result(a[6], "out", n.dev, n.x.sizes(), ys);
  const Tensor s = norm_sum(n, a[7]);
  on_stream(n.dev, "wkv_rms_norm", [&](void* st) {
    return lib.rms_norm(n.N, n.C, n.groups, n.eps, n.x.data_ptr(), n.xt, n.xs, ptr(n.residual), n.rt, n.rs,
                        (const float*)n.weight.data_ptr(), y.data_ptr(), yt, ptr(s), st);
  });
  written(a[6], y);
  written(a[7], s);
  return tuple_of({y, s});
}

// (x, weight, residual, eps, groups, block, residual_out)
PyObject* rms_norm_quant(PyObject* const* a) {
  const Norm n = norm_inputs(a[0], a[1], a[2], a[3], a[4]);
  const int64_t block = integer(a[5]);
  if ((block != 0 && block != 32 && block != 64 && block != 128) || (block && n.C % block))
    bad_value("block must be 0 (a whole row), or 32, 64 or 128 and divide the columns");
  const Tensor q = fresh(n.dev, n.x.sizes(), at::kFloat8_e4m3fn);
  auto shape = n.x.sizes().vec();
  shape.back() = block ? n.C / block : 1;
  const Tensor scale = fresh(n.dev, shape, at::kFloat);
  const Tensor s = norm_sum(n, a[6]);
  on_stream(n.dev, "wkv_rms_norm_quant", [&](void* st) {
    return lib.rms_norm_quant(n.N, n.C, n.groups, n.eps, n.x.data_ptr(), n.xt, n.xs, ptr(n.residual), n.rt, n.rs,
                              (const float*)n.weight.data_ptr(), q.data_ptr(), (float*)scale.data_ptr(), block, ptr(s),
                              st);
  });
  written(a[6], s);
  return tuple_of({q, scale, s});
}

// (gy, s, weight, gs, eps, groups, workspace)
PyObject* rms_norm_backward(PyObject* const* a) {
  const Tensor& s = cuda_tensor(a[1], "s");
  const wkv_dtype sc = value_type(s, "s");
  if (s.dim() < 1) bad_value("s must be [..., C]");
  const c10::Device dev = s.device();
  const Tensor& any = cuda_tensor(a[0], "gy");
  const wkv_dtype gc = value_type(any, "gy");
  const Tensor& gy = exact(a[0], "gy", dev, s.sizes(), any.scalar_type());
  if (gc == WKV_F32 && sc != WKV_F32) bad_type("s must be float32 beside a float32 gy");
  const int64_t C = s.size(-1), groups = integer(a[5]);
  const double eps = number(a[4]);
  norm_scalars(eps, groups, C);
  const Tensor& w = exact(a[2], "weight", dev, {C}, at::kFloat);
  const Tensor gs = optional(a[3], "gs", dev, s.sizes(), s.scalar_type());
  int64_t N, ss;
  rows_of(s, "s", &N, &ss);
  const size_t need = lib.norm_workspace_size(N, C, groups);
  if (need == 0) bad_value("invalid sizes");
  Tensor ws;
  if (a[6] == Py_None) {
    ws = fresh(dev, {(int64_t)need}, at::kByte);
  } else {
    ws = cuda_tensor(a[6], "workspace");
    workspace_of_caller(ws, dev);
  }
  const Tensor ds = fresh(dev, s.sizes(), s.scalar_type()), dw = fresh(dev, {C}, at::kFloat);
  on_stream(dev, "wkv_rms_norm_backward", [&](void* st) {
    return lib.rms_norm_backward(N, C, groups, (float)eps, gy.data_ptr(), gc, s.data_ptr(), sc, ss,
                                 (const float*)w.data_ptr(), ptr(gs), ds.data_ptr(), (float*)dw.data_ptr(),
                                 ws.data_ptr(), bytes_of(ws), st);
  });
  return tuple_of({ds, dw});
}

// ---------------------------------------------------------------------------
// the module
// ---------------------------------------------------------------------------
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", N, n);
    return nullptr;
  }
  if (!lib.check) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(lib.out_of_memory, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// bind(addresses by name, check, out of memory): the loaded library's entry
// points and the exceptions of the package and of torch
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3 || !PyDict_Check(args[0]) || !PyCallable_Check(args[1]) || !PyExceptionClass_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "bind(dict of addresses, check, exception)");
    return nullptr;
  }
  auto take = [&](const char* name, auto* to) {
    PyObject* o = PyDict_GetItemString(args[0], name);
    void* p = o ? PyLong_AsVoidPtr(o) : nullptr;
    *to = reinterpret_cast<std::remove_pointer_t<decltype(to)>>(p);
    return p != nullptr;
  };
  if (!take("wkv_gated_workspace_size", &lib.gated_workspace_size) || !take("wkv_gated_forward", &lib.gated_forward) ||
      !take("wkv_gated_backward", &lib.gated_backward) || !take("wkv_gated_step", &lib.gated_step) ||
      !take("wkv_rms_norm", &lib.rms_norm) || !take("wkv_rms_norm_quant", &lib.rms_norm_quant) ||
      !take("wkv_rms_norm_backward_workspace_size", &lib.norm_workspace_size) ||
      !take("wkv_rms_norm_backward", &lib.rms_norm_backward)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, "an entry point is missing");
    return nullptr;
  }
  Py_XDECREF(lib.check);
  Py_XDECREF(lib.out_of_memory);
  lib.check = Py_NewRef(args[1]);
  lib.out_of_memory = Py_NewRef(args[2]);
  Py_RETURN_NONE;
}

// what the object was compiled against (build.py: ext_key)
PyObject* built_for(PyObject*, PyObject*) { return PyUnicode_FromString(WKV_EXT_KEY); }

#define WKV_ENTRY(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    {"built_for", &built_for, METH_NOARGS, nullptr},
    WKV_ENTRY(gated_kept_workspace, 1),
    WKV_ENTRY(gated_checkpoints, 1),
    WKV_ENTRY(gated_forward, 9),
    WKV_ENTRY(gated_backward, 8),
    WKV_ENTRY(gated_step, 8),
    WKV_ENTRY(rms_norm, 8),
    WKV_ENTRY(rms_norm_quant, 7),
    WKV_ENTRY(rms_norm_backward, 7),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_wkv_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__wkv_torch(void) { return PyModule_Create(&module); }
