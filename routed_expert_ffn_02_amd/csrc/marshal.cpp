// Torch tensors to the C entry points around the experts (moe_dispatch ... moe_block_norm_backward):
// checks of type, shape, stride and device, the current stream, and the call.  A Python
// extension module, since those checks in Python cost more than the launch they precede
// (0.4 us a tensor, 4 to 14 tensors a call, against 3 us): nothing is computed here.
#include <hip/hip_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <c10/hip/HIPStream.h>
#include <torch/csrc/api/include/torch/version.h>

#include <initializer_list>
#include <limits>
#include <string>

#include "../../include/routed_moe.h"

namespace {

PyObject* g_error = nullptr;  // the package's MoeError(status, where, message)

struct Refusal {
  moe_status status;
  std::string message;
};
[[noreturn]] void refuse(const std::string& message) { throw Refusal{MOE_EINVAL, message}; }

std::string shape_text(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

int32_t int_arg(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  if (v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max())
    refuse(std::string(name) + " is out of range");
  return (int32_t)v;
}
int64_t long_arg(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  return v;
}
float float_arg(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return (float)v;
}

// A [rows, H] matrix whose rows are contiguous; all zero for None.
struct Rows {
  void* p = nullptr;
  int32_t fmt = MOE_AFMT_F32, n = 0, h = 0;
  int64_t ld = 0;
};

// The tensors of one call: each is checked as it is read, and their devices once at the end.
class Call {
 public:
  // What a matrix has to agree with: rows and width where they are not zero, no gaps
  // between rows, the format and stride of `like`.
  struct Want {
    int64_t n = 0, h = 0;
    bool dense = false;
    const Rows* like = nullptr;
  };

  Rows rows(PyObject* o, const char* name, const Want& want) {
    if (o == Py_None) return {};
    return need_rows(o, name, want);
  }
  Rows need_rows(PyObject* o, const char* name, const Want& want) {
    const at::Tensor& t = tensor(o, name);
    const auto type = t.scalar_type();
    if (t.dim() != 2 || (type != at::kFloat && type != at::kBFloat16))
      refuse(std::string(name) + " must be a two-dimensional fp32 or bf16 tensor");
    const int64_t n = t.size(0), h = t.size(1), step = t.stride(1);
    constexpr int64_t most = std::numeric_limits<int32_t>::max();
    if (n < 1 || h < 1 || n > most || h > most || (want.n && n != want.n) || (want.h && h != want.h))
      refuse(std::string(name) + " has shape " + shape_text(t.sizes()) + ", not (" +
             (want.n ? std::to_string(want.n) : "T") + ", " + (want.h ? std::to_string(want.h) : "H") + ")");
    const int64_t ld = n == 1 ? h : t.stride(0);
    if ((step != 1 && h > 1) || ld < h || (want.dense && ld != h))
      refuse(std::string(name) + " needs contiguous rows" + (want.dense ? " without gaps" : ""));
    const int32_t fmt = type == at::kBFloat16 ? MOE_AFMT_BF16 : MOE_AFMT_F32;
    if (want.like && want.like->p && (fmt != want.like->fmt || ld != want.like->ld))
      refuse(std::string(name) + " must have the type and row stride of the tensor it belongs to");
    return {t.data_ptr(), fmt, (int32_t)n, (int32_t)h, ld};
  }

  // A dense tensor of this type and shape (one number: that many elements); nullptr for None.
  template <typename T>
  T* flat(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (o == Py_None) return nullptr;
    return need_flat<T>(o, name, type, shape);
  }
  template <typename T>
  T* need_flat(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || !t.is_contiguous())
      refuse(std::string(name) + " must be a contiguous " + (type == at::kInt ? "int32" : "float32") + " tensor");
    const c10::IntArrayRef want(shape.begin(), shape.size());
    if (t.sizes() != want && !(shape.size() == 1 && t.numel() == want[0]))
      refuse(std::string(name) + " has shape " + shape_text(t.sizes()) + ", not " + shape_text(want));
    return static_cast<T*>(t.data_ptr());
  }

  // T rows of H elements of format fmt, ld elements apart (0: H); of any shape without gaps where
  // the rows have none.
  void block_rows(PyObject* o, const char* name, int32_t T, int32_t H, int32_t fmt, int64_t ld) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != (fmt == MOE_AFMT_BF16 ? at::kBFloat16 : at::kFloat))
      refuse(std::string(name) + " must have the type that norm gives it");
    const bool matrix = t.dim() == 2 && t.size(0) == T && t.size(1) == H && (H == 1 || t.stride(1) == 1) &&
                        (T == 1 || t.stride(0) == (ld ? ld : H));
    const bool dense = t.numel() == (int64_t)T * H && t.is_contiguous() && (T == 1 || ld == 0 || ld == H);
    if (!matrix && !dense)
      refuse(std::string(name) + " has shape " + shape_text(t.sizes()) + " or strides that are not norm's");
  }

  // An int32 table [T, k].
  int32_t* pairs(PyObject* o, const char* name, int32_t* T, int32_t* k) {
    const at::Tensor& t = tensor(o, name);
    constexpr int64_t most = std::numeric_limits<int32_t>::max();
    if (t.dim() != 2 || t.numel() < 1 || t.size(0) > most || t.size(1) > most)
      refuse(std::string(name) + " must be an int32 tensor [T, k]");
    *T = (int32_t)t.size(0);
    *k = (int32_t)t.size(1);
    return need_flat<int32_t>(o, name, at::kInt, {t.size(0), t.size(1)});
  }

  // The caller's workspace.
  void* workspace(PyObject* o, size_t* bytes) {
    *bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, "ws");
    if (!t.is_contiguous()) refuse("ws must be a contiguous tensor");
    *bytes = (size_t)t.numel() * t.element_size();
    return *bytes ? t.data_ptr() : nullptr;
  }

  void on_one_gpu() const {
    if (off_gpu_) refuse(std::string(off_gpu_) + " must be on the GPU");
    if (other_)
      refuse(std::string(other_) + " is on cuda:" + std::to_string(other_device_) + ", other tensors on cuda:" +
             std::to_string(device_));
  }

  // The stream of the call: `o` (a handle, or a torch stream), or the current one of the
  // tensors' device, which becomes the current device until the call is over.
  moe_stream_t stream(PyObject* o) {
    on_one_gpu();
    void* s = nullptr;
    if (o == Py_None) {
      s = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device_).stream();
    } else if (PyLong_Check(o)) {
      s = PyLong_AsVoidPtr(o);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("stream is no handle");
      }
    } else {
      const int64_t device = attribute(o, "device_index");
      if (device != device_)
        refuse("stream is on cuda:" + std::to_string(device) + ", tensors on cuda:" + std::to_string(device_));
      s = reinterpret_cast<void*>(attribute(o, "cuda_stream"));
    }
    int now = -1;
    if (hipGetDevice(&now) == hipSuccess && now != device_ && hipSetDevice(device_) == hipSuccess) before_ = now;
    // a handle's device, but for the reserved ones, which belong to the current device
    hipDevice_t of = device_;
    const hipStream_t h = static_cast<hipStream_t>(s);
    if (PyLong_Check(o) && h && h != hipStreamLegacy && h != hipStreamPerThread && hipStreamGetDevice(h, &of) == hipSuccess &&
        of != device_)
      refuse("stream is on cuda:" + std::to_string(of) + ", tensors on cuda:" + std::to_string(device_));
    return s;
  }

  ~Call() {
    if (before_ >= 0) (void)hipSetDevice(before_);
  }

 private:
  const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) refuse(std::string(name) + " must be a strided tensor");
    if (!t.is_cuda()) {
      if (!off_gpu_) off_gpu_ = name;
    } else if (device_ < 0) {
      device_ = t.get_device();
    } else if (t.get_device() != device_ && !other_) {
      other_ = name;
      other_device_ = t.get_device();
    }
    return t;
  }
  static int64_t attribute(PyObject* o, const char* name) {
    PyObject* v = PyObject_GetAttrString(o, name);
    const long long n = v ? PyLong_AsLongLong(v) : -1;
    Py_XDECREF(v);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse("stream must be a torch stream or a stream handle");
    }
    return n;
  }

  int device_ = -1, other_device_ = -1, before_ = -1;
  const char *off_gpu_ = nullptr, *other_ = nullptr;
};

// One entry point: N arguments, the body's status, and every error as the package's MoeError.
template <Py_ssize_t N, typename F>
PyObject* entry(const char* where, PyObject* const* a, Py_ssize_t n, F body) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", where, N);
  moe_status status = MOE_OK;
  std::string message;
  try {
    status = body(a);
    if (status == MOE_EHIP) message = "launch failure";
    else if (status != MOE_OK) message = "shape out of range, overlapping tensors, missing argument or short workspace";
  } catch (const Refusal& r) {
    status = r.status;
    message = r.message;
  } catch (const std::exception& e) {
    status = MOE_EINVAL;
    message = e.what();
  }
  if (status == MOE_OK) Py_RETURN_NONE;
  if (PyObject* e = PyObject_CallFunction(g_error, "iss", (int)status, where, message.c_str())) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// The call itself, without the interpreter's lock (a launch waits where the queue is full).
template <typename F>
moe_status unlocked(F call) {
  PyThreadState* state = PyEval_SaveThread();
  const moe_status status = call();
  PyEval_RestoreThread(state);
  return status;
}

constexpr auto kI32 = at::kInt;
constexpr auto kF32 = at::kFloat;

// (topk_idx, n_experts, x, xs, perm, inv, offsets, ws, stream)
PyObject* dispatch(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<9>("moe_dispatch", args, n, [](PyObject* const* a) {
    Call c;
    int32_t T, k;
    size_t bytes;
    const int32_t* idx = c.pairs(a[0], "topk_idx", &T, &k);
    const int32_t E = int_arg(a[1], "n_experts");
    const int64_t P = (int64_t)T * k;
    Rows x, xs;
    if (a[2] != Py_None || a[3] != Py_None) {
      x = c.need_rows(a[2], "x", {T});
      xs = c.need_rows(a[3], "xs", {P, x.h, true});
      if (xs.fmt != x.fmt) refuse("xs must have x's type");
    }
    int32_t* perm = c.need_flat<int32_t>(a[4], "perm", kI32, {P});
    int32_t* inv = c.need_flat<int32_t>(a[5], "inv", kI32, {T, k});
    int32_t* offsets = c.need_flat<int32_t>(a[6], "offsets", kI32, {(int64_t)E + 1});
    void* ws = c.workspace(a[7], &bytes);
    const moe_stream_t s = c.stream(a[8]);
    return unlocked([&] {
      return moe_dispatch(idx, T, k, E, x.p, x.fmt, x.h, x.ld, xs.p, perm, inv, offsets, ws, bytes, s);
    });
  });
}

// (dxs, inv, dx, stream)
PyObject* dispatch_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<4>("moe_dispatch_backward", args, n, [](PyObject* const* a) {
    Call c;
    int32_t T, k;
    const int32_t* inv = c.pairs(a[1], "inv", &T, &k);
    const Rows g = c.need_rows(a[0], "dxs", {(int64_t)T * k, 0, true});
    const Rows o = c.need_rows(a[2], "dx", {T, g.h});
    const moe_stream_t s = c.stream(a[3]);
    return unlocked([&] {
      return moe_dispatch_backward(g.p, g.fmt, inv, T, k, g.h, o.p, o.fmt, o.ld, s);
    });
  });
}

// (ys, inv, w, y, stream)
PyObject* combine(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<5>("moe_combine", args, n, [](PyObject* const* a) {
    Call c;
    int32_t T, k;
    const int32_t* inv = c.pairs(a[1], "inv", &T, &k);
    const Rows r = c.need_rows(a[0], "ys", {(int64_t)T * k, 0, true});
    const float* w = c.need_flat<float>(a[2], "w", kF32, {T, k});
    const Rows o = c.need_rows(a[3], "y", {T, r.h});
    const moe_stream_t s = c.stream(a[4]);
    return unlocked([&] {
      return moe_combine(r.p, r.fmt, inv, w, T, k, r.h, o.p, o.fmt, o.ld, s);
    });
  });
}

// (dy, ys, inv, w, dys, dw, stream)
PyObject* combine_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<7>("moe_combine_backward", args, n, [](PyObject* const* a) {
    Call c;
    int32_t T, k;
    const int32_t* inv = c.pairs(a[2], "inv", &T, &k);
    const Rows d = c.need_rows(a[0], "dy", {T});
    const int64_t P = (int64_t)T * k;
    const Rows o = c.rows(a[4], "dys", {P, d.h, true});
    float* dw = c.flat<float>(a[5], "dw", kF32, {T, k});
    const float* w = o.p ? c.need_flat<float>(a[3], "w", kF32, {T, k}) : nullptr;
    const Rows r = dw ? c.need_rows(a[1], "ys", {P, d.h, true}) : Rows{};
    if (o.p && r.p && o.fmt != r.fmt) refuse("dys must have ys's type");
    const moe_stream_t s = c.stream(a[6]);
    return unlocked([&] {
      return moe_combine_backward(d.p, d.fmt, d.ld, r.p, r.p ? r.fmt : o.fmt, inv, w, T, k, d.h, o.p, dw, s);
    });
  });
}

// (logits, topk_idx, dw, renorm, dlogits, stream)
PyObject* topk_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<6>("moe_topk_backward", args, n, [](PyObject* const* a) {
    Call c;
    int32_t T, k;
    const int32_t* idx = c.pairs(a[1], "topk_idx", &T, &k);
    const Rows z = c.need_rows(a[0], "logits", {T, 0, true});
    if (z.fmt != MOE_AFMT_F32) refuse("logits must be fp32");
    const float* dw = c.need_flat<float>(a[2], "dw", kF32, {T, k});
    const int32_t renorm = int_arg(a[3], "renorm");
    float* o = c.need_flat<float>(a[4], "dlogits", kF32, {T, z.h});
    const moe_stream_t s = c.stream(a[5]);
    return unlocked([&] {
      return moe_topk_backward(static_cast<float*>(z.p), T, z.h, idx, k, dw, renorm, o, s);
    });
  });
}

struct NormWeights {
  float *post, *gate, *pre;
};
NormWeights norm_weights(Call& c, PyObject* post, PyObject* gate, PyObject* pre, int32_t T, int32_t H, int32_t kind) {
  NormWeights w;
  w.post = c.flat<float>(post, "w_post", kF32, {H});
  w.pre = c.flat<float>(pre, "w_pre", kF32, {H});
  if ((gate == Py_None) != (kind == MOE_GATE_NONE)) refuse("gate and gate_kind must go together");
  w.gate = c.flat<float>(gate, "gate", kF32, {kind == MOE_GATE_TOKEN ? T : H});
  return w;
}

// (h, y, w_post, gate, w_pre, h_out, x_out, gate_kind, alpha, eps, stream)
PyObject* block_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<11>("moe_block_norm", args, n, [](PyObject* const* a) {
    Call c;
    const Rows h = c.need_rows(a[0], "h", {});
    const int32_t T = h.n, H = h.h, kind = int_arg(a[7], "gate_kind");
    const Rows y = c.rows(a[1], "y", {T, H}), ho = c.rows(a[5], "h_out", {T, H, false, &h});
    const Rows xo = c.rows(a[6], "x_out", {T, H});
    const NormWeights w = norm_weights(c, a[2], a[3], a[4], T, H, kind);
    const moe_norm_config cfg = {T, H, h.fmt, y.fmt, xo.fmt, kind, float_arg(a[8], "alpha"), float_arg(a[9], "eps"),
                                 h.ld, y.ld, xo.ld};
    const moe_stream_t s = c.stream(a[10]);
    return unlocked([&] {
      return moe_block_norm(&cfg, h.p, y.p, w.post, w.gate, w.pre, ho.p, xo.p, s);
    });
  });
}

// (h_out, y, w_post, gate, w_pre, dh_out, dx, dh, dy, dw_post, dgate, dw_pre, ws, gate_kind, alpha, eps, stream)
PyObject* block_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<17>("moe_block_norm_backward", args, n, [](PyObject* const* a) {
    Call c;
    if (a[5] == Py_None && a[6] == Py_None) refuse("dh_out or dx must be given");
    const int32_t kind = int_arg(a[13], "gate_kind");
    const Rows dh_out = c.rows(a[5], "dh_out", {}), dx = c.rows(a[6], "dx", {dh_out.n, dh_out.h});
    const int32_t T = dx.p ? dx.n : dh_out.n, H = dx.p ? dx.h : dh_out.h;
    // h_out, dh_out and dh share a format and a stride, y and dy likewise
    const Rows h_out = c.rows(a[0], "h_out", {T, H, false, &dh_out});
    const Rows& h_like = dh_out.p ? dh_out : h_out;
    const Rows dh = c.rows(a[7], "dh", {T, H, false, &h_like});
    const Rows y = c.rows(a[1], "y", {T, H}), dy = c.rows(a[8], "dy", {T, H, false, &y});
    const NormWeights w = norm_weights(c, a[2], a[3], a[4], T, H, kind);
    float* dw_post = c.flat<float>(a[9], "dw_post", kF32, {H});
    float* dgate = c.flat<float>(a[10], "dgate", kF32, {kind == MOE_GATE_TOKEN ? T : H});
    float* dw_pre = c.flat<float>(a[11], "dw_pre", kF32, {H});
    size_t bytes;
    void* ws = c.workspace(a[12], &bytes);
    const Rows& h_any = h_like.p ? h_like : dh;
    const moe_norm_config cfg = {T, H, h_any.fmt, y.fmt, dx.fmt, kind, float_arg(a[14], "alpha"),
                                 float_arg(a[15], "eps"), h_any.ld, y.ld, dx.ld};
    const moe_stream_t s = c.stream(a[16]);
    return unlocked([&] {
      return moe_block_norm_backward(&cfg, h_out.p, y.p, w.post, w.gate, w.pre, dh_out.p, dx.p, dh.p, dy.p, dw_post, dgate,
                                   dw_pre, ws, bytes, s);
    });
  });
}

// (T, H, h_fmt, x_fmt, gate_kind, ld_h, ld_x, h, w_post, gate, w_pre, x_next): the norm's tensors of
// moe_decode_block against its configuration.  That call goes through ctypes with the rest of a context's, so
// an address (an int) stands for a tensor there and is taken as it is.
PyObject* check_block(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<12>("moe_decode_block", args, n, [](PyObject* const* a) {
    Call c;
    const int32_t T = int_arg(a[0], "T"), H = int_arg(a[1], "H"), kind = int_arg(a[4], "gate_kind");
    const auto given = [](PyObject* o) { return o != Py_None && !PyLong_Check(o); };
    if (given(a[7])) c.block_rows(a[7], "h", T, H, int_arg(a[2], "h_fmt"), long_arg(a[5], "ld_h"));
    if (given(a[11])) c.block_rows(a[11], "x_next", T, H, int_arg(a[3], "x_fmt"), long_arg(a[6], "ld_x"));
    if (given(a[8])) c.need_flat<float>(a[8], "w_post", kF32, {H});
    if (given(a[9])) c.need_flat<float>(a[9], "gate", kF32, {kind == MOE_GATE_TOKEN ? T : H});
    if (given(a[10])) c.need_flat<float>(a[10], "w_pre", kF32, {H});
    c.on_one_gpu();
    return MOE_OK;
  });
}

// (MoeError)
PyObject* set_error(PyObject*, PyObject* o) {
  Py_INCREF(o);
  Py_XSETREF(g_error, o);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(dispatch), FAST(dispatch_backward), FAST(combine), FAST(combine_backward),
                           FAST(topk_backward), FAST(block_norm), FAST(block_norm_backward), FAST(check_block),
                           {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", "Tensors to the C entry points around the experts", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch that this was compiled against (its C++ interface has no other tag)
PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
