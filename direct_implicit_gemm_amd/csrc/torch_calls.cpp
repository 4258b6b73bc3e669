// torch_calls.cpp -- the calls of the attention-layer operators on torch
// tensors: argument checks, outputs and workspaces, strides, stream.  A CPython
// module (_torch_calls), because a small call takes less time on the GPU than
// Python takes to look its tensors over.  Measured, calls in a row: norms and
// rotation of 8 tokens of 60 heads of 64 (4.8 us of GPU) 5.4 us, through
// attributes in Python and ctypes 12.1; 8 rows of 640 -> 1920 with adapters of
// rank 8 (two kernels, 7.9 us) 8.9 and 13.5.  It links no GPU library: the
// operators' addresses come from the loaded libconv (see bind).
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/core/StreamGuard.h>
#include <c10/core/impl/VirtualGuardImpl.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <string>

#include "libconv.h"

namespace {

decltype(&libconv_qk_norm_rope) rope_call;
decltype(&libconv_prefix_attention) attention_call;
decltype(&libconv_prefix_attention_workspace) attention_workspace;
decltype(&libconv_lora_linear) lora_call;
decltype(&libconv_lora_workspace) lora_workspace;
// raw_stream(device) -> handle of the current stream; stream_id(handle, device)
// -> torch's number of any stream; fail(status, name) raises
PyObject *raw_stream, *stream_id, *fail;

constexpr const char* kOperands =
    "operands must be device tensors of one device and dtype, their last axis dense";

[[noreturn]] void refuse(const char* what, const char* why) {
  C10_THROW_ERROR(ValueError, std::string(what) + ": " + why);
}

[[noreturn]] void refuse_type(const char* what, const char* why) {
  throw torch::TypeError(std::string(what) + ": " + why);
}

const at::Tensor* tensor(const char* what, PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse_type(what, "expected a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(const char* what, PyObject* o) {
  const at::Tensor* t = tensor(what, o);
  if (!t) refuse_type(what, "expected a tensor");
  return *t;
}

// What the first operand sets for all others.
struct Kind {
  c10::Device device;
  at::ScalarType type;
  int code;
};
Kind kind_of(const char* what, const at::Tensor& t, int64_t dims) {
  const at::ScalarType s = t.scalar_type();
  const int code = s == at::kFloat ? LIBCONV_F32 : s == at::kHalf ? LIBCONV_F16
                   : s == at::kBFloat16 ? LIBCONV_BF16 : -1;
  if (!t.is_cuda() || code < 0 || t.dim() != dims ||
      (t.size(dims - 1) > 1 && t.stride(dims - 1) != 1))
    refuse(what, kOperands);
  return {t.device(), s, code};
}
bool bad(const at::Tensor& t, const Kind& k, std::initializer_list<int64_t> shape) {
  return t.device() != k.device || t.scalar_type() != k.type ||
         t.sizes() != c10::IntArrayRef(shape) ||
         (t.size(-1) > 1 && t.stride(-1) != 1);
}
bool bad_array(const at::Tensor& t, const Kind& k, at::ScalarType type,
               std::initializer_list<int64_t> shape) {
  return t.device() != k.device || t.scalar_type() != type ||
         t.sizes() != c10::IntArrayRef(shape) || !t.is_contiguous();
}
// There is no backward pass: a caller who may expect one is told (once an operator).
bool wants_grad(std::initializer_list<const at::Tensor*> operands) {
  if (!c10::GradMode::is_enabled()) return false;
  for (const at::Tensor* t : operands)
    if (t && t->requires_grad()) return true;
  return false;
}
#define LIBCONV_FORWARD_ONLY(what, ...)                                                       \
  do {                                                                                        \
    if (wants_grad({__VA_ARGS__})) {                                                          \
      TORCH_WARN_ONCE(what, ": an operand requires gradients, but the operator has no "       \
                      "backward pass: its outputs require none (torch.no_grad() says so)");   \
    }                                                                                         \
  } while (0)

const void* address(const at::Tensor* t) { return t ? t->const_data_ptr() : nullptr; }
template <class T> const T* address_of(const at::Tensor& t) {
  return static_cast<const T*>(t.const_data_ptr());
}
int as_int(const char* what, int64_t v) {
  if (v < 0 || v > INT32_MAX) refuse(what, "a size past 31 bits");
  return static_cast<int>(v);
}

// A launch waits when its queue is full: without the interpreter's lock.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The stream of a call, its outputs and, where it is asked for, its workspace.
// torch's allocator hands freed memory out again in the order of the stream it
// was allocated on: outputs and workspaces of a call are allocated with the
// call's stream as the current one, so that neither work still queued on the
// caller's stream nor the call itself meets another user of the same memory.
struct Call {
  c10::DeviceGuard guard;
  const Kind& kind;
  c10::OptionalStreamGuard on_stream;
  std::optional<c10::Stream> callers;   // the caller's stream, where it is another one
  void* stream = nullptr;
  at::Tensor buffer;
  void* ws = nullptr;
  long long bytes = 0;

  Call(const Kind& k, PyObject* given) : guard(k.device), kind(k) {
    PyObject* index = PyLong_FromLong(k.device.index());
    PyObject* handle = index ? PyObject_CallOneArg(raw_stream, index) : nullptr;
    Py_XDECREF(index);
    if (!handle) throw python_error();
    stream = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (PyErr_Occurred()) throw python_error();
    if (given == Py_None) return;
    void* const current = stream;
    stream = PyLong_AsVoidPtr(given);
    if (PyErr_Occurred()) throw python_error();
    if (stream == current) return;
    PyObject* id = PyObject_CallFunction(stream_id, "Oi", given, (int)k.device.index());
    const long long number = id ? PyLong_AsLongLong(id) : -1;
    Py_XDECREF(id);
    if (PyErr_Occurred()) throw python_error();
    callers = c10::impl::VirtualGuardImpl(k.device.type()).getStream(k.device);
    on_stream.reset_stream(c10::Stream::unpack3(number, k.device.index(), k.device.type()));
  }
  // An output: the caller, who reads it on a stream of theirs, may drop it while
  // that stream still does.
  at::Tensor fresh(at::ScalarType type, std::initializer_list<int64_t> shape) {
    at::Tensor t = at::empty(c10::IntArrayRef(shape),
                             at::TensorOptions().dtype(type).device(kind.device));
    if (callers)
      c10::impl::VirtualGuardImpl(kind.device.type())
          .recordDataPtrOnStream(t.storage().data_ptr(), *callers);
    return t;
  }
  // workspace: True (allocate `need` bytes), None or False (none), or a tensor
  void workspace(const char* what, PyObject* o, long long need) {
    if (o == Py_True) {
      if (need <= 0) return;   // none, or invalid sizes: the call says which
      buffer = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(kind.device));
      ws = buffer.mutable_data_ptr();
      bytes = need;
    } else if (o != Py_None && o != Py_False) {
      const at::Tensor& t = needed(what, o);
      if (t.device() != kind.device || !t.is_contiguous())
        refuse(what, "the workspace must be a contiguous device tensor");
      ws = t.mutable_data_ptr();
      bytes = static_cast<long long>(t.nbytes());
    }
  }
  template <class F> void run(const char* name, F&& enqueue) {
    libconv_status status;
    {
      Unlocked other_threads_run;
      status = enqueue();
    }
    if (status != LIBCONV_OK) {
      PyObject* r = PyObject_CallFunction(fail, "is", (int)status, name);
      Py_XDECREF(r);
      throw python_error();
    }
  }
};

// The caller's tensor again, or the one made for the call.
PyObject* result(PyObject* given, const at::Tensor& t) {
  if (given == Py_None) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) throw python_error();
    return o;
  }
  Py_INCREF(given);
  return given;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// q, k, positions, freqs, q_weight, k_weight, eps, sections, interleaved, v,
// slots, q_out, k_out, v_out, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* what = "qk_norm_rope";
  if (n != 15) refuse_type(what, "15 arguments");
  const at::Tensor &q = needed(what, a[0]), &k = needed(what, a[1]), &pos = needed(what, a[2]),
                   &freqs = needed(what, a[3]);
  const Kind kind = kind_of(what, q, 3);
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
  if (k.dim() != 3) refuse(what, kOperands);
  const int64_t Hk = k.size(1);
  if (bad(k, kind, {T, Hk, D})) refuse(what, "q [T, Hq, D], k and v [T, Hk, D]");
  const at::Tensor *qw = tensor(what, a[4]), *kw = tensor(what, a[5]), *v = tensor(what, a[9]),
                   *slots = tensor(what, a[10]), *qo = tensor(what, a[11]),
                   *ko = tensor(what, a[12]), *vo = tensor(what, a[13]);
  if (slots && (!ko || (v && !vo))) refuse(what, "slots need k_out (and v_out)");
  if (vo && !v) refuse(what, "v_out without v");
  const int64_t pairs = freqs.numel();
  int64_t part[3] = {pairs, 0, 0};
  if (a[7] != Py_None) {
    PyObject* s = PySequence_Fast(a[7], "sections: a sequence of numbers of pairs");
    if (!s) throw python_error();
    part[0] = 0;
    bool fits = true;
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(s); ++i) {
      const long long m = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(s, i));
      if (m == -1 && PyErr_Occurred()) {
        Py_DECREF(s);
        throw python_error();
      }
      fits = fits && m >= 0 && (i < 3 || m == 0);
      if (i < 3) part[i] = m;
    }
    Py_DECREF(s);
    if (!fits || part[0] + part[1] + part[2] != pairs)
      refuse(what, "up to 3 sections that add up to the pairs of freqs");
  }
  const int64_t axes = part[2] ? 3 : part[1] ? 2 : 1;
  const int64_t rows_pos = pos.dim() == 1 ? 1 : pos.dim() == 2 ? pos.size(0) : 0;
  if (2 * pairs > D || rows_pos < axes)
    refuse(what, "a row of positions for each section, and at most D / 2 pairs");
  if (pos.device() != kind.device || pos.scalar_type() != at::kInt || pos.size(-1) != T ||
      !pos.is_contiguous())
    refuse(what, "positions must be a contiguous int32 device tensor [axes, T]");
  if (freqs.device() != kind.device || freqs.scalar_type() != at::kDouble ||
      !freqs.is_contiguous())
    refuse(what, "freqs must be a contiguous float64 device tensor");
  if ((qw && bad(*qw, kind, {D})) || (kw && bad(*kw, kind, {D})))
    refuse(what, "weights [D] as the operands");
  if (slots && ko->dim() != 3) refuse(what, "k_out [rows, Hk, D]");
  const int64_t rows = slots ? ko->size(0) : T;
  if (slots && bad_array(*slots, kind, at::kInt, {T}))
    refuse(what, "slots must be a contiguous int32 device tensor [T]");
  if (v && bad(*v, kind, {T, Hk, D})) refuse(what, "v [T, Hk, D] as the operands");
  if ((qo && bad(*qo, kind, {T, Hq, D})) || (ko && bad(*ko, kind, {rows, Hk, D})) ||
      (vo && bad(*vo, kind, {rows, Hk, D})))
    refuse(what, "bad output tensor");
  LIBCONV_FORWARD_ONLY(what, &q, &k, v, qw, kw, &freqs);
  Call call(kind, a[14]);
  at::Tensor made[3];
  if (!qo) qo = &(made[0] = call.fresh(kind.type, {T, Hq, D}));
  if (!ko) ko = &(made[1] = call.fresh(kind.type, {T, Hk, D}));
  if (v && !vo) vo = &(made[2] = call.fresh(kind.type, {T, Hk, D}));
  if (T > 0) {
    const at::Tensor* in[6] = {&q, &k, v, qo, ko, vo};
    long long strides[12] = {};
    for (int i = 0; i < 6; ++i)
      if (in[i]) {
        strides[2 * i] = in[i]->stride(0);
        strides[2 * i + 1] = in[i]->stride(1);
      }
    const int t = as_int(what, T), hq = as_int(what, Hq), hk = as_int(what, Hk),
              d = as_int(what, D), out_rows = as_int(what, rows), interleaved = truth(a[8]);
    const float eps = (float)number(a[6]);
    call.run("libconv_qk_norm_rope", [&] {
      return rope_call(q.const_data_ptr(), k.const_data_ptr(), address(v), qo->mutable_data_ptr(),
                       ko->mutable_data_ptr(), vo ? vo->mutable_data_ptr() : nullptr, address(qw),
                       address(kw), address_of<double>(freqs), address_of<int>(pos),
                       slots ? address_of<int>(*slots) : nullptr, strides, t, hq, hk, d,
                       (int)(2 * pairs), (int)part[0], (int)part[1], (int)part[2], interleaved,
                       out_rows, eps, kind.code, call.stream);
    });
  }
  PyObject* out = PyTuple_New(v ? 3 : 2);
  if (!out) throw python_error();
  PyTuple_SET_ITEM(out, 0, result(a[11], *qo));
  PyTuple_SET_ITEM(out, 1, result(a[12], *ko));
  if (v) PyTuple_SET_ITEM(out, 2, result(a[13], *vo));
  return out;
  END_HANDLE_TH_ERRORS
}

// q, k_prefix, v_prefix, k, v, lengths, scale, causal, out, return_lse, stream,
// workspace
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* what = "prefix_attention";
  if (n != 12) refuse_type(what, "12 arguments");
  const at::Tensor &q = needed(what, a[0]), &lengths = needed(what, a[5]);
  const at::Tensor *kp = tensor(what, a[1]), *vp = tensor(what, a[2]), *k = tensor(what, a[3]),
                   *v = tensor(what, a[4]), *out = tensor(what, a[8]);
  const Kind kind = kind_of(what, q, 4);
  const int64_t B = q.size(0), Sq = q.size(1), Hq = q.size(2), D = q.size(3);
  if (!k != !v || !kp != !vp) refuse(what, "keys and values come together");
  if (!k && !kp) refuse(what, "neither a prefix nor own keys");
  int64_t P = 0, S = 0, Hk = 0;
  if (k) {
    if (k->dim() != 4) refuse(what, "k, v [B, S, Hk, D]");
    S = k->size(1);
    Hk = k->size(2);
    if (bad(*k, kind, {B, S, Hk, D}) || bad(*v, kind, {B, S, Hk, D}))
      refuse(what, "k, v [B, S, Hk, D] as q");
  }
  if (kp) {
    if (kp->dim() != 3) refuse(what, "k_prefix, v_prefix [P, Hk, D]");
    P = kp->size(0);
    if (!k) Hk = kp->size(1);
    if (bad(*kp, kind, {P, Hk, D}) || bad(*vp, kind, {P, Hk, D}))
      refuse(what, "k_prefix, v_prefix [P, Hk, D] as q");
  }
  if (bad_array(lengths, kind, at::kInt, {B}))
    refuse(what, "lengths must be a contiguous int32 device tensor [B]");
  if (out && bad(*out, kind, {B, Sq, Hq, D})) refuse(what, "bad output tensor");
  const bool with_lse = truth(a[9]);
  LIBCONV_FORWARD_ONLY(what, &q, kp, vp, k, v);
  Call call(kind, a[10]);
  at::Tensor made, lse;
  if (!out) out = &(made = call.fresh(kind.type, {B, Sq, Hq, D}));
  if (with_lse) lse = call.fresh(at::kFloat, {B, Hq, Sq});
  if (B > 0 && Sq > 0) {
    long long strides[16] = {};
    auto put = [&](int at, const at::Tensor* t, int axes) {
      for (int i = 0; t && i < axes; ++i) strides[at + i] = t->stride(i);
    };
    put(0, &q, 3);
    put(3, kp, 2);
    put(5, vp, 2);
    put(7, k, 3);
    put(10, v, 3);
    put(13, out, 3);
    const int b = as_int(what, B), sq = as_int(what, Sq), p = as_int(what, P), s = as_int(what, S),
              hq = as_int(what, Hq), hk = as_int(what, Hk), d = as_int(what, D);
    const float scale = a[6] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)number(a[6]);
    const int with_causal = truth(a[7]);
    call.workspace(what, a[11],
                   a[11] == Py_True ? attention_workspace(b, sq, p, s, hq, hk, d, kind.code) : 0);
    call.run("libconv_prefix_attention", [&] {
      return attention_call(q.const_data_ptr(), address(kp), address(vp), address(k), address(v),
                            address_of<int>(lengths), out->mutable_data_ptr(),
                            with_lse ? static_cast<float*>(lse.mutable_data_ptr()) : nullptr,
                            strides, b, sq, p, s, hq, hk, d, scale, with_causal, kind.code,
                            call.ws, call.bytes, call.stream);
    });
  }
  if (!with_lse) return result(a[8], *out);
  PyObject* pair = PyTuple_New(2);
  if (!pair) throw python_error();
  PyTuple_SET_ITEM(pair, 0, result(a[8], *out));
  PyTuple_SET_ITEM(pair, 1, result(Py_None, lse));
  return pair;
  END_HANDLE_TH_ERRORS
}

// x, w, bias, a, b, scales, row_starts, adapters, out, stream, workspace
PyObject* lora_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* what = "lora_linear";
  if (n != 11) refuse_type(what, "11 arguments");
  const at::Tensor &x = needed(what, a[0]), &w = needed(what, a[1]);
  const at::Tensor *bias = tensor(what, a[2]), *la = tensor(what, a[3]), *lb = tensor(what, a[4]),
                   *scales = tensor(what, a[5]), *starts = tensor(what, a[6]),
                   *ids = tensor(what, a[7]), *out = tensor(what, a[8]);
  const Kind kind = kind_of(what, x, 2);
  const int64_t T = x.size(0), K = x.size(1);
  const int64_t N = w.dim() == 2 ? w.size(0) : -1;
  if (N < 0 || bad(w, kind, {N, K}) || !w.is_contiguous())
    refuse(what, "w must be a contiguous [N, K] as x");
  if (bias && bad(*bias, kind, {N})) refuse(what, "bias must be [N] as x");
  int64_t count = 0, rank = 0, R = 0;
  if (la && lb && scales && starts && ids) {
    if (la->dim() != 3 || ids->dim() != 1) refuse(what, "a [n, rank, K], adapters [R]");
    count = la->size(0);
    rank = la->size(1);
    R = ids->size(0);
    if (bad(*la, kind, {count, rank, K}) || !la->is_contiguous() ||
        bad(*lb, kind, {count, N, rank}) || !lb->is_contiguous())
      refuse(what, "contiguous a [n, rank, K] and b [n, N, rank] as x");
    if (bad_array(*scales, kind, at::kFloat, {count}))
      refuse(what, "scales must be a contiguous float32 device tensor [n]");
    if (bad_array(*ids, kind, at::kInt, {R}) || bad_array(*starts, kind, at::kInt, {R + 1}))
      refuse(what, "row_starts [R + 1] and adapters [R] must be contiguous int32 device tensors");
  } else if (la || lb || scales || starts || ids) {
    refuse(what, "a, b, scales, row_starts and adapters come together");
  }
  if (out && bad(*out, kind, {T, N})) refuse(what, "bad output tensor");
  LIBCONV_FORWARD_ONLY(what, &x, &w, bias, la, lb, scales);
  Call call(kind, a[9]);
  at::Tensor made;
  if (!out) out = &(made = call.fresh(kind.type, {T, N}));
  if (T > 0) {
    const int t = as_int(what, T), kk = as_int(what, K), nn = as_int(what, N),
              r = as_int(what, rank), c = as_int(what, count), q = as_int(what, R);
    call.workspace(what, a[10],
                   a[10] == Py_True ? lora_workspace(t, kk, nn, r, c, q, kind.code) : 0);
    call.run("libconv_lora_linear", [&] {
      return lora_call(x.const_data_ptr(), w.const_data_ptr(), address(bias), address(la),
                       address(lb), scales ? address_of<float>(*scales) : nullptr,
                       starts ? address_of<int>(*starts) : nullptr,
                       ids ? address_of<int>(*ids) : nullptr, out->mutable_data_ptr(), t, kk, nn,
                       r, c, q, x.stride(0), out->stride(0), kind.code, call.ws, call.bytes,
                       call.stream);
    });
  }
  return result(a[8], *out);
  END_HANDLE_TH_ERRORS
}

// The addresses of the five functions (in the order above), raw_stream,
// stream_id, fail.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) refuse_type("bind", "8 arguments");
  void* f[5];
  for (int i = 0; i < 5; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) throw python_error();
  rope_call = reinterpret_cast<decltype(rope_call)>(f[0]);
  attention_call = reinterpret_cast<decltype(attention_call)>(f[1]);
  attention_workspace = reinterpret_cast<decltype(attention_workspace)>(f[2]);
  lora_call = reinterpret_cast<decltype(lora_call)>(f[3]);
  lora_workspace = reinterpret_cast<decltype(lora_workspace)>(f[4]);
  PyObject** keep[3] = {&raw_stream, &stream_id, &fail};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(a[5 + i]);
    Py_XDECREF(*keep[i]);
    *keep[i] = a[5 + i];
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define LIBCONV_METHOD(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LIBCONV_METHOD(qk_norm_rope), LIBCONV_METHOD(prefix_attention),
                         LIBCONV_METHOD(lora_linear), LIBCONV_METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
