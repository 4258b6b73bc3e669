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
#include <ATen/ops/zeros.h>
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
decltype(&libconv_kv_cache_write) cache_write_call;
decltype(&libconv_kv_cache_read) cache_read_call;
decltype(&libconv_cache_attention) cache_attention_call;
decltype(&libconv_cache_attention_workspace) cache_attention_workspace;
decltype(&libconv_linear) linear_call;
decltype(&libconv_linear_workspace) linear_workspace;
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
int code_of(at::ScalarType s) {
  return s == at::kFloat ? LIBCONV_F32 : s == at::kHalf ? LIBCONV_F16
         : s == at::kBFloat16 ? LIBCONV_BF16 : -1;
}
Kind kind_of(const char* what, const at::Tensor& t, int64_t dims) {
  const at::ScalarType s = t.scalar_type();
  const int code = code_of(s);
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
  at::Tensor fresh(at::ScalarType type, std::initializer_list<int64_t> shape, bool zeros = false) {
    const at::TensorOptions options = at::TensorOptions().dtype(type).device(kind.device);
    at::Tensor t = zeros ? at::zeros(c10::IntArrayRef(shape), options)
                         : at::empty(c10::IntArrayRef(shape), options);
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

// A cache in 8 bits: k_cache, v_cache, k_scale, v_scale from a[at] on, and
// lengths and block_table.
struct Cache {
  const at::Tensor &k, &v, &ks, &vs, &lengths, &table;
  int64_t blocks, size, heads, dim, width, entries;
  int format;

  Cache(const char* what, PyObject* const* a, PyObject* lengths_, PyObject* table_)
      : k(needed(what, a[0])), v(needed(what, a[1])), ks(needed(what, a[2])),
        vs(needed(what, a[3])), lengths(needed(what, lengths_)), table(needed(what, table_)) {
    const at::ScalarType t = k.scalar_type();
    format = t == at::kChar ? LIBCONV_CACHE_I8 : t == at::kFloat8_e4m3fn ? LIBCONV_CACHE_E4M3 : -1;
    if (!k.is_cuda() || format < 0 || k.dim() != 4 || (k.size(3) > 1 && k.stride(3) != 1))
      refuse(what, "k_cache [blocks, block, Hk, D] must be an int8 or float8_e4m3fn device tensor, "
                   "its last axis dense");
    blocks = k.size(0);
    size = k.size(1);
    heads = k.size(2);
    dim = k.size(3);
    const Kind of_codes = {k.device(), t, format}, of_scales = {k.device(), at::kFloat, 0};
    if (bad(v, of_codes, {blocks, size, heads, dim})) refuse(what, "v_cache must be as k_cache");
    if (bad_array(ks, of_scales, at::kFloat, {blocks, heads}) ||
        bad_array(vs, of_scales, at::kFloat, {blocks, heads}))
      refuse(what, "k_scale, v_scale must be contiguous float32 device tensors [blocks, Hk]");
    if (lengths.dim() != 1 || table.dim() != 2) refuse(what, "lengths [B], block_table [B, blocks]");
    entries = lengths.size(0);
    width = table.size(1);
    if (bad_array(lengths, of_codes, at::kInt, {entries}) ||
        bad_array(table, of_codes, at::kInt, {entries, width}))
      refuse(what, "lengths [B] and block_table [B, blocks] must be contiguous int32 device tensors");
  }
  void check_starts(const char* what, const at::Tensor& starts) const {
    const Kind any = {k.device(), at::kInt, 0};
    if (bad_array(starts, any, at::kInt, {entries + 1}))
      refuse(what, "row_starts must be a contiguous int32 device tensor [B + 1]");
  }
  void put_strides(long long* s) const {
    for (int i = 0; i < 3; ++i) {
      s[i] = k.stride(i);
      s[3 + i] = v.stride(i);
    }
  }
};

// k, v, k_cache, v_cache, k_scale, v_scale, row_starts, lengths, block_table, stream
PyObject* kv_cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* what = "kv_cache_write";
  if (n != 10) refuse_type(what, "10 arguments");
  const at::Tensor &k = needed(what, a[0]), &v = needed(what, a[1]), &starts = needed(what, a[6]);
  const Kind kind = kind_of(what, k, 3);
  const Cache c(what, a + 2, a[7], a[8]);
  const int64_t T = k.size(0);
  if (c.k.device() != kind.device) refuse(what, kOperands);
  if (bad(k, kind, {T, c.heads, c.dim}) || bad(v, kind, {T, c.heads, c.dim}))
    refuse(what, "k, v [T, Hk, D] with the cache's heads");
  c.check_starts(what, starts);
  LIBCONV_FORWARD_ONLY(what, &k, &v);
  Call call(kind, a[9]);
  if (T > 0 && c.entries > 0) {
    long long strides[10] = {k.stride(0), k.stride(1), v.stride(0), v.stride(1)};
    c.put_strides(strides + 4);
    const int t = as_int(what, T), b = as_int(what, c.entries), blocks = as_int(what, c.blocks),
              size = as_int(what, c.size), width = as_int(what, c.width),
              heads = as_int(what, c.heads), dim = as_int(what, c.dim);
    call.run("libconv_kv_cache_write", [&] {
      return cache_write_call(k.const_data_ptr(), v.const_data_ptr(), c.k.mutable_data_ptr(),
                              c.v.mutable_data_ptr(), static_cast<float*>(c.ks.mutable_data_ptr()),
                              static_cast<float*>(c.vs.mutable_data_ptr()),
                              address_of<int>(starts), address_of<int>(c.lengths),
                              address_of<int>(c.table), strides, b, t, blocks, size, width, heads,
                              dim, c.format, kind.code, call.stream);
    });
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, k_scale, v_scale, lengths, block_table, k_out, v_out, like (an
// empty tensor of the type of outputs made here), rows, stream
PyObject* kv_cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* what = "kv_cache_read";
  if (n != 11) refuse_type(what, "11 arguments");
  const Cache c(what, a, a[4], a[5]);
  const at::Tensor *ko = tensor(what, a[6]), *vo = tensor(what, a[7]);
  const at::ScalarType type = ko ? ko->scalar_type() : vo ? vo->scalar_type()
                                                          : needed(what, a[8]).scalar_type();
  const Kind kind = {c.k.device(), type, code_of(type)};
  if (kind.code < 0) refuse(what, "outputs are float32, float16 or bfloat16");
  int64_t S = ko && ko->dim() == 4 ? ko->size(1) : vo && vo->dim() == 4 ? vo->size(1) : -1;
  if (S < 0) {
    S = c.width * c.size;
    if (a[9] != Py_None) {
      const long long rows = PyLong_AsLongLong(a[9]);
      if (rows == -1 && PyErr_Occurred()) throw python_error();
      S = as_int(what, rows);
    }
  }
  if ((ko && bad(*ko, kind, {c.entries, S, c.heads, c.dim})) ||
      (vo && bad(*vo, kind, {c.entries, S, c.heads, c.dim})))
    refuse(what, "bad output tensor");
  Call call(kind, a[10]);
  at::Tensor made[2];
  if (!ko) ko = &(made[0] = call.fresh(type, {c.entries, S, c.heads, c.dim}, true));
  if (!vo) vo = &(made[1] = call.fresh(type, {c.entries, S, c.heads, c.dim}, true));
  if (c.entries > 0 && S > 0) {
    long long strides[12] = {};
    c.put_strides(strides);
    for (int i = 0; i < 3; ++i) {
      strides[6 + i] = ko->stride(i);
      strides[9 + i] = vo->stride(i);
    }
    const int s = as_int(what, S), b = as_int(what, c.entries), blocks = as_int(what, c.blocks),
              size = as_int(what, c.size), width = as_int(what, c.width),
              heads = as_int(what, c.heads), dim = as_int(what, c.dim);
    call.run("libconv_kv_cache_read", [&] {
      return cache_read_call(c.k.const_data_ptr(), c.v.const_data_ptr(), address_of<float>(c.ks),
                             address_of<float>(c.vs), address_of<int>(c.lengths),
                             address_of<int>(c.table), ko->mutable_data_ptr(),
                             vo->mutable_data_ptr(), strides, b, s, blocks, size, width, heads, dim,
                             c.format, kind.code, call.stream);
    });
  }
  PyObject* pair = PyTuple_New(2);
  if (!pair) throw python_error();
  PyTuple_SET_ITEM(pair, 0, result(a[6], *ko));
  PyTuple_SET_ITEM(pair, 1, result(a[7], *vo));
  return pair;
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, k_scale, v_scale, row_starts, lengths, block_table, max_rows,
// scale, causal, out, return_lse, stream, workspace
PyObject* cache_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* what = "cache_attention";
  if (n != 15) refuse_type(what, "15 arguments");
  const at::Tensor &q = needed(what, a[0]), &starts = needed(what, a[5]);
  const Kind kind = kind_of(what, q, 3);
  const Cache c(what, a + 1, a[6], a[7]);
  const int64_t T = q.size(0), Hq = q.size(1);
  if (c.k.device() != kind.device) refuse(what, kOperands);
  if (q.size(2) != c.dim) refuse(what, "q [T, Hq, D] with the cache's head size");
  c.check_starts(what, starts);
  const at::Tensor* out = tensor(what, a[11]);
  if (out && bad(*out, kind, {T, Hq, c.dim})) refuse(what, "bad output tensor");
  long long most = T;
  if (a[8] != Py_None) {
    most = PyLong_AsLongLong(a[8]);
    if (most == -1 && PyErr_Occurred()) throw python_error();
    if (most < 0) refuse(what, "max_rows: the largest number of rows of an entry");
  }
  const bool with_lse = truth(a[12]);
  LIBCONV_FORWARD_ONLY(what, &q);
  Call call(kind, a[13]);
  at::Tensor made, lse;
  if (!out) out = &(made = call.fresh(kind.type, {T, Hq, c.dim}));
  if (with_lse) lse = call.fresh(at::kFloat, {T, Hq});
  if (T > 0 && c.entries > 0) {
    long long strides[10] = {q.stride(0), q.stride(1), out->stride(0), out->stride(1)};
    c.put_strides(strides + 4);
    const int t = as_int(what, T), hq = as_int(what, Hq), rows = as_int(what, most),
              b = as_int(what, c.entries), blocks = as_int(what, c.blocks),
              size = as_int(what, c.size), width = as_int(what, c.width),
              heads = as_int(what, c.heads), dim = as_int(what, c.dim);
    const float scale =
        a[9] == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : (float)number(a[9]);
    const int causal = truth(a[10]);
    call.workspace(what, a[14],
                   a[14] == Py_True ? cache_attention_workspace(b, t, rows, size, width, hq, heads,
                                                                dim, kind.code)
                                    : 0);
    call.run("libconv_cache_attention", [&] {
      return cache_attention_call(
          q.const_data_ptr(), c.k.const_data_ptr(), c.v.const_data_ptr(),
          address_of<float>(c.ks), address_of<float>(c.vs), address_of<int>(starts),
          address_of<int>(c.lengths), address_of<int>(c.table), out->mutable_data_ptr(),
          with_lse ? static_cast<float*>(lse.mutable_data_ptr()) : nullptr, strides, b, t, rows,
          blocks, size, width, hq, heads, dim, scale, causal, c.format, kind.code, call.ws,
          call.bytes, call.stream);
    });
  }
  if (!with_lse) return result(a[11], *out);
  PyObject* pair = PyTuple_New(2);
  if (!pair) throw python_error();
  PyTuple_SET_ITEM(pair, 0, result(a[11], *out));
  PyTuple_SET_ITEM(pair, 1, result(Py_None, lse));
  return pair;
  END_HANDLE_TH_ERRORS
}

// x, w, bias, act (a number), residual, out, stream, workspace
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* what = "linear";
  if (n != 8) refuse_type(what, "8 arguments");
  const at::Tensor &x = needed(what, a[0]), &w = needed(what, a[1]);
  const at::Tensor *bias = tensor(what, a[2]), *residual = tensor(what, a[4]),
                   *out = tensor(what, a[5]);
  const Kind kind = kind_of(what, x, 2);
  const int64_t T = x.size(0), K = x.size(1);
  const int64_t N = w.dim() == 2 ? w.size(0) : -1;
  if (N < 0 || bad(w, kind, {N, K}) || !w.is_contiguous())
    refuse(what, "w must be a contiguous [N, K] as x");
  if (bias && bad(*bias, kind, {N})) refuse(what, "bias must be [N] as x");
  if (residual && bad(*residual, kind, {T, N})) refuse(what, "residual must be [T, N] as x");
  if (out && bad(*out, kind, {T, N})) refuse(what, "bad output tensor");
  const long long act = PyLong_AsLongLong(a[3]);
  if (act == -1 && PyErr_Occurred()) throw python_error();
  LIBCONV_FORWARD_ONLY(what, &x, &w, bias, residual);
  Call call(kind, a[6]);
  at::Tensor made;
  if (!out) out = &(made = call.fresh(kind.type, {T, N}));
  if (T > 0) {
    const int t = as_int(what, T), kk = as_int(what, K), nn = as_int(what, N);
    call.workspace(what, a[7], a[7] == Py_True ? linear_workspace(t, kk, nn, kind.code) : 0);
    call.run("libconv_linear", [&] {
      return linear_call(x.const_data_ptr(), w.const_data_ptr(), address(bias), address(residual),
                         out->mutable_data_ptr(), t, kk, nn, x.stride(0),
                         residual ? residual->stride(0) : 0, out->stride(0), (int)act, kind.code,
                         call.ws, call.bytes, call.stream);
    });
  }
  return result(a[5], *out);
  END_HANDLE_TH_ERRORS
}

// The addresses of the functions, in the order of `calls`, raw_stream, stream_id,
// fail.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  void** const calls[] = {
      reinterpret_cast<void**>(&rope_call), reinterpret_cast<void**>(&attention_call),
      reinterpret_cast<void**>(&attention_workspace), reinterpret_cast<void**>(&lora_call),
      reinterpret_cast<void**>(&lora_workspace), reinterpret_cast<void**>(&cache_write_call),
      reinterpret_cast<void**>(&cache_read_call), reinterpret_cast<void**>(&cache_attention_call),
      reinterpret_cast<void**>(&cache_attention_workspace), reinterpret_cast<void**>(&linear_call),
      reinterpret_cast<void**>(&linear_workspace)};
  constexpr int count = sizeof(calls) / sizeof(*calls);
  if (n != count + 3) refuse_type("bind", "another number of functions");
  void* f[count];
  for (int i = 0; i < count; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) throw python_error();
  for (int i = 0; i < count; ++i) *calls[i] = f[i];
  PyObject** keep[3] = {&raw_stream, &stream_id, &fail};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(a[count + i]);
    Py_XDECREF(*keep[i]);
    *keep[i] = a[count + i];
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define LIBCONV_METHOD(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LIBCONV_METHOD(qk_norm_rope), LIBCONV_METHOD(prefix_attention),
                         LIBCONV_METHOD(lora_linear), LIBCONV_METHOD(kv_cache_write),
                         LIBCONV_METHOD(kv_cache_read), LIBCONV_METHOD(cache_attention),
                         LIBCONV_METHOD(linear), LIBCONV_METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
