// binding.cpp -- the Python side of the FP8 block-128, router and combine-gradient calls: checks
// torch tensors, allocates the outputs that the caller does not bring, takes the current stream or the given one
// and calls the C ABI (include/fme.h).
//
// These calls take a few microseconds on the GPU in a decode step, less than their Python checks
// and allocations took on a Grace core (moe_gate of 16 tokens: 11 us a call through ctypes).
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <string>

#include "../../include/fme.h"

namespace {

PyObject *g_fme_error = nullptr;  // FmeError(status, where, detail)

struct PythonError {};                      // a Python exception is set
struct Refused : std::runtime_error {       // ValueError
  using std::runtime_error::runtime_error;
};

using Shape = at::IntArrayRef;

std::string describe(Shape shape) {
  std::ostringstream s;
  s << "(";
  for (size_t i = 0; i < shape.size(); ++i) s << (i ? ", " : "") << shape[i];
  s << (shape.size() == 1 ? ",)" : ")");
  return s.str();
}

const char *name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kBool: return "torch.bool";
    default: return c10::toString(t);
  }
}

// A call: its name, and the device that all its tensors must share.
struct Call {
  const char *where;
  const char *first = nullptr;  // the argument whose device it is
  int device = -1;
};

const at::Tensor &tensor(const Call &c, const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) throw Refused(std::string(c.where) + ": " + name + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The kernels get plain addresses, so one of another GPU's would be an illegal access there.
void on_one_device(Call &c, const char *name, const at::Tensor &t) {
  const int device = t.device().index();
  if (!c.first) {
    c.first = name;
    c.device = device;
  } else if (device != c.device) {
    std::ostringstream s;
    s << c.where << ": " << name << " is on " << t.device() << ", " << c.first << " on cuda:" << c.device;
    throw Refused(s.str());
  }
}

void need(Call &c, const char *name, const at::Tensor &t, at::ScalarType type, Shape shape) {
  if (t.scalar_type() == type && t.sizes() == shape && t.is_cuda() && t.is_contiguous()) {
    on_one_device(c, name, t);
    return;
  }
  std::ostringstream s;
  s << c.where << ": " << name << " must be a contiguous CUDA tensor of " << name_of(type) << " " << describe(shape)
    << ", got " << name_of(t.scalar_type()) << " " << describe(t.sizes()) << " on " << t.device()
    << (t.is_contiguous() ? "" : " (not contiguous)");
  throw Refused(s.str());
}

const at::Tensor &input(Call &c, const char *name, PyObject *o, at::ScalarType type, Shape shape) {
  const at::Tensor &t = tensor(c, name, o);
  need(c, name, t, type, shape);
  return t;
}

// Dimensions of an argument that the others' shapes follow from.
Shape dims(const Call &c, const char *name, PyObject *o, size_t n) {
  const at::Tensor &t = tensor(c, name, o);
  if (t.dim() != static_cast<int64_t>(n))
    throw Refused(std::string(c.where) + ": " + name + " must have " + std::to_string(n) + " dimensions, got " +
                  describe(t.sizes()));
  return t.sizes();
}

template <typename T = void>
T *ptr(const at::Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}

int32_t *status_ptr(Call &c, PyObject *o) {
  if (o == Py_None) return nullptr;
  const at::Tensor &t = tensor(c, "status", o);
  if (t.scalar_type() != at::kInt || !t.is_cuda() || t.numel() < 1)
    throw Refused(std::string(c.where) + ": status must be a CUDA tensor of torch.int32");
  on_one_device(c, "status", t);
  return ptr<int32_t>(t);
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
// Past 32 bits: a value that the library refuses.
int32_t integer32(PyObject *o) {
  const int64_t v = integer(o);
  return v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : static_cast<int32_t>(v);
}
float real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(v);
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}

// The stream of a call: a raw one, or None for the current one.  The tensors' device must be the current one: its
// streams, properties and launches are the call's.  What the call allocates while this lives comes from the pool
// of its own stream: a block of another's, just freed, may still be used by work queued there.
class OnStream {
 public:
  OnStream(const Call &c, PyObject *o) : outer_(c10::cuda::getCurrentCUDAStream()), own_(outer_) {
    if (c.device != outer_.device_index()) {
      std::ostringstream s;
      s << c.where << ": " << c.first << " is on cuda:" << c.device << ", the current device is cuda:"
        << static_cast<int>(outer_.device_index());
      throw Refused(s.str());
    }
    if (o == Py_None) return;
    void *raw = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw PythonError{};
    own_ = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), outer_.device_index());
    if (raw == outer_.stream()) return;
    other_ = true;
    c10::cuda::setCurrentCUDAStream(own_);
  }
  ~OnStream() {
    if (other_) c10::cuda::setCurrentCUDAStream(outer_);
  }
  OnStream(const OnStream &) = delete;
  OnStream &operator=(const OnStream &) = delete;
  void *raw() const { return own_.stream(); }
  // The caller goes on with an output on its own stream: freed, its memory waits for that one as well.
  at::Tensor shared(at::Tensor t) const {
    if (other_) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), outer_);
    return t;
  }

 private:
  c10::cuda::CUDAStream outer_, own_;
  bool other_ = false;
};

// The caller's output tensor, checked, or a new one.
at::Tensor output(Call &c, const OnStream &on, const char *name, PyObject *o, at::ScalarType type, Shape shape,
                  const at::Tensor &like) {
  if (o == Py_None) return on.shared(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
  return input(c, name, o, type, shape);
}

template <typename F>
void call(const Call &c, F f) {
  fme_status st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS if (st == FME_OK) return;
  PyObject *e = PyObject_CallFunction(g_fme_error, "iss", st, c.where, st == FME_ERR_CUDA ? fme_last_cuda_error() : "");
  if (e) {
    PyErr_SetObject(g_fme_error, e);
    Py_DECREF(e);
  }
  throw PythonError{};
}

// Outputs as Python objects: the caller's own where it brought them.
PyObject *one(PyObject *given, const at::Tensor &t) {
  if (given == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(given);
  return given;
}
struct Result {
  PyObject *given;
  const at::Tensor &t;
};
PyObject *tuple(std::initializer_list<Result> results) {
  PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(results.size()));
  if (!r) throw PythonError{};
  Py_ssize_t i = 0;
  for (const Result &x : results) {
    PyObject *o = one(x.given, x.t);
    if (!o) {
      Py_DECREF(r);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Wraps f(args) as a Python function of exactly N positional arguments.
template <int N, PyObject *(*F)(PyObject *const *)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PythonError &) {
  } catch (const Refused &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception &e) {  // allocation failures among them
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;
constexpr auto kU8 = at::kByte;

// ------------------------------------------------------------------ quantizers --
// x, src_row, top_k, codes, scale, status, stream
PyObject *quantize_rows(PyObject *const *a) {
  Call w{"quantize_fp8_block128"};
  const Shape s = dims(w, "x", a[0], 2);
  const int64_t rows = s[0], cols = s[1];
  const at::Tensor &x = input(w, "x", a[0], kBf16, {rows, cols});
  const int32_t top_k = integer32(a[2]);
  const bool gather = a[1] != Py_None;
  const int64_t out = gather ? rows * top_k : rows;
  const int32_t *src = gather ? ptr<int32_t>(input(w, "src_row", a[1], kI32, {out})) : nullptr;
  int32_t *st = status_ptr(w, a[5]);
  const OnStream on(w, a[6]);
  const at::Tensor codes = output(w, on, "codes", a[3], kU8, {out, cols}, x);
  const at::Tensor scale = output(w, on, "scale", a[4], kF32, {(cols + 127) / 128, out}, x);
  call(w, [&] {
    return gather ? permute_quantize_fp8_block128(ptr(x), rows, cols, src, top_k, ptr<uint8_t>(codes), ptr<float>(scale),
                                                  st, on.raw())
                  : quantize_fp8_block128(ptr(x), rows, cols, FME_ROWWISE, nullptr, 1, ptr<uint8_t>(codes),
                                          ptr<float>(scale), nullptr, st, on.raw());
  });
  return tuple({{a[3], codes}, {a[4], scale}});
}

// The groups of a column-wise call: offsets (or None) and their number (or None).
int32_t groups_of(Call &w, PyObject *offsets, PyObject *num_groups, const int32_t **out) {
  *out = nullptr;
  if (offsets == Py_None) return num_groups == Py_None ? 1 : integer32(num_groups);
  const int64_t n = num_groups == Py_None ? dims(w, "offsets", offsets, 1)[0] - 1 : integer(num_groups);
  *out = ptr<int32_t>(input(w, "offsets", offsets, kI32, {n + 1}));
  return static_cast<int32_t>(n);
}

// x, offsets, num_groups, codes, scale, padded_offsets, status, stream
PyObject *quantize_cols(PyObject *const *a) {
  Call w{"quantize_fp8_block128"};
  const Shape s = dims(w, "x", a[0], 2);
  const int64_t rows = s[0], cols = s[1];
  const at::Tensor &x = input(w, "x", a[0], kBf16, {rows, cols});
  const int32_t *off;
  const int32_t g = groups_of(w, a[1], a[2], &off);
  const int64_t ld = fme_colwise_ld(rows, g);
  int32_t *st = status_ptr(w, a[6]);
  const OnStream on(w, a[7]);
  const at::Tensor codes = output(w, on, "codes", a[3], kU8, {ld, cols}, x);
  const at::Tensor scale = output(w, on, "scale", a[4], kF32, {ld / 128, cols}, x);
  const at::Tensor po = output(w, on, "padded_offsets", a[5], kI32, {g < 0 ? 0 : int64_t(g) + 1}, x);
  call(w, [&] {
    return quantize_fp8_block128(ptr(x), rows, cols, FME_COLWISE, off, g, ptr<uint8_t>(codes), ptr<float>(scale),
                                 ptr<int32_t>(po), st, on.raw());
  });
  return tuple({{a[3], codes}, {a[4], scale}, {a[5], po}});
}

// x, offsets, num_groups, row_codes, row_scale, col_codes, col_scale, padded_offsets, status, stream
PyObject *quantize_rowcol(PyObject *const *a) {
  Call w{"quantize_fp8_block128_rowcol"};
  const Shape s = dims(w, "x", a[0], 2);
  const int64_t rows = s[0], cols = s[1];
  const at::Tensor &x = input(w, "x", a[0], kBf16, {rows, cols});
  const int32_t *off;
  const int32_t g = groups_of(w, a[1], a[2], &off);
  const int64_t ld = fme_colwise_ld(rows, g);
  int32_t *st = status_ptr(w, a[8]);
  const OnStream on(w, a[9]);
  const at::Tensor rc = output(w, on, "row_codes", a[3], kU8, {rows, cols}, x);
  const at::Tensor rs = output(w, on, "row_scale", a[4], kF32, {(cols + 127) / 128, rows}, x);
  const at::Tensor cc = output(w, on, "col_codes", a[5], kU8, {ld, cols}, x);
  const at::Tensor cs = output(w, on, "col_scale", a[6], kF32, {ld / 128, cols}, x);
  const at::Tensor po = output(w, on, "padded_offsets", a[7], kI32, {g < 0 ? 0 : int64_t(g) + 1}, x);
  call(w, [&] {
    return quantize_fp8_block128_rowcol(ptr(x), rows, cols, off, g, ptr<uint8_t>(rc), ptr<float>(rs), ptr<uint8_t>(cc),
                                        ptr<float>(cs), ptr<int32_t>(po), st, on.raw());
  });
  return tuple({{a[3], rc}, {a[4], rs}, {a[5], cc}, {a[6], cs}, {a[7], po}});
}

// w, codes, scale, stream
PyObject *quantize_weights(PyObject *const *a) {
  Call w{"quantize_fp8_block128_weights"};
  const Shape s = dims(w, "w", a[0], 3);
  const int64_t e = s[0], n = s[1], k = s[2];
  const at::Tensor &x = input(w, "w", a[0], kBf16, {e, n, k});
  const OnStream on(w, a[3]);
  const at::Tensor codes = output(w, on, "codes", a[1], kU8, {e, n, k}, x);
  const at::Tensor scale = output(w, on, "scale", a[2], kF32, {e, (n + 127) / 128, (k + 127) / 128}, x);
  const int32_t experts = e > INT32_MAX ? INT32_MAX : static_cast<int32_t>(e);
  call(w, [&] {
    return quantize_fp8_block128_weights(ptr(x), experts, n, k, ptr<uint8_t>(codes), ptr<float>(scale), on.raw());
  });
  return tuple({{a[1], codes}, {a[2], scale}});
}

// -------------------------------------------------------------------- products --
// a_codes, a_scale, w_codes, w_scale, offsets, y, status, stream
template <bool kDgrad>
PyObject *rows_gemm(PyObject *const *a) {
  Call w{kDgrad ? "grouped_gemm_dgrad_fp8_block128" : "grouped_gemm_fwd_fp8_block128"};
  const Shape ws = dims(w, "w_codes", a[2], 3);
  const int64_t e = ws[0], n = ws[1], k = ws[2];
  const char *codes = kDgrad ? "dy_codes" : "a_codes";
  const int64_t m = dims(w, codes, a[0], 2)[0];
  const int64_t inner = kDgrad ? n : k, cols = kDgrad ? k : n;
  const at::Tensor &ac = input(w, codes, a[0], kU8, {m, inner});
  const at::Tensor &as = input(w, kDgrad ? "dy_scale" : "a_scale", a[1], kF32, {(inner + 127) / 128, m});
  const at::Tensor &wc = input(w, "w_codes", a[2], kU8, {e, n, k});
  const at::Tensor &wsc = input(w, "w_scale", a[3], kF32, {e, (n + 127) / 128, (k + 127) / 128});
  const at::Tensor &off = input(w, "offsets", a[4], kI32, {e + 1});
  int32_t *st = status_ptr(w, a[6]);
  const OnStream on(w, a[7]);
  const at::Tensor y = output(w, on, kDgrad ? "dx" : "y", a[5], kBf16, {m, cols}, ac);
  const int32_t experts = static_cast<int32_t>(e);
  call(w, [&] {
    return (kDgrad ? grouped_gemm_dgrad_fp8_block128 : grouped_gemm_fwd_fp8_block128)(
        ptr<uint8_t>(ac), ptr<float>(as), ptr<uint8_t>(wc), ptr<float>(wsc), ptr<int32_t>(off), experts, m, n, k, ptr(y),
        st, on.raw());
  });
  return one(a[5], y);
}

// dy_codes, dy_scale, x_codes, x_scale, padded_offsets, dw, mode (FME_DW_*), status, stream
PyObject *wgrad(PyObject *const *a) {
  Call w{"grouped_gemm_wgrad_fp8_block128"};
  const Shape ds = dims(w, "dy_codes", a[0], 2);
  const int64_t ld = ds[0], n = ds[1], k = dims(w, "x_codes", a[2], 2)[1];
  const int64_t e = dims(w, "padded_offsets", a[4], 1)[0] - 1;
  const at::Tensor &dc = input(w, "dy_codes", a[0], kU8, {ld, n});
  const at::Tensor &dsc = input(w, "dy_scale", a[1], kF32, {ld / 128, n});
  const at::Tensor &xc = input(w, "x_codes", a[2], kU8, {ld, k});
  const at::Tensor &xs = input(w, "x_scale", a[3], kF32, {ld / 128, k});
  const at::Tensor &po = input(w, "padded_offsets", a[4], kI32, {e + 1});
  const int32_t mode = integer32(a[6]);
  if (e < 1) throw Refused(std::string(w.where) + ": padded_offsets must have at least 2 elements");
  int32_t *st = status_ptr(w, a[7]);
  const OnStream on(w, a[8]);
  const at::Tensor dw = output(w, on, "dw", a[5], mode == FME_DW_BF16 ? kBf16 : kF32, {e, n, k}, dc);
  call(w, [&] {
    return grouped_gemm_wgrad_fp8_block128(ptr<uint8_t>(dc), ptr<float>(dsc), ptr<uint8_t>(xc), ptr<float>(xs), ld,
                                           ptr<int32_t>(po), static_cast<int32_t>(e), n, k, ptr(dw), mode, st,
                                           on.raw());
  });
  return one(a[5], dw);
}

// ---------------------------------------------------------------------- router --
struct Logits {
  const at::Tensor &t;
  int64_t tokens, experts;
  int32_t experts32, dtype;
};
Logits logits_of(Call &w, PyObject *o) {
  const Shape s = dims(w, "logits", o, 2);
  const at::Tensor &t = THPVariable_Unpack(o);
  const auto type = t.scalar_type();
  if (type != kBf16 && type != kF32)
    throw Refused(std::string(w.where) + ": logits must be bfloat16 or float32, got " + name_of(type));
  need(w, "logits", t, type, s);
  return {t, s[0], s[1], s[1] > INT32_MAX ? INT32_MAX : static_cast<int32_t>(s[1]), type == kBf16 ? FME_BF16 : FME_FP32};
}
int32_t score_of(const Call &w, PyObject *o) {
  const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  if (s && std::string(s) == "softmax") return FME_SCORE_SOFTMAX;
  if (s && std::string(s) == "sigmoid") return FME_SCORE_SIGMOID;
  PyErr_Clear();
  throw Refused(std::string(w.where) + ": score must be 'softmax' or 'sigmoid'");
}

// logits, top_k, score, bias, normalize, scale, ids, weights, stream
PyObject *gate(PyObject *const *a) {
  Call w{"moe_gate"};
  const Logits l = logits_of(w, a[0]);
  const int32_t top_k = integer32(a[1]), score = score_of(w, a[2]);
  const float *bias = a[3] == Py_None ? nullptr : ptr<float>(input(w, "bias", a[3], kF32, {l.experts}));
  if (top_k < 0) throw Refused(std::string(w.where) + ": top_k must not be negative");
  const OnStream on(w, a[8]);
  const at::Tensor ids = output(w, on, "ids", a[6], kI32, {l.tokens, top_k}, l.t);
  const at::Tensor weights = output(w, on, "weights", a[7], kF32, {l.tokens, top_k}, l.t);
  const int32_t normalize = truth(a[4]);
  const float scale = real(a[5]);
  call(w, [&] {
    return moe_gate(ptr(l.t), l.dtype, l.tokens, l.experts32, top_k, score, normalize, scale, bias, ptr<int32_t>(ids),
                    ptr<float>(weights), on.raw());
  });
  return tuple({{a[6], ids}, {a[7], weights}});
}

// logits, ids, d_weights, score, normalize, scale, d_logits, status, stream
PyObject *gate_backward(PyObject *const *a) {
  Call w{"moe_gate_backward"};
  const Logits l = logits_of(w, a[0]);
  const int64_t top_k = dims(w, "ids", a[1], 2)[1];
  const at::Tensor &ids = input(w, "ids", a[1], kI32, {l.tokens, top_k});
  const at::Tensor &d = input(w, "d_weights", a[2], kF32, {l.tokens, top_k});
  const int32_t score = score_of(w, a[3]), normalize = truth(a[4]);
  const float scale = real(a[5]);
  int32_t *st = status_ptr(w, a[7]);
  const OnStream on(w, a[8]);
  const at::Tensor out = output(w, on, "d_logits", a[6], l.t.scalar_type(), {l.tokens, l.experts}, l.t);
  const int32_t k = top_k > INT32_MAX ? INT32_MAX : static_cast<int32_t>(top_k);
  call(w, [&] {
    return moe_gate_backward(ptr(l.t), l.dtype, ptr<int32_t>(ids), ptr<float>(d), l.tokens, l.experts32, k, score,
                             normalize, scale, ptr(out), st, on.raw());
  });
  return one(a[6], out);
}

struct Sequences {
  const int32_t *offsets;
  int64_t count;
  const uint8_t *mask;
};
Sequences sequences_of(Call &w, PyObject *offsets, PyObject *mask, int64_t tokens) {
  Sequences s{nullptr, 1, nullptr};
  if (offsets != Py_None) {
    const int64_t n = dims(w, "seq_offsets", offsets, 1)[0];
    s.offsets = ptr<int32_t>(input(w, "seq_offsets", offsets, kI32, {n}));
    s.count = n - 1;
  }
  if (mask != Py_None) {
    const at::Tensor &t = tensor(w, "token_mask", mask);
    if (t.scalar_type() != at::kBool && t.scalar_type() != kU8)
      throw Refused(std::string(w.where) + ": token_mask must be bool or uint8, got " + name_of(t.scalar_type()));
    need(w, "token_mask", t, t.scalar_type(), {tokens});
    s.mask = ptr<uint8_t>(t);
  }
  return s;
}

// logits, ids, score, alpha, seq_offsets, token_mask, loss, counts, seq_tokens, workspace, status, stream
PyObject *balance_loss(PyObject *const *a) {
  Call w{"moe_balance_loss"};
  const Logits l = logits_of(w, a[0]);
  const int64_t top_k = dims(w, "ids", a[1], 2)[1];
  const at::Tensor &ids = input(w, "ids", a[1], kI32, {l.tokens, top_k});
  const int32_t score = score_of(w, a[2]);
  const float alpha = real(a[3]);
  const Sequences s = sequences_of(w, a[4], a[5], l.tokens);
  if (s.count < 1) throw Refused(std::string(w.where) + ": seq_offsets must have at least 2 elements");
  int32_t *st = status_ptr(w, a[10]);
  const OnStream on(w, a[11]);
  const at::Tensor loss = output(w, on, "loss", a[6], kF32, {1}, l.t);
  const at::Tensor counts = output(w, on, "counts", a[7], kI32, {s.count, l.experts}, l.t);
  const at::Tensor n = output(w, on, "seq_tokens", a[8], kI32, {s.count}, l.t);
  at::Tensor ws;
  if (a[9] == Py_None)
    ws = at::detail::empty_cuda({fme_balance_workspace_bytes(l.tokens, s.count, l.experts32)}, kU8, l.t.device(),
                                std::nullopt);
  else
    ws = tensor(w, "workspace", a[9]);
  if (!ws.is_cuda() || !ws.is_contiguous()) throw Refused(std::string(w.where) + ": workspace must be a contiguous CUDA tensor");
  on_one_device(w, "workspace", ws);
  const int32_t k = top_k > INT32_MAX ? INT32_MAX : static_cast<int32_t>(top_k);
  call(w, [&] {
    return moe_balance_loss(ptr(l.t), l.dtype, ptr<int32_t>(ids), l.tokens, l.experts32, k, score, alpha, s.offsets,
                            s.count, s.mask, ptr<float>(loss), ptr<int32_t>(counts), ptr<int32_t>(n), ptr(ws),
                            static_cast<int64_t>(ws.nbytes()), st, on.raw());
  });
  return tuple({{a[6], loss}, {a[7], counts}, {a[8], n}});
}

// logits, counts, seq_tokens, d_loss, top_k, score, alpha, seq_offsets, token_mask, d_logits, accumulate, stream
PyObject *balance_loss_backward(PyObject *const *a) {
  Call w{"moe_balance_loss_backward"};
  const Logits l = logits_of(w, a[0]);
  const Sequences s = sequences_of(w, a[7], a[8], l.tokens);
  const at::Tensor &counts = input(w, "counts", a[1], kI32, {s.count, l.experts});
  const at::Tensor &n = input(w, "seq_tokens", a[2], kI32, {s.count});
  const at::Tensor &d = input(w, "d_loss", a[3], kF32, {1});
  const int32_t top_k = integer32(a[4]), score = score_of(w, a[5]);
  const float alpha = real(a[6]);
  const bool accumulate = truth(a[10]);
  if (accumulate && a[9] == Py_None) throw Refused(std::string(w.where) + ": accumulate needs the d_logits to add to");
  const OnStream on(w, a[11]);
  const at::Tensor out = output(w, on, "d_logits", a[9], l.t.scalar_type(), {l.tokens, l.experts}, l.t);
  call(w, [&] {
    return moe_balance_loss_backward(ptr(l.t), l.dtype, ptr<int32_t>(counts), ptr<int32_t>(n), ptr<float>(d), l.tokens,
                                     l.experts32, top_k, score, alpha, s.offsets, s.count, s.mask, ptr(out), accumulate,
                                     on.raw());
  });
  return one(a[9], out);
}

// d_out, y, row_of, weights, d_y, d_weights, status, stream
PyObject *combine_backward(PyObject *const *a) {
  Call w{"moe_combine_backward"};
  const Shape ys = dims(w, "y", a[1], 2), rs = dims(w, "row_of", a[2], 2);
  const int64_t rows = ys[0], n = ys[1], tokens = rs[0], top_k = rs[1];
  const at::Tensor &d = input(w, "d_out", a[0], kBf16, {tokens, n});
  const at::Tensor &y = input(w, "y", a[1], kBf16, {rows, n});
  const at::Tensor &row_of = input(w, "row_of", a[2], kI32, {tokens, top_k});
  const at::Tensor &weights = input(w, "weights", a[3], kF32, {tokens, top_k});
  int32_t *st = status_ptr(w, a[6]);
  const OnStream on(w, a[7]);
  const at::Tensor dy = output(w, on, "d_y", a[4], kBf16, {rows, n}, y);
  const at::Tensor dw = output(w, on, "d_weights", a[5], kF32, {tokens, top_k}, y);
  const int32_t k = top_k > INT32_MAX ? INT32_MAX : static_cast<int32_t>(top_k);
  call(w, [&] {
    return moe_combine_backward(ptr(d), ptr(y), rows, ptr<int32_t>(row_of), ptr<float>(weights), tokens, k, n, ptr(dy),
                                ptr<float>(dw), st, on.raw());
  });
  return tuple({{a[4], dy}, {a[5], dw}});
}

// error class
PyObject *set_error(PyObject *, PyObject *cls) {
  Py_XDECREF(g_fme_error);
  Py_INCREF(cls);
  g_fme_error = cls;
  Py_RETURN_NONE;
}

template <int N, PyObject *(*F)(PyObject *const *)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<N, F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<7, quantize_rows>("quantize_rows"),
    method<8, quantize_cols>("quantize_cols"),
    method<10, quantize_rowcol>("quantize_rowcol"),
    method<4, quantize_weights>("quantize_weights"),
    method<8, rows_gemm<false>>("fwd"),
    method<8, rows_gemm<true>>("dgrad"),
    method<9, wgrad>("wgrad"),
    method<9, gate>("gate"),
    method<9, gate_backward>("gate_backward"),
    method<12, balance_loss>("balance_loss"),
    method<12, balance_loss_backward>("balance_loss_backward"),
    method<8, combine_backward>("combine_backward"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__binding(void) {
  PyObject *m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "built_for", FME_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
