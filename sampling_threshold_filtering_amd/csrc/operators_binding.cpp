// The language-model operators for Python: argument checks, output and scratch tensors and
// the library's call, in one compiled step.
//
// At the smallest sizes the GPU's part of a call is 3 to 5 us, and the same steps taken from
// Python (five tensors of 1.4 us each, checks, the foreign call) took 14 us of the caller's
// time for a router, 9 us for a gradient.
//
// Every function gets the current stream's handle last and returns its outputs, or the
// library's status as a number when that is not 0.  A wrong argument raises ValueError.
#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>

#include "profk.h"

namespace {

struct Refused {
  std::string text;
};

void refuse(const std::string& text) { throw Refused{text}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  return v;
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return v;
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(std::string(name) + " must be true or false");
  }
  return v;
}

// Forward-mode derivatives would be lost without a word.
void no_tangent(const at::Tensor& t, const char* name) {
  if (t.defined() && t._fw_grad(/*level=*/0).defined())
    refuse(std::string(name) + " has a forward-mode tangent, and this operator has no forward-mode derivative: detach it");
}

void* stream_of(PyObject* o) { return PyLong_AsVoidPtr(o); }

// torch's device allocator, as its own tensors have it; it allocates on the current device,
// which the caller has made the logits' one, for the current stream.
c10::Allocator* allocator(at::Device d) {
  static c10::Allocator* const a =
      at::Tensor(at::detail::empty_cuda({1}, at::kByte, d, std::nullopt)).storage().allocator();
  return a;
}

// A matrix of logits with unit column stride.
struct Logits {
  at::Tensor x;
  int dtype;
  int64_t rows, cols, ld;

  explicit Logits(PyObject* o) : x(tensor(o, "logits")) {
    const auto t = x.scalar_type();
    dtype = t == at::kFloat ? PROFK_FP32 : t == at::kHalf ? PROFK_FP16 : t == at::kBFloat16 ? PROFK_BF16 : -1;
    if (dtype < 0 || x.dim() != 2 || !x.is_cuda())
      refuse("logits must be a 2-D float32, float16 or bfloat16 device tensor");
    rows = x.size(0);
    cols = x.size(1);
    if (cols < 1) refuse("logits must have at least one column");
    // rows that overlap (broadcast ones too) or run backwards, and strided columns, are laid out anew
    if ((cols > 1 && x.stride(1) != 1) || (rows > 1 && x.stride(0) < cols)) x = x.contiguous();
    ld = rows > 1 ? x.stride(0) : cols;
    if (ld < cols) ld = cols;
  }
  // An output, with a storage of its own: kept, saved or resized, it takes no other one along.
  // Made without torch's dispatcher, which takes half of the 0.9 us of at::empty.
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::detail::empty_generic(shape, allocator(x.device()), c10::DispatchKeySet(c10::DispatchKey::CUDA), t,
                                     std::nullopt);
  }
};

// Scratch of one call, given back at its end: the allocator hands it out again behind the
// call's kernels, on their stream.  (A tensor for it takes 0.5 us more of the caller's time.)
struct Scratch {
  c10::DataPtr memory;
  int64_t bytes;
  Scratch(const Logits& like, int64_t n) : memory(allocator(like.x.device())->allocate(n)), bytes(n) {}
  void* get() const { return memory.get(); }
};

// A tensor of one dimension with n values of a type, unit stride; None: undefined.
at::Tensor vector(PyObject* o, const char* name, const char* what, int64_t n, at::ScalarType t, const Logits& like) {
  if (o == Py_None) return {};
  const at::Tensor& v = tensor(o, name);
  if (v.dim() != 1 || v.size(0) != n || v.scalar_type() != t || v.device() != like.x.device())
    refuse(std::string(name) + " must be " + std::to_string(n) + " " + what + " values on " + like.x.device().str());
  return n > 1 && v.stride(0) != 1 ? v.contiguous() : v;
}

at::Tensor shaped(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType t, const Logits& like) {
  const at::Tensor& v = tensor(o, name);
  if (v.sizes() != shape || v.scalar_type() != t || v.device() != like.x.device())
    refuse(std::string(name) + " must be a " + c10::toString(t) + " tensor of shape " + shape_text(shape) + " on " +
           like.x.device().str());
  return v.is_contiguous() ? v : v.contiguous();
}

template <class T>
T* address(const at::Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

PyObject* result(std::initializer_list<at::Tensor> out) {
  PyObject* r = PyTuple_New((Py_ssize_t)out.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : out) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

PyObject* status(int64_t rc) { return PyLong_FromLongLong(rc); }

int32_t scores_of(PyObject* o) {
  const char* text = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  if (!text) PyErr_Clear();
  if (text && !std::strcmp(text, "softmax")) return PROFK_SOFTMAX;
  if (text && !std::strcmp(text, "sigmoid")) return PROFK_SIGMOID;
  refuse("scores must be \"softmax\" or \"sigmoid\"");
  return 0;
}

float finite(PyObject* o, const char* name) {
  const double v = number(o, name);
  if (!(std::abs(v) < 3e38)) refuse(std::string(name) + " must be finite");
  return (float)v;
}

// A sampling setting: a number for all rows, or a tensor of one value per row.
struct Setting {
  at::Tensor rows;
  double value = 0;
  int64_t whole = 0;

  Setting(PyObject* o, const char* name, at::ScalarType t, const Logits& like) {
    const bool is_float = t == at::kFloat;
    if (!THPVariable_Check(o)) {
      if (is_float)
        value = number(o, name);
      else
        whole = integer(o, name);
      return;
    }
    const at::Tensor& v = THPVariable_Unpack(o);
    if (v.dim() != 1 || v.size(0) != like.rows || v.device() != like.x.device() ||
        v.is_floating_point() != is_float || v.is_complex() || v.scalar_type() == at::kBool)
      refuse(std::string(name) + " must be a number or a 1-D tensor of " + std::to_string(like.rows) + " values on " +
             like.x.device().str());
    rows = v.scalar_type() == t && (like.rows <= 1 || v.stride(0) == 1) ? v : v.to(t).contiguous();
  }
};

// sample(logits, u, temperature, top_k, top_p, min_p, out, stream)
PyObject* sample(PyObject* const* a) {
  const Logits x(a[0]);
  if (a[1] == Py_None) refuse("u must be a tensor");
  const at::Tensor u = vector(a[1], "u", "float32", x.rows, at::kFloat, x);
  const Setting t(a[2], "temperature", at::kFloat, x), k(a[3], "top_k", at::kLong, x),
      p(a[4], "top_p", at::kFloat, x), m(a[5], "min_p", at::kFloat, x);
  if (!(t.value >= 0 && k.whole >= 0 && p.value >= 0 && p.value <= 1 && m.value >= 0 && m.value <= 1))
    refuse("need temperature >= 0, top_k >= 0, 0 <= top_p <= 1 and 0 <= min_p <= 1");
  at::Tensor tokens, logprobs;
  if (a[6] == Py_None) {
    tokens = x.empty({x.rows}, at::kLong);
    logprobs = x.empty({x.rows}, at::kFloat);
  } else {
    if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 2) refuse("out must be (tokens, logprobs)");
    tokens = tensor(PyTuple_GET_ITEM(a[6], 0), "out[0]");
    logprobs = tensor(PyTuple_GET_ITEM(a[6], 1), "out[1]");
    const std::array<int64_t, 1> shape{x.rows};
    if (tokens.sizes() != at::IntArrayRef(shape) || logprobs.sizes() != at::IntArrayRef(shape) ||
        tokens.scalar_type() != at::kLong || logprobs.scalar_type() != at::kFloat ||
        tokens.device() != x.x.device() || logprobs.device() != x.x.device() || !tokens.is_contiguous() ||
        !logprobs.is_contiguous())
      refuse("out must be contiguous int64 / float32 tensors of shape " + shape_text(shape) + " on " +
             x.x.device().str());
  }
  const profk_sampling how = {(float)t.value,         (float)p.value,           (float)m.value,
                              0,                      k.whole,                  address<const float>(t.rows),
                              address<const int64_t>(k.rows), address<const float>(p.rows), address<const float>(m.rows)};
  const int rc = profk_sample_tokens(x.x.data_ptr(), x.dtype, x.rows, x.cols, x.ld, address<const float>(u), &how,
                                     address<int64_t>(tokens), address<float>(logprobs), nullptr, 0, stream_of(a[7]));
  return rc ? status(rc) : result({tokens, logprobs});
}

// route(logits, k, normalize, mask, balance, stream)
PyObject* route(PyObject* const* a) {
  const Logits x(a[0]);
  no_tangent(x.x, "logits");
  const int64_t k = integer(a[1], "k");
  if (k < 1 || k > x.cols) refuse("k must be in 1.." + std::to_string(x.cols));
  const bool normalize = truth(a[2], "normalize"), balance = truth(a[4], "balance");
  const at::Tensor mask = vector(a[3], "mask", "bool", x.rows, at::kBool, x);
  const int64_t need = profk_route_scratch(x.rows, x.cols);
  if (need < 0) return status(x.cols > PROFK_ROUTE_MAX_EXPERTS ? PROFK_EUNSUPPORTED : need);
  const Scratch scratch(x, need);
  const at::Tensor weights = x.empty({x.rows, k}, at::kFloat), experts = x.empty({x.rows, k}, at::kLong),
                   counts = x.empty({x.cols}, at::kLong), rows = x.empty({}, at::kLong),
                   loss = balance ? x.empty({}, at::kFloat) : at::Tensor();
  const int rc = profk_route_tokens(x.x.data_ptr(), x.dtype, x.rows, x.cols, x.ld, address<const uint8_t>(mask), k,
                                    normalize, address<float>(weights), address<int64_t>(experts),
                                    address<int64_t>(counts), address<int64_t>(rows), address<float>(loss),
                                    scratch.get(), scratch.bytes, stream_of(a[5]));
  return rc ? status(rc) : result({weights, experts, counts, rows, loss});
}

// A loss gradient given as a number or a one-element float32 tensor.
struct LossScale {
  at::Tensor value;
  double factor = 1;
  LossScale(PyObject* o, const Logits& like) {
    if (!THPVariable_Check(o)) {
      factor = number(o, "d_loss");
      return;
    }
    value = THPVariable_Unpack(o);
    if (value.numel() != 1 || value.scalar_type() != at::kFloat || value.device() != like.x.device())
      refuse("d_loss must be a number or one float32 value on " + like.x.device().str());
    no_tangent(value, "d_loss");
  }
};

// route_grad(logits, experts, counts, rows, d_weights, d_loss, normalize, mask, scores, scale, stream)
PyObject* route_grad(PyObject* const* a) {
  const Logits x(a[0]);
  no_tangent(x.x, "logits");
  const at::Tensor& choice = tensor(a[1], "experts");
  const int64_t k = choice.dim() == 2 ? choice.size(1) : 0;
  const at::Tensor mask = vector(a[7], "mask", "bool", x.rows, at::kBool, x);
  const bool normalize = truth(a[6], "normalize");
  const int32_t scores = scores_of(a[8]);
  const float scale = finite(a[9], "scale");
  at::Tensor experts, d_weights, counts, rows, d_loss;
  double factor = 0;
  if (a[4] != Py_None) {
    d_weights = shaped(a[4], "d_weights", {x.rows, k}, at::kFloat, x);
    no_tangent(d_weights, "d_weights");
    experts = shaped(a[1], "experts", {x.rows, k}, at::kLong, x);
  }
  if (a[5] != Py_None) {
    counts = shaped(a[2], "counts", {x.cols}, at::kLong, x);
    rows = shaped(a[3], "rows", {}, at::kLong, x);
    const LossScale s(a[5], x);
    d_loss = s.value;
    factor = s.factor;
  }
  const at::Tensor dx = x.empty({x.rows, x.cols}, x.x.scalar_type());
  const int rc = profk_route_scored_grad(x.x.data_ptr(), x.dtype, x.rows, x.cols, x.ld, address<const uint8_t>(mask), k,
                                         normalize, scores, scale, address<const int64_t>(experts),
                                         address<const float>(d_weights), address<const int64_t>(counts),
                                         address<const int64_t>(rows), address<const float>(d_loss), (float)factor,
                                         dx.data_ptr(), stream_of(a[10]));
  return rc ? status(rc) : THPVariable_Wrap(dx);
}

// scored(logits, k, normalize, mask, balance, scores, bias, groups, top_groups, group_best, scale, stream)
PyObject* scored(PyObject* const* a) {
  const Logits x(a[0]);
  no_tangent(x.x, "logits");
  const int64_t k = integer(a[1], "k");
  if (k < 1 || k > x.cols) refuse("k must be in 1.." + std::to_string(x.cols));
  const bool normalize = truth(a[2], "normalize"), balance = truth(a[4], "balance");
  const at::Tensor mask = vector(a[3], "mask", "bool", x.rows, at::kBool, x),
                   bias = vector(a[6], "bias", "float32", x.cols, at::kFloat, x);
  no_tangent(bias, "bias");
  const int64_t groups = integer(a[7], "groups"), top = a[8] == Py_None ? groups : integer(a[8], "top_groups"),
                best = integer(a[9], "group_best");
  if (groups < 1 || x.cols % groups) refuse("groups must divide the " + std::to_string(x.cols) + " experts");
  if (top < 1 || top > groups) refuse("top_groups must be in 1.." + std::to_string(groups));
  if (best != 1 && best != 2) refuse("group_best must be 1 or 2");
  const int32_t scores = scores_of(a[5]);
  const float scale = finite(a[10], "scale");
  const int64_t need = profk_route_scratch(x.rows, x.cols);
  if (need < 0) return status(x.cols > PROFK_ROUTE_MAX_EXPERTS ? PROFK_EUNSUPPORTED : need);
  if (groups > PROFK_ROUTE_MAX_GROUPS) return status(PROFK_EUNSUPPORTED);
  const Scratch scratch(x, need);
  const at::Tensor weights = x.empty({x.rows, k}, at::kFloat), experts = x.empty({x.rows, k}, at::kLong),
                   counts = x.empty({x.cols}, at::kLong), rows = x.empty({}, at::kLong),
                   loss = balance ? x.empty({}, at::kFloat) : at::Tensor();
  const profk_scoring how = {scores, (int32_t)groups, (int32_t)top, (int32_t)best, scale, normalize,
                             address<const float>(bias)};
  const int rc = profk_route_scored(x.x.data_ptr(), x.dtype, x.rows, x.cols, x.ld, address<const uint8_t>(mask), k,
                                    &how, address<float>(weights), address<int64_t>(experts),
                                    address<int64_t>(counts), address<int64_t>(rows), address<float>(loss),
                                    scratch.get(), scratch.bytes, stream_of(a[11]));
  return rc ? status(rc) : result({weights, experts, counts, rows, loss});
}

// balance(logits, experts, mask, stream)
PyObject* balance(PyObject* const* a) {
  const Logits x(a[0]);
  no_tangent(x.x, "logits");
  const at::Tensor& choice = tensor(a[1], "experts");
  if (choice.dim() != 2 || choice.size(1) < 1) refuse("experts must be a 2-D int64 tensor with a row per token");
  const int64_t k = choice.size(1);
  const at::Tensor experts = shaped(a[1], "experts", {x.rows, k}, at::kLong, x),
                   mask = vector(a[2], "mask", "bool", x.rows, at::kBool, x);
  const int64_t need = profk_route_scratch(x.rows, x.cols);
  if (need < 0) return status(x.cols > PROFK_ROUTE_MAX_EXPERTS ? PROFK_EUNSUPPORTED : need);
  const Scratch scratch(x, need);
  const at::Tensor counts = x.empty({x.cols}, at::kLong), rows = x.empty({}, at::kLong), loss = x.empty({}, at::kFloat);
  const int rc = profk_balance_loss(x.x.data_ptr(), x.dtype, x.rows, x.cols, x.ld, address<const uint8_t>(mask),
                                    address<const int64_t>(experts), k, address<int64_t>(counts),
                                    address<int64_t>(rows), address<float>(loss), scratch.get(), scratch.bytes,
                                    stream_of(a[3]));
  return rc ? status(rc) : result({loss, counts, rows});
}

// balance_grad(logits, k, counts, rows, d_loss, mask, stream)
PyObject* balance_grad(PyObject* const* a) {
  const Logits x(a[0]);
  no_tangent(x.x, "logits");
  const at::Tensor mask = vector(a[5], "mask", "bool", x.rows, at::kBool, x),
                   counts = shaped(a[2], "counts", {x.cols}, at::kLong, x),
                   rows = shaped(a[3], "rows", {}, at::kLong, x);
  const LossScale s(a[4], x);
  const at::Tensor dx = x.empty({x.rows, x.cols}, x.x.scalar_type());
  const int rc = profk_balance_loss_grad(x.x.data_ptr(), x.dtype, x.rows, x.cols, x.ld, address<const uint8_t>(mask),
                                         integer(a[1], "k"), address<const int64_t>(counts),
                                         address<const int64_t>(rows), address<const float>(s.value), (float)s.factor,
                                         dx.data_ptr(), stream_of(a[6]));
  return rc ? status(rc) : THPVariable_Wrap(dx);
}

double temperature_of(PyObject* o) {
  const double t = number(o, "temperature");
  if (!(t >= 0x1p-20 && t <= 0x1p20)) refuse("temperature must be within 2^-20 .. 2^20");
  return t;
}

// What the losses over given tokens have in common: one token per row, the mask, scratch.
struct TokenRows {
  Logits x;
  at::Tensor tokens, mask;
  double temperature;
  int64_t need;
  TokenRows(PyObject* logits, PyObject* tok, PyObject* m, PyObject* temp) : x(logits) {
    no_tangent(x.x, "logits");
    if (tok == Py_None) refuse("tokens must be a tensor");
    tokens = vector(tok, "tokens", "int64", x.rows, at::kLong, x);
    mask = vector(m, "mask", "bool", x.rows, at::kBool, x);
    temperature = temperature_of(temp);
    need = profk_token_loss_scratch(x.rows, x.cols);
  }
  at::Tensor row_values(PyObject* o, const char* name, bool needed) const {
    if (needed && o == Py_None) refuse(std::string(name) + " must be a tensor");
    const at::Tensor v = vector(o, name, "float32", x.rows, at::kFloat, x);
    no_tangent(v, name);
    return v;
  }
};

// token_logprobs(logits, tokens, mask, temperature, stream)
PyObject* token_logprobs(PyObject* const* a) {
  const TokenRows r(a[0], a[1], a[2], a[3]);
  if (r.need < 0) return status(PROFK_EUNSUPPORTED);
  const Scratch scratch(r.x, r.need);
  const at::Tensor logprobs = r.x.empty({r.x.rows}, at::kFloat);
  const int rc = profk_token_logprobs(r.x.x.data_ptr(), r.x.dtype, r.x.rows, r.x.cols, r.x.ld,
                                      address<const int64_t>(r.tokens), address<const uint8_t>(r.mask), r.temperature,
                                      address<float>(logprobs), scratch.get(), scratch.bytes, stream_of(a[4]));
  return rc ? status(rc) : THPVariable_Wrap(logprobs);
}

// token_logprobs_grad(logits, tokens, d_logprobs, d_loss, mask, temperature, stream)
PyObject* token_logprobs_grad(PyObject* const* a) {
  const TokenRows r(a[0], a[1], a[4], a[5]);
  if (r.need < 0) return status(PROFK_EUNSUPPORTED);
  const at::Tensor d = r.row_values(a[2], "d_logprobs", true);
  const LossScale s(a[3], r.x);
  const Scratch scratch(r.x, r.need);
  const at::Tensor dx = r.x.empty({r.x.rows, r.x.cols}, r.x.x.scalar_type());
  const int rc = profk_token_logprobs_grad(
      r.x.x.data_ptr(), r.x.dtype, r.x.rows, r.x.cols, r.x.ld, address<const int64_t>(r.tokens),
      address<const uint8_t>(r.mask), r.temperature, address<const float>(d), address<const float>(s.value),
      (float)s.factor, dx.data_ptr(), scratch.get(), scratch.bytes, stream_of(a[6]));
  return rc ? status(rc) : THPVariable_Wrap(dx);
}

// policy(logits, tokens, old, advantages, ref, weights, mask, clip_low, clip_high, kl_weight, temperature, d_loss,
// stream); d_loss None: no gradient
PyObject* policy(PyObject* const* a) {
  const TokenRows r(a[0], a[1], a[6], a[10]);
  if (r.need < 0) return status(PROFK_EUNSUPPORTED);
  const at::Tensor old = r.row_values(a[2], "old_logprobs", true), adv = r.row_values(a[3], "advantages", true),
                   ref = r.row_values(a[4], "ref_logprobs", false), weights = r.row_values(a[5], "weights", false);
  const double low = number(a[7], "clip_low"), high = number(a[8], "clip_high"), kl = number(a[9], "kl_weight");
  if (!(low >= 0 && high >= 0 && kl >= 0 && std::isfinite(kl))) refuse("need clip_low >= 0, clip_high >= 0 and a finite kl_weight >= 0");
  if (kl > 0 && !ref.defined()) refuse("a kl_weight needs ref_logprobs");
  const bool grad = a[11] != Py_None;
  at::Tensor d_loss, dx;
  double factor = 1;
  if (grad) {
    const LossScale s(a[11], r.x);
    d_loss = s.value;
    factor = s.factor;
    dx = r.x.empty({r.x.rows, r.x.cols}, r.x.x.scalar_type());
  }
  const Scratch scratch(r.x, r.need);
  const at::Tensor loss = r.x.empty({}, at::kFloat), logprobs = r.x.empty({r.x.rows}, at::kFloat),
                   gap = r.x.empty({}, at::kFloat), clipped = r.x.empty({}, at::kLong), rows = r.x.empty({}, at::kLong);
  const profk_policy how = {address<const float>(old), address<const float>(adv), address<const float>(ref),
                            address<const float>(weights), low, high, kl};
  const int rc = profk_policy_loss(
      r.x.x.data_ptr(), r.x.dtype, r.x.rows, r.x.cols, r.x.ld, address<const int64_t>(r.tokens),
      address<const uint8_t>(r.mask), r.temperature, &how, address<float>(loss), address<float>(gap),
      address<int64_t>(clipped), address<int64_t>(rows), address<float>(logprobs), address<const float>(d_loss),
      (float)factor, address<void>(dx), scratch.get(), scratch.bytes, stream_of(a[12]));
  return rc ? status(rc) : result({loss, logprobs, gap, clipped, rows, dx});
}

// preference(logits, tokens, offsets, ref, mask, beta, smoothing, margin, average, temperature, stream)
PyObject* preference(PyObject* const* a) {
  const TokenRows r(a[0], a[1], a[4], a[9]);
  if (r.need < 0) return status(PROFK_EUNSUPPORTED);
  at::Tensor offsets = tensor(a[2], "offsets");
  if (offsets.dim() != 1 || offsets.size(0) < 3 || offsets.size(0) % 2 == 0 || offsets.scalar_type() != at::kLong ||
      offsets.device() != r.x.x.device())
    refuse("offsets must be 2 * pairs + 1 int64 values on " + r.x.x.device().str());
  offsets = offsets.contiguous();
  const int64_t pairs = offsets.size(0) / 2;
  const at::Tensor ref = r.row_values(a[3], "ref_logprobs", false);
  const double beta = number(a[5], "beta"), smoothing = number(a[6], "smoothing"), margin = number(a[7], "margin");
  if (!(std::isfinite(beta) && std::isfinite(margin) && smoothing >= 0 && smoothing <= 1))
    refuse("need a finite beta and margin and 0 <= smoothing <= 1");
  const profk_preference how = {address<const int64_t>(offsets), address<const float>(ref), pairs, beta, smoothing, margin,
                                truth(a[8], "average"), 0};
  const Scratch scratch(r.x, r.need);
  const at::Tensor loss = r.x.empty({}, at::kFloat), margins = r.x.empty({pairs}, at::kFloat),
                   sums = r.x.empty({2 * pairs}, at::kFloat), rows = r.x.empty({}, at::kLong),
                   logprobs = r.x.empty({r.x.rows}, at::kFloat), coefficients = r.x.empty({r.x.rows}, at::kFloat);
  const int rc = profk_preference_loss(
      r.x.x.data_ptr(), r.x.dtype, r.x.rows, r.x.cols, r.x.ld, address<const int64_t>(r.tokens),
      address<const uint8_t>(r.mask), r.temperature, &how, address<float>(loss), address<float>(margins),
      address<float>(sums), address<int64_t>(rows), address<float>(logprobs), address<float>(coefficients),
      scratch.get(), scratch.bytes, stream_of(a[10]));
  return rc ? status(rc) : result({loss, margins, sums, rows, logprobs, coefficients});
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)(void))call<F, N>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<sample, 8>("sample"),       method<route, 6>("route"), method<scored, 12>("scored"),
                         method<route_grad, 11>("route_grad"), method<balance, 4>("balance"),
                         method<balance_grad, 7>("balance_grad"),
                         method<token_logprobs, 5>("token_logprobs"),
                         method<token_logprobs_grad, 7>("token_logprobs_grad"), method<policy, 13>("policy"),
                         method<preference, 11>("preference"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operators", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__operators() { return PyModule_Create(&module); }
