// torch_bind.cpp -- argument checks, output allocation and marshalling of the operators in block.py
// and of optim.AdamW's calls, as a CPython extension over the C ABI.  These operators take a few
// microseconds on the GPU, less than the same checks and allocations take in Python: a forward of
// the residual norm took 19 us of host time there and 6 to 7 here.  Nothing is computed here.
//
// Every function takes its arguments by position, in the order of its caller in block.py, which
// documents them.  A wrong argument raises ValueError, a status of the library QLoraError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <sstream>
#include <utility>

#include "../../include/qlora_nf4.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // abi.QLoraError

// A status raised as QLoraError(function, code); false where there is nothing to raise.
bool failed(const char* fn, qlora_status st) {
  if (st == QLORA_OK) return false;
  PyObject* e = PyObject_CallFunction(g_error, "si", fn, static_cast<int>(st));
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return true;
}

// An optional tensor argument; the reference stays with the caller's tuple.
const Tensor* opt(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
  return &THPVariable_Unpack(o);
}
const Tensor& need(PyObject* o, const char* name) {
  const Tensor* t = opt(o, name);
  TORCH_CHECK_VALUE(t, name, ": expected a tensor, got None");
  return *t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

std::string shown(const Tensor& t) {
  std::ostringstream s;
  s << t.scalar_type() << " " << t.sizes() << " (strides " << t.strides() << ") on " << t.device();
  return s.str();
}
bool here(const Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
bool either(at::ScalarType t) { return t == kBf16 || t == kF32; }

// Contiguous, on the current device, of this type (Undefined: bf16 or fp32) and shape.
void want(const Tensor& t, at::ScalarType type, at::IntArrayRef shape, const char* name, int dev) {
  const auto have = t.scalar_type();
  const bool ok = (type == at::ScalarType::Undefined ? either(have) : have == type) &&
                  t.sizes() == shape && t.is_contiguous() && here(t, dev);
  if (!ok)
    TORCH_CHECK_VALUE(false, name, ": expected contiguous ",
                      type == at::ScalarType::Undefined ? "bf16 or fp32" : c10::toString(type), " ",
                      shape, " on the current CUDA device ", dev, ", got ", shown(t));
}
constexpr auto kEither = at::ScalarType::Undefined;

Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, dev), std::nullopt);
}
// A given output, checked, or a new one.
Tensor out(const Tensor* given, at::IntArrayRef shape, at::ScalarType type, const char* name,
           int dev) {
  if (!given) return fresh(shape, type, dev);
  want(*given, type, shape, name, dev);
  return *given;
}

// Address, null for no tensor.  An empty tensor's is null too: with no tokens the library looks at
// no data, but tells what is there by its pointer.
constexpr uintptr_t kNoData = 16;
void* ptr(const Tensor* t) {
  if (!t) return nullptr;
  void* p = const_cast<void*>(t->const_data_ptr());
  return p || t->numel() ? p : reinterpret_cast<void*>(kNoData);
}
void* ptr(const Tensor& t) { return t.defined() ? ptr(&t) : nullptr; }
template <typename T>
T* as(void* p) {
  return static_cast<T*>(p);
}

qlora_stream_t stream(int dev) {
  return static_cast<qlora_stream_t>(
      c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}

// The bytes of a contiguous tensor, empty for none.
std::pair<uintptr_t, uintptr_t> span(const Tensor* t) {
  if (!t || !t->defined()) return {0, 0};
  const auto p = reinterpret_cast<uintptr_t>(t->const_data_ptr());
  return {p, p + t->nbytes()};
}
// Given outputs share no memory with the inputs or with each other, but as a pair of `same` says
// {output, input}: those may start at the same address.
struct Named {
  const char* name;
  const Tensor* t;
};
void apart(at::ArrayRef<Named> outs, at::ArrayRef<Named> ins,
           at::ArrayRef<std::pair<const Tensor*, const Tensor*>> same) {
  auto meet = [](const Tensor* a, const Tensor* b) {
    const auto x = span(a), y = span(b);
    return x.first < y.second && y.first < x.second;
  };
  for (size_t i = 0; i < outs.size(); ++i) {
    const Tensor* o = outs[i].t;
    if (!o) continue;
    for (const Named& in : ins)
      if (meet(o, in.t)) {
        bool allowed = false;
        for (const auto& [a, b] : same)
          allowed |= a == o && b == in.t && span(a) == span(b);
        TORCH_CHECK_VALUE(allowed, outs[i].name, ": shares memory with ", in.name);
      }
    for (size_t j = 0; j < i; ++j)
      TORCH_CHECK_VALUE(!meet(o, outs[j].t), outs[i].name, ": shares memory with ", outs[j].name);
  }
}

// New references into a tuple; undefined tensors as None, a given tensor as the object it came as.
PyObject* object(const Tensor& t, PyObject* given) {
  if (given && given != Py_None) return Py_NewRef(given);
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

// The weights and the gate that both directions share.
struct Norm {
  const Tensor *w_pre, *w_post, *gate;
  int types, kind;
};
Norm norm_args(PyObject* w_pre, PyObject* w_post, PyObject* gate, at::ScalarType resid, int64_t M,
               int64_t D, int dev) {
  Norm n = {opt(w_pre, "w_pre"), opt(w_post, "w_post"), opt(gate, "gate"),
            resid == kF32 ? QLORA_F32_RESIDUAL : 0, QLORA_GATE_NONE};
  if (n.w_pre) want(*n.w_pre, kEither, {D}, "w_pre", dev);
  if (n.w_post) want(*n.w_post, n.w_pre ? n.w_pre->scalar_type() : kEither, {D}, "w_post", dev);
  const Tensor* w = n.w_pre ? n.w_pre : n.w_post;
  if (w && w->scalar_type() == kF32) n.types |= QLORA_F32_WEIGHTS;
  if (n.gate) {
    const Tensor& g = *n.gate;
    if (g.dim() == 1) {
      n.kind = QLORA_GATE_CHANNEL;
      want(g, kEither, {D}, "gate", dev);
    } else if (g.dim() == 2 && g.size(1) == 1 && D > 1) {
      n.kind = QLORA_GATE_TOKEN;
      want(g, kEither, {M, 1}, "gate", dev);
    } else {
      n.kind = QLORA_GATE_FULL;
      want(g, kEither, {M, D}, "gate", dev);
    }
    if (g.scalar_type() == kF32) n.types |= QLORA_F32_GATE;
  }
  return n;
}

int count(const char* fn, Py_ssize_t have, Py_ssize_t wanted) {
  TORCH_CHECK_TYPE(have == wanted, fn, ": ", wanted, " arguments, got ", have);
  return 0;
}

// (h, y, w_pre, w_post, gate, eps, res_scale, branch_scale, weight_offset, h_out, n, rstd_pre,
//  rstd_post, save_rstd)
PyObject* residual_norm_forward(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS
  count("residual_norm_forward", na, 14);
  const int dev = c10::cuda::current_device();
  const Tensor& h = need(a[0], "h");
  TORCH_CHECK_VALUE(h.dim() == 2, "h: expected [M, D], got ", shown(h));
  const int64_t M = h.size(0), D = h.size(1);
  const auto R = h.scalar_type();
  want(h, kEither, {M, D}, "h", dev);
  const Norm w = norm_args(a[2], a[3], a[4], R, M, D, dev);
  const Tensor* y = opt(a[1], "y");
  const Tensor *given_h = opt(a[9], "h_out"), *given_n = opt(a[10], "n"),
               *given_pre = opt(a[11], "rstd_pre"), *given_post = opt(a[12], "rstd_post");
  const double res = number(a[6]), br = number(a[7]);
  const bool save = truth(a[13]);
  Tensor h_out, n, rstd_pre, rstd_post;
  if (!y) {
    TORCH_CHECK_VALUE(w.w_pre, "residual_norm_forward: nothing to do without y and w_pre");
    TORCH_CHECK_VALUE(!w.w_post && !w.gate && !given_h,
                      "residual_norm_forward: w_post, gate and h_out need y");
    TORCH_CHECK_VALUE(res == 1.0 && br == 1.0, "residual_norm_forward: the scales need y");
  } else {
    want(*y, kBf16, {M, D}, "y", dev);
    h_out = out(given_h, {M, D}, R, "h_out", dev);
  }
  if (w.w_pre) {
    n = out(given_n, {M, D}, kBf16, "n", dev);
    if (given_pre || save) rstd_pre = out(given_pre, {M}, kF32, "rstd_pre", dev);
  } else {
    TORCH_CHECK_VALUE(!given_n && !given_pre, "residual_norm_forward: n and rstd_pre need w_pre");
  }
  if (w.w_post) {
    if (given_post || save) rstd_post = out(given_post, {M}, kF32, "rstd_post", dev);
  } else {
    TORCH_CHECK_VALUE(!given_post, "residual_norm_forward: rstd_post needs w_post");
  }
  TORCH_CHECK_VALUE(D <= INT32_MAX, "h: too wide");
  if (given_h || given_n || given_pre || given_post)
    apart({{"h_out", given_h}, {"n", given_n}, {"rstd_pre", given_pre}, {"rstd_post", given_post}},
          {{"h", &h}, {"y", y}, {"w_pre", w.w_pre}, {"w_post", w.w_post}, {"gate", w.gate}},
          {{given_h, &h}, {given_n, y}});
  if (failed("qlora_residual_norm_fwd",
             qlora_residual_norm_fwd(ptr(h), ptr(y), ptr(w.w_pre), ptr(w.w_post), ptr(w.gate),
                                     w.kind, M, static_cast<int>(D), w.types,
                                     static_cast<float>(number(a[5])), static_cast<float>(res),
                                     static_cast<float>(br), static_cast<float>(number(a[8])),
                                     ptr(h_out), ptr(n), as<float>(ptr(rstd_pre)),
                                     as<float>(ptr(rstd_post)), stream(dev))))
    return nullptr;
  PyObject* t = PyTuple_New(4);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, y ? object(h_out, a[9]) : Py_NewRef(a[0]));
  PyTuple_SET_ITEM(t, 1, object(n, a[10]));
  PyTuple_SET_ITEM(t, 2, object(rstd_pre, a[11]));
  PyTuple_SET_ITEM(t, 3, object(rstd_post, a[12]));
  return t;
  END_HANDLE_TH_ERRORS
}

// (dn, dh_out, h_out, y, rstd_pre, rstd_post, w_pre, w_post, gate, res_scale, branch_scale,
//  weight_offset, need_dw, need_dgate, branch, dh, dy, dw_pre, dw_post, dgate, ws)
PyObject* residual_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS
  count("residual_norm_backward", na, 21);
  const int dev = c10::cuda::current_device();
  const Tensor *dn = opt(a[0], "dn"), *dh_out = opt(a[1], "dh_out"), *h_out = opt(a[2], "h_out"),
               *y = opt(a[3], "y"), *rstd_pre = opt(a[4], "rstd_pre"),
               *rstd_post = opt(a[5], "rstd_post");
  const Tensor* lead = dh_out ? dh_out : h_out;
  const char* lead_name = dh_out ? "dh_out" : "h_out";
  TORCH_CHECK_VALUE(lead,
                    "residual_norm_backward: one of dh_out and h_out gives the residual's type");
  TORCH_CHECK_VALUE(lead->dim() == 2, lead_name, ": expected [M, D], got ", shown(*lead));
  const int64_t M = lead->size(0), D = lead->size(1);
  const auto R = lead->scalar_type();
  want(*lead, kEither, {M, D}, lead_name, dev);
  const Norm w = norm_args(a[6], a[7], a[8], R, M, D, dev);
  if (w.w_pre) {
    TORCH_CHECK_VALUE(dn && h_out && rstd_pre,
                      "residual_norm_backward: w_pre needs dn, h_out and rstd_pre");
    want(*dn, kBf16, {M, D}, "dn", dev);
    want(*h_out, R, {M, D}, "h_out", dev);
    want(*rstd_pre, kF32, {M}, "rstd_pre", dev);
  } else {
    TORCH_CHECK_VALUE(!dn, "residual_norm_backward: dn needs w_pre");
    TORCH_CHECK_VALUE(dh_out, "residual_norm_backward: no gradient comes in");
  }
  const bool branch = a[14] == Py_None ? (y || w.gate || w.w_post) : truth(a[14]);
  const bool need_dw = truth(a[12]), need_dgate = truth(a[13]) && w.gate;
  if (y)
    want(*y, kBf16, {M, D}, "y", dev);
  else
    TORCH_CHECK_VALUE(!w.w_post && !need_dgate,
                      "residual_norm_backward: w_post and the gate's gradient need y");
  TORCH_CHECK_VALUE(branch || (!w.gate && !w.w_post && !y),
                    "residual_norm_backward: y, gate and w_post belong to a branch");
  if (w.w_post) {
    TORCH_CHECK_VALUE(rstd_post, "residual_norm_backward: w_post needs rstd_post");
    want(*rstd_post, kF32, {M}, "rstd_post", dev);
  }
  TORCH_CHECK_VALUE(D <= INT32_MAX, lead_name, ": too wide");
  Tensor dy, dw_pre, dw_post, dgate, ws;
  Tensor dh = out(opt(a[15], "dh"), {M, D}, R, "dh", dev);
  if (branch) dy = out(opt(a[16], "dy"), {M, D}, kBf16, "dy", dev);
  if (need_dw && w.w_pre) dw_pre = out(opt(a[17], "dw_pre"), {D}, kF32, "dw_pre", dev);
  if (need_dw && w.w_post) dw_post = out(opt(a[18], "dw_post"), {D}, kF32, "dw_post", dev);
  if (need_dgate) {
    const Tensor* g = opt(a[19], "dgate");
    dgate = w.kind == QLORA_GATE_CHANNEL ? out(g, {D}, kF32, "dgate", dev)
            : w.kind == QLORA_GATE_TOKEN ? out(g, {M, 1}, kF32, "dgate", dev)
                                         : out(g, {M, D}, w.gate->scalar_type(), "dgate", dev);
  }
  bool given = false;
  for (int i = 15; i < 21; ++i) given |= a[i] != Py_None;
  if (given) {
    auto of = [&](int i, const Tensor& used) { return used.defined() ? opt(a[i], "") : nullptr; };
    const Tensor *gh = of(15, dh), *gy = of(16, dy);
    apart({{"dh", gh}, {"dy", gy}, {"dw_pre", of(17, dw_pre)}, {"dw_post", of(18, dw_post)},
           {"dgate", of(19, dgate)}, {"ws", opt(a[20], "ws")}},
          {{"dn", dn}, {"dh_out", dh_out}, {"h_out", h_out}, {"y", y}, {"rstd_pre", rstd_pre},
           {"rstd_post", rstd_post}, {"w_pre", w.w_pre}, {"w_post", w.w_post}, {"gate", w.gate}},
          {{gh, dh_out}, {gy, y}, {gy, dn}});
  }
  size_t ws_bytes = 0;
  if (dw_pre.defined() || dw_post.defined() ||
      (dgate.defined() && w.kind == QLORA_GATE_CHANNEL)) {
    if (const Tensor* given = opt(a[20], "ws")) {
      TORCH_CHECK_VALUE(given->scalar_type() == at::kByte && given->is_contiguous() &&
                            here(*given, dev),
                        "ws: expected contiguous uint8 on the current CUDA device, got ",
                        shown(*given));
      ws = *given;
    } else if (M > 0) {
      ws = fresh({static_cast<int64_t>(
                     qlora_residual_norm_workspace_bytes(M, static_cast<int>(D)))},
                 at::kByte, dev);
    }
    ws_bytes = ws.defined() ? static_cast<size_t>(ws.numel()) : 0;
  }
  if (failed("qlora_residual_norm_bwd",
             qlora_residual_norm_bwd(
                 ptr(dn), ptr(dh_out), w.w_pre ? ptr(h_out) : nullptr, ptr(y),
                 w.w_pre ? as<float>(ptr(rstd_pre)) : nullptr,
                 w.w_post ? as<float>(ptr(rstd_post)) : nullptr, ptr(w.w_pre), ptr(w.w_post),
                 ptr(w.gate), w.kind, M, static_cast<int>(D), w.types,
                 static_cast<float>(number(a[9])), static_cast<float>(number(a[10])),
                 static_cast<float>(number(a[11])), ptr(dh), ptr(dy), as<float>(ptr(dw_pre)),
                 as<float>(ptr(dw_post)), ptr(dgate), ptr(ws), ws_bytes, stream(dev))))
    return nullptr;
  PyObject* t = PyTuple_New(5);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, object(dh, a[15]));
  PyTuple_SET_ITEM(t, 1, object(dy, dy.defined() ? a[16] : nullptr));
  PyTuple_SET_ITEM(t, 2, object(dw_pre, dw_pre.defined() ? a[17] : nullptr));
  PyTuple_SET_ITEM(t, 3, object(dw_post, dw_post.defined() ? a[18] : nullptr));
  PyTuple_SET_ITEM(t, 4, object(dgate, dgate.defined() ? a[19] : nullptr));
  return t;
  END_HANDLE_TH_ERRORS
}

// A tensor of heads as [B, S, n, head_dim].
struct Heads {
  int64_t B, S, n, batch, token, head;
};
Heads heads_of(const Tensor& x, int64_t n_heads, int64_t hd, const char* name, int dev) {
  TORCH_CHECK_VALUE(here(x, dev), name, ": expected a tensor on the current CUDA device ", dev,
                    ", got ", x.device());
  Heads h = {1, 0, 0, 0, 0, 0};
  bool ok = false;
  const int64_t d = x.dim();
  if (d == 2) {
    h.n = n_heads < 0 ? x.size(1) / hd : n_heads;
    ok = h.n * hd <= x.size(1) && (n_heads >= 0 || x.size(1) % hd == 0);
    h.S = x.size(0);
    h.token = x.stride(0);
    h.head = hd;
  } else if (d == 3 || d == 4) {
    h.n = n_heads < 0 ? x.size(d - 2) : n_heads;
    ok = x.size(d - 1) == hd && h.n <= x.size(d - 2);
    h.S = x.size(d - 3);
    h.token = x.stride(d - 3);
    h.head = x.stride(d - 2);
    if (d == 4) {
      h.B = x.size(0);
      h.batch = x.stride(0);
    }
  }
  if (!ok || h.n < 1 || (x.numel() && x.stride(d - 1) != 1))
    TORCH_CHECK_VALUE(false, name, ": expected [M, n * ", hd, "], [M, n, ", hd, "] or [B, S, n, ",
                      hd, "] with unit stride in the head and n >= ", std::max<int64_t>(n_heads, 1),
                      ", got ", shown(x));
  return h;
}
// Whether no two elements share an address, as far as sorted strides tell.
bool distinct(const Heads& h, int64_t hd) {
  std::pair<int64_t, int64_t> d[3] = {{h.batch, h.B}, {h.token, h.S}, {h.head, h.n}};
  std::sort(d, d + 3);
  int64_t reach = hd;
  for (const auto& [stride, size] : d) {
    if (size <= 1) continue;
    if (stride < reach) return false;
    reach += stride * (size - 1);
  }
  return true;
}

// The distance from the first element of the heads to behind the last.
int64_t reach(const Heads& h, int64_t hd) {
  return h.B && h.S ? (h.B - 1) * h.batch + (h.S - 1) * h.token + (h.n - 1) * h.head + hd : 0;
}
// Whether two tensors of heads share no element: apart altogether, or in different parts of one of
// the strides (such as of a packed row), of which all strides that reach further are multiples.
bool apart(const Tensor& x, const Heads& a, const Tensor& y, const Heads& b, int64_t hd) {
  const auto e = static_cast<int64_t>(x.element_size());
  const auto p = reinterpret_cast<intptr_t>(x.const_data_ptr()),
             q = reinterpret_cast<intptr_t>(y.const_data_ptr());
  if (p + reach(a, hd) * e <= q || q + reach(b, hd) * e <= p) return true;
  for (const int64_t s : {a.head, a.token, a.batch}) {
    if (s < 1) continue;
    auto part = [&](const Heads& h) {
      int64_t r = hd;
      if (h.B > 1 && h.batch % s) r += (h.B - 1) * h.batch;
      if (h.S > 1 && h.token % s) r += (h.S - 1) * h.token;
      if (h.n > 1 && h.head % s) r += (h.n - 1) * h.head;
      return r * e;
    };
    const int64_t d = ((q - p) % (s * e) + s * e) % (s * e);
    if (d >= part(a) && d + part(b) <= s * e) return true;
  }
  return false;
}

// (x, positions, phase, scale, head_dim, rotary_dim, interleaved, n_heads, k, n_heads_k, inverse,
//  inplace, out, out_k)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS
  count("rope", na, 14);
  const int dev = c10::cuda::current_device();
  const Tensor& x = need(a[0], "x");
  const Tensor* k = opt(a[8], "k");
  const Tensor& phase = need(a[2], "plan.phase");
  const int64_t hd = integer(a[4]), rd = integer(a[5]);
  const auto type = x.scalar_type();
  TORCH_CHECK_VALUE(hd >= 2 && rd >= 2 && rd <= hd, "plan: a head of ", hd, " with ", rd,
                    " rotary elements");
  TORCH_CHECK_VALUE(either(type), "x: expected bf16 or fp32, got ", type);
  auto heads_arg = [](PyObject* o) { return o == Py_None ? int64_t{-1} : integer(o); };
  if (a[7] != Py_None)
    TORCH_CHECK_VALUE(integer(a[7]) >= 1, "n_heads: expected at least 1, got ", integer(a[7]));
  const Tensor* given[2] = {opt(a[12], "out"), opt(a[13], "out_k")};
  TORCH_CHECK_VALUE(k || (!given[1] && a[9] == Py_None), "rope: out_k and n_heads_k need k");
  TORCH_CHECK_VALUE(here(phase, dev) && phase.scalar_type() == at::kLong &&
                        phase.is_contiguous() && phase.numel() == rd / 2,
                    "plan: expected its phases on the current CUDA device ", dev, ", got ",
                    shown(phase));
  const bool inplace = truth(a[11]) && !given[0] && !given[1];
  const Tensor* in[2] = {&x, k};
  static const char* names[2] = {"x", "k"};
  static const char* out_names[2] = {"out", "out_k"};
  qlora_rope_heads q[2];
  Tensor outs[2];
  Heads from[2], to[2];
  int64_t B = 0, S = 0;
  for (int i = 0; i < (k ? 2 : 1); ++i) {
    const Tensor& t = *in[i];
    TORCH_CHECK_VALUE(t.scalar_type() == type, names[i], ": expected ", type, " as x, got ",
                      t.scalar_type());
    const Heads h = heads_of(t, heads_arg(a[i ? 9 : 7]), hd, names[i], dev);
    if (i == 0) {
      B = h.B;
      S = h.S;
    }
    TORCH_CHECK_VALUE(h.B == B && h.S == S, names[i], ": expected ", B, " x ", S,
                      " tokens as x, got ", h.B, " x ", h.S);
    Heads o = h;
    if (inplace) {
      outs[i] = t;
    } else {
      c10::SmallVector<int64_t, 4> shape;
      if (t.dim() == 2) {
        shape = {S, h.n * hd};
      } else {
        if (t.dim() == 4) shape.push_back(B);
        shape.append({S, h.n, hd});
      }
      if (given[i]) {
        TORCH_CHECK_VALUE(given[i]->scalar_type() == type &&
                              given[i]->sizes() == at::IntArrayRef(shape),
                          out_names[i], ": expected ", type, " ", at::IntArrayRef(shape),
                          ", got ", shown(*given[i]));
        outs[i] = *given[i];
      } else {
        outs[i] = fresh(shape, type, dev);
      }
      o = heads_of(outs[i], h.n, hd, out_names[i], dev);
    }
    TORCH_CHECK_VALUE(distinct(o, hd), "rope: elements of ", inplace ? names[i] : out_names[i],
                      " share an address");
    TORCH_CHECK_VALUE(h.n <= INT32_MAX, names[i], ": too many heads");
    from[i] = h;
    to[i] = o;
    q[i] = {ptr(t),   ptr(outs[i]), h.batch, h.token, h.head,
            o.batch, o.token,      o.head,  static_cast<int>(h.n)};
  }
  // What is written shares no element with anything else: in place x with k, otherwise given
  // outputs with the inputs (but one with its own, which is in place too) and each other.
  if (inplace) {
    if (k) TORCH_CHECK_VALUE(apart(x, from[0], *k, from[1], hd), "rope: x and k share elements");
  } else if (given[0] || given[1]) {
    for (int i = 0; i < (k ? 2 : 1); ++i)
      for (int j = 0; given[i] && j < (k ? 2 : 1); ++j) {
        const bool own = i == j && q[i].x == q[i].out && from[i].batch == to[i].batch &&
                         from[i].token == to[i].token && from[i].head == to[i].head;
        TORCH_CHECK_VALUE(own || apart(outs[i], to[i], *in[j], from[j], hd), out_names[i],
                          ": shares elements with ", names[j]);
      }
    if (k)
      TORCH_CHECK_VALUE(apart(outs[0], to[0], outs[1], to[1], hd),
                        "rope: out and out_k share elements");
  }
  const void* pos = nullptr;
  bool pos64 = false;
  int64_t start = 0;
  if (PyLong_Check(a[1])) {
    start = integer(a[1]);
  } else {
    const Tensor& p = need(a[1], "positions");
    pos64 = p.scalar_type() == at::kLong;
    const bool shape = p.dim() == 2 ? p.size(0) == B && p.size(1) == S
                                    : p.dim() == 1 && p.size(0) == B * S;
    if (!shape || (!pos64 && p.scalar_type() != at::kInt) || !p.is_contiguous() || !here(p, dev))
      TORCH_CHECK_VALUE(false, "positions: expected contiguous int32 or int64 [", B * S, "] or [",
                        B, ", ", S, "] on the current CUDA device ", dev, ", got ", shown(p));
    pos = p.const_data_ptr();
  }
  if (B > 0 && S > 0 &&
      failed("qlora_rope",
             qlora_rope(&q[0], k ? &q[1] : nullptr, B, S, static_cast<int>(hd),
                        static_cast<int>(rd), type == kF32, pos, pos64, start,
                        static_cast<const uint64_t*>(phase.const_data_ptr()),
                        static_cast<float>(number(a[3])), truth(a[6]), truth(a[10]),
                        stream(dev))))
    return nullptr;
  auto result = [&](int i) {
    return object(outs[i], inplace ? a[i ? 8 : 0] : a[i ? 13 : 12]);
  };
  if (!k) return result(0);
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, result(0));
  PyTuple_SET_ITEM(t, 1, result(1));
  return t;
  END_HANDLE_TH_ERRORS
}

// (m, v, m_scale, v_scale, f32): the values that 8-bit moments stand for.
PyObject* adamw_moments(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS
  count("adamw_moments", na, 5);
  const int dev = c10::cuda::current_device();
  const Tensor &m = need(a[0], "m"), &v = need(a[1], "v"), &ms = need(a[2], "m_scale"),
               &vs = need(a[3], "v_scale");
  const int64_t n = m.numel();
  want(m, at::kByte, {n}, "m", dev);
  want(v, at::kByte, {n}, "v", dev);
  want(ms, kF32, {n / 256}, "m_scale", dev);
  want(vs, kF32, {n / 256}, "v_scale", dev);
  const bool f32 = truth(a[4]);
  const Tensor mo = fresh({n}, f32 ? kF32 : kBf16, dev), vo = fresh({n}, f32 ? kF32 : kBf16, dev);
  if (failed("qlora_adamw_moments",
             qlora_adamw_moments(ptr(m), ptr(v), as<float>(ptr(ms)), as<float>(ptr(vs)), n / 256,
                                 f32, ptr(mo), ptr(vo), stream(dev))))
    return nullptr;
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(mo));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(vo));
  return t;
  END_HANDLE_TH_ERRORS
}

// (device index): the current stream's handle where that device is current, else None.
PyObject* current_stream(PyObject*, PyObject* o) {
  HANDLE_TH_ERRORS
  const int64_t dev = integer(o);
  if (c10::cuda::current_device() != dev) Py_RETURN_NONE;
  return PyLong_FromVoidPtr(stream(static_cast<int>(dev)));
  END_HANDLE_TH_ERRORS
}

// (class): what a status is raised as.
PyObject* set_error(PyObject*, PyObject* o) {
  Py_XSETREF(g_error, Py_NewRef(o));
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace

PyMODINIT_FUNC PyInit__torch_bind() {
  static PyMethodDef methods[] = {
      {"residual_norm_forward", method(residual_norm_forward), METH_FASTCALL, nullptr},
      {"residual_norm_backward", method(residual_norm_backward), METH_FASTCALL, nullptr},
      {"rope", method(rope), METH_FASTCALL, nullptr},
      {"adamw_moments", method(adamw_moments), METH_FASTCALL, nullptr},
      {"current_stream", current_stream, METH_O, nullptr},
      {"set_error", set_error, METH_O, nullptr},
      {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_torch_bind", nullptr, -1, methods,
                            nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&def);
}
