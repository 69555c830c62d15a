// Argument marshalling of the operators around the Muon step: checks tensors,
// allocates the outputs that the caller did not give and calls the C entry
// points of libmuon.  It exists because these operators take a few microseconds
// on the GPU, and the same checks and allocations in Python take 10 to 20.
//
// The C functions are handed over by address (bind), so that whichever build of
// the library is loaded is the one that runs.  Every function returns its
// outputs, or the muon_status as an integer when the call was refused.
//
// Outputs are allocated with the call's stream as PyTorch's current one: its
// allocator hands a block out again to the stream that it was made for without
// waiting, so a block made for any other stream could still be read by that
// stream's work, or be handed on while this call writes it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "muon.h"

namespace {

struct Error {
  PyObject *type;
  std::string text;
};

[[noreturn]] void type_error(const std::string &s) { throw Error{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string &s) { throw Error{PyExc_ValueError, s}; }

decltype(&muon_gated_ffn) p_gated_ffn;
decltype(&muon_gated_ffn_backward) p_gated_ffn_backward;
decltype(&muon_block_norm) p_block_norm;
decltype(&muon_block_norm_backward) p_block_norm_backward;
decltype(&muon_token_logprobs) p_token_logprobs;
decltype(&muon_token_logprobs_backward) p_token_logprobs_backward;
decltype(&muon_route) p_route;
decltype(&muon_route_backward) p_route_backward;
decltype(&muon_dispatch) p_dispatch;
decltype(&muon_dispatch_backward) p_dispatch_backward;
decltype(&muon_combine) p_combine;
decltype(&muon_combine_backward) p_combine_backward;
decltype(&muon_head_loss) p_head_loss;
decltype(&muon_head_loss_backward) p_head_loss_backward;

using Sizes = std::initializer_list<int64_t>;

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Error{nullptr, ""};
  return v;
}
long long integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Error{nullptr, ""};
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Error{nullptr, ""};
  return v != 0;
}

// One call's stream and tensors, all on one device.
struct Call {
  int device;
  cudaStream_t handle;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  bool entered = false;

  // (handle, device, whether both are PyTorch's current ones), or a handle on the current device
  explicit Call(PyObject *stream) {
    const bool all = PyTuple_Check(stream) && PyTuple_GET_SIZE(stream) == 3;
    handle = reinterpret_cast<cudaStream_t>((uintptr_t)integer(all ? PyTuple_GET_ITEM(stream, 0) : stream));
    device = all ? (int)integer(PyTuple_GET_ITEM(stream, 1)) : -1;
    entered = all && PyTuple_GET_ITEM(stream, 2) == Py_True;
  }

  // From here to the call's end its stream and device are PyTorch's current ones.  Where
  // they are known to be, nothing is asked: asking costs 1 to 3 us between launches.
  void enter() {
    if (entered) return;
    entered = true;
    if (c10::cuda::current_device() != device || c10::cuda::getCurrentCUDAStream(device).stream() != handle)
      guard.emplace(c10::cuda::getStreamFromExternal(handle, device));
  }
  at::Tensor empty(at::IntArrayRef sizes, const at::TensorOptions &options) {
    enter();
    return at::empty(sizes, options);
  }
  muon_stream_t stream() {
    enter();
    return reinterpret_cast<muon_stream_t>(handle);
  }

  const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
    if (device < 0) device = c10::cuda::current_device();
    if (t.get_device() != device)   // a launch on one device with another's memory
      value_error(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", the call's stream on cuda:" +
                  std::to_string(device));
    return t;
  }

  void check(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape) {
    if (t.scalar_type() != type)
      type_error(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
      value_error(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
  }

  // a dense tensor
  const at::Tensor &dense(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, shape);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t;
  }
  // rows x cols whose last axis is dense; its row stride in *stride
  const at::Tensor &rows(PyObject *o, const char *name, at::ScalarType type, int64_t n, int64_t cols, int64_t *stride) {
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, {n, cols});
    *stride = cols;
    if (!t.is_contiguous()) {
      if ((t.stride(1) != 1 && cols > 1) || (t.stride(0) < cols && n > 1))
        value_error(std::string(name) + " must be dense along its last axis, with rows that do not overlap");
      *stride = std::max(t.stride(0), cols);   // the stride of a single row says nothing
    }
    return t;
  }
  void *workspace(PyObject *o, size_t *bytes) {
    *bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "workspace");
    if (t.scalar_type() != at::kByte) type_error("workspace must be torch.uint8");
    if (!t.is_contiguous()) value_error("workspace must be contiguous");
    *bytes = (size_t)t.numel();
    return t.data_ptr();
  }
};

void *opt(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

int type_code(const at::Tensor &t, const char *name) {
  if (t.scalar_type() == at::kBFloat16) return MUON_BF16;
  if (t.scalar_type() == at::kFloat) return MUON_F32;
  type_error(std::string(name) + " must be torch.bfloat16 or torch.float32, got " + c10::toString(t.scalar_type()));
}

// An output: the caller's object, or a tensor made here.
struct Out {
  at::Tensor t;
  PyObject *given = nullptr;

  PyObject *object() const {
    if (given) {
      Py_INCREF(given);
      return given;
    }
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
  }
};

Out out_rows(Call &c, PyObject *o, const char *name, const at::Tensor &like, int64_t n, int64_t cols, int64_t *stride) {
  Out r;
  if (o == Py_None) {
    r.t = c.empty({n, cols}, like.options());
    *stride = cols;
  } else {
    r.t = c.rows(o, name, like.scalar_type(), n, cols, stride);
    r.given = o;
  }
  return r;
}

PyObject *tuple_of(std::initializer_list<const Out *> outs) {
  PyObject *r = PyTuple_New((Py_ssize_t)outs.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Out *o : outs) {
    PyObject *v = o->object();
    if (!v) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, v);
  }
  return r;
}

// Runs a function's body; its exceptions become Python's.
template <typename F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F &&body) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
    return nullptr;
  }
  try {
    return body();
  } catch (const Error &e) {
    if (e.type) PyErr_SetString(e.type, e.text.c_str());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ---------------------------------------------------------------------------- feed-forward
struct Ffn {
  int64_t T, E, H, F, ldx;
  const at::Tensor *x, *w1, *w3, *w2;
  const int64_t *offsets = nullptr;

  Ffn(Call &c, PyObject *x_, PyObject *w1_, PyObject *w3_, PyObject *w2_, PyObject *off) {
    const at::Tensor &xt = c.tensor(x_, "x"), &w = c.tensor(w1_, "w1");
    if (w.dim() != 2 && w.dim() != 3) value_error("w1 must be (experts, hidden, ffn) or (hidden, ffn)");
    if (xt.dim() != 2) value_error("x must be (rows, hidden)");
    const bool many = w.dim() == 3;
    E = many ? w.size(0) : 1, H = w.size(-2), F = w.size(-1), T = xt.size(0);
    x = &c.rows(x_, "x", at::kBFloat16, T, H, &ldx);
    w1 = &c.dense(w1_, "w1", at::kBFloat16, w.sizes());
    w3 = &c.dense(w3_, "w3", at::kBFloat16, w.sizes());
    const int64_t s3[3] = {E, F, H};
    w2 = &c.dense(w2_, "w2", at::kBFloat16, at::IntArrayRef(many ? s3 : s3 + 1, many ? 3 : 2));
    if (off != Py_None)
      offsets = static_cast<const int64_t *>(c.dense(off, "offsets", at::kLong, {E + 1}).data_ptr());
    else if (E != 1)
      value_error("offsets are needed with more than one expert");
  }
};

// (x, w1, w3, w2, offsets, act, keep, out, workspace, stream)
PyObject *gated_ffn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    Call c(a[9]);
    const Ffn f(c, a[0], a[1], a[2], a[3], a[4]);
    const bool keep = truth(a[6]);
    int64_t ldy;
    const Out y = out_rows(c, a[7], "out", *f.x, f.T, f.H, &ldy);
    Out gate, up;
    if (keep) {
      gate.t = c.empty({f.T, f.F}, f.x->options());
      up.t = c.empty({f.T, f.F}, f.x->options());
    }
    size_t bytes;
    void *ws = c.workspace(a[8], &bytes);
    const int st = p_gated_ffn(f.x->data_ptr(), f.ldx, f.w1->data_ptr(), f.w3->data_ptr(), f.w2->data_ptr(), f.offsets,
                               f.T, f.E, f.H, f.F, (int)integer(a[5]), y.t.data_ptr(), ldy, opt(gate.t), opt(up.t), ws,
                               bytes, c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return keep ? tuple_of({&y, &gate, &up}) : y.object();
  });
}

// (dy, x, gate, up, w1, w3, w2, offsets, act, dx, dw, need_dx, need_dw, workspace, stream)
PyObject *gated_ffn_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject * {
    Call c(a[14]);
    const Ffn f(c, a[1], a[4], a[5], a[6], a[7]);
    int64_t lddy, lddx = f.H;
    const at::Tensor &dy = c.rows(a[0], "dy", at::kBFloat16, f.T, f.H, &lddy);
    const at::Tensor &gate = c.dense(a[2], "gate", at::kBFloat16, {f.T, f.F});
    const at::Tensor &up = c.dense(a[3], "up", at::kBFloat16, {f.T, f.F});
    Out dx, dw[3];
    if (truth(a[11])) dx = out_rows(c, a[9], "dx", *f.x, f.T, f.H, &lddx);
    const at::Tensor *w[3] = {f.w1, f.w3, f.w2};
    if (truth(a[12])) {
      static const char *names[3] = {"dw1", "dw3", "dw2"};
      if (a[10] == Py_None) {
        for (int i = 0; i < 3; ++i) dw[i].t = c.empty(w[i]->sizes(), w[i]->options());
      } else {
        if (!PyTuple_Check(a[10]) || PyTuple_GET_SIZE(a[10]) != 3) value_error("dw must be (dw1, dw3, dw2)");
        for (int i = 0; i < 3; ++i) {
          dw[i].given = PyTuple_GET_ITEM(a[10], i);
          dw[i].t = c.dense(dw[i].given, names[i], at::kBFloat16, w[i]->sizes());
        }
      }
    }
    size_t bytes;
    void *ws = c.workspace(a[13], &bytes);
    const int st = p_gated_ffn_backward(dy.data_ptr(), lddy, f.x->data_ptr(), f.ldx, gate.data_ptr(), up.data_ptr(),
                                        f.w1->data_ptr(), f.w3->data_ptr(), f.w2->data_ptr(), f.offsets, f.T, f.E, f.H,
                                        f.F, (int)integer(a[8]), opt(dx.t), lddx, opt(dw[0].t), opt(dw[1].t),
                                        opt(dw[2].t), ws, bytes, c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({&dx, &dw[0], &dw[1], &dw[2]});
  });
}

// ---------------------------------------------------------------------------- norms
// a gate's row stride: 0 for one gate for all rows
const at::Tensor &gate_of(Call &c, PyObject *o, at::ScalarType type, int64_t T, int64_t H, int64_t *stride) {
  *stride = 0;
  if (c.tensor(o, "gate").dim() == 1) return c.dense(o, "gate", type, {H});
  return c.rows(o, "gate", type, T, H, stride);
}

bool given(PyObject *o) { return o != Py_None; }

// (residual, block, w_post, gate, w_pre, scale, eps, norm_next, out, normed, stream)
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    Call c(a[10]);
    const at::Tensor &res = c.tensor(a[0], "residual");
    if (res.dim() != 2) value_error("residual must be (rows, hidden)");
    const int64_t T = res.size(0), H = res.size(1);
    const bool post = given(a[1]), pre = truth(a[7]);
    const at::Tensor &branch = post ? c.tensor(a[1], "block") : given(a[4]) ? c.tensor(a[4], "w_pre")
                               : given(a[9]) ? c.tensor(a[9], "normed") : res;
    const at::ScalarType bt = branch.scalar_type();
    muon_block_norm_args k{};
    k.rows = T, k.hidden = H;
    k.residual_type = type_code(res, "residual"), k.branch_type = type_code(branch, "block");
    k.scale = (float)number(a[5]), k.eps = (float)number(a[6]);
    k.residual = c.rows(a[0], "residual", res.scalar_type(), T, H, &k.residual_stride).data_ptr();
    Out out, normed, rstd_post, rstd_pre;
    const auto f32 = res.options().dtype(at::kFloat);
    if (post) {
      k.block = c.rows(a[1], "block", bt, T, H, &k.block_stride).data_ptr();
      if (given(a[2])) k.w_post = c.dense(a[2], "w_post", bt, {H}).data_ptr();
      if (given(a[3])) k.gate = gate_of(c, a[3], bt, T, H, &k.gate_stride).data_ptr();
      out = out_rows(c, a[8], "out", res, T, H, &k.residual_out_stride);
      k.residual_out = out.t.data_ptr();
      rstd_post.t = c.empty({T}, f32);
      k.rstd_post = rstd_post.t.data_ptr<float>();
    } else {
      if (given(a[2]) || given(a[3]) || given(a[8])) value_error("w_post, gate and out belong to a block");
      if (!pre) value_error("there is nothing to compute without a block and without norm_next");
      out.given = a[0];
    }
    if (pre) {
      if (given(a[4])) k.w_pre = c.dense(a[4], "w_pre", bt, {H}).data_ptr();
      normed = out_rows(c, a[9], "normed", branch, T, H, &k.normed_stride);
      k.normed = normed.t.data_ptr();
      rstd_pre.t = c.empty({T}, f32);
      k.rstd_pre = rstd_pre.t.data_ptr<float>();
    } else if (given(a[4]) || given(a[9])) {
      value_error("w_pre and normed belong to the norm before the next block");
    }
    const int st = p_block_norm(&k, c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({&out, &normed, &rstd_post, &rstd_pre});
  });
}

// (dresidual, dnormed, residual, block, rstd_post, rstd_pre, w_post, gate, w_pre, scale, workspace, stream)
PyObject *block_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject * {
    Call c(a[11]);
    const at::Tensor &res = c.tensor(a[2], "residual");
    if (res.dim() != 2) value_error("residual must be (rows, hidden)");
    const int64_t T = res.size(0), H = res.size(1);
    const bool pre = given(a[1]), post = given(a[3]);
    if (!given(a[0]) && !pre) value_error("dresidual or dnormed must be given");
    const at::Tensor &branch = pre ? c.tensor(a[1], "dnormed") : post ? c.tensor(a[3], "block") : res;
    const at::ScalarType rt = res.scalar_type(), bt = branch.scalar_type();
    muon_block_norm_backward_args k{};
    k.rows = T, k.hidden = H;
    k.residual_type = type_code(res, "residual"), k.branch_type = type_code(branch, "block");
    k.scale = (float)number(a[9]);
    k.residual = c.rows(a[2], "residual", rt, T, H, &k.residual_stride).data_ptr();
    if (given(a[0])) k.dresidual_out = c.rows(a[0], "dresidual", rt, T, H, &k.dresidual_out_stride).data_ptr();
    Out dr, dblock, dw_post, dgate, dw_pre;
    if (pre) {
      k.dnormed = c.rows(a[1], "dnormed", bt, T, H, &k.dnormed_stride).data_ptr();
      k.rstd_pre = static_cast<const float *>(c.dense(a[5], "rstd_pre", at::kFloat, {T}).data_ptr());
      if (given(a[8])) {
        k.w_pre = c.dense(a[8], "w_pre", bt, {H}).data_ptr();
        dw_pre.t = c.empty({H}, branch.options());
        k.dw_pre = dw_pre.t.data_ptr();
      }
    } else if (given(a[8])) {
      value_error("w_pre belongs to the norm before the next block");
    }
    if (post) {
      k.block = c.rows(a[3], "block", bt, T, H, &k.block_stride).data_ptr();
      k.rstd_post = static_cast<const float *>(c.dense(a[4], "rstd_post", at::kFloat, {T}).data_ptr());
      dblock.t = c.empty({T, H}, branch.options());
      k.dblock = dblock.t.data_ptr(), k.dblock_stride = H;
      if (given(a[6])) {
        k.w_post = c.dense(a[6], "w_post", bt, {H}).data_ptr();
        dw_post.t = c.empty({H}, branch.options());
        k.dw_post = dw_post.t.data_ptr();
      }
      if (given(a[7])) {
        const at::Tensor &g = gate_of(c, a[7], bt, T, H, &k.gate_stride);
        k.gate = g.data_ptr();
        dgate.t = c.empty(g.sizes(), branch.options());
        k.dgate = dgate.t.data_ptr(), k.dgate_stride = H;
      }
    } else if (given(a[6]) || given(a[7])) {
      value_error("w_post and gate belong to a block");
    }
    dr.t = c.empty({T, H}, res.options());
    k.dresidual = dr.t.data_ptr(), k.dresidual_stride = H;
    size_t bytes;
    void *ws = c.workspace(a[10], &bytes);
    const int st = p_block_norm_backward(&k, ws, bytes, c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({&dr, &dblock, &dw_post, &dgate, &dw_pre});
  });
}

// ---------------------------------------------------------------------------- log probabilities
const at::Tensor &logits_of(Call &c, PyObject *o, int64_t *T, int64_t *V, int64_t *stride, int *code) {
  const at::Tensor &x = c.tensor(o, "logits");
  if (x.dim() != 2) value_error("logits must be (rows, vocab)");
  *code = type_code(x, "logits");
  *T = x.size(0), *V = x.size(1);
  return c.rows(o, "logits", x.scalar_type(), *T, *V, stride);
}

const int64_t *tokens_of(Call &c, PyObject *o, int64_t T) {
  if (!given(o)) return nullptr;
  return static_cast<const int64_t *>(c.dense(o, "tokens", at::kLong, {T}).data_ptr());
}

// (logits, tokens, top, stream)
PyObject *token_logprobs(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject * {
    Call c(a[3]);
    int64_t T, V, stride;
    int code;
    const at::Tensor &x = logits_of(c, a[0], &T, &V, &stride, &code);
    const int64_t *tokens = tokens_of(c, a[1], T);
    const long long top = integer(a[2]);
    if (top < -1000000 || top > 1000000) value_error("top is out of range");
    const auto f32 = x.options().dtype(at::kFloat);
    Out logp, entropy, lse, ids, values;
    if (given(a[1])) logp.t = c.empty({T}, f32);
    entropy.t = c.empty({T}, f32);
    lse.t = c.empty({T}, f32);
    if (top > 0) {
      ids.t = c.empty({T, top}, x.options().dtype(at::kLong));
      values.t = c.empty({T, top}, f32);
    }
    const int st = p_token_logprobs(x.data_ptr(), stride, tokens, T, V, code, static_cast<float *>(opt(logp.t)),
                                    entropy.t.data_ptr<float>(), lse.t.data_ptr<float>(), (int)top,
                                    static_cast<int64_t *>(opt(ids.t)), static_cast<float *>(opt(values.t)),
                                    c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({&logp, &entropy, &lse, &ids, &values});
  });
}

// (logits, tokens, lse, entropy, dlogp, dentropy, out, stream)
PyObject *token_logprobs_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    Call c(a[7]);
    int64_t T, V, stride, out_stride;
    int code;
    const at::Tensor &x = logits_of(c, a[0], &T, &V, &stride, &code);
    const int64_t *tokens = tokens_of(c, a[1], T);
    if (given(a[4]) && !tokens && T) value_error("dlogp needs tokens");
    if (given(a[5]) && !given(a[3])) value_error("dentropy needs entropy");
    const float *in[4] = {};
    static const char *names[4] = {"lse", "entropy", "dlogp", "dentropy"};
    for (int i = 0; i < 4; ++i)
      if (given(a[2 + i]) || i == 0)
        in[i] = static_cast<const float *>(c.dense(a[2 + i], names[i], at::kFloat, {T}).data_ptr());
    const Out out = out_rows(c, a[6], "out", x, T, V, &out_stride);
    const int st = p_token_logprobs_backward(x.data_ptr(), stride, tokens, in[0], in[1], in[2], in[3], T, V, code,
                                             out.t.data_ptr(), out_stride, c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return out.object();
  });
}

// ---------------------------------------------------------------------------- routing
// a size or count that has to fit an int (what it may be beyond that is the library's to say)
int small_integer(PyObject *o, const char *name) {
  const long long v = integer(o);
  if (v < -1000000 || v > 1000000) value_error(std::string(name) + " is out of range");
  return (int)v;
}

const at::Tensor &route_logits(Call &c, PyObject *o, int64_t *T, int64_t *E, int64_t *stride, int *code) {
  const at::Tensor &x = c.tensor(o, "logits");
  if (x.dim() != 2) value_error("logits must be (rows, experts)");
  *code = type_code(x, "logits");
  *T = x.size(0), *E = x.size(1);
  return c.rows(o, "logits", x.scalar_type(), *T, *E, stride);
}

// (logits, top, bias, score, normalize, scale, stream)
PyObject *route(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject * {
    Call c(a[6]);
    int64_t T, E, stride;
    int code;
    const at::Tensor &x = route_logits(c, a[0], &T, &E, &stride, &code);
    const int top = small_integer(a[1], "top");
    const float *bias =
        given(a[2]) ? static_cast<const float *>(c.dense(a[2], "bias", at::kFloat, {E}).data_ptr()) : nullptr;
    const int score = (int)integer(a[3]), normalize = truth(a[4]);
    const float scale = (float)number(a[5]);
    Out ids, weights;
    const int64_t k = std::min(std::max(top, 0), 32);   // the library refuses more
    ids.t = c.empty({T, k}, x.options().dtype(at::kLong));
    weights.t = c.empty({T, k}, x.options().dtype(at::kFloat));
    const int st = p_route(x.data_ptr(), stride, bias, T, E, code, top, score, normalize, scale,
                           ids.t.data_ptr<int64_t>(), weights.t.data_ptr<float>(), c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({&ids, &weights});
  });
}

// (dweights, logits, ids, score, normalize, scale, out, stream)
PyObject *route_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    Call c(a[7]);
    int64_t T, E, stride, out_stride;
    int code;
    const at::Tensor &x = route_logits(c, a[1], &T, &E, &stride, &code), &ids = c.tensor(a[2], "ids");
    if (ids.dim() != 2) value_error("ids must be (rows, top)");
    const int64_t top = ids.size(1);
    if (top > 1000000) value_error("top is out of range");
    c.dense(a[2], "ids", at::kLong, {T, top});
    const at::Tensor &dw = c.dense(a[0], "dweights", at::kFloat, {T, top});
    const int score = (int)integer(a[3]), normalize = truth(a[4]);
    const float scale = (float)number(a[5]);
    const Out out = out_rows(c, a[6], "out", x, T, E, &out_stride);
    const int st = p_route_backward(dw.data_ptr<float>(), x.data_ptr(), stride, ids.data_ptr<int64_t>(), T, E, code,
                                    (int)top, score, normalize, scale, out.t.data_ptr(), out_stride, c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return out.object();
  });
}

// ---------------------------------------------------------------------------- tokens by expert and back
// (tokens, slots), int64
const at::Tensor &slots_of(Call &c, PyObject *o, const char *name, int64_t *T, int64_t *k) {
  const at::Tensor &t = c.tensor(o, name);
  if (t.dim() != 2) value_error(std::string(name) + " must be (tokens, slots)");
  *T = t.size(0), *k = t.size(1);
  return c.dense(o, name, at::kLong, {*T, *k});
}

// rows by expert, dense
const at::Tensor &sorted_rows(Call &c, PyObject *o, const char *name, int64_t n, int64_t *H, int *code) {
  const at::Tensor &t = c.tensor(o, name);
  if (t.dim() != 2) value_error(std::string(name) + " must be (tokens * slots, hidden)");
  *code = type_code(t, name);
  *H = t.size(1);
  return c.dense(o, name, t.scalar_type(), {n, *H});
}

// (x, ids, experts, out, stream)
PyObject *dispatch(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    Call c(a[4]);
    int64_t T, k, ldx;
    const at::Tensor &ids = slots_of(c, a[1], "ids", &T, &k), &xt = c.tensor(a[0], "x");
    if (xt.dim() != 2) value_error("x must be (tokens, hidden)");
    const int code = type_code(xt, "x");
    const int64_t H = xt.size(1);
    const at::Tensor &x = c.rows(a[0], "x", xt.scalar_type(), T, H, &ldx);
    const int experts = small_integer(a[2], "experts");
    if (k > 32) return PyLong_FromLong(MUON_ERR_UNSUPPORTED);   // before the rows of so many slots are allocated
    Out rows, offsets, place;
    if (given(a[3])) {
      rows.t = c.dense(a[3], "out", x.scalar_type(), {T * k, H});
      rows.given = a[3];
    } else {
      rows.t = c.empty({T * k, H}, x.options());
    }
    offsets.t = c.empty({std::max(experts, 0) + 1}, ids.options());
    place.t = c.empty({T, k}, ids.options());
    const int st = p_dispatch(x.data_ptr(), ldx, ids.data_ptr<int64_t>(), T, k, experts, H, code, rows.t.data_ptr(),
                              offsets.t.data_ptr<int64_t>(), place.t.data_ptr<int64_t>(), c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({&rows, &offsets, &place});
  });
}

// (drows, place, out, stream)
PyObject *dispatch_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject * {
    Call c(a[3]);
    int64_t T, k, H, ldo;
    int code;
    const at::Tensor &place = slots_of(c, a[1], "place", &T, &k);
    const at::Tensor &drows = sorted_rows(c, a[0], "drows", T * k, &H, &code);
    const Out out = out_rows(c, a[2], "out", drows, T, H, &ldo);
    const int st = p_dispatch_backward(drows.data_ptr(), place.data_ptr<int64_t>(), T, k, H, code, out.t.data_ptr(), ldo,
                                       c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return out.object();
  });
}

// (y, place, weights, out, stream)
PyObject *combine(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    Call c(a[4]);
    int64_t T, k, H, ldo;
    int code;
    const at::Tensor &place = slots_of(c, a[1], "place", &T, &k);
    const at::Tensor &y = sorted_rows(c, a[0], "y", T * k, &H, &code);
    const float *w =
        given(a[2]) ? static_cast<const float *>(c.dense(a[2], "weights", at::kFloat, {T, k}).data_ptr()) : nullptr;
    const Out out = out_rows(c, a[3], "out", y, T, H, &ldo);
    const int st = p_combine(y.data_ptr(), place.data_ptr<int64_t>(), w, T, k, H, code, out.t.data_ptr(), ldo, c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return out.object();
  });
}

// (dout, y, place, weights, dy, need_dy, need_dweights, stream)
PyObject *combine_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    Call c(a[7]);
    int64_t T, k, ldd;
    const at::Tensor &place = slots_of(c, a[2], "place", &T, &k), &dt = c.tensor(a[0], "dout");
    if (dt.dim() != 2) value_error("dout must be (tokens, hidden)");
    const int code = type_code(dt, "dout");
    const int64_t H = dt.size(1);
    const at::Tensor &dout = c.rows(a[0], "dout", dt.scalar_type(), T, H, &ldd);
    const float *w =
        given(a[3]) ? static_cast<const float *>(c.dense(a[3], "weights", at::kFloat, {T, k}).data_ptr()) : nullptr;
    Out dy, dweights;
    const void *y = nullptr;
    if (truth(a[5])) {
      if (given(a[4])) {
        dy.t = c.dense(a[4], "dy", dout.scalar_type(), {T * k, H});
        dy.given = a[4];
      } else {
        dy.t = c.empty({T * k, H}, dout.options());
      }
    }
    if (given(a[3]) && truth(a[6])) {
      y = c.dense(a[1], "y", dout.scalar_type(), {T * k, H}).data_ptr();
      dweights.t = c.empty({T, k}, dout.options().dtype(at::kFloat));
    }
    const int st = p_combine_backward(dout.data_ptr(), ldd, y, place.data_ptr<int64_t>(), w, T, k, H, code, opt(dy.t),
                                      static_cast<float *>(opt(dweights.t)), c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({&dy, &dweights});
  });
}

// ---------------------------------------------------------------------------- loss over a head matrix
struct Head {
  int64_t T, V, H, ldx;
  const at::Tensor *x, *w;
  const int64_t *targets;

  Head(Call &c, PyObject *x_, PyObject *w_, PyObject *t_) {
    const at::Tensor &xt = c.tensor(x_, "x"), &wt = c.tensor(w_, "weight");
    if (xt.dim() != 2) value_error("x must be (rows, hidden)");
    if (wt.dim() != 2) value_error("weight must be (vocab, hidden)");
    T = xt.size(0), H = xt.size(1), V = wt.size(0);
    x = &c.rows(x_, "x", at::kBFloat16, T, H, &ldx);
    w = &c.dense(w_, "weight", at::kBFloat16, {V, H});
    targets = static_cast<const int64_t *>(c.dense(t_, "targets", at::kLong, {T}).data_ptr());
  }
};

// (x, weight, targets, workspace, stream)
PyObject *head_loss(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    Call c(a[4]);
    const Head h(c, a[0], a[1], a[2]);
    size_t bytes;
    void *ws = c.workspace(a[3], &bytes);
    const auto f32 = h.x->options().dtype(at::kFloat);
    Out loss, lse;
    loss.t = c.empty({h.T}, f32);
    lse.t = c.empty({h.T}, f32);
    const int st = p_head_loss(h.x->data_ptr(), h.ldx, h.w->data_ptr(), h.targets, h.T, h.V, h.H,
                               loss.t.data_ptr<float>(), lse.t.data_ptr<float>(), ws, bytes, c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({&loss, &lse});
  });
}

// (dloss, x, weight, targets, lse, dlse, dx, dweight, need_dx, need_dweight, workspace, stream)
PyObject *head_loss_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject * {
    Call c(a[11]);
    const Head h(c, a[1], a[2], a[3]);
    const float *dloss = static_cast<const float *>(c.dense(a[0], "dloss", at::kFloat, {h.T}).data_ptr());
    const float *lse = static_cast<const float *>(c.dense(a[4], "lse", at::kFloat, {h.T}).data_ptr());
    const float *dlse =
        given(a[5]) ? static_cast<const float *>(c.dense(a[5], "dlse", at::kFloat, {h.T}).data_ptr()) : nullptr;
    int64_t lddx = h.H;
    Out dx, dw;
    if (truth(a[8])) dx = out_rows(c, a[6], "dx", *h.x, h.T, h.H, &lddx);
    if (truth(a[9])) {
      if (given(a[7])) {
        dw.t = c.dense(a[7], "dweight", at::kBFloat16, {h.V, h.H});
        dw.given = a[7];
      } else {
        dw.t = c.empty({h.V, h.H}, h.w->options());
      }
    }
    size_t bytes;
    void *ws = c.workspace(a[10], &bytes);
    const int st = p_head_loss_backward(dloss, dlse, h.x->data_ptr(), h.ldx, h.w->data_ptr(), h.targets, lse, h.T, h.V,
                                        h.H, opt(dx.t), lddx, opt(dw.t), ws, bytes, c.stream());
    if (st != MUON_OK) return PyLong_FromLong(st);
    return tuple_of({&dx, &dw});
  });
}

// bind({name: address}): the library's entry points
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject * {
    auto address = [&](const char *name) {
      PyObject *v = PyDict_Check(a[0]) ? PyDict_GetItemString(a[0], name) : nullptr;
      if (!v) value_error(std::string("no address of ") + name);
      return reinterpret_cast<void *>((uintptr_t)integer(v));
    };
#define MUON_BIND(f) p_##f = reinterpret_cast<decltype(p_##f)>(address("muon_" #f))
    MUON_BIND(gated_ffn);
    MUON_BIND(gated_ffn_backward);
    MUON_BIND(block_norm);
    MUON_BIND(block_norm_backward);
    MUON_BIND(token_logprobs);
    MUON_BIND(token_logprobs_backward);
    MUON_BIND(route);
    MUON_BIND(route_backward);
    MUON_BIND(dispatch);
    MUON_BIND(dispatch_backward);
    MUON_BIND(combine);
    MUON_BIND(combine_backward);
    MUON_BIND(head_loss);
    MUON_BIND(head_loss_backward);
#undef MUON_BIND
    Py_RETURN_NONE;
  });
}

#define MUON_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MUON_METHOD(bind),
                         MUON_METHOD(gated_ffn),
                         MUON_METHOD(gated_ffn_backward),
                         MUON_METHOD(block_norm),
                         MUON_METHOD(block_norm_backward),
                         MUON_METHOD(token_logprobs),
                         MUON_METHOD(token_logprobs_backward),
                         MUON_METHOD(route),
                         MUON_METHOD(route_backward),
                         MUON_METHOD(dispatch),
                         MUON_METHOD(dispatch_backward),
                         MUON_METHOD(combine),
                         MUON_METHOD(combine_backward),
                         MUON_METHOD(head_loss),
                         MUON_METHOD(head_loss_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "muon_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_muon_ops() { return PyModule_Create(&module); }
