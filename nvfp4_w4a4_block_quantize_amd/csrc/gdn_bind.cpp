// Native side of the gated delta layer's Python binding (gdn.py), in the module of
// kv_bind.cpp and by its rules: arguments by position, the stream last (None:
// torch's current one), ValueError for a tensor that does not fit, and the C status
// as the result.
#include "bind_common.h"
#include "nvfp4_gdn.h"

namespace nvfp4_bind {
namespace {

// a dense float32 tensor of `shape`, or None where that is allowed
float* floats(PyObject* o, at::IntArrayRef shape, const char* name, const at::Tensor& like, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kFloat || t.sizes() != shape) {
    std::string want;
    for (int64_t n : shape) want += (want.empty() ? "" : ", ") + std::to_string(n);
    refuse("%s must be float32 [%s], got %s %s", name, want.c_str(), at::toString(t.scalar_type()),
           shape_of(t).c_str());
  }
  if (!t.is_contiguous()) refuse("%s must be contiguous", name);
  on_device(t, name, like);
  return static_cast<float*>(t.data_ptr());
}

// rows of `columns` elements with any stride between them
struct Rows {
  void* p;
  int64_t rows, columns, ld;
  Rows(PyObject* o, const char* name, const at::Tensor& like, int64_t rows_, int64_t columns_) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != like.scalar_type() || t.dim() != 2 || t.size(0) != rows_ || t.size(1) != columns_)
      refuse("%s must be %s [%lld, %lld], got %s %s", name, at::toString(like.scalar_type()), (long long)rows_,
             (long long)columns_, at::toString(t.scalar_type()), shape_of(t).c_str());
    if (t.stride(1) != 1 && columns_ != 1) refuse("%s must have unit column stride", name);
    on_device(t, name, like);
    rows = rows_;
    columns = columns_;
    ld = rows > 1 ? t.stride(0) : columns;
    p = t.data_ptr();
  }
};

// a state and where it goes, dense tensors of one shape whose first axis is the slots
struct States {
  void *in, *out;
  int64_t slots;
  States(PyObject* state, PyObject* state_out, at::ScalarType type, at::IntArrayRef of_slot, const at::Tensor& like) {
    const at::Tensor& t = tensor(state, "state");
    slots = t.dim() > 0 ? t.size(0) : 0;
    in = dense(t, "state", type, of_slot, like);
    out = dense(tensor(state_out, "state_out"), "state_out", type, of_slot, like);
  }
  void* dense(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef of_slot,
              const at::Tensor& like) const {
    bool fits = t.scalar_type() == type && t.dim() == (int64_t)of_slot.size() + 1 && t.size(0) == slots;
    std::string want = std::to_string(slots);
    for (size_t i = 0; i < of_slot.size(); ++i) {
      fits = fits && t.size(i + 1) == of_slot[i];
      want += ", " + std::to_string(of_slot[i]);
    }
    if (!fits)
      refuse("%s must be %s [%s], got %s %s", name, at::toString(type), want.c_str(), at::toString(t.scalar_type()),
             shape_of(t).c_str());
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    on_device(t, name, like);
    return t.data_ptr();
  }
};

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)v;
}

// sequences of ragged prompts: slots, token_starts, cached_lens or None
struct Ragged {
  int64_t n;
  const int32_t *slots, *starts, *cached;
  Ragged(PyObject* slots_, PyObject* starts_, PyObject* cached_, const at::Tensor& like) {
    const at::Tensor& t = tensor(slots_, "slots");
    n = t.dim() > 0 ? t.size(0) : 0;
    slots = ints(slots_, n, "slots", like);
    starts = ints(starts_, n + 1, "token_starts", like);
    cached = cached_ == Py_None ? nullptr : ints(cached_, n, "cached_lens", like);
  }
};

const at::Tensor& rows_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 2) refuse("%s must be [tokens, channels], got %s", name, shape_of(t).c_str());
  return t;
}

struct ConvTensors {
  Rows x, out;
  int64_t width;
  const float *weight, *bias;
  States states;
  int32_t dtype;
  ConvTensors(PyObject* x_, PyObject* weight_, PyObject* bias_, PyObject* state, PyObject* state_out, PyObject* out_,
              const at::Tensor& xt)
      : x(x_, "x", xt, xt.size(0), xt.size(1)),
        out(out_, "out", xt, xt.size(0), xt.size(1)),
        width(width_of(weight_)),
        weight(floats(weight_, {x.columns, width}, "weight", xt)),
        bias(floats(bias_, {x.columns}, "bias", xt, true)),
        states(state, state_out, xt.scalar_type(), {width - 1, x.columns}, xt),
        dtype(dtype_code(xt)) {}
  static int64_t width_of(PyObject* o) {
    const at::Tensor& t = tensor(o, "weight");
    if (t.dim() != 2 || t.size(1) < 1) refuse("weight must be [channels, width], got %s", shape_of(t).c_str());
    return t.size(1);
  }
};

struct DeltaTensors {
  Heads q, k, v, out;
  Rows a, b;
  const float *a_log, *dt_bias;
  States states;
  float scale, eps;
  int32_t dtype;
  // q k v a b a_log dt_bias state state_out scale eps out
  DeltaTensors(PyObject* const* o, const at::Tensor& qt, const at::Tensor& vt)
      : q(o[0], "q", qt),
        k(o[1], "k", qt, &qt),
        v(o[2], "v", qt),
        out(o[11], "out", qt, &vt),
        a(o[3], "a", qt, q.tokens, v.heads),
        b(o[4], "b", qt, q.tokens, v.heads),
        a_log(floats(o[5], {v.heads}, "a_log", qt)),
        dt_bias(floats(o[6], {v.heads}, "dt_bias", qt)),
        states(o[7], o[8], at::kFloat, {v.heads, q.dim, v.dim}, qt),
        scale(number(o[9])),
        eps(number(o[10])),
        dtype(dtype_code(qt)) {
    if (v.tokens != q.tokens)
      refuse("v must have %lld tokens, got %s", (long long)q.tokens, shape_of(vt).c_str());
  }
};

}  // namespace

PyObject* causal_conv(PyObject*, PyObject* const* o, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 11);
    const at::Tensor& xt = rows_of(o[0], "x");
    const ConvTensors c(o[0], o[1], o[2], o[4], o[5], o[9], xt);
    const int32_t act = (int32_t)integer(o[3]);
    const Ragged r(o[6], o[7], o[8], xt);
    return launch("nvfp4_causal_conv", xt, o[10], [&](void* stream) {
      return nvfp4_causal_conv(c.x.rows, c.x.columns, c.width, c.dtype, c.x.p, c.x.ld, c.weight, c.bias, act, r.n,
                               r.starts, r.cached, r.slots, c.states.in, c.states.out, c.states.slots, c.out.p,
                               c.out.ld, stream);
    });
  });
}

PyObject* causal_conv_step(PyObject*, PyObject* const* o, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 9);
    const at::Tensor& xt = rows_of(o[0], "x");
    const ConvTensors c(o[0], o[1], o[2], o[4], o[5], o[7], xt);
    const int32_t act = (int32_t)integer(o[3]);
    const int32_t* slots = ints(o[6], c.x.rows, "slots", xt);
    return launch("nvfp4_causal_conv_step", xt, o[8], [&](void* stream) {
      return nvfp4_causal_conv_step(c.x.rows, c.x.columns, c.width, c.dtype, c.x.p, c.x.ld, c.weight, c.bias, act,
                                    slots, c.states.in, c.states.out, c.states.slots, c.out.p, c.out.ld, stream);
    });
  });
}

PyObject* gated_delta_chunked(PyObject*, PyObject* const* o, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 17);
    const at::Tensor &qt = tensor(o[0], "q"), &vt = tensor(o[2], "v");
    const DeltaTensors d(o, qt, vt);
    const Ragged r(o[12], o[13], o[14], qt);
    const at::Tensor& ws = tensor(o[15], "workspace");
    if (ws.scalar_type() != at::kByte || !ws.is_contiguous()) refuse("workspace must be a contiguous uint8 tensor");
    on_device(ws, "workspace", qt);
    return launch("nvfp4_gated_delta_chunked", qt, o[16], [&](void* stream) {
      return nvfp4_gated_delta_chunked(
          d.q.tokens, d.q.heads, d.v.heads, d.q.dim, d.v.dim, d.dtype, d.q.p, d.q.token, d.q.head, d.k.p, d.k.token,
          d.k.head, d.v.p, d.v.token, d.v.head, d.a.p, d.a.ld, d.b.p, d.b.ld, d.a_log, d.dt_bias, d.scale, d.eps, r.n,
          r.starts, r.cached, r.slots, static_cast<const float*>(d.states.in), static_cast<float*>(d.states.out),
          d.states.slots, d.out.p, d.out.token, d.out.head, ws.data_ptr(), ws.numel(), stream);
    });
  });
}

PyObject* gated_delta_step(PyObject*, PyObject* const* o, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 14);
    const at::Tensor &qt = tensor(o[0], "q"), &vt = tensor(o[2], "v");
    const DeltaTensors d(o, qt, vt);
    const int32_t* slots = ints(o[12], d.q.tokens, "slots", qt);
    return launch("nvfp4_gated_delta_step", qt, o[13], [&](void* stream) {
      return nvfp4_gated_delta_step(
          d.q.tokens, d.q.heads, d.v.heads, d.q.dim, d.v.dim, d.dtype, d.q.p, d.q.token, d.q.head, d.k.p, d.k.token,
          d.k.head, d.v.p, d.v.token, d.v.head, d.a.p, d.a.ld, d.b.p, d.b.ld, d.a_log, d.dt_bias, d.scale, d.eps,
          slots, static_cast<const float*>(d.states.in), static_cast<float*>(d.states.out), d.states.slots, d.out.p,
          d.out.token, d.out.head, stream);
    });
  });
}

PyObject* group_norm(PyObject*, PyObject* const* o, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 9);
    const at::Tensor& xt = tensor(o[0], "x");
    const Heads x(o[0], "x", xt), out(o[7], "out", xt, &xt);
    const at::Tensor& wt = tensor(o[1], "weight");
    const bool shared = wt.dim() == 1;
    const std::vector<int64_t> shape =
        shared ? std::vector<int64_t>{x.dim} : std::vector<int64_t>{x.heads, x.dim};
    const float *weight = floats(o[1], shape, "weight", xt), *bias = floats(o[2], shape, "bias", xt, true);
    Heads gate;
    if (o[3] != Py_None) gate = Heads(o[3], "gate", xt, &xt);
    const int32_t act = (int32_t)integer(o[4]);
    const int centred = PyObject_IsTrue(o[5]);
    if (centred < 0) throw Refused();
    const float eps = number(o[6]);
    const int32_t dtype = dtype_code(xt);
    return launch("nvfp4_group_norm", xt, o[8], [&](void* stream) {
      return nvfp4_group_norm(x.tokens, x.heads, x.dim, dtype, x.p, x.token, x.head, weight, shared ? 0 : x.dim, bias,
                              gate.p, gate.token, gate.head, act, centred, eps, out.p, out.token, out.head, stream);
    });
  });
}

}  // namespace nvfp4_bind
