// Native side of the paged KV cache's Python binding (kv.py): reads what the C ABI
// wants to know out of the tensors, checks it and makes the call.  A decode step's
// calls take 3 to 7 us on the GPU; the same checks in Python took 5 us of host time
// a call, and passing the arguments through ctypes one more.
//
// Each function takes its arguments by position, the stream last (None: torch's
// current one), raises ValueError for a tensor that does not fit, and returns the
// C status.  The module also holds the gated delta layer's functions (gdn_bind.cpp).
#include "bind_common.h"
#include "nvfp4_kv.h"

namespace {

using namespace nvfp4_bind;

// int32 rows with unit column stride
struct Table {
  int32_t* p;
  int64_t columns, ld;
  Table(PyObject* o, int64_t rows, const at::Tensor& like) {
    const at::Tensor& t = tensor(o, "block_table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != rows)
      refuse("block_table must be int32 [%lld, pages], got %s %s", (long long)rows, at::toString(t.scalar_type()),
             shape_of(t).c_str());
    columns = t.size(1);
    if (t.stride(1) != 1 && columns != 1) refuse("block_table must have unit column stride");
    on_device(t, "block_table", like);
    p = static_cast<int32_t*>(t.data_ptr());
    ld = rows > 1 ? t.stride(0) : columns;
  }
};

// two [num_pages][kv_heads][page_size][head_dim] byte tensors
struct Caches {
  uint8_t *k, *v;
  int64_t pages, heads, page_size, dim;
  Caches(PyObject* ko, PyObject* vo, const at::Tensor& like) {
    const at::Tensor &kt = tensor(ko, "k_cache"), &vt = tensor(vo, "v_cache");
    if (kt.dim() != 4)
      refuse("k_cache must be [num_pages, kv_heads, page_size, head_dim], got %s", shape_of(kt).c_str());
    k = bytes(kt, "k_cache", kt, like);
    v = bytes(vt, "v_cache", kt, like);
    pages = kt.size(0);
    heads = kt.size(1);
    page_size = kt.size(2);
    dim = kt.size(3);
  }
  static uint8_t* bytes(const at::Tensor& t, const char* name, const at::Tensor& same, const at::Tensor& like) {
    if (t.scalar_type() != at::kByte) refuse("%s must be uint8, got %s", name, at::toString(t.scalar_type()));
    if (t.sizes() != same.sizes())
      refuse("%s must have shape %s, got %s", name, shape_of(same).c_str(), shape_of(t).c_str());
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    on_device(t, name, like);
    return static_cast<uint8_t*>(t.data_ptr());
  }
};

PyObject* block_table(PyObject*, PyObject* const* o, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 12);
    const at::Tensor &lens = tensor(o[0], "cached_lens"), &free = tensor(o[3], "free_pages"),
                     &slots = tensor(o[6], "slot_map");
    if (lens.dim() != 1 || free.dim() != 1 || slots.dim() != 1)
      refuse("cached_lens, free_pages and slot_map must be 1-D");
    const int64_t n = lens.size(0), n_free = free.size(0), tokens = slots.size(0);
    const int32_t *cached = ints(o[0], n, "cached_lens", lens), *added = ints(o[1], n, "new_lens", lens);
    const int64_t page_size = integer(o[2]);
    const int32_t *pages = ints(o[3], n_free, "free_pages", lens), *used = ints(o[4], 1, "free_used", lens);
    const Table table(o[5], n, lens);
    int32_t *slot_map = ints(o[6], tokens, "slot_map", lens), *seq_lens = ints(o[7], n, "seq_lens", lens);
    int32_t *starts = ints(o[8], n + 1, "token_starts", lens), *first = ints(o[9], n, "first_pages", lens);
    int32_t* used_out = ints(o[10], 1, "free_used_out", lens);
    return launch("nvfp4_kv_block_table", lens, o[11], [&](void* stream) {
      return nvfp4_kv_block_table(n, cached, added, page_size, pages, n_free, used, table.p, table.columns, table.ld,
                                  slot_map, tokens, seq_lens, starts, first, used_out, stream);
    });
  });
}

PyObject* rope(PyObject*, PyObject* const* o, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 9);
    const at::Tensor& qt = tensor(o[0], "q");
    const Heads q(o[0], "q", qt), q_out(o[6], "q_out", qt, &qt);
    const at::Tensor &pos = tensor(o[2], "positions"), &freq = tensor(o[3], "inv_freq");
    if (pos.dim() != 2 || pos.scalar_type() != at::kInt || pos.size(1) != q.tokens)
      refuse("positions must be int32 [axes, %lld], got %s %s", (long long)q.tokens, at::toString(pos.scalar_type()),
             shape_of(pos).c_str());
    if (pos.stride(1) != 1 && q.tokens != 1) refuse("positions must have unit stride along tokens");
    if (freq.dim() != 1 || freq.scalar_type() != at::kFloat || !freq.is_contiguous())
      refuse("inv_freq must be float32 [rot_dim / 2], contiguous");
    on_device(pos, "positions", qt);
    on_device(freq, "inv_freq", qt);
    const int64_t pairs = freq.size(0), n_axes = pos.size(0);
    const int32_t* axes = ints(o[4], pairs, "axes", qt);
    const int adjacent = PyObject_IsTrue(o[5]);
    if (adjacent < 0) throw Refused();
    Heads k, k_out;
    if (o[1] != Py_None) {
      const at::Tensor& kt = tensor(o[1], "k");
      if (kt.dim() != 3 || kt.scalar_type() != qt.scalar_type() || kt.size(0) != q.tokens || kt.size(2) != q.dim)
        refuse("k must be %s [%lld, heads, %lld], got %s %s", at::toString(qt.scalar_type()), (long long)q.tokens,
               (long long)q.dim, at::toString(kt.scalar_type()), shape_of(kt).c_str());
      k = Heads(o[1], "k", qt);
      k_out = Heads(o[7], "k_out", qt, &kt);
    } else if (o[7] != Py_None) {
      refuse("k_out without k");
    }
    const int32_t dtype = dtype_code(qt);
    return launch("nvfp4_rope", qt, o[8], [&](void* stream) {
      return nvfp4_rope(q.tokens, q.dim, 2 * pairs, dtype, adjacent, static_cast<const int32_t*>(pos.data_ptr()),
                        n_axes, n_axes > 1 ? pos.stride(0) : q.tokens, static_cast<const float*>(freq.data_ptr()),
                        axes, q.p, q_out.p, q.heads, q.token, q.head, q_out.token, q_out.head, k.p, k_out.p, k.heads,
                        k.token, k.head, k_out.token, k_out.head, stream);
    });
  });
}

PyObject* cache_write(PyObject*, PyObject* const* o, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 8);
    const at::Tensor& kt = tensor(o[0], "k");
    const Heads k(o[0], "k", kt), v(o[1], "v", kt, &kt);
    const float *k_scale = scale(o[2], "k_scale", kt), *v_scale = scale(o[3], "v_scale", kt);
    const int32_t* slots = ints(o[4], k.tokens, "slot_map", kt);
    const Caches c(o[5], o[6], kt);
    if (c.heads != k.heads || c.dim != k.dim)
      refuse("k_cache must be [pages, %lld, page_size, %lld], got [%lld, %lld, %lld, %lld]", (long long)k.heads,
             (long long)k.dim, (long long)c.pages, (long long)c.heads, (long long)c.page_size, (long long)c.dim);
    const int32_t dtype = dtype_code(kt);
    return launch("nvfp4_kv_cache_write", kt, o[7], [&](void* stream) {
      return nvfp4_kv_cache_write(k.tokens, k.heads, k.dim, dtype, k.p, k.token, k.head, v.p, v.token, v.head, k_scale,
                                  v_scale, slots, c.k, c.v, c.pages, c.page_size, stream);
    });
  });
}

PyObject* paged_attention(PyObject*, PyObject* const* o, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    count(n_args, 13);
    const at::Tensor& qt = tensor(o[0], "q");
    const Heads q(o[0], "q", qt), out(o[9], "out", qt, &qt);
    const Caches c(o[1], o[2], qt);
    if (c.dim != q.dim) refuse("k_cache has head_dim %lld, q has %lld", (long long)c.dim, (long long)q.dim);
    const float *k_scale = scale(o[3], "k_scale", qt), *v_scale = scale(o[4], "v_scale", qt);
    const Table table(o[5], q.tokens, qt);
    const int32_t* lens = ints(o[6], q.tokens, "seq_lens", qt);
    const double softmax_scale = PyFloat_AsDouble(o[7]);
    if (softmax_scale == -1.0 && PyErr_Occurred()) throw Refused();
    const int64_t window = integer(o[8]);
    float* lse = nullptr;
    if (o[10] != Py_None) {
      const at::Tensor& t = tensor(o[10], "lse");
      if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != q.tokens || t.size(1) != q.heads ||
          !t.is_contiguous())
        refuse("lse must be float32 [%lld, %lld], contiguous", (long long)q.tokens, (long long)q.heads);
      on_device(t, "lse", qt);
      lse = static_cast<float*>(t.data_ptr());
    }
    const at::Tensor& ws = tensor(o[11], "workspace");
    if (ws.scalar_type() != at::kByte || !ws.is_contiguous()) refuse("workspace must be a contiguous uint8 tensor");
    on_device(ws, "workspace", qt);
    const int32_t dtype = dtype_code(qt);
    return launch("nvfp4_paged_attention", qt, o[12], [&](void* stream) {
      return nvfp4_paged_attention(q.tokens, q.heads, c.heads, q.dim, dtype, q.p, q.token, q.head, c.k, c.v, c.pages,
                                   c.page_size, k_scale, v_scale, table.p, table.columns, table.ld, lens,
                                   (float)softmax_scale, window, out.p, out.token, out.head, lse, ws.data_ptr(),
                                   ws.numel(), stream);
    });
  });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(block_table), METHOD(rope), METHOD(cache_write), METHOD(paged_attention),
                         METHOD(causal_conv), METHOD(causal_conv_step), METHOD(gated_delta_chunked), METHOD(gated_delta_step),
                         METHOD(group_norm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_bind() {
  PyObject* c = PyImport_ImportModule("torch._C");
  if (!c) return nullptr;
  get_device = PyObject_GetAttrString(c, "_cuda_getDevice");
  exchange_device = PyObject_GetAttrString(c, "_cuda_exchangeDevice");
  raw_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  Py_DECREF(c);
  if (!get_device || !exchange_device || !raw_stream) return nullptr;
  return PyModule_Create(&module);
}
