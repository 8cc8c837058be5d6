// C ABI of the gated delta layer (include/nvfp4_gdn.h): argument validation (pure,
// before any HIP call) and dispatch onto the caller's stream.
#include "nvfp4_gdn.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "abi_checks.h"
#include "gdn_internal.h"

namespace {

using namespace nvfp4;

constexpr int64_t kMaxTokenHeads = (int64_t)1 << 37;  // tokens times value heads
constexpr int64_t kMaxSeqHeads = (int64_t)1 << 28;    // sequences times value heads

inline bool switch_ok(int32_t v) { return v == 0 || v == 1; }

inline bool delta_heads_ok(int64_t k_heads, int64_t v_heads, int64_t head_k, int64_t head_v) {
  return (head_k == 64 || head_k == 128) && head_v > 0 && head_v % 64 == 0 && head_v <= NVFP4_DELTA_MAX_HEAD_V &&
         row_ok(k_heads, head_k) && row_ok(v_heads, head_v) && v_heads % k_heads == 0;
}

inline bool heads16(const void* p, int64_t token, int64_t head, int es) {
  return aligned(p, 16) && by16(token, es) && by16(head, es);
}

nvfp4_status conv_check(const ConvArgs& a, int64_t tokens, int64_t channels, int64_t width, int64_t n_seqs,
                        int64_t num_slots) {
  if (!a.x || !a.weight || !a.slots || !a.state || !a.state_out || !a.out) return NVFP4_ERR_NULL;
  const int es = dtype_size(a.dtype);
  if (es == 0 || !switch_ok(a.activation)) return NVFP4_ERR_DTYPE;
  if (!size_ok(tokens) || channels <= 0 || channels > kMaxRow || width < 2 || width > NVFP4_CONV_MAX_WIDTH ||
      n_seqs <= 0 || n_seqs >= kMaxDim - 1 || !size_ok(num_slots) || a.ldx < channels || a.ldx >= kMaxStride ||
      a.ldo < channels || a.ldo >= kMaxStride || a.x == a.out)
    return NVFP4_ERR_SHAPE;
  if (!aligned(a.x, es) || !aligned(a.out, es) || !aligned(a.state, es) || !aligned(a.state_out, es) ||
      !aligned(a.weight, 4) || !aligned(a.bias, 4) || !aligned(a.slots, 4) || !aligned(a.token_starts, 4) ||
      !aligned(a.cached_lens, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// what the chunked call and the step have in common; sizes are 64-bit as the caller gave them
struct DeltaSizes {
  int64_t tokens, k_heads, v_heads, head_k, head_v, n_seqs, num_slots;
};

nvfp4_status delta_check(const DeltaArgs& a, const DeltaSizes& n) {
  if (!a.q.p || !a.k.p || !a.v.p || !a.a || !a.b || !a.a_log || !a.dt_bias || !a.slots || !a.state || !a.state_out ||
      !a.out.p)
    return NVFP4_ERR_NULL;
  const int es = dtype_size(a.dtype);
  if (es == 0) return NVFP4_ERR_DTYPE;
  if (!std::isfinite(a.scale) || !(a.scale > 0.0f) || !std::isfinite(a.eps) || !(a.eps >= 0.0f)) return NVFP4_ERR_RANGE;
  if (!size_ok(n.tokens) || n.n_seqs <= 0 || n.n_seqs >= kMaxDim - 1 || !size_ok(n.num_slots) ||
      !delta_heads_ok(n.k_heads, n.v_heads, n.head_k, n.head_v) || n.tokens * n.v_heads > kMaxTokenHeads ||
      n.n_seqs * n.v_heads > kMaxSeqHeads || a.out.p == a.v.p ||
      !strides_ok(n.k_heads, n.head_k, a.q.token, a.q.head) || !strides_ok(n.k_heads, n.head_k, a.k.token, a.k.head) ||
      !strides_ok(n.v_heads, n.head_v, a.v.token, a.v.head) ||
      !strides_ok(n.v_heads, n.head_v, a.out.token, a.out.head) || a.a_token < n.v_heads || a.a_token >= kMaxStride ||
      a.b_token < n.v_heads || a.b_token >= kMaxStride)
    return NVFP4_ERR_SHAPE;
  if (!heads16(a.q.p, a.q.token, a.q.head, es) || !heads16(a.k.p, a.k.token, a.k.head, es) ||
      !heads16(a.v.p, a.v.token, a.v.head, es) || !heads16(a.out.p, a.out.token, a.out.head, es) ||
      !aligned(a.a, es) || !aligned(a.b, es) || !aligned(a.a_log, 4) || !aligned(a.dt_bias, 4) ||
      !aligned(a.slots, 4) || !aligned(a.token_starts, 4) || !aligned(a.cached_lens, 4) || !aligned(a.state, 16) ||
      !aligned(a.state_out, 16) || !aligned(a.workspace, 16))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

void set_sizes(DeltaArgs& a, const DeltaSizes& n) {
  a.tokens = n.tokens;
  a.k_heads = (int)n.k_heads;
  a.v_heads = (int)n.v_heads;
  a.head_k = (int)n.head_k;
  a.head_v = (int)n.head_v;
  a.n_seqs = (int)n.n_seqs;
  a.num_slots = (int)n.num_slots;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_causal_conv(int64_t tokens, int64_t channels, int64_t width, int32_t dtype, const void* x,
                               int64_t ldx, const float* weight, const float* bias, int32_t activation,
                               int64_t n_seqs, const int32_t* token_starts, const int32_t* cached_lens,
                               const int32_t* slots, const void* state, void* state_out, int64_t num_slots, void* out,
                               int64_t ldo, void* stream) {
  if (!token_starts) return NVFP4_ERR_NULL;
  ConvArgs a = {tokens, 0, 0, dtype, x, ldx, weight, bias, activation, 0, token_starts, cached_lens, slots, state,
                state_out, 0, out, ldo};
  const nvfp4_status s = conv_check(a, tokens, channels, width, n_seqs, num_slots);
  if (s != NVFP4_OK) return s;
  a.channels = (int)channels;
  a.width = (int)width;
  a.n_seqs = (int)n_seqs;
  a.num_slots = (int)num_slots;
  if (!device_ok()) return NVFP4_ERR_DEVICE;
  return done(launch_causal_conv(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_causal_conv_step(int64_t n_seqs, int64_t channels, int64_t width, int32_t dtype, const void* x,
                                    int64_t ldx, const float* weight, const float* bias, int32_t activation,
                                    const int32_t* slots, const void* state, void* state_out, int64_t num_slots,
                                    void* out, int64_t ldo, void* stream) {
  ConvArgs a = {n_seqs, 0, 0, dtype, x, ldx, weight, bias, activation, 0, nullptr, nullptr, slots, state,
                state_out, 0, out, ldo};
  const nvfp4_status s = conv_check(a, n_seqs, channels, width, n_seqs, num_slots);
  if (s != NVFP4_OK) return s;
  a.channels = (int)channels;
  a.width = (int)width;
  a.n_seqs = (int)n_seqs;
  a.num_slots = (int)num_slots;
  if (!device_ok()) return NVFP4_ERR_DEVICE;
  return done(launch_causal_conv_step(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_gated_delta_workspace(int64_t tokens, int64_t n_seqs, int64_t k_heads, int64_t v_heads,
                                         int64_t head_k, int64_t head_v, int32_t dtype, int64_t* bytes) {
  if (!bytes) return NVFP4_ERR_NULL;
  if (dtype_size(dtype) == 0) return NVFP4_ERR_DTYPE;
  if (!size_ok(tokens) || n_seqs <= 0 || n_seqs >= kMaxDim - 1 || !delta_heads_ok(k_heads, v_heads, head_k, head_v) ||
      tokens * v_heads > kMaxTokenHeads || n_seqs * v_heads > kMaxSeqHeads)
    return NVFP4_ERR_SHAPE;
  *bytes = gated_delta_workspace_bytes(tokens, n_seqs, (int)k_heads, (int)v_heads, (int)head_k, (int)head_v, dtype);
  return NVFP4_OK;
}

nvfp4_status nvfp4_gated_delta_chunked(int64_t tokens, int64_t k_heads, int64_t v_heads, int64_t head_k,
                                       int64_t head_v, int32_t dtype, const void* q, int64_t q_token, int64_t q_head,
                                       const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                                       int64_t v_head, const void* a, int64_t a_token, const void* b, int64_t b_token,
                                       const float* a_log, const float* dt_bias, float scale, float eps,
                                       int64_t n_seqs, const int32_t* token_starts, const int32_t* cached_lens,
                                       const int32_t* slots, const float* state, float* state_out, int64_t num_slots,
                                       void* out, int64_t out_token, int64_t out_head, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
  if (!token_starts || !workspace) return NVFP4_ERR_NULL;
  DeltaArgs d = {0, 0, 0, 0, 0, dtype, {q, q_token, q_head}, {k, k_token, k_head}, {v, v_token, v_head}, a, a_token, b,
                 b_token, a_log, dt_bias, scale, eps, 0, token_starts, cached_lens, slots, state, state_out, 0,
                 {out, out_token, out_head}, workspace};
  const DeltaSizes n = {tokens, k_heads, v_heads, head_k, head_v, n_seqs, num_slots};
  const nvfp4_status s = delta_check(d, n);
  if (s != NVFP4_OK) return s;
  set_sizes(d, n);
  if (workspace_bytes < gated_delta_workspace_bytes(tokens, n_seqs, d.k_heads, d.v_heads, d.head_k, d.head_v, dtype))
    return NVFP4_ERR_SHAPE;
  if (!device_ok()) return NVFP4_ERR_DEVICE;
  return done(launch_gated_delta_chunked(d, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_gated_delta_step(int64_t n_seqs, int64_t k_heads, int64_t v_heads, int64_t head_k, int64_t head_v,
                                    int32_t dtype, const void* q, int64_t q_token, int64_t q_head, const void* k,
                                    int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                                    const void* a, int64_t a_token, const void* b, int64_t b_token,
                                    const float* a_log, const float* dt_bias, float scale, float eps,
                                    const int32_t* slots, const float* state, float* state_out, int64_t num_slots,
                                    void* out, int64_t out_token, int64_t out_head, void* stream) {
  DeltaArgs d = {0, 0, 0, 0, 0, dtype, {q, q_token, q_head}, {k, k_token, k_head}, {v, v_token, v_head}, a, a_token, b,
                 b_token, a_log, dt_bias, scale, eps, 0, nullptr, nullptr, slots, state, state_out, 0,
                 {out, out_token, out_head}, nullptr};
  const DeltaSizes n = {n_seqs, k_heads, v_heads, head_k, head_v, n_seqs, num_slots};
  const nvfp4_status s = delta_check(d, n);
  if (s != NVFP4_OK) return s;
  set_sizes(d, n);
  if (!device_ok()) return NVFP4_ERR_DEVICE;
  return done(launch_gated_delta_step(d, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_group_norm(int64_t tokens, int64_t groups, int64_t group_dim, int32_t dtype, const void* x,
                              int64_t x_token, int64_t x_group, const float* weight, int64_t weight_group,
                              const float* bias, const void* gate, int64_t gate_token, int64_t gate_group,
                              int32_t activation, int32_t centred, float eps, void* out, int64_t out_token,
                              int64_t out_group, void* stream) {
  if (!x || !weight || !out) return NVFP4_ERR_NULL;
  const int es = dtype_size(dtype);
  if (es == 0 || !switch_ok(activation) || !switch_ok(centred)) return NVFP4_ERR_DTYPE;
  if (!std::isfinite(eps) || !(eps >= 0.0f)) return NVFP4_ERR_RANGE;
  auto same = [&](const void* p, int64_t token, int64_t group) {
    return out == p && (token != out_token || group != out_group);
  };
  if (!size_ok(tokens) || !row_ok(groups, group_dim) || group_dim > NVFP4_NORM_MAX_GROUP ||
      (weight_group != 0 && weight_group != group_dim) || !strides_ok(groups, group_dim, x_token, x_group) ||
      !strides_ok(groups, group_dim, out_token, out_group) || same(x, x_token, x_group) ||
      (gate && (!strides_ok(groups, group_dim, gate_token, gate_group) || same(gate, gate_token, gate_group))))
    return NVFP4_ERR_SHAPE;
  if (!aligned(x, es) || !aligned(gate, es) || !aligned(out, es) || !aligned(weight, 4) || !aligned(bias, 4))
    return NVFP4_ERR_ALIGN;
  if (!device_ok()) return NVFP4_ERR_DEVICE;
  const NormArgs a = {tokens, (int)groups, (int)group_dim, dtype, {x, x_token, x_group}, {gate, gate_token, gate_group},
                      {out, out_token, out_group}, weight, (int)weight_group, bias, activation, centred, eps};
  return done(launch_group_norm(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
