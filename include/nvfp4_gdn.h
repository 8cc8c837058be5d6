/*
 * nvfp4_gdn.h — C ABI of what stands between the fused input projection and
 * the output projection of a Gated DeltaNet layer (MI355X, gfx950).
 *
 * The news article "Qwen3.8-27B最激进4bit量化开源，权重显存暴降2.9倍！" describes
 * these layers in section 01: a gated delta rule on L2-normalised queries and
 * keys, a forget gate held in log space, a write strength, and a state of fixed
 * size.  nvfp4.h holds the layer's two matrix products; here is the rest:
 *
 *   nvfp4_causal_conv          causal depthwise convolution of ragged prompts
 *   nvfp4_causal_conv_step     the same for one new token a sequence
 *   nvfp4_gated_delta_chunked  the gated delta rule over ragged prompts
 *   nvfp4_gated_delta_step     the same for one new token a sequence
 *   nvfp4_group_norm           a norm of each head with a gate or an activation
 *
 * All conventions of nvfp4.h hold (device pointers unless "host", the caller
 * owns every buffer, work enqueued on `stream`, validation before any HIP
 * call, status codes, NaN/Inf inputs unspecified but every access in bounds).
 * Besides:
 *   - The stream's device is the current device of the calling thread.
 *   - An output may not overlap another argument unless its comment says so.
 *   - Strides are in elements, below 2^40.  Tensors of heads are addressed by
 *     (token, head) strides with head_dim consecutive elements.  A token's heads
 *     lie one behind another and end before the next token (token >= (heads - 1) *
 *     head + head_dim), as in nvfp4_kv.h: other strides, those of tensors laid out
 *     by heads first among them, are refused.
 *   - Values that live on the device (slots, starts) cannot be refused by the
 *     call.  What a wrong one does is part of the description; none leads to an
 *     access outside the buffers.
 *
 * Ragged prompts
 *   The tokens of n_seqs sequences lie one after another.
 *   token_starts int32 [n_seqs + 1]: sequence r has the rows token_starts[r] to
 *                token_starts[r+1] - 1 (nvfp4_kv_block_table writes it so).
 *                Starts outside 0..tokens count as the nearer end; a sequence
 *                whose end is not behind its start has no rows.  Rows of no
 *                sequence are not read, and their outputs stay as they were.
 *                Starts that fall again make the results unspecified.
 *   cached_lens  int32 [n_seqs] or NULL: a sequence with cached_lens[r] <= 0
 *                starts from a state of zeros, one with more (every one, where it
 *                is NULL) from the state in its slot.
 *
 * States
 *   Every sequence has a slot: slots, int32 [n_seqs], in 0..num_slots-1.
 *   state        [num_slots][...]: read at the sequence's slot
 *   state_out    of the same shape: written at the sequence's slot, nowhere else.
 *                May be state itself; else it may not overlap it.
 *   A sequence without rows, or whose slot is not in 0..num_slots-1 (as -1 in
 *   rows that pad a batch), is left out: its outputs and states stay as they
 *   were.  No two sequences of a call may have the same slot: what is then in
 *   the slot, and with state_out = state their outputs, are unspecified.
 */
#ifndef NVFP4_GDN_H
#define NVFP4_GDN_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { NVFP4_ACT_NONE = 0, NVFP4_ACT_SILU = 1 };

enum {
  NVFP4_CONV_MAX_WIDTH = 4,
  NVFP4_NORM_MAX_GROUP = 8192,  /* elements of a group */
  NVFP4_DELTA_MAX_HEAD_V = 256
};

/*
 * nvfp4_causal_conv — for each sequence, with x_t = its inputs,
 *
 *   out_t[c] = act(bias[c] + sum_{j<width} weight[c][j] x_{t - (width-1) + j}[c])
 *
 * where inputs before the sequence's first token are the width - 1 rows of its
 * state (zeros for a sequence that starts from zeros).  Its last width - 1
 * inputs are the state it leaves.
 *
 *   x, out     [tokens][ldx], [tokens][ldo] elements of dtype, channels of each
 *              row used; any element alignment (16-byte rows are faster)
 *   weight     fp32 [channels][width], width 2..4; the last column meets the
 *              newest input
 *   bias       fp32 [channels] or NULL
 *   activation NVFP4_ACT_NONE or NVFP4_ACT_SILU: y / (1 + e^-y)
 *   state, state_out  [num_slots][width-1][channels] of dtype, dense, the newest
 *              input last; exact copies of inputs
 *
 * Sums in fp32, one rounding to dtype.
 *
 * Errors: NULL pointers -> ERR_NULL; sizes <= 0 or >= 2^31, channels > 2^26,
 * width outside 2..4, ldx or ldo < channels, out = x -> ERR_SHAPE; pointers not
 * aligned to their elements -> ERR_ALIGN; dtype, activation -> ERR_DTYPE.
 */
nvfp4_status nvfp4_causal_conv(int64_t tokens, int64_t channels, int64_t width, int32_t dtype, const void* x,
                               int64_t ldx, const float* weight, const float* bias, int32_t activation,
                               int64_t n_seqs, const int32_t* token_starts, const int32_t* cached_lens,
                               const int32_t* slots, const void* state, void* state_out, int64_t num_slots, void* out,
                               int64_t ldo, void* stream);

/*
 * nvfp4_causal_conv_step — the same for one new token a sequence: row r of x and
 * out belongs to the sequence in slot slots[r], which starts from its state.
 */
nvfp4_status nvfp4_causal_conv_step(int64_t n_seqs, int64_t channels, int64_t width, int32_t dtype, const void* x,
                                    int64_t ldx, const float* weight, const float* bias, int32_t activation,
                                    const int32_t* slots, const void* state, void* state_out, int64_t num_slots,
                                    void* out, int64_t ldo, void* stream);

/*
 * nvfp4_gated_delta_chunked — for each sequence and value head h, token after
 * token, with the state S [head_k][head_v]:
 *
 *   k~ = k / sqrt(|k|^2 + eps),  q~ = q / sqrt(|q|^2 + eps)   of key head
 *                                                      h / (v_heads / k_heads)
 *   g = -e^a_log[h] ln(1 + e^(a[h] + dt_bias[h])),  beta = 1 / (1 + e^-b[h])
 *   S <- e^g S;  S <- S + k~ (beta (v - S^T k~))^T;  out = scale S^T q~
 *
 * Finite rows of q and k of any size are normalised; a row of zeros is one of
 * zeros, also where eps is 0.  A NaN in a, b, k or v is never lost: the state
 * behind it has NaNs (which outputs have them is unspecified).
 *
 *   q, k       [tokens][k_heads][head_k], v and out [tokens][v_heads][head_v],
 *              elements of dtype; pointers 16-byte aligned, strides multiples of
 *              16 bytes; the rows of a tensor may not overlap.  v_heads is a
 *              multiple of k_heads, head_k is 64 or 128, head_v a multiple of 64
 *              up to 256.
 *   a, b       [tokens][v_heads] of dtype, rows a_token and b_token elements
 *              apart; any element alignment
 *   a_log, dt_bias  fp32 [v_heads]
 *   state, state_out  fp32 [num_slots][v_heads][head_k][head_v], dense, 16-byte
 *              aligned
 *   workspace  device buffer of at least nvfp4_gated_delta_workspace()'s bytes,
 *              16-byte aligned.  Its contents need no preparation and mean
 *              nothing afterwards.  Calls that may run at the same time need one
 *              each.
 *
 * Tokens are taken in chunks of 64: what a chunk's tokens write into each other
 * is solved for at once (a unit lower triangular system), and only the chunks
 * follow one another.  Products run on the matrix units with operands cut into
 * fp16 parts: q, k, scaled by a power of two a row (exact but for 2^-29 of the
 * row's length; float32 in two parts), states, decays, solutions and values in
 * two (2^-22 of an element's value, or 2^-29 of the largest of its column, of the
 * state and of beta v).  Sums, states and gates are fp32, sums of log decays 64
 * bits.  Where heads are few, parts of a sequence are taken at once and joined in
 * fp32.  nvfp4_gated_delta_step has fp32 throughout.  The
 * result is the same in every call on cards with as many CUs.
 *
 * Errors: NULL pointers -> ERR_NULL; sizes <= 0 or >= 2^31, head counts and
 * sizes other than above, heads * head_dim > 2^26, tokens * v_heads > 2^37,
 * n_seqs * v_heads > 2^28, other strides than above, out = v, workspace_bytes
 * too small -> ERR_SHAPE; alignment -> ERR_ALIGN; dtype -> ERR_DTYPE; scale not finite
 * or <= 0, eps not finite or < 0 -> ERR_RANGE.
 */
nvfp4_status nvfp4_gated_delta_chunked(int64_t tokens, int64_t k_heads, int64_t v_heads, int64_t head_k,
                                       int64_t head_v, int32_t dtype, const void* q, int64_t q_token, int64_t q_head,
                                       const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                                       int64_t v_head, const void* a, int64_t a_token, const void* b, int64_t b_token,
                                       const float* a_log, const float* dt_bias, float scale, float eps,
                                       int64_t n_seqs, const int32_t* token_starts, const int32_t* cached_lens,
                                       const int32_t* slots, const float* state, float* state_out, int64_t num_slots,
                                       void* out, int64_t out_token, int64_t out_head, void* workspace,
                                       int64_t workspace_bytes, void* stream);

/*
 * Bytes of workspace that nvfp4_gated_delta_chunked wants for calls of up to
 * these many tokens and sequences.  *bytes is host memory, written before the
 * call returns.  About 26 KiB a value head and 53 KiB a key head (16-bit types,
 * head_k 128) for each chunk of 64 tokens and each sequence, and what parts want: 243
 * MiB for 8192 tokens of 8 and 48 heads of 128, 3.3 GiB for 131072.
 *
 * Errors: NULL bytes -> ERR_NULL; sizes and heads as above -> ERR_SHAPE; dtype ->
 * ERR_DTYPE.
 */
nvfp4_status nvfp4_gated_delta_workspace(int64_t tokens, int64_t n_seqs, int64_t k_heads, int64_t v_heads,
                                         int64_t head_k, int64_t head_v, int32_t dtype, int64_t* bytes);

/*
 * nvfp4_gated_delta_step — the same rule for one new token a sequence: row r of
 * q, k, v, a, b and out belongs to the sequence in slot slots[r], which starts
 * from its state.  Everything in fp32.  Errors as above.
 */
nvfp4_status nvfp4_gated_delta_step(int64_t n_seqs, int64_t k_heads, int64_t v_heads, int64_t head_k, int64_t head_v,
                                    int32_t dtype, const void* q, int64_t q_token, int64_t q_head, const void* k,
                                    int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                                    const void* a, int64_t a_token, const void* b, int64_t b_token,
                                    const float* a_log, const float* dt_bias, float scale, float eps,
                                    const int32_t* slots, const float* state, float* state_out, int64_t num_slots,
                                    void* out, int64_t out_token, int64_t out_head, void* stream);

/*
 * nvfp4_group_norm — each token's channels, last and consecutive in groups, are
 * normalised group by group:
 *
 *   m = mean(x) where centred, else 0;  y = (x - m) / sqrt(mean((x-m)^2) + eps)
 *   y = y weight + bias;  out = y act(gate), or act(y) without a gate
 *
 *   x, gate, out  [tokens][groups][group_dim] of dtype; any element alignment
 *              (16-byte rows of groups are faster).  gate may be NULL.  out may
 *              be x or gate itself, with that tensor's strides.
 *   weight     fp32, of group i from weight + i * weight_group; weight_group is
 *              group_dim, or 0 where all groups share one row
 *   bias       fp32, laid out like weight, or NULL
 *   activation NVFP4_ACT_NONE or NVFP4_ACT_SILU
 *   group_dim  up to 8192
 *
 * Everything in fp32, the mean taken off before squares are summed; one rounding
 * to dtype.  Finite groups of any size are normalised; where the squares are all 0
 * and eps is too, (x - m) / 0 counts as 0.
 *
 * Errors: NULL pointers -> ERR_NULL; sizes <= 0 or >= 2^31, group_dim > 8192,
 * groups * group_dim > 2^26, weight_group, other strides than above, out = x or
 * gate with other strides -> ERR_SHAPE; pointers not aligned to their elements ->
 * ERR_ALIGN; dtype, activation, centred not 0 or 1 -> ERR_DTYPE; eps not finite
 * or < 0 -> ERR_RANGE.
 */
nvfp4_status nvfp4_group_norm(int64_t tokens, int64_t groups, int64_t group_dim, int32_t dtype, const void* x,
                              int64_t x_token, int64_t x_group, const float* weight, int64_t weight_group,
                              const float* bias, const void* gate, int64_t gate_token, int64_t gate_group,
                              int32_t activation, int32_t centred, float eps, void* out, int64_t out_token,
                              int64_t out_group, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_GDN_H */
