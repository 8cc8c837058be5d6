/*
 * nvfp4_kv.h — C ABI of the paged FP8 KV cache that stands between the qkv
 * and the output projection of an attention layer (MI355X, gfx950).
 *
 * The news article "Qwen3.8-27B最激进4bit量化开源，权重显存暴降2.9倍！" keeps the
 * KV cache in FP8 with static calibrated scales (sections 03 and 04).  nvfp4.h
 * holds that quantiser on dense rows; here are the cache in pages, what fills
 * it and what reads it:
 *
 *   nvfp4_kv_block_table    block tables and slot maps from request lengths
 *   nvfp4_rope              rotary positions with several axes (q and k heads)
 *   nvfp4_kv_cache_write    K and V rows to E4M3, into cache pages
 *   nvfp4_paged_attention   one new token per sequence against its pages
 *
 * All conventions of nvfp4.h hold (device pointers unless "host", the caller
 * owns every buffer, work enqueued on `stream`, validation before any HIP
 * call, status codes, NaN/Inf inputs unspecified but every access in bounds).
 * Besides:
 *   - The stream's device is the current device of the calling thread.
 *   - An output may not overlap another argument unless its comment says so.
 *   - heads * head_dim is at most 2^26, strides are below 2^40 elements.
 *   - Values that live on the device (lengths, page numbers, slots) cannot be
 *     refused by the call.  What each kernel does with a wrong one is part of
 *     its description; none of them reads or writes outside its buffers.
 *
 * The cache
 *   k_cache, v_cache : uint8 [num_pages][kv_heads][page_size][head_dim], dense,
 *                16-byte aligned, OCP E4M3FN bytes; the value of a byte is
 *                e4m3(byte) / scale with one static ENCODE scale per tensor
 *                (nvfp4_kv_scale_from_amax).  One head's tokens of a page are
 *                consecutive rows.  page_size: a multiple of 8, up to 1024.
 *   slot       : int32, page * page_size + offset of one token's place; a
 *                negative one means "no place".
 *   block table: int32 [n_seqs][ld_table], row r's entry j is the page that
 *                holds tokens [j*page_size, (j+1)*page_size) of sequence r.
 */
#ifndef NVFP4_KV_H
#define NVFP4_KV_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  NVFP4_KV_MAX_PAGE_SIZE = 1024,   /* tokens */
  NVFP4_KV_MAX_SEQ_LEN = 1 << 28,  /* max_pages * page_size of a block table */
  NVFP4_ROPE_MAX_AXES = 8,
  NVFP4_ROPE_MAX_HEAD_DIM = 1024
};

/*
 * nvfp4_kv_block_table — room in the cache for each request's new tokens.
 *
 * Request r holds cached_lens[r] = c tokens and brings new_lens[r] = n.  With
 * held = ceil(c/P) and all = ceil((c+n)/P) pages (P = page_size) it wants
 * need = all - held fresh pages, taken from the free list in request order:
 *
 *   fits_r   = c >= 0, n >= 0, all <= max_pages, and its last token's place in
 *              the slot map, sum_{i<=r} max(n_i, 0), is <= max_tokens
 *   upto_r   = used + sum of need over the fitting requests up to r
 *   served_r = fits_r and (need = 0 or upto_r <= n_free)
 *
 * A request is served whole or not at all.  Once the list is too short for one
 * request, later requests that need pages are not served either; those that
 * need none still are.
 *
 *   cached_lens, new_lens  int32 [n_seqs]
 *   free_pages   int32 [n_free] page numbers; NULL is allowed when n_free is 0
 *   free_used    int32 [1], how many entries of free_pages are already taken
 *                (a negative value counts as 0)
 *   block_table  int32 [n_seqs][ld_table], ld_table >= max_pages; the served
 *                requests' fresh pages are written behind their held ones,
 *                nothing else in it changes
 *   slot_map     int32 [max_tokens] (output): for the requests' new tokens one
 *                after another, each token's slot.  -1 for the tokens of a
 *                request that is not served, for a token whose held page is a
 *                negative table entry or whose slot passes 2^31 - 1, and
 *                behind the last token.
 *   seq_lens     int32 [n_seqs] (output): c + n where served, c elsewhere.
 *                May be cached_lens itself.
 *   token_starts int32 [n_seqs + 1] (output): where each request's tokens begin
 *                in slot_map, and where the last ones end; capped at max_tokens.
 *   first_pages  int32 [n_seqs] (output): -1 where not served, else the place in
 *                free_pages of its first fresh page (where it took none: of the
 *                next page that was free then, at most n_free).
 *   free_used_out int32 [1] (output): free_used plus the pages taken.  May be
 *                free_used itself.
 *
 * Errors: NULL pointers -> ERR_NULL; n_seqs, max_tokens, max_pages <= 0,
 * n_free < 0, sizes >= 2^31, page_size not a multiple of 8 in 8..1024,
 * max_pages * page_size > 2^28, ld_table < max_pages -> ERR_SHAPE; pointers
 * not 4-byte aligned -> ERR_ALIGN.
 */
nvfp4_status nvfp4_kv_block_table(int64_t n_seqs, const int32_t* cached_lens, const int32_t* new_lens,
                                  int64_t page_size, const int32_t* free_pages, int64_t n_free,
                                  const int32_t* free_used, int32_t* block_table, int64_t max_pages,
                                  int64_t ld_table, int32_t* slot_map, int64_t max_tokens, int32_t* seq_lens,
                                  int32_t* token_starts, int32_t* first_pages, int32_t* free_used_out,
                                  void* stream);

/*
 * nvfp4_rope — rotary positions on the query heads and, in the same call, the
 * key heads.  Pair i of a head (i < rot_dim/2) turns by the angle
 *
 *   angle = positions[axes[i]][token] * inv_freq[i]     (in 64 bits)
 *   (a, b) -> (a cos - b sin, b cos + a sin)            (in 32 bits, rounded once)
 *
 * with several position axes (time, height, width of images and video; text has
 * the same number on all).  adjacent = 0 pairs element i with i + rot_dim/2,
 * adjacent = 1 pairs 2i with 2i + 1.  Elements from rot_dim on are copied.
 *
 *   positions  int32 [n_axes][ld_pos], ld_pos >= tokens, or 0: one row for all
 *              axes, as text has it; any value
 *   inv_freq   fp32 [rot_dim/2]
 *   axes       int32 [rot_dim/2], each in 0..n_axes-1 (a value outside counts as
 *              the nearest one inside)
 *   q, q_out   [tokens][q_heads][head_dim] of type dtype (NVFP4_F32/BF16/F16);
 *              element (t, h, d) at t * *_token + h * *_head + d.  q_out may be
 *              q itself (same pointer and strides): then only the first rot_dim
 *              elements of each head are read and written.
 *   k, k_out   likewise with k_heads; k_heads = 0 leaves the keys out (k and
 *              k_out may be NULL).  16-byte aligned pointers and strides that
 *              are multiples of 16 bytes run fastest; element alignment is
 *              enough.
 *
 * Errors: NULL pointers -> ERR_NULL; tokens, q_heads, head_dim <= 0, k_heads <
 * 0, head_dim odd or > 1024, rot_dim odd, < 2 or > head_dim, n_axes outside 1..8,
 * strides below head_dim or that make heads or tokens overlap (*_head <
 * head_dim; *_token < (heads-1) * *_head + head_dim), sizes >= 2^31 ->
 * ERR_SHAPE; element alignment -> ERR_ALIGN; dtype or adjacent -> ERR_DTYPE.
 */
nvfp4_status nvfp4_rope(int64_t tokens, int64_t head_dim, int64_t rot_dim, int32_t dtype, int32_t adjacent,
                        const int32_t* positions, int64_t n_axes, int64_t ld_pos, const float* inv_freq,
                        const int32_t* axes, const void* q, void* q_out, int64_t q_heads, int64_t q_token,
                        int64_t q_head, int64_t q_out_token, int64_t q_out_head, const void* k, void* k_out,
                        int64_t k_heads, int64_t k_token, int64_t k_head, int64_t k_out_token, int64_t k_out_head,
                        void* stream);

/*
 * nvfp4_kv_cache_write — the new tokens' K and V rows, quantised by the rule of
 * nvfp4_kv_quantize_fp8 (y = fp32(x * s), E4M3 nearest-even, saturating at
 * 448), into the cache at their slots.
 *
 *   k, v       [tokens][kv_heads][head_dim] of type dtype; element (t, h, d) at
 *              t * *_token + h * *_head + d.  16-byte aligned, strides multiples
 *              of 16 bytes, head_dim a multiple of 8.
 *   k_scale, v_scale  device fp32[1], ENCODE scales (448 / calibrated amax)
 *   slot_map   int32 [tokens].  A token whose slot is negative or at least
 *              num_pages * page_size is left out.  Slots are distinct: if two
 *              tokens name the same one, it holds parts of either.
 *   k_cache, v_cache  the cache (see above).  Only the named slots change.
 *
 * Errors: NULL pointers -> ERR_NULL; tokens, kv_heads, head_dim, num_pages <=
 * 0, head_dim % 8 != 0, page_size not a multiple of 8 in 8..1024, overlapping
 * strides, sizes >= 2^31, num_pages * page_size >= 2^31 -> ERR_SHAPE;
 * alignment -> ERR_ALIGN; dtype -> ERR_DTYPE.
 */
nvfp4_status nvfp4_kv_cache_write(int64_t tokens, int64_t kv_heads, int64_t head_dim, int32_t dtype, const void* k,
                                  int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                                  const float* k_scale, const float* v_scale, const int32_t* slot_map,
                                  uint8_t* k_cache, uint8_t* v_cache, int64_t num_pages, int64_t page_size,
                                  void* stream);

/*
 * nvfp4_paged_attention — softmax attention of ONE new token per sequence over
 * its cached tokens (decode), grouped query heads:
 *
 *   s_j   = softmax_scale * sum_d q[d] * e4m3(k_j[d]) / k_scale
 *   out   = sum_j exp(s_j - lse) * e4m3(v_j) / v_scale,   lse = ln sum_j exp(s_j)
 *
 * over the seen tokens j of sequence r: max(0, len - window) <= j < len with len
 * = seq_lens[r] (window = 0: all of them).  len counts the new token when its K
 * and V were written to the cache before, as is usual.  Query head h reads KV
 * head h / (q_heads / kv_heads).  Where no token is seen (len <= 0), out is 0
 * and lse is -inf.
 *
 *   q, out     [n_seqs][q_heads][head_dim] of type dtype (NVFP4_F32/BF16/F16);
 *              element (r, h, d) at r * *_token + h * *_head + d; 16-byte
 *              aligned, strides multiples of 16 bytes
 *   head_dim   64, 128, 192 or 256
 *   block_table int32 [n_seqs][ld_table], of which max_pages columns are used.
 *              A length past max_pages * page_size counts as that many.  Tokens
 *              of a page number outside 0..num_pages-1 are not seen.
 *   seq_lens   int32 [n_seqs]
 *   lse        fp32 [n_seqs][q_heads] (output) or NULL
 *   workspace  device buffer of at least nvfp4_paged_attention_workspace()'s
 *              bytes, 16-byte aligned, for partial results.  Its contents need
 *              no preparation and mean nothing afterwards.  Calls that may run
 *              at the same time need one each.
 *
 * q, probabilities and values meet in matrix instructions: cache bytes are
 * exact in their 16-bit types, float32 queries are split into three bf16 parts
 * (nothing is lost), probabilities into two fp16 parts (22 bits), sums, maxima
 * and outputs are held in fp32.  The result depends on the lengths, the window,
 * the table's width and the device's CU count, and is the same in every call.
 *
 * Errors: NULL pointers -> ERR_NULL; sizes <= 0, head_dim not one of the four,
 * q_heads % kv_heads != 0, n_seqs * q_heads >= 2^31, max_pages * page_size *
 * q_heads > 2^37, window < 0, page_size and max_pages as above,
 * num_pages * page_size >= 2^31, ld_table < max_pages, overlapping strides,
 * out = q, workspace_bytes too small -> ERR_SHAPE; alignment -> ERR_ALIGN; dtype ->
 * ERR_DTYPE; softmax_scale not finite or <= 0 -> ERR_RANGE.
 */
nvfp4_status nvfp4_paged_attention(int64_t n_seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                   int32_t dtype, const void* q, int64_t q_token, int64_t q_head,
                                   const uint8_t* k_cache, const uint8_t* v_cache, int64_t num_pages,
                                   int64_t page_size, const float* k_scale, const float* v_scale,
                                   const int32_t* block_table, int64_t max_pages, int64_t ld_table,
                                   const int32_t* seq_lens, float softmax_scale, int64_t window, void* out,
                                   int64_t out_token, int64_t out_head, float* lse, void* workspace,
                                   int64_t workspace_bytes, void* stream);

/*
 * Bytes of workspace that nvfp4_paged_attention wants for these heads, whatever
 * the number and length of the sequences.  *bytes is host memory, written before
 * the call returns.
 *
 * Errors: NULL bytes -> ERR_NULL; heads and head_dim as above -> ERR_SHAPE.
 */
nvfp4_status nvfp4_paged_attention_workspace(int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_KV_H */
