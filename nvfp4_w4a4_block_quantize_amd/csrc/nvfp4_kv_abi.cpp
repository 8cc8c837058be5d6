// C ABI of the paged KV cache (include/nvfp4_kv.h): argument validation (pure,
// before any HIP call) and dispatch onto the caller's stream.
#include "nvfp4_kv.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kv_internal.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int dtype_size(int32_t dt) { return dt == NVFP4_F32 ? 4 : (dt == NVFP4_BF16 || dt == NVFP4_F16) ? 2 : 0; }

// true when a GPU is usable from this thread (checked only after validation)
inline bool device_ok() {
  int dev = -1;
  return hipGetDevice(&dev) == hipSuccess && dev >= 0;
}

constexpr int64_t kMaxDim = (int64_t)1 << 31;     // sizes are below 2^31
constexpr int64_t kMaxStride = (int64_t)1 << 40;  // strides too large for a byte offset are refused
constexpr int64_t kMaxRow = (int64_t)1 << 26;     // elements of one token's heads

constexpr int64_t kMaxReach = (int64_t)1 << 37;   // tokens of a full table row times query heads

inline bool size_ok(int64_t n) { return n > 0 && n < kMaxDim; }

// heads * head_dim elements of a token; both factors are checked before they are multiplied
inline bool row_ok(int64_t heads, int64_t head_dim) {
  return heads > 0 && head_dim > 0 && heads < kMaxRow && head_dim < kMaxRow && heads * head_dim <= kMaxRow;
}

// no two elements of a [tokens][heads][head_dim] tensor share a place
inline bool strides_ok(int64_t heads, int64_t head_dim, int64_t token, int64_t head) {
  if (token >= kMaxStride || head >= kMaxStride || head < head_dim || token < head_dim) return false;
  return (heads - 1) * head + head_dim <= token;
}

inline bool page_ok(int64_t page_size) {
  return page_size >= 8 && page_size <= NVFP4_KV_MAX_PAGE_SIZE && page_size % 8 == 0;
}

inline bool table_ok(int64_t max_pages, int64_t page_size, int64_t ld_table) {
  return max_pages > 0 && max_pages <= NVFP4_KV_MAX_SEQ_LEN && max_pages * page_size <= NVFP4_KV_MAX_SEQ_LEN &&
         ld_table >= max_pages && ld_table < kMaxStride;
}

inline bool cache_ok(int64_t num_pages, int64_t page_size) {
  return size_ok(num_pages) && page_ok(page_size) && num_pages * page_size < kMaxDim;
}

inline bool attention_heads_ok(int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 192 && head_dim != 256) return false;
  return row_ok(q_heads, head_dim) && row_ok(kv_heads, head_dim) && q_heads % kv_heads == 0;
}

inline bool by16(int64_t stride, int es) { return (stride * es) % 16 == 0; }

inline nvfp4_status done(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_DEVICE; }

}  // namespace

extern "C" {

nvfp4_status nvfp4_kv_block_table(int64_t n_seqs, const int32_t* cached_lens, const int32_t* new_lens,
                                  int64_t page_size, const int32_t* free_pages, int64_t n_free,
                                  const int32_t* free_used, int32_t* block_table, int64_t max_pages,
                                  int64_t ld_table, int32_t* slot_map, int64_t max_tokens, int32_t* seq_lens,
                                  int32_t* token_starts, int32_t* first_pages, int32_t* free_used_out,
                                  void* stream) {
  if (!cached_lens || !new_lens || !free_used || !block_table || !slot_map || !seq_lens || !token_starts ||
      !first_pages || !free_used_out || (!free_pages && n_free != 0))
    return NVFP4_ERR_NULL;
  if (n_seqs <= 0 || n_seqs >= kMaxDim - 1 || !size_ok(max_tokens) || n_free < 0 || n_free >= kMaxDim ||
      !page_ok(page_size) || !table_ok(max_pages, page_size, ld_table))
    return NVFP4_ERR_SHAPE;
  if (!aligned(cached_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(free_used, 4) ||
      !aligned(block_table, 4) || !aligned(slot_map, 4) || !aligned(seq_lens, 4) || !aligned(token_starts, 4) ||
      !aligned(first_pages, 4) || !aligned(free_used_out, 4))
    return NVFP4_ERR_ALIGN;
  if (!device_ok()) return NVFP4_ERR_DEVICE;
  nvfp4::BlockTableArgs a;
  a.n_seqs = (int)n_seqs;
  a.cached_lens = cached_lens;
  a.new_lens = new_lens;
  a.page_size = (int)page_size;
  a.free_pages = free_pages;
  a.n_free = (int)n_free;
  a.free_used = free_used;
  a.block_table = block_table;
  a.max_pages = (int)max_pages;
  a.ld_table = ld_table;
  a.slot_map = slot_map;
  a.max_tokens = (int)max_tokens;
  a.seq_lens = seq_lens;
  a.token_starts = token_starts;
  a.first_pages = first_pages;
  a.free_used_out = free_used_out;
  return done(nvfp4::launch_kv_block_table(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_rope(int64_t tokens, int64_t head_dim, int64_t rot_dim, int32_t dtype, int32_t adjacent,
                        const int32_t* positions, int64_t n_axes, int64_t ld_pos, const float* inv_freq,
                        const int32_t* axes, const void* q, void* q_out, int64_t q_heads, int64_t q_token,
                        int64_t q_head, int64_t q_out_token, int64_t q_out_head, const void* k, void* k_out,
                        int64_t k_heads, int64_t k_token, int64_t k_head, int64_t k_out_token, int64_t k_out_head,
                        void* stream) {
  if (!positions || !inv_freq || !axes || !q || !q_out || (k_heads != 0 && (!k || !k_out))) return NVFP4_ERR_NULL;
  const int es = dtype_size(dtype);
  if (es == 0 || (adjacent != 0 && adjacent != 1)) return NVFP4_ERR_DTYPE;
  if (!size_ok(tokens) || head_dim <= 0 || head_dim > NVFP4_ROPE_MAX_HEAD_DIM || head_dim % 2 != 0 || rot_dim < 2 ||
      rot_dim % 2 != 0 || rot_dim > head_dim || n_axes < 1 || n_axes > NVFP4_ROPE_MAX_AXES ||
      (ld_pos < tokens && ld_pos != 0) || ld_pos >= kMaxStride || !row_ok(q_heads, head_dim) || k_heads < 0 ||
      (k_heads > 0 && !row_ok(k_heads, head_dim)))
    return NVFP4_ERR_SHAPE;
  if (!strides_ok(q_heads, head_dim, q_token, q_head) || !strides_ok(q_heads, head_dim, q_out_token, q_out_head) ||
      (q == q_out && (q_token != q_out_token || q_head != q_out_head)))
    return NVFP4_ERR_SHAPE;
  if (k_heads > 0 &&
      (!strides_ok(k_heads, head_dim, k_token, k_head) || !strides_ok(k_heads, head_dim, k_out_token, k_out_head) ||
       (k == k_out && (k_token != k_out_token || k_head != k_out_head))))
    return NVFP4_ERR_SHAPE;
  if (!aligned(positions, 4) || !aligned(inv_freq, 4) || !aligned(axes, 4) || !aligned(q, es) || !aligned(q_out, es) ||
      (k_heads > 0 && (!aligned(k, es) || !aligned(k_out, es))))
    return NVFP4_ERR_ALIGN;
  if (!device_ok()) return NVFP4_ERR_DEVICE;
  nvfp4::RopeArgs a;
  a.tokens = tokens;
  a.head_dim = (int)head_dim;
  a.rot_dim = (int)rot_dim;
  a.dtype = dtype;
  a.adjacent = adjacent;
  a.positions = positions;
  a.n_axes = (int)n_axes;
  a.ld_pos = ld_pos;
  a.inv_freq = inv_freq;
  a.axes = axes;
  a.q = {q, q_token, q_head};
  a.q_out = {q_out, q_out_token, q_out_head};
  a.q_heads = (int)q_heads;
  a.k = {k, k_token, k_head};
  a.k_out = {k_out, k_out_token, k_out_head};
  a.k_heads = (int)k_heads;
  return done(nvfp4::launch_rope(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_cache_write(int64_t tokens, int64_t kv_heads, int64_t head_dim, int32_t dtype, const void* k,
                                  int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                                  const float* k_scale, const float* v_scale, const int32_t* slot_map,
                                  uint8_t* k_cache, uint8_t* v_cache, int64_t num_pages, int64_t page_size,
                                  void* stream) {
  if (!k || !v || !k_scale || !v_scale || !slot_map || !k_cache || !v_cache) return NVFP4_ERR_NULL;
  const int es = dtype_size(dtype);
  if (es == 0) return NVFP4_ERR_DTYPE;
  if (!size_ok(tokens) || !row_ok(kv_heads, head_dim) || head_dim % 8 != 0 || !cache_ok(num_pages, page_size) ||
      !strides_ok(kv_heads, head_dim, k_token, k_head) || !strides_ok(kv_heads, head_dim, v_token, v_head) ||
      k_cache == v_cache)
    return NVFP4_ERR_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16) || !by16(k_token, es) || !by16(k_head, es) || !by16(v_token, es) ||
      !by16(v_head, es) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(slot_map, 4) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return NVFP4_ERR_ALIGN;
  if (!device_ok()) return NVFP4_ERR_DEVICE;
  nvfp4::CacheWriteArgs a;
  a.tokens = tokens;
  a.kv_heads = (int)kv_heads;
  a.head_dim = (int)head_dim;
  a.dtype = dtype;
  a.k = {k, k_token, k_head};
  a.v = {v, v_token, v_head};
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.slot_map = slot_map;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_pages = (int)num_pages;
  a.page_size = (int)page_size;
  return done(nvfp4::launch_kv_cache_write(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_paged_attention_workspace(int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t* bytes) {
  if (!bytes) return NVFP4_ERR_NULL;
  if (!attention_heads_ok(q_heads, kv_heads, head_dim)) return NVFP4_ERR_SHAPE;
  *bytes = nvfp4::attention_workspace_bytes((int)q_heads, (int)kv_heads, (int)head_dim);
  return NVFP4_OK;
}

nvfp4_status nvfp4_paged_attention(int64_t n_seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                   int32_t dtype, const void* q, int64_t q_token, int64_t q_head,
                                   const uint8_t* k_cache, const uint8_t* v_cache, int64_t num_pages,
                                   int64_t page_size, const float* k_scale, const float* v_scale,
                                   const int32_t* block_table, int64_t max_pages, int64_t ld_table,
                                   const int32_t* seq_lens, float softmax_scale, int64_t window, void* out,
                                   int64_t out_token, int64_t out_head, float* lse, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out || !workspace)
    return NVFP4_ERR_NULL;
  const int es = dtype_size(dtype);
  if (es == 0) return NVFP4_ERR_DTYPE;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.0f)) return NVFP4_ERR_RANGE;
  if (!size_ok(n_seqs) || !attention_heads_ok(q_heads, kv_heads, head_dim) || n_seqs * q_heads >= kMaxDim ||
      window < 0 || q == out || !cache_ok(num_pages, page_size) || !table_ok(max_pages, page_size, ld_table) ||
      max_pages * page_size * q_heads > kMaxReach ||
      !strides_ok(q_heads, head_dim, q_token, q_head) || !strides_ok(q_heads, head_dim, out_token, out_head))
    return NVFP4_ERR_SHAPE;
  if (!aligned(q, 16) || !by16(q_token, es) || !by16(q_head, es) || !aligned(out, 16) || !by16(out_token, es) ||
      !by16(out_head, es) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  if (workspace_bytes < nvfp4::attention_workspace_bytes((int)q_heads, (int)kv_heads, (int)head_dim))
    return NVFP4_ERR_SHAPE;
  if (!device_ok()) return NVFP4_ERR_DEVICE;
  nvfp4::PagedAttentionArgs a;
  a.n_seqs = (int)n_seqs;
  a.q_heads = (int)q_heads;
  a.kv_heads = (int)kv_heads;
  a.head_dim = (int)head_dim;
  a.dtype = dtype;
  a.q = {q, q_token, q_head};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_pages = (int)num_pages;
  a.page_size = (int)page_size;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_table = block_table;
  a.max_pages = (int)max_pages;
  a.ld_table = ld_table;
  a.seq_lens = seq_lens;
  a.softmax_scale = softmax_scale;
  a.window = window;
  a.out = {out, out_token, out_head};
  a.lse = lse;
  a.workspace = workspace;
  return done(nvfp4::launch_paged_attention(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
