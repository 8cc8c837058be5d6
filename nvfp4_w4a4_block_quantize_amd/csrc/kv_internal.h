// Launchers of the paged KV cache's kernels (include/nvfp4_kv.h).  Arguments are
// validated by the caller (nvfp4_kv_abi.cpp); these only launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// n / d for n below 2^31 as one high multiply and a shift.  With 2^s < d <= 2^(s+1)
// and mul = ceil(2^(32+s) / d) (below 2^32, since d > 2^s), mul * d exceeds
// 2^(32+s) by less than d <= 2^(s+1), so n * mul / 2^(32+s) exceeds n / d by less
// than n / (2^31 d): for n < 2^31 never enough to reach the next multiple of 1/d.
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div), mul(0), shift(0) {
    if (div < 2) return;
    while ((2ull << shift) < div) ++shift;
    mul = (uint32_t)(((1ull << (32 + shift)) + div - 1) / div);
  }
#if defined(__HIPCC__)
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return d == 1 ? n : __umulhi(n, mul) >> shift; }
#endif
};

// of a launch: the grid's threads are counted in 32 bits, and larger calls go in pieces
constexpr int64_t kMostWorkgroups = 1 << 20;

struct BlockTableArgs {
  int n_seqs;
  const int32_t *cached_lens, *new_lens;
  int page_size;
  const int32_t* free_pages;
  int n_free;
  const int32_t* free_used;
  int32_t* block_table;
  int max_pages;
  int64_t ld_table;
  int32_t* slot_map;
  int max_tokens;
  int32_t *seq_lens, *token_starts, *first_pages, *free_used_out;
};
int device_cu_count();  // of the current device, cached

hipError_t launch_kv_block_table(const BlockTableArgs& a, hipStream_t stream);

// one tensor of heads: element (t, h, d) at t * token + h * head + d
struct HeadsIn {
  const void* p;
  int64_t token, head;
};
struct HeadsOut {
  void* p;
  int64_t token, head;
};

struct RopeArgs {
  int64_t tokens;
  int head_dim, rot_dim, dtype, adjacent;
  const int32_t* positions;
  int n_axes;
  int64_t ld_pos;
  const float* inv_freq;
  const int32_t* axes;
  HeadsIn q;
  HeadsOut q_out;
  int q_heads;
  HeadsIn k;
  HeadsOut k_out;
  int k_heads;
};

// The heads (queries, then keys) whose elements past rot_dim are copied: those that are not turned in place.
struct RopeCopied {
  int first, count;
};
inline RopeCopied rope_copied(const RopeArgs& a) {
  const int q = a.q_out.p == a.q.p ? 0 : a.q_heads, k = a.k_heads == 0 || a.k_out.p == a.k.p ? 0 : a.k_heads;
  return {a.q_heads - q, q + k};
}
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);

struct CacheWriteArgs {
  int64_t tokens;
  int kv_heads, head_dim, dtype;
  HeadsIn k, v;
  const float *k_scale, *v_scale;
  const int32_t* slot_map;
  uint8_t *k_cache, *v_cache;
  int num_pages, page_size;
};
hipError_t launch_kv_cache_write(const CacheWriteArgs& a, hipStream_t stream);

struct PagedAttentionArgs {
  int n_seqs, q_heads, kv_heads, head_dim, dtype;
  HeadsIn q;
  const uint8_t *k_cache, *v_cache;
  int num_pages, page_size;
  const float *k_scale, *v_scale;
  const int32_t* block_table;
  int max_pages;
  int64_t ld_table;
  const int32_t* seq_lens;
  float softmax_scale;
  int64_t window;
  HeadsOut out;
  float* lse;
  void* workspace;
};
hipError_t launch_paged_attention(const PagedAttentionArgs& a, hipStream_t stream);

// Workgroups of an attention call that leave partial results: up to four on each of an MI355X's CUs.  A number of its
// own, so that the workspace's size can be checked without asking HIP.
constexpr int kMaxCus = 256, kMaxWorkersPerCu = 4, kMostWorkers = kMaxCus * kMaxWorkersPerCu;

// Query heads of an item: two tiles of 16 where the registers hold them, so that more queries meet each row that is
// read.  They do not for float32 queries, which take three times the room, nor for heads of 256.  32 contexts up to
// 16000, 32 bf16 query heads on one KV head, with 16 rows and 32: heads of 192 50 and 42 us, of 256 62 and 63 (spilled).
inline int attention_rows_of_item(int group, bool f32, int head_dim) {
  const int most = f32 || head_dim > 192 ? 16 : 32;
  return group < most ? group : most;
}

// of the workspace: for each worker an entry of 16 bytes and two partial results of a maximum, a sum and outputs a row
inline int64_t attention_workspace_bytes(int q_heads, int kv_heads, int head_dim) {
  const int64_t rows = attention_rows_of_item(q_heads / kv_heads, false, head_dim);
  return kMostWorkers * (16 + 2 * rows * (8 + 4 * (int64_t)head_dim));
}

}  // namespace nvfp4
