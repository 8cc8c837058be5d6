// Launchers of the gated delta layer's kernels (include/nvfp4_gdn.h).  Arguments
// are validated by the caller (nvfp4_gdn_abi.cpp); these only launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kv_internal.h"

namespace nvfp4 {

struct ConvArgs {
  int64_t tokens;  // rows of x; a step has one for each sequence
  int channels, width, dtype;
  const void* x;
  int64_t ldx;
  const float *weight, *bias;
  int activation;
  int n_seqs;
  const int32_t *token_starts, *cached_lens;  // NULL in a step
  const int32_t* slots;
  const void* state;
  void* state_out;
  int num_slots;
  void* out;
  int64_t ldo;
};
// Tokens a thread of the convolution of prompts takes; `columns` workgroups of a wave hold a row.  With more of them fewer
// rows are loaded twice, with fewer the card is filled: 32, in vectors of 16 bytes and past the caches, from 5 1/2
// waves a CU on, else 16 from 4 waves a CU on, else 8.  us:
//   tokens, channels     waves a CU of 32    8      16     32
//   1024 x 8192, bf16    2                   10.7   10.2   12.1
//   2048 x 8192, bf16    4                   17.6   15.9   14.7
//   1024 x 8192, f32     4                   15.8   15.3   16.4
//   7069 x 2568, f16     5.2                 18.9   16.7   18.4
//   13 prompts, 7069     5.2                 19.2   18.3   20.1
//   3000 x 8192, bf16    5.9                 26.2   22.9   20.7
//   1500 x 8192, f32     5.9                 22.9   22.9   20.3
//   10000 x 2568, f16    7.3                 28.7   25.6   21.6
//   13 prompts, 10400    7.6                 30.0   27.8   25.0
//   8192 x 8192, bf16    16                  69.8   64.9   59.0 (through the caches 63.2)
// (2568 channels: width 3, else 4)
inline int conv_rows(int64_t tokens, int64_t columns, bool vectors, int cus) {
  if (vectors && tokens / 32 * columns * 2 >= 11 * cus) return 32;
  return tokens / 16 * columns >= 4 * cus ? 16 : 8;
}
hipError_t launch_causal_conv(const ConvArgs& a, hipStream_t stream);
hipError_t launch_causal_conv_step(const ConvArgs& a, hipStream_t stream);

struct DeltaArgs {
  int64_t tokens;  // rows of q, k, v; a step has one for each sequence
  int k_heads, v_heads, head_k, head_v, dtype;
  HeadsIn q, k, v;
  const void* a;
  int64_t a_token;
  const void* b;
  int64_t b_token;
  const float *a_log, *dt_bias;
  float scale, eps;
  int n_seqs;
  const int32_t *token_starts, *cached_lens;  // NULL in a step
  const int32_t* slots;
  const float* state;
  float* state_out;
  int num_slots;
  HeadsOut out;
  void* workspace;
};
hipError_t launch_gated_delta_chunked(const DeltaArgs& a, hipStream_t stream);
hipError_t launch_gated_delta_step(const DeltaArgs& a, hipStream_t stream);

struct NormArgs {
  int64_t tokens;
  int groups, group_dim, dtype;
  HeadsIn x, gate;  // gate.p may be NULL
  HeadsOut out;
  const float* weight;
  int weight_group;
  const float* bias;
  int activation, centred;
  float eps;
};
hipError_t launch_group_norm(const NormArgs& a, hipStream_t stream);

// The workspace of nvfp4_gated_delta_chunked: for each chunk of 64 tokens of a sequence the normalised keys and queries of
// every key head, then what ties the chunk's tokens together for every value head.  Chunk i of sequence r has place
// floor(start_r / 64) + r + i, which no other chunk has.
constexpr int kDeltaChunk = 64;
constexpr int kDeltaTieBytes = 26 << 10;
constexpr int64_t delta_key_bytes(int head_k, int dtype) {  // float32: two fp16 parts; then norms (padded) and products
  return (int64_t)2 * kDeltaChunk * head_k * (dtype == 0 ? 4 : 2) + (21 << 10);
}
constexpr int64_t delta_chunk_bytes(int k_heads, int v_heads, int head_k, int dtype) {
  return k_heads * delta_key_bytes(head_k, dtype) + (int64_t)v_heads * kDeltaTieBytes;
}
inline int64_t delta_chunk_places(int64_t tokens, int64_t n_seqs) { return tokens / kDeltaChunk + n_seqs; }

// Behind the chunks: where heads are few, sequences are taken in parts, and each part of a sequence and head has the state
// it starts from, and what it does to any.  Of 64 columns of states a CU in all parts (as many as run at once, with as
// many again for what parts do) if those are 8 parts or more, else of twice that; a part has 8 chunks or more but for the
// last.
//
// And only where that is not slower: both passes over a part take 2.4 times as long a chunk as the whole chain takes, 4.3
// times where a CU has more than 64 columns meanwhile, and each part adds a join, all together two launches.  Lengths are
// not known here: the longest of n sequences is between 1 / n of the tokens and all of them, 1 / sqrt(n) is taken, and all
// are cut alike.  In us, whole and in parts, bf16 and heads of 128 if not said:
//   6 heads, 1024 tokens: 55, 65 in 2           1536: 75, 70 in 3              2048: 95, 75 in 4
//   6 heads, 16411: 615, 158 in 21, 181 in 32   8 heads, 2048: 97, 81 in 4     16 heads, 4096: 172, 102 in 8
//   24 heads, 16411: 664, 384 in 10             32 heads, 2048: 97, 92 in 4    32 heads, 8192: 340, 256 in 8
//   40 heads, 3000: 136, 149 in 5               40 heads, 8192: 351, 319 in 5  48 heads, 3000: 139, 154 in 5
//   48 heads, 4096: 178, 186 in 5               48 heads, 6000: 266, 262 in 5  48 heads, 8192: 355, 332 in 5
//   56 heads, 8192: 360, 385 in 4               64 heads, 16411: 726, 779 in 4
//   float32: 6 heads, 1536: 120, 95 in 3        40 heads, 3000: 226, 258 in 5  48 heads, 8192: 740, 671 in 5
//   heads of 64: 48 heads, 2048: 82, 74 in 4    96 heads, 4096: 156, 172 in 5  96 heads, 8192: 317, 334 in 5
//   8 sequences of 6 heads, the longest 1024: 63, 95    2048: 101, 121    4096: 175, 162    3 of them, 4096: 170, 106
//   16 of one head of 64, 1024: 45, 57          2048: 76, 63
// It misses 6 heads of 1536 tokens, 96 heads of 64, the 8 sequences up to 2048 and the 16 up to 1024.
constexpr int kDeltaPartColumns = kMaxCus * 128, kDeltaPartChunks = 8, kDeltaMostParts = 32;
inline int64_t delta_parts(int64_t tokens, int64_t n_seqs, int v_heads, int head_v) {
  const int64_t of_seq = (int64_t)v_heads * head_v, columns = n_seqs * of_seq;
  int64_t parts = kDeltaPartColumns / 2 / columns;
  if (parts < 8) parts = kDeltaPartColumns / columns;
  if (parts > tokens / (kDeltaChunk * kDeltaPartChunks)) parts = tokens / (kDeltaChunk * kDeltaPartChunks);
  if (parts > kDeltaMostParts) parts = kDeltaMostParts;
  if (parts < 2) return 0;
  const int64_t all = (tokens + kDeltaChunk - 1) / kDeltaChunk, longest = (int64_t)((double)all / std::sqrt((double)n_seqs));
  int64_t each = (longest + parts - 1) / parts;
  if (each < kDeltaPartChunks) each = kDeltaPartChunks;
  auto cut = [&](int64_t chunks) { return (chunks + each - 1) / each; };
  // in tenths of a chunk of the whole chain
  const int64_t pass = (cut(all) + n_seqs - 1) * of_seq > 64 * kMaxCus ? 43 : 24, join = 15, launches = 15;
  return each * pass + cut(longest) * join + launches < longest * 10 ? parts : 0;
}
inline int64_t delta_part_bytes(int head_k, int head_v) { return (int64_t)4 * head_k * (head_v + head_k); }
// enough for any number of sequences up to n_seqs
inline int64_t gated_delta_workspace_bytes(int64_t tokens, int64_t n_seqs, int k_heads, int v_heads, int head_k, int head_v,
                                           int dtype) {
  const int64_t by_columns = kDeltaPartColumns / head_v, by_chunks = tokens / (kDeltaChunk * kDeltaPartChunks) * n_seqs * v_heads;
  const int64_t order = 4 * (n_seqs < 512 ? (n_seqs + 3) / 4 * 4 : 512);  // of sequences by their lengths, in calls without parts
  return delta_chunk_places(tokens, n_seqs) * delta_chunk_bytes(k_heads, v_heads, head_k, dtype) +
         (by_columns < by_chunks ? by_columns : by_chunks) * delta_part_bytes(head_k, head_v) + order;
}

}  // namespace nvfp4
