// Launchers of the gated delta layer's kernels (include/nvfp4_gdn.h).  Arguments
// are validated by the caller (nvfp4_gdn_abi.cpp); these only launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

// of the workspace of nvfp4_gated_delta_chunked
inline int64_t gated_delta_workspace_bytes(int64_t, int64_t, int, int, int, int, int) { return 16; }

}  // namespace nvfp4
