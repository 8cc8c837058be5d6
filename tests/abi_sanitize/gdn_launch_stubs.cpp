// Kernel launchers for a host-only build of the gated delta layer's C ABI layer
// (nvfp4_gdn_abi.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer: the
// argument checks run as in the real library, and any call that gets past them
// finds no device here.  Used by tests/test_gdn_abi_sanitized.py only.
#include "gdn_internal.h"

namespace nvfp4 {

hipError_t launch_causal_conv(const ConvArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_causal_conv_step(const ConvArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_gated_delta_chunked(const DeltaArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_gated_delta_step(const DeltaArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_group_norm(const NormArgs&, hipStream_t) { return hipErrorNoDevice; }

}  // namespace nvfp4

// What the chunked rule takes from its workspace: returns the bytes that a call of these sizes uses, of chunks, parts and the
// order of sequences.
extern "C" int64_t gdn_test_used(int64_t tokens, int64_t n_seqs, int k_heads, int v_heads, int head_k, int head_v, int dtype) {
  const int64_t chunks = nvfp4::delta_chunk_places(tokens, n_seqs) * nvfp4::delta_chunk_bytes(k_heads, v_heads, head_k, dtype);
  const int64_t parts = nvfp4::delta_parts(tokens, n_seqs, v_heads, head_v);
  if (parts) return chunks + n_seqs * v_heads * parts * nvfp4::delta_part_bytes(head_k, head_v);
  return chunks + (n_seqs > 1 && n_seqs <= 512 ? 4 * n_seqs : 0);
}
extern "C" int64_t gdn_test_parts(int64_t tokens, int64_t n_seqs, int v_heads, int head_v) {
  return nvfp4::delta_parts(tokens, n_seqs, v_heads, head_v);
}
extern "C" int gdn_test_conv_rows(int64_t tokens, int64_t columns, int vectors, int cus) {
  return nvfp4::conv_rows(tokens, columns, vectors != 0, cus);
}
