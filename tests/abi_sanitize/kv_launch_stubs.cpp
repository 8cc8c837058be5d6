// Kernel launchers for a host-only build of the paged KV cache's C ABI layer
// (nvfp4_kv_abi.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer: the
// argument checks run as in the real library, and any call that gets past them
// finds no device here.  Used by tests/test_kv_abi_sanitized.py only, which
// also reaches the kernels' division through it.
#include "kv_internal.h"

namespace nvfp4 {

int device_cu_count() { return 256; }
hipError_t launch_kv_block_table(const BlockTableArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_rope(const RopeArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_kv_cache_write(const CacheWriteArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_paged_attention(const PagedAttentionArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t paged_attention_workspace(int q_heads, int kv_heads, int head_dim) {
  const int64_t rows = q_heads / kv_heads < 32 ? q_heads / kv_heads : 32;
  return 1024 * (16 + 2 * rows * (8 + 4 * (int64_t)head_dim));
}

}  // namespace nvfp4

extern "C" uint32_t kv_test_fastdiv(uint32_t d, uint32_t n) {
  const nvfp4::FastDiv f(d);
  return f.d == 1 ? n : (uint32_t)(((uint64_t)n * f.mul) >> 32) >> f.shift;
}
