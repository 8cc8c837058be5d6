// What the paged KV cache's C ABI layer (nvfp4_kv_abi.cpp) does before a launch,
// for a host-only build without the HIP runtime: the device query counts its
// calls, and the launchers keep what they were given.  Used by tests/test_kv_host.py.
#include "kv_internal.h"

namespace {
int64_t hip_calls = 0;
nvfp4::RopeArgs last_rope;
}  // namespace

extern "C" hipError_t hipGetDevice(int* device) {
  ++hip_calls;
  *device = 0;
  return hipSuccess;
}

namespace nvfp4 {

int device_cu_count() {
  ++hip_calls;
  return 256;
}
hipError_t launch_kv_block_table(const BlockTableArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_rope(const RopeArgs& a, hipStream_t) {
  last_rope = a;
  return hipSuccess;
}
hipError_t launch_kv_cache_write(const CacheWriteArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_paged_attention(const PagedAttentionArgs&, hipStream_t) { return hipSuccess; }

}  // namespace nvfp4

extern "C" int64_t kv_test_hip_calls() { return hip_calls; }
extern "C" void kv_test_rope_copied(int32_t* first, int32_t* count) {
  const nvfp4::RopeCopied c = nvfp4::rope_copied(last_rope);
  *first = c.first;
  *count = c.count;
}
