// Argument checks that the C ABI layers share: pure functions of the arguments,
// made before any HIP call.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "nvfp4.h"

namespace nvfp4 {

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

inline bool size_ok(int64_t n) { return n > 0 && n < kMaxDim; }

// heads * head_dim elements of a token; both factors are checked before they are multiplied
inline bool row_ok(int64_t heads, int64_t head_dim) {
  return heads > 0 && head_dim > 0 && heads < kMaxRow && head_dim < kMaxRow && heads * head_dim <= kMaxRow;
}

// a token's heads lie one behind another and end before the next token; (heads - 1) * head may pass 2^63
inline bool strides_ok(int64_t heads, int64_t head_dim, int64_t token, int64_t head) {
  if (token >= kMaxStride || head >= kMaxStride || head < head_dim || token < head_dim) return false;
  return heads == 1 || head <= (token - head_dim) / (heads - 1);
}

inline bool by16(int64_t stride, int es) { return (stride * es) % 16 == 0; }

inline nvfp4_status done(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_DEVICE; }

}  // namespace nvfp4
