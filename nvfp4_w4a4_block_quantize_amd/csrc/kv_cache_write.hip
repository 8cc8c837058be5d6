// K and V rows to E4M3 bytes in cache pages (nvfp4_kv_cache_write).
//
// Per element the rule of the dense quantiser: y = fp32(x * s), clamped to
// [-448, 448], v_cvt_pk_fp8_f32 (nearest even; checked on every fp32 input by
// conformance_cvt).  The row of one token and head goes to
//   cache[page][head][offset][:], slot = page * page_size + offset,
// head_dim consecutive bytes.
//
// Bandwidth kernel: 2 B read and 1 B written per bf16 element.  A thread owns
// kUnroll chunks of 8 elements (16 B in, 8 B out), kThreads apart in the flat
// list (tensor, token, chunk of the token's row), and has all its loads in
// flight before it converts.
#include <algorithm>

#include "nvfp4_device.h"
#include "kv_internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// eight elements as fp32, from one (16-bit types) or two 16-byte loads
template <int DT>
struct Raw {
  u32x4_t w[DT == 0 ? 2 : 1];
  __device__ __forceinline__ void load(const void* x, int64_t elem) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(x) + elem * (DT == 0 ? 4 : 2));
    w[0] = __builtin_nontemporal_load(p);
    if constexpr (DT == 0) w[1] = __builtin_nontemporal_load(p + 1);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == 0) {
      return __uint_as_float(w[i >> 2][i & 3]);
    } else {
      const uint32_t v = w[0][i >> 1];
      if constexpr (DT == 1) return __uint_as_float(i & 1 ? v & 0xFFFF0000u : v << 16);
      const uint16_t h = (uint16_t)(i & 1 ? v >> 16 : v & 0xFFFFu);
      _Float16 f;
      __builtin_memcpy(&f, &h, 2);
      return (float)f;
    }
  }
};

__device__ __forceinline__ uint32_t e4m3x4(float y0, float y1, float y2, float y3) {
  auto clamp = [](float y) { return __builtin_amdgcn_fmed3f(y, -448.0f, 448.0f); };
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(clamp(y0), clamp(y1), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp(y2), clamp(y3), lo, true);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void kv_cache_write_kernel(CacheWriteArgs a, FastDiv by_row, FastDiv by_head,
                                                                  FastDiv by_page, int64_t chunks) {
  const bool value = blockIdx.y != 0;  // K, then V
  const HeadsIn in = value ? a.v : a.k;
  uint8_t* cache = value ? a.v_cache : a.k_cache;
  const float s = value ? *a.v_scale : *a.k_scale;
  const int slots = a.num_pages * a.page_size;

  const int64_t first = (int64_t)blockIdx.x * (kThreads * kUnroll);
  const int64_t token0 = first / by_row.d;  // one division for the workgroup; the rest fits 32 bits
  const uint32_t skip = (uint32_t)(first - token0 * by_row.d) + threadIdx.x;

  Raw<DT> raw[kUnroll];
  uint8_t* out[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    out[u] = nullptr;
    if (first + threadIdx.x + u * kThreads >= chunks) continue;
    const uint32_t at = skip + u * kThreads;
    const uint32_t t = by_row.div(at), in_row = at - t * by_row.d;
    const uint32_t head = by_head.div(in_row), chunk = in_row - head * by_head.d;
    const int64_t token = token0 + t;
    const int slot = a.slot_map[token];
    raw[u].load(in.p, token * in.token + head * in.head + chunk * 8);
    if (slot >= 0 && slot < slots) {
      const uint32_t page = by_page.div((uint32_t)slot), off = (uint32_t)slot - page * by_page.d;
      out[u] = cache + (((int64_t)page * a.kv_heads + head) * a.page_size + off) * a.head_dim + chunk * 8;
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (!out[u]) continue;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = raw[u].get(i) * s;
    const u32x2_t w = {e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7])};
    *reinterpret_cast<u32x2_t*>(out[u]) = w;
  }
}

template <int DT>
hipError_t launch_typed(const CacheWriteArgs& a, hipStream_t stream) {
  const uint32_t row = (uint32_t)a.kv_heads * (uint32_t)(a.head_dim / 8);
  const int64_t chunks = a.tokens * row, per_block = (int64_t)kThreads * kUnroll;
  const int64_t blocks = (chunks + per_block - 1) / per_block;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  kv_cache_write_kernel<DT><<<dim3((unsigned)blocks, 2), kThreads, 0, stream>>>(
      a, FastDiv(row), FastDiv((uint32_t)(a.head_dim / 8)), FastDiv((uint32_t)a.page_size), chunks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_cache_write(const CacheWriteArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case 0: return launch_typed<0>(a, stream);
    case 1: return launch_typed<1>(a, stream);
    default: return launch_typed<2>(a, stream);
  }
}

}  // namespace nvfp4
