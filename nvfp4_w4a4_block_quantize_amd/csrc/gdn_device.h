// Device-side helpers of the gated delta layer's kernels: elements of the three
// types in vectors, the functions of gates and activations, and ragged prompts.
#pragma once

#include "gdn_internal.h"
#include "nvfp4_device.h"

namespace nvfp4 {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int element_size(int dt) { return dt == 0 ? 4 : 2; }

// two floats as two elements of a 16-bit type, each to nearest even
template <int DT>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (DT == 1) return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{x, y}, bf16x2_t));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{x, y}, half2_t));
}

// E consecutive elements: 16-byte accesses where E elements are a multiple of 16 bytes, else one element (E = 1)
template <int DT, int E>
struct Elements {
  static constexpr int kWords = E == 1 ? 1 : E * element_size(DT) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    const char* p = static_cast<const char*>(base) + elem * element_size(DT);
    if constexpr (E == 1) {
      if constexpr (DT == 0)
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      else
        w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const u32x4_t v = reinterpret_cast<const u32x4_t*>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
      }
    }
  }
  // PAST: past the caches, where vectors are stored
  template <bool PAST = false>
  __device__ __forceinline__ void store(void* base, int64_t elem) const {
    char* p = static_cast<char*>(base) + elem * element_size(DT);
    if constexpr (E == 1) {
      if constexpr (DT == 0)
        *reinterpret_cast<uint32_t*>(p) = w[0];
      else
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const u32x4_t v = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        if constexpr (PAST)
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p) + i);
        else
          reinterpret_cast<u32x4_t*>(p)[i] = v;
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == 0) {
      return __uint_as_float(w[i]);
    } else {
      const uint32_t v = w[i >> 1];
      if constexpr (DT == 1) return __uint_as_float(i & 1 ? v & 0xFFFF0000u : v << 16);
      const uint16_t h = (uint16_t)(i & 1 ? v >> 16 : v & 0xFFFFu);
      return (float)__builtin_bit_cast(_Float16, h);
    }
  }
  // all elements at once
  __device__ __forceinline__ void set(const float (&x)[E]) {
    if constexpr (DT == 0) {
#pragma unroll
      for (int i = 0; i < E; ++i) w[i] = __float_as_uint(x[i]);
    } else if constexpr (E == 1) {
      w[0] = pack2<DT>(x[0], 0.0f) & 0xFFFFu;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = pack2<DT>(x[2 * i], x[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
};

template <int DT>
__device__ __forceinline__ float element(const void* base, int64_t elem) {
  Elements<DT, 1> e;
  e.load(base, elem);
  return e.get(0);
}

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLog2eRest = 1.925963033500e-08f;  // log2(e) less its rounding to 32 bits
constexpr float kLn2 = 0.693147180559945309f;

// e^x.  v_exp_f32 gives 2^t; where 32 bits are asked for, what t = x log2(e) drops in rounding (up to |t| 2^-24) is
// added to first order.
template <bool FULL>
__device__ __forceinline__ float exp_of(float x) {
  const float t = x * kLog2e;
  const float e = __builtin_amdgcn_exp2f(t);
  if constexpr (!FULL) return e;
  const float rest = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -t));
  // where e is infinite or 0 the rest is of no use, and infinity times 0 would be NaN
  return fabsf(t) < 126.0f ? __builtin_fmaf(e, rest * kLn2, e) : e;
}

// 1 / (1 + e^-x), 0 and 1 at the ends
template <bool FULL>
__device__ __forceinline__ float sigmoid(float x) {
  const float d = 1.0f + exp_of<FULL>(-x);
  if constexpr (FULL) return 1.0f / d;
  return __builtin_amdgcn_rcpf(d);
}

// ln(1 + e^x)
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

// What a row x 2^up whose squares sum to `squares` is multiplied by to be x / sqrt(|x|^2 + eps).  A row of zeros stays one,
// also where eps is 0.
__device__ __forceinline__ float norm_of(float squares, int up, float eps) {
  if (squares == 0.0f) return 0.0f;
  const float more = __builtin_amdgcn_ldexpf(eps, 2 * up);
  // where that is infinite, x is nothing beside eps
  return more > 3e38f ? __builtin_amdgcn_ldexpf(1.0f / sqrtf(eps), -up) : 1.0f / sqrtf(squares + more);
}

// first row and end of sequence r, inside the buffers whatever the starts hold
__device__ __forceinline__ int64_t start_of(const int32_t* starts, int r, int64_t tokens) {
  const int64_t s = starts[r];
  return s < 0 ? 0 : s > tokens ? tokens : s;
}

__device__ __forceinline__ bool slot_ok(int slot, int num_slots) { return slot >= 0 && slot < num_slots; }

}  // namespace nvfp4
