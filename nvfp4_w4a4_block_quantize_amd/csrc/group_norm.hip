// Norm of each token's groups of channels, with a gate or an activation
// (nvfp4_group_norm).
//
//   y = (x - m) / sqrt(mean((x - m)^2) + eps) * weight + bias,  out = y act(gate) or act(y)
//
// Bandwidth kernel: x and gate are read once and stay in registers, so the mean can be
// taken off before squares are summed, and out may be either of them.  LANES lanes
// share a group: 16 of them (a group of 128 in 16-bit types is one 16-byte load each),
// a wave, or a workgroup, whatever holds it.  Rows that are not whole 16-byte pieces are
// taken element by element, 16 lanes of up to 8.  Sums go round rows of 16 lanes without
// LDS.  8192 tokens of 48 groups of 128, bf16, with a gate: 59 us, 5.1 TB/s (weights
// loaded one by one 122; two groups a thread 59, at 1024 tokens 11.0 and not 9.5); 4099 of
// 20 of 121 in float32: 21.8 (two groups a thread 23.1; through LDS and 64 lanes 36).
//
// Groups whose squares leave the range of fp32 are normalised again by a path of their own;
// what it is in the way costs 1%, and 3% of the widest bf16 groups (8192 of 4096: 42.9 ->
// 44.3), whose 100 registers leave four waves a SIMD and not five.
#include <algorithm>

#include "gdn_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

// `v` of the lane `by` places on, around each row of 16
template <int BY>
__device__ __forceinline__ float turned(float v) {
  constexpr int kRowRor = 0x120;
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kRowRor + BY, 0xF, 0xF, false));
}

// of a group's lanes, the same in all of them
template <int LANES, typename F>
__device__ __forceinline__ float joined(float v, float* lds, F join) {
  v = join(v, turned<8>(v));
  v = join(v, turned<4>(v));
  v = join(v, turned<2>(v));
  v = join(v, turned<1>(v));
  if constexpr (LANES > 16) {
    const auto rows = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = join(__uint_as_float(rows[0]), __uint_as_float(rows[1]));
    const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = join(__uint_as_float(halves[0]), __uint_as_float(halves[1]));
  }
  if constexpr (LANES > 64) {
    __syncthreads();  // what the last one left in lds is read
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = join(join(join(lds[0], lds[1]), lds[2]), lds[3]);
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ float sum_of(float v, float* lds) {
  return joined<LANES>(v, lds, [](float a, float b) { return a + b; });
}

// A group's sum of squares is taken as it is below 2^126, and from 2^-80 on or beside an eps of 2^-100 and more: what
// squares lose below the normal range is nothing then.
constexpr float kMostSquares = 0x1p126f, kLeastSquares = 0x1p-80f, kLeastEps = 0x1p-100f;

// A group: where its elements are, and its weights.
struct Group {
  int64_t x, gate, out, weight;
};

// elements `at` of a group, normalised, on to the output
template <int DT, int E>
__device__ __forceinline__ void put(const NormArgs& a, const Group& group, int at, float (&y)[E], const Elements<DT, E>& gate) {
  const bool gated = a.gate.p != nullptr;
  Elements<0, E> w, b;
  w.load(a.weight, group.weight + at);
  if (a.bias) b.load(a.bias, group.weight + at);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    y[e] *= w.get(e);
    if (a.bias) y[e] += b.get(e);
    const float g = gated ? gate.get(e) : y[e];
    const float act = a.activation ? g * sigmoid<DT == 0>(g) : g;
    y[e] = gated ? y[e] * act : act;
  }
  Elements<DT, E> out;
  out.set(y);
  out.store(a.out.p, group.out + at);
}

// A group whose squares leave the range: times a power of two that takes the largest element into [1/4, 1/2), an element at a
// time and from memory each time, so that the common case's registers are its own.
template <int DT, int LANES>
__device__ __forceinline__ void norm_scaled(const NormArgs& a, const Group& group, int lane, float over_dim, float* lds) {
  int up = 0;
  auto each = [&](auto f) {
#pragma unroll 1
    for (int at = lane; at < a.group_dim; at += LANES) f(at, __builtin_amdgcn_ldexpf(element<DT>(a.x.p, group.x + at), up));
  };
  float top = 0.0f, mean = 0.0f, s = 0.0f;
  each([&](int, float x) { top = fmaxf(top, fabsf(x)); });
  up = -1 - __builtin_amdgcn_frexp_expf(joined<LANES>(top, lds, [](float a, float b) { return fmaxf(a, b); }));
  if (a.centred) {
    each([&](int, float x) { mean += x; });
    mean = sum_of<LANES>(mean, lds) * over_dim;
  }
  each([&](int, float x) { s = __builtin_fmaf(x - mean, x - mean, s); });
  const float over = norm_of(sum_of<LANES>(s, lds) * over_dim, up, a.eps);
  each([&](int at, float x) {
    Elements<DT, 1> z;
    if (a.gate.p) z.load(a.gate.p, group.gate + at);
    float y[1] = {(x - mean) * over};
    put<DT, 1>(a, group, at, y, z);
  });
}

// Groups of up to LANES * N * E elements, E of them at a time.
template <int DT, int E, int LANES, int N>
__global__ __launch_bounds__(kThreads) void group_norm_kernel(NormArgs a, FastDiv by_groups, uint32_t items, float over_dim) {
  __shared__ float lds[4];
  const int lane = threadIdx.x % LANES;
  const bool gated = a.gate.p != nullptr;
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const bool live = item < items;  // the others keep step with their wave
  const uint32_t t = by_groups.div(live ? item : 0);
  const int64_t token = t;
  const int of_token = live ? (int)(item - t * by_groups.d) : 0;
  const Group group = {token * a.x.token + of_token * a.x.head, token * a.gate.token + of_token * a.gate.head,
                       token * a.out.token + of_token * a.out.head, (int64_t)of_token * a.weight_group};
  Elements<DT, E> x[N], z[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = (i * LANES + lane) * E;
    if (at < a.group_dim) {
      x[i].load(a.x.p, group.x + at);
      if (gated) z[i].load(a.gate.p, group.gate + at);
    } else {
      x[i].zero();
    }
  }
  float mean = 0.0f;
  if (a.centred) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) s += x[i].get(e);
    mean = sum_of<LANES>(s, lds) * over_dim;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool inside = (i * LANES + lane) * E < a.group_dim;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float y = inside ? x[i].get(e) - mean : 0.0f;
      s = __builtin_fmaf(y, y, s);
    }
  }
  s = sum_of<LANES>(s, lds);
  float over = 1.0f / sqrtf(__builtin_fmaf(s, over_dim, a.eps));
  if constexpr (DT == 2) {  // squares of fp16 are in range, or all zeros
    if (s == 0.0f) over = fminf(over, 1.0f);
  } else if (__builtin_expect(!(s < kMostSquares && (s >= kLeastSquares || a.eps >= kLeastEps)), 0)) {  // a group's lanes agree
    if (live) norm_scaled<DT, LANES>(a, group, lane, over_dim, lds);
    return;
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = (i * LANES + lane) * E;
    if (at >= a.group_dim) continue;
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = (x[i].get(e) - mean) * over;
    put<DT, E>(a, group, at, y, z[i]);
  }
}

template <int DT, int E, int LANES, int N>
hipError_t launch_lanes(NormArgs a, hipStream_t stream) {
  constexpr int kPer = kThreads / LANES;
  const FastDiv by_groups((uint32_t)a.groups);
  // a launch takes whole tokens, of fewer than 2^31 groups in all
  const int64_t most = std::max<int64_t>(kMostWorkgroups * kPer / a.groups, 1);
  for (int64_t left = a.tokens;;) {
    const int64_t tokens = std::min(left, most);
    const uint32_t items = (uint32_t)(tokens * a.groups);
    group_norm_kernel<DT, E, LANES, N>
        <<<(items + kPer - 1) / kPer, kThreads, 0, stream>>>(a, by_groups, items, 1.0f / (float)a.group_dim);
    const hipError_t e = hipGetLastError();
    left -= tokens;
    if (e != hipSuccess || left == 0) return e;
    auto behind = [&](int64_t stride) { return tokens * stride * element_size(DT); };
    a.x.p = static_cast<const char*>(a.x.p) + behind(a.x.token);
    if (a.gate.p) a.gate.p = static_cast<const char*>(a.gate.p) + behind(a.gate.token);
    a.out.p = static_cast<char*>(a.out.p) + behind(a.out.token);
  }
}

template <int DT>
hipError_t launch_typed(const NormArgs& a, hipStream_t stream) {
  constexpr int kE = 16 / element_size(DT);
  auto whole = [&](const void* p, int64_t token, int64_t group) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token % kE == 0 && group % kE == 0;
  };
  const int n = a.group_dim;
  if (n % kE == 0 && whole(a.x.p, a.x.token, a.x.head) && whole(a.out.p, a.out.token, a.out.head) &&
      whole(a.weight, 0, a.weight_group) && whole(a.bias, 0, 0) &&
      (!a.gate.p || whole(a.gate.p, a.gate.token, a.gate.head))) {
    if (n <= 16 * kE) return launch_lanes<DT, kE, 16, 1>(a, stream);
    if (n <= 32 * kE) return launch_lanes<DT, kE, 16, 2>(a, stream);
    if (n <= 128 * kE) return launch_lanes<DT, kE, 64, 2>(a, stream);
    return launch_lanes<DT, kE, 256, 8192 / (256 * kE)>(a, stream);
  }
  if (n <= 64) return launch_lanes<DT, 1, 16, 4>(a, stream);
  if (n <= 128) return launch_lanes<DT, 1, 16, 8>(a, stream);
  if (n <= 512) return launch_lanes<DT, 1, 64, 8>(a, stream);
  return launch_lanes<DT, 1, 256, 32>(a, stream);
}

}  // namespace

hipError_t launch_group_norm(const NormArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case 0: return launch_typed<0>(a, stream);
    case 1: return launch_typed<1>(a, stream);
    default: return launch_typed<2>(a, stream);
  }
}

}  // namespace nvfp4
