// Norm of each token's groups of channels, with a gate or an activation
// (nvfp4_group_norm).
//
//   y = (x - m) / sqrt(mean((x - m)^2) + eps) * weight + bias,  out = y act(gate) or act(y)
//
// Bandwidth kernel: x and gate are read once and stay in registers, so the mean can be
// taken off before squares are summed, and out may be either of them.  LANES lanes
// share a group: 16 of them (a group of 128 in 16-bit types is one 16-byte load each),
// a wave, or a workgroup, whatever holds it.
#include <algorithm>

#include "gdn_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

template <int LANES>
__device__ __forceinline__ float sum_of(float v, float* lds) {
#pragma unroll
  for (int m = 1; m < std::min(LANES, 64); m *= 2) v += __shfl_xor(v, m);
  if constexpr (LANES > 64) {
    __syncthreads();  // what the last sum left in lds is read
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0] + lds[1] + lds[2] + lds[3];
  }
  return v;
}

// a group of up to LANES * N * E elements, E of them at a time
template <int DT, int E, int LANES, int N>
__global__ __launch_bounds__(kThreads) void group_norm_kernel(NormArgs a, int64_t first, int64_t items, float over_dim) {
  __shared__ float lds[4];
  constexpr int kPer = kThreads / LANES;
  const int64_t item = first + (int64_t)blockIdx.x * kPer + threadIdx.x / LANES;
  const bool live = item < items;  // the others keep step with their wave
  const int64_t token = live ? item / a.groups : 0;
  const int group = live ? (int)(item - token * a.groups) : 0;
  const int lane = threadIdx.x % LANES;
  const int64_t xo = token * a.x.token + group * a.x.head, zo = token * a.gate.token + group * a.gate.head;
  Elements<DT, E> x[N], z[N];
  const bool gated = a.gate.p != nullptr;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = (i * LANES + lane) * E;
    if (at < a.group_dim) {
      x[i].load(a.x.p, xo + at);
      if (gated) z[i].load(a.gate.p, zo + at);
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
  const float var = __builtin_fmaf(sum_of<LANES>(s, lds), over_dim, a.eps);
  const float over = 1.0f / sqrtf(var);
  if (!live) return;
  const float* weight = a.weight + (int64_t)group * a.weight_group;
  const float* bias = a.bias ? a.bias + (int64_t)group * a.weight_group : nullptr;
  const int64_t oo = token * a.out.token + group * a.out.head;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = (i * LANES + lane) * E;
    if (at >= a.group_dim) continue;
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      y[e] = (x[i].get(e) - mean) * over * weight[at + e];
      if (bias) y[e] += bias[at + e];
      const float g = gated ? z[i].get(e) : y[e];
      const float act = a.activation ? g * sigmoid<DT == 0>(g) : g;
      y[e] = gated ? y[e] * act : act;
    }
    Elements<DT, E> out;
    out.set(y);
    out.store(a.out.p, oo + at);
  }
}

template <int DT, int E, int LANES, int N>
hipError_t launch_lanes(const NormArgs& a, hipStream_t stream) {
  const int64_t items = a.tokens * a.groups, per = kThreads / LANES, most = kMostWorkgroups * per;
  for (int64_t first = 0; first < items; first += most) {
    const int64_t left = std::min(items - first, most);
    group_norm_kernel<DT, E, LANES, N>
        <<<(uint32_t)((left + per - 1) / per), kThreads, 0, stream>>>(a, first, items, 1.0f / (float)a.group_dim);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t launch_typed(const NormArgs& a, hipStream_t stream) {
  constexpr int kE = 16 / element_size(DT);
  auto whole = [&](const void* p, int64_t token, int64_t group) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token % kE == 0 && group % kE == 0;
  };
  const int n = a.group_dim;
  if (n % kE == 0 && whole(a.x.p, a.x.token, a.x.head) && whole(a.out.p, a.out.token, a.out.head) &&
      (!a.gate.p || whole(a.gate.p, a.gate.token, a.gate.head))) {
    if (n <= 16 * kE) return launch_lanes<DT, kE, 16, 1>(a, stream);
    if (n <= 32 * kE) return launch_lanes<DT, kE, 16, 2>(a, stream);
    if (n <= 128 * kE) return launch_lanes<DT, kE, 64, 2>(a, stream);
    return launch_lanes<DT, kE, 256, 8192 / (256 * kE)>(a, stream);
  }
  if (n <= 64) return launch_lanes<DT, 1, 16, 4>(a, stream);
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
