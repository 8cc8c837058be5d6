// The gated delta rule over ragged prompts (nvfp4_gated_delta_chunked), token by token.
//
//   S' = e^g S;  d = beta (v - S'^T k~);  S_new = S' + k~ d^T;  out = scale S_new^T q~
//
// A workgroup holds 64 columns of one head's state in its threads' registers and walks
// the sequence's tokens; each token costs a sum over the rows through LDS.
#include <algorithm>

#include "gdn_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

template <int DT, int DK>
__global__ __launch_bounds__(kThreads) void gated_delta_kernel(DeltaArgs a, FastDiv by_group, int64_t first) {
  constexpr int kLanes = kCols / 4;
  constexpr int kGroups = kThreads / kLanes;
  constexpr int kRows = DK / kGroups;
  constexpr int kWaves = kThreads / 64;
  __shared__ float lds_k[2][DK], lds_q[2][DK];
  __shared__ float4_t lds_sum[2][2][kWaves][kLanes];
  const int slices = a.head_v / kCols;
  const int64_t item = first + blockIdx.x;
  const int64_t pair = item / slices;
  const int column = (int)(item - pair * slices) * kCols;
  const int64_t r = pair / a.v_heads;
  const int h = (int)(pair - r * a.v_heads);
  const int slot = a.slots[r];
  const int64_t begin = start_of(a.token_starts, (int)r, a.tokens), end = start_of(a.token_starts, (int)r + 1, a.tokens);
  if (!slot_ok(slot, a.num_slots) || begin >= end) return;
  const int thread = threadIdx.x, lane = thread & 63, wave = thread >> 6;
  const int col = thread % kLanes, row = thread / kLanes;
  const int64_t state = (((int64_t)slot * a.v_heads + h) * DK) * a.head_v + column + 4 * col;
  const bool carried = !a.cached_lens || a.cached_lens[r] > 0;
  float4_t s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    s[i] = carried ? *reinterpret_cast<const float4_t*>(a.state + state + (int64_t)(row + i * kGroups) * a.head_v)
                   : float4_t{0, 0, 0, 0};
  const int kh = (int)by_group.div((uint32_t)h);
  const float rate = expf(a.a_log[h]), dt = a.dt_bias[h];
  constexpr int kOf = DK / 64;
  for (int64_t t = begin; t < end; ++t) {
    const int turn = (int)(t & 1);
    float kv[kOf], qv[kOf], kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int i = 0; i < kOf; ++i) {
      kv[i] = element<DT>(a.k.p, t * a.k.token + kh * a.k.head + lane + 64 * i);
      qv[i] = element<DT>(a.q.p, t * a.q.token + kh * a.q.head + lane + 64 * i);
      kk = __builtin_fmaf(kv[i], kv[i], kk);
      qq = __builtin_fmaf(qv[i], qv[i], qq);
      kq = __builtin_fmaf(kv[i], qv[i], kq);
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      kk += __shfl_xor(kk, m);
      qq += __shfl_xor(qq, m);
      kq += __shfl_xor(kq, m);
    }
    const float kn = 1.0f / sqrtf(kk + a.eps), qn = 1.0f / sqrtf(qq + a.eps);
    kq *= kn * qn;
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < kOf; ++i) {
        lds_k[turn][lane + 64 * i] = kv[i] * kn;
        lds_q[turn][lane + 64 * i] = qv[i] * qn;
      }
    }
    const float alpha = expf(-rate * softplus(element<DT>(a.a, t * a.a_token + h) + dt));
    const float beta = sigmoid<true>(element<DT>(a.b, t * a.b_token + h));
    __syncthreads();
    float4_t u = {0, 0, 0, 0}, w = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float kr = lds_k[turn][row + i * kGroups], qr = lds_q[turn][row + i * kGroups];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[j] = __builtin_fmaf(s[i][j], kr, u[j]);
        w[j] = __builtin_fmaf(s[i][j], qr, w[j]);
      }
    }
#pragma unroll
    for (int m = kLanes; m < 64; m *= 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[j] += __shfl_xor(u[j], m);
        w[j] += __shfl_xor(w[j], m);
      }
    }
    if (lane < kLanes) {
      lds_sum[turn][0][wave][lane] = u;
      lds_sum[turn][1][wave][lane] = w;
    }
    __syncthreads();
    u = lds_sum[turn][0][0][col];
    w = lds_sum[turn][1][0][col];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
      u += lds_sum[turn][0][i][col];
      w += lds_sum[turn][1][i][col];
    }
    float4_t d;
    const int64_t vo = t * a.v.token + h * a.v.head + column + 4 * col;
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = beta * (element<DT>(a.v.p, vo + j) - alpha * u[j]);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float kr = lds_k[turn][row + i * kGroups];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = __builtin_fmaf(kr, d[j], alpha * s[i][j]);
    }
    if (row == 0) {
      const int64_t o = t * a.out.token + h * a.out.head + column + 4 * col;
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = a.scale * __builtin_fmaf(kq, d[j], alpha * w[j]);
      if constexpr (DT == 0)
        *reinterpret_cast<float4_t*>(static_cast<float*>(a.out.p) + o) = float4_t{y[0], y[1], y[2], y[3]};
      else
        *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out.p) + o) =
            u32x2_t{pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3])};
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    *reinterpret_cast<float4_t*>(a.state_out + state + (int64_t)(row + i * kGroups) * a.head_v) = s[i];
}

template <int DT, int DK>
hipError_t launch_sized(const DeltaArgs& a, hipStream_t stream) {
  const int64_t items = (int64_t)a.n_seqs * a.v_heads * (a.head_v / kCols);
  const FastDiv by_group((uint32_t)(a.v_heads / a.k_heads));
  for (int64_t first = 0; first < items; first += kMostWorkgroups) {
    const uint32_t grid = (uint32_t)std::min<int64_t>(kMostWorkgroups, items - first);
    gated_delta_kernel<DT, DK><<<grid, kThreads, 0, stream>>>(a, by_group, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t launch_typed(const DeltaArgs& a, hipStream_t stream) {
  return a.head_k == 64 ? launch_sized<DT, 64>(a, stream) : launch_sized<DT, 128>(a, stream);
}

}  // namespace

hipError_t launch_gated_delta_chunked(const DeltaArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case 0: return launch_typed<0>(a, stream);
    case 1: return launch_typed<1>(a, stream);
    default: return launch_typed<2>(a, stream);
  }
}

}  // namespace nvfp4
