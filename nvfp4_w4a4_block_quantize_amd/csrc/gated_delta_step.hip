// The gated delta rule for one new token a sequence (nvfp4_gated_delta_step).
//
//   S' = e^g S;  d = beta (v - S'^T k~);  S_new = S' + k~ d^T;  out = scale S_new^T q~
//
// Bandwidth kernel: 4 head_k head_v bytes of state read and written a head, 7 flop an
// element.  A workgroup takes COLS columns of one head's state.  All of its rows are
// in the threads' registers at once, so the state is read once: S^T k~ and S^T q~ are
// summed together, and out = scale (e^g S^T q~ + (k~ . q~) d) needs no second sum.
//
// 48 heads of 128 x 128, us a call in a graph:    1 sequence    8     32    128
//   64 columns a workgroup                        4.78        11.9   40.7  150.9
//   32                                            4.63        12.9   42.2  159.4
//   128                                           5.27        11.6   40.9  154.6
//   64, states loaded and stored past the caches  4.75         9.7   36.4  143.8
// The last is taken: 5.2 TB/s at 32 sequences, 5.6 at 128.  A step's states are not met
// again before every other layer's.
#include <algorithm>

#include "gdn_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sum_of_wave(float x) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) x += __shfl_xor(x, m);
  return x;
}

// sums of squares between which neither they, their products nor the squares of what counts in them leave the normal range
constexpr float kLeastSquares = 0x1p-80f, kMostSquares = 0x1p120f;

// A row of a wave, N elements a lane, times the power of two that takes its largest element into [1/2, 1); returns what
// then makes it a unit row.
template <int N>
__device__ __forceinline__ float unit_norm(float (&x)[N], float eps) {
  float top = 0.0f, squares = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
  for (int m = 1; m < 64; m *= 2) top = fmaxf(top, __shfl_xor(top, m));
  const int up = -__builtin_amdgcn_frexp_expf(top);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = __builtin_amdgcn_ldexpf(x[i], up);
    squares = __builtin_fmaf(x[i], x[i], squares);
  }
  return norm_of(sum_of_wave(squares), up, eps);
}

// Four waves a SIMD where a state's head has 128 rows: with the five that its registers allow, 128 sequences take 145.9 us
// and not 144.3.  Heads of 64 rows take as many as fit (21.5 us at 32 sequences in float32, with four 21.9).
template <int DT, int DK, int COLS>
__global__ __launch_bounds__(kThreads)
    __attribute__((amdgpu_waves_per_eu(4, DK == 128 ? 4 : 8))) void gated_delta_step_kernel(DeltaArgs a, FastDiv by_group, int64_t first) {
  constexpr int kLanes = COLS / 4;            // of a row
  constexpr int kGroups = kThreads / kLanes;  // rows at a time
  constexpr int kRows = DK / kGroups;
  constexpr int kWaves = kThreads / 64;
  __shared__ float lds_k[DK], lds_q[DK];
  __shared__ float4_t lds_sum[2][kWaves][kLanes];

  const int slices = a.head_v / COLS;
  const int64_t item = first + blockIdx.x;
  const int64_t pair = item / slices;
  const int column = (int)(item - pair * slices) * COLS;
  const int64_t r = pair / a.v_heads;
  const int h = (int)(pair - r * a.v_heads);
  const int slot = a.slots[r];
  if (!slot_ok(slot, a.num_slots)) return;
  const int thread = threadIdx.x, lane = thread & 63, wave = thread >> 6;
  const int col = thread % kLanes, row = thread / kLanes;

  const int64_t state = (((int64_t)slot * a.v_heads + h) * DK) * a.head_v + column + 4 * col;
  float4_t s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    s[i] = __builtin_nontemporal_load(reinterpret_cast<const float4_t*>(a.state + state + (int64_t)(row + i * kGroups) * a.head_v));

  // k~, q~: each wave makes them for itself, DK / 64 elements a lane
  const int kh = (int)by_group.div((uint32_t)h);
  constexpr int kOf = DK / 64;
  float kv[kOf], qv[kOf], kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
  for (int i = 0; i < kOf; ++i) {
    kv[i] = element<DT>(a.k.p, r * a.k.token + kh * a.k.head + lane + 64 * i);
    qv[i] = element<DT>(a.q.p, r * a.q.token + kh * a.q.head + lane + 64 * i);
  }
  const float av = element<DT>(a.a, r * a.a_token + h), bv = element<DT>(a.b, r * a.b_token + h);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = element<DT>(a.v.p, r * a.v.token + h * a.v.head + column + 4 * col + i);
#pragma unroll
  for (int i = 0; i < kOf; ++i) {
    kk = __builtin_fmaf(kv[i], kv[i], kk);
    qq = __builtin_fmaf(qv[i], qv[i], qq);
    kq = __builtin_fmaf(kv[i], qv[i], kq);
  }
  kk = sum_of_wave(kk);
  qq = sum_of_wave(qq);
  kq = sum_of_wave(kq);
  float kn, qn;
  if (kk > kLeastSquares && kk < kMostSquares && qq > kLeastSquares && qq < kMostSquares) {
    kn = 1.0f / sqrtf(kk + a.eps);
    qn = 1.0f / sqrtf(qq + a.eps);
    kq *= kn * qn;
  } else {  // squares that overflowed or vanished: the rows by a power of two first
    kn = unit_norm(kv, a.eps);
    qn = unit_norm(qv, a.eps);
    kq = 0.0f;
#pragma unroll
    for (int i = 0; i < kOf; ++i) kq = __builtin_fmaf(kv[i] * kn, qv[i] * qn, kq);
    kq = sum_of_wave(kq);
  }
  if (wave == 0) {
#pragma unroll
    for (int i = 0; i < kOf; ++i) {
      lds_k[lane + 64 * i] = kv[i] * kn;
      lds_q[lane + 64 * i] = qv[i] * qn;
    }
  }
  const float alpha = expf(-expf(a.a_log[h]) * softplus(av + a.dt_bias[h]));
  const float beta = sigmoid<true>(bv);
  __syncthreads();

  float4_t u = {0, 0, 0, 0}, w = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float kr = lds_k[row + i * kGroups], qr = lds_q[row + i * kGroups];
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
    lds_sum[0][wave][lane] = u;
    lds_sum[1][wave][lane] = w;
  }
  __syncthreads();
  u = lds_sum[0][0][col];
  w = lds_sum[1][0][col];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    u += lds_sum[0][i][col];
    w += lds_sum[1][i][col];
  }
  float4_t d;
#pragma unroll
  for (int j = 0; j < 4; ++j) d[j] = beta * (v[j] - alpha * u[j]);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float kr = lds_k[row + i * kGroups];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = __builtin_fmaf(kr, d[j], alpha * s[i][j]);
    __builtin_nontemporal_store(s[i], reinterpret_cast<float4_t*>(a.state_out + state + (int64_t)(row + i * kGroups) * a.head_v));
  }
  if (row == 0) {
    const int64_t o = r * a.out.token + h * a.out.head + column + 4 * col;
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = a.scale * __builtin_fmaf(kq, d[j], alpha * w[j]);
    if constexpr (DT == 0) {
      *reinterpret_cast<float4_t*>(static_cast<float*>(a.out.p) + o) = float4_t{y[0], y[1], y[2], y[3]};
    } else {
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out.p) + o) =
          u32x2_t{pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3])};
    }
  }
}

template <int DT, int DK>
hipError_t launch_sized(const DeltaArgs& a, hipStream_t stream) {
  constexpr int kCols = 64;
  const int64_t items = (int64_t)a.n_seqs * a.v_heads * (a.head_v / kCols);
  const FastDiv by_group((uint32_t)(a.v_heads / a.k_heads));
  for (int64_t first = 0; first < items; first += kMostWorkgroups) {
    const uint32_t grid = (uint32_t)std::min<int64_t>(kMostWorkgroups, items - first);
    gated_delta_step_kernel<DT, DK, kCols><<<grid, kThreads, 0, stream>>>(a, by_group, first);
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

hipError_t launch_gated_delta_step(const DeltaArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case 0: return launch_typed<0>(a, stream);
    case 1: return launch_typed<1>(a, stream);
    default: return launch_typed<2>(a, stream);
  }
}

}  // namespace nvfp4
