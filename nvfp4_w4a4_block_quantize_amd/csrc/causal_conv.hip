// Causal depthwise convolution of ragged prompts, and of one token a sequence
// (nvfp4_causal_conv, nvfp4_causal_conv_step).
//
//   y_t[c] = act(bias[c] + sum_j w[c][j] x_{t-(W-1)+j}[c])
//
// Bandwidth kernel: each input read once and each output written once.  A thread
// owns E neighbouring channels (16 bytes) and walks ROWS tokens with the last
// W - 1 inputs and its weights in registers, so an input is loaded by one thread but
// for the W - 1 rows before its first token.
//
// A sequence's state is read only by the workgroup that holds its first token, which
// also takes the tokens behind it that still see the state (they may lie past its own
// rows) and writes the new state, after reading the old one.  So state_out may be
// state.
#include <algorithm>

#include "gdn_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 64;

template <int DT, int E, int W>
struct Taps {
  float w[W][E], bias[E];
  __device__ __forceinline__ void load(const ConvArgs& a, int c) {
    float flat[E * W];
    if constexpr (E == 1) {
#pragma unroll
      for (int i = 0; i < W; ++i) flat[i] = a.weight[(int64_t)c * W + i];
      bias[0] = a.bias ? a.bias[c] : 0.0f;
    } else {
      Elements<0, E * W> all;
      all.load(a.weight, (int64_t)c * W);
#pragma unroll
      for (int i = 0; i < E * W; ++i) flat[i] = all.get(i);
      Elements<0, E> b;
      b.zero();
      if (a.bias) b.load(a.bias, c);
#pragma unroll
      for (int e = 0; e < E; ++e) bias[e] = b.get(e);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][e] = flat[e * W + j];
  }
  // rows[0] is the oldest
  __device__ __forceinline__ Elements<DT, E> at(const Elements<DT, E> (&rows)[W], int activation) const {
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float s = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) s = __builtin_fmaf(w[j][e], rows[j].get(e), s);
      y[e] = activation ? s * sigmoid<DT == 0>(s) : s;
    }
    Elements<DT, E> out;
    out.set(y);
    return out;
  }
};

// the last sequence from `low` on that starts at or before row t; `low` if none does
__device__ __forceinline__ int sequence_at(const int32_t* starts, int low, int n, int64_t t) {
  int high = n;  // the answer is in [low, high)
  while (high - low > 1) {
    const int mid = low + (high - low) / 2;
    if (starts[mid] <= t) low = mid; else high = mid;
  }
  return low;
}

template <int DT, int E, int W, int ROWS, bool PAST>
__global__ __launch_bounds__(kThreads) void causal_conv_kernel(ConvArgs a, int64_t first_block) {
  const int c = (blockIdx.y * kThreads + threadIdx.x) * E;
  if (c >= a.channels) return;
  const int64_t begin = (first_block + blockIdx.x) * ROWS, behind = std::min(begin + ROWS, a.tokens);
  Taps<DT, E, W> taps;
  taps.load(a, c);
  int r = sequence_at(a.token_starts, 0, a.n_seqs, begin);
  int64_t low = start_of(a.token_starts, r, a.tokens), high = start_of(a.token_starts, r + 1, a.tokens);
  // tokens that see a sequence's state belong to the workgroup of its first one
  int64_t t = low >= begin ? low : std::max(begin, std::min(low + W - 1, high));
  for (;;) {
    while (t >= high) {  // on to the next sequence with rows
      if (high >= behind || ++r >= a.n_seqs) return;
      low = std::max(high, start_of(a.token_starts, r, a.tokens));
      high = start_of(a.token_starts, r + 1, a.tokens);
      if (high <= low && r + 1 < a.n_seqs) {  // none, nor maybe have many behind it: the last one that starts here
        r = sequence_at(a.token_starts, r + 1, a.n_seqs, low);
        low = std::max(low, start_of(a.token_starts, r, a.tokens));
        high = start_of(a.token_starts, r + 1, a.tokens);
      }
      t = low;
    }
    const bool mine = t == low;  // its first token
    if (t >= behind) return;
    const int slot = a.slots[r];
    if (!slot_ok(slot, a.num_slots)) {
      t = high;
      continue;
    }
    Elements<DT, E> rows[W];
    const int64_t state = (int64_t)slot * (W - 1) * a.channels + c;
    if (mine) {
      const bool carried = !a.cached_lens || a.cached_lens[r] > 0;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        if (carried) rows[j].load(a.state, state + (int64_t)j * a.channels);
        else rows[j].zero();
      }
      const int64_t n = high - low;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        Elements<DT, E> last;
        if (n >= W - 1 - j) {
          last.load(a.x, (high - (W - 1) + j) * a.ldx + c);
        } else {  // of the old state: row j + n, and n is at least 1
          last = rows[W - 2];
#pragma unroll
          for (int i = 1; i < W - 2; ++i)
            if (j + n == i) last = rows[i];
        }
        last.store(a.state_out, state + (int64_t)j * a.channels);
      }
    } else {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) rows[j].load(a.x, (t - (W - 1) + j) * a.ldx + c);
    }
    const int64_t end = std::min(high, std::max(behind, mine ? std::min(low + W - 1, high) : behind));
    constexpr int kAhead = 8;  // rows under way at a time
    for (; t + kAhead <= end; t += kAhead) {
      Elements<DT, E> next[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next[i].load(a.x, (t + i) * a.ldx + c);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        rows[W - 1] = next[i];
        taps.at(rows, a.activation).template store<PAST>(a.out, (t + i) * a.ldo + c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) rows[j] = rows[j + 1];
      }
    }
    if (t < end) {
      Elements<DT, E> next[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next[i].load(a.x, std::min(t + i, end - 1) * a.ldx + c);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        rows[W - 1] = next[i];
        if (t + i < end) taps.at(rows, a.activation).template store<PAST>(a.out, (t + i) * a.ldo + c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) rows[j] = rows[j + 1];
      }
    }
    t = end;
    if (t >= behind) return;
  }
}

template <int DT, int E, int W>
__global__ __launch_bounds__(kThreads) void causal_conv_step_kernel(ConvArgs a, int64_t first) {
  const int c = (blockIdx.y * kThreads + threadIdx.x) * E;
  if (c >= a.channels) return;
  const int64_t r = first + blockIdx.x;
  const int slot = a.slots[r];
  if (!slot_ok(slot, a.num_slots)) return;
  Elements<DT, E> rows[W];
  const int64_t state = (int64_t)slot * (W - 1) * a.channels + c;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j].load(a.state, state + (int64_t)j * a.channels);
  rows[W - 1].load(a.x, r * a.ldx + c);
  Taps<DT, E, W> taps;
  taps.load(a, c);
  taps.at(rows, a.activation).store(a.out, r * a.ldo + c);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j + 1].store(a.state_out, state + (int64_t)j * a.channels);
}

// `launch(blocks, columns, first block)`, so many blocks at a time
template <typename F>
hipError_t for_blocks(int64_t blocks, uint32_t columns, F launch) {
  const int64_t most = std::max<int64_t>(kMostWorkgroups / columns, 1);
  for (int64_t first = 0; first < blocks; first += most) {
    launch(dim3((uint32_t)std::min(most, blocks - first), columns), first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int E, int W, int ROWS, bool PAST>
hipError_t launch_rows(const ConvArgs& a, uint32_t columns, hipStream_t stream) {
  return for_blocks((a.tokens + ROWS - 1) / ROWS, columns, [&](dim3 grid, int64_t first) {
    causal_conv_kernel<DT, E, W, ROWS, PAST><<<grid, kThreads, 0, stream>>>(a, first);
  });
}

template <int DT, int E, int W>
hipError_t launch_width(const ConvArgs& a, bool step, hipStream_t stream) {
  const uint32_t columns = (uint32_t)((a.channels + (int64_t)kThreads * E - 1) / (kThreads * E));
  if (step)
    return for_blocks(a.tokens, columns, [&](dim3 grid, int64_t first) {
      causal_conv_step_kernel<DT, E, W><<<grid, kThreads, 0, stream>>>(a, first);
    });
  const int rows = conv_rows(a.tokens, columns, E > 1, device_cu_count());
  if constexpr (E > 1) {
    if (rows == 32) return launch_rows<DT, E, W, 32, true>(a, columns, stream);
  }
  return rows == 16 ? launch_rows<DT, E, W, 16, false>(a, columns, stream) : launch_rows<DT, E, W, 8, false>(a, columns, stream);
}

template <int DT, int E>
hipError_t launch_elements(const ConvArgs& a, bool step, hipStream_t stream) {
  switch (a.width) {
    case 2: return launch_width<DT, E, 2>(a, step, stream);
    case 3: return launch_width<DT, E, 3>(a, step, stream);
    default: return launch_width<DT, E, 4>(a, step, stream);
  }
}

template <int DT>
hipError_t launch_typed(const ConvArgs& a, bool step, hipStream_t stream) {
  constexpr int kElements = 16 / element_size(DT);
  auto whole = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  if (a.channels % kElements == 0 && a.ldx % kElements == 0 && a.ldo % kElements == 0 && whole(a.x) && whole(a.out) &&
      whole(a.state) && whole(a.state_out) && whole(a.weight) && whole(a.bias))
    return launch_elements<DT, kElements>(a, step, stream);
  return launch_elements<DT, 1>(a, step, stream);
}

hipError_t launch(const ConvArgs& a, bool step, hipStream_t stream) {
  switch (a.dtype) {
    case 0: return launch_typed<0>(a, step, stream);
    case 1: return launch_typed<1>(a, step, stream);
    default: return launch_typed<2>(a, step, stream);
  }
}

}  // namespace

hipError_t launch_causal_conv(const ConvArgs& a, hipStream_t stream) { return launch(a, false, stream); }
hipError_t launch_causal_conv_step(const ConvArgs& a, hipStream_t stream) { return launch(a, true, stream); }

}  // namespace nvfp4
