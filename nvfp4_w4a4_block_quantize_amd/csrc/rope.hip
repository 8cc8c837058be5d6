// Rotary positions with several axes (nvfp4_rope): pair i of every head turns by
//   angle = positions[axis_i][token] * inv_freq_i,
//   (a, b) -> (a cos - b sin, b cos + a sin).
//
// The angle is held in 64 bits as a number of turns, its whole part is dropped
// there, and what is left (at most half a turn) goes to the 32-bit sine and
// cosine of pi*x: a far position loses nothing.  An angle belongs to a token and
// a pair, not to a head, so a workgroup computes the angles of its tokens once,
// into LDS, and all heads of q and k use them.
//
// Bandwidth kernel: every element is read once and written once.  A workgroup
// owns a run of consecutive items of the flat list (token, head, item of the
// head), each thread four of them with all loads in flight before the first is
// used (one, where few heads share an angle and four items' angles would fill
// the LDS).  An item is two vectors of a head that turn together, or one vector
// past rot_dim that is copied; a vector is the widest of 16, 8, 4 or 2 bytes that
// pointers, strides and the two parts of a head allow.
#include <algorithm>

#include "nvfp4_device.h"
#include "kv_internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr size_t kLdsMost = 32 * 1024;  // of angles in a workgroup, so that four fit a CU

struct Plan {
  int pairs;          // rot_dim / 2
  int turn_items;     // items of a head that turn
  int head_items;     // and with those that are copied
  uint32_t token_items;
  int64_t items;
  FastDiv by_token, by_head;
};

template <int DT>
struct Elem;
template <>
struct Elem<0> {
  typedef float type;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<1> {
  typedef __bf16 type;
  static __device__ __forceinline__ float get(__bf16 v) { return (float)v; }
  static __device__ __forceinline__ __bf16 put(float v) { return (__bf16)v; }  // nearest even
};
template <>
struct Elem<2> {
  typedef _Float16 type;
  static __device__ __forceinline__ float get(_Float16 v) { return (float)v; }
  static __device__ __forceinline__ _Float16 put(float v) { return (_Float16)v; }
};

// VEC elements, moved as one access; ALIGNED false: at element alignment, in as many accesses as it takes
template <typename T, int VEC, bool ALIGNED>
struct alignas(ALIGNED ? sizeof(T) * VEC : sizeof(T)) Pack {
  T v[VEC];
};

template <int DT, int VEC, bool ADJACENT, bool ALIGNED, int kUnroll>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, Plan p) {
  typedef typename Elem<DT>::type T;
  typedef Pack<T, VEC, ALIGNED> V;
  constexpr int kItems = kThreads * kUnroll;
  extern __shared__ float2 turns[];  // [token of this workgroup][pair] cosine and sine

  const int64_t item0 = (int64_t)blockIdx.x * kItems;
  const int64_t token0 = item0 / p.token_items;
  const uint32_t skip = (uint32_t)(item0 - token0 * p.token_items);
  const int count = (int)min((int64_t)kItems, p.items - item0);
  const int tokens = (int)(p.by_token.div(skip + count - 1)) + 1;

  constexpr double kPerTurn = 0.15915494309189533576888;  // 1 / (2 pi)
  for (int i = threadIdx.x; i < tokens * p.pairs; i += kThreads) {
    const int t = i / p.pairs, pair = i - t * p.pairs;
    const int axis = min(max(a.axes[pair], 0), a.n_axes - 1);
    const double turn = (double)a.positions[axis * a.ld_pos + token0 + t] * ((double)a.inv_freq[pair] * kPerTurn);
    float s, c;
    sincospif((float)((turn - rint(turn)) * 2.0), &s, &c);
    turns[i] = make_float2(c, s);
  }
  __syncthreads();

  V x[kUnroll], y[kUnroll];
  T* out[kUnroll];
  int kind[kUnroll];  // 0 nothing, 1 turn, 2 copy
  int angle[kUnroll];
  constexpr bool kTwo = !ADJACENT;  // the halves of a turning item lie rot_dim/2 apart
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int n = threadIdx.x + u * kThreads;
    kind[u] = 0;
    if (n >= count) continue;
    const uint32_t at = skip + n;
    const uint32_t t = p.by_token.div(at), in_token = at - t * p.token_items;
    uint32_t head = p.by_head.div(in_token);
    const int item = (int)(in_token - head * p.head_items);
    const bool key = head >= (uint32_t)a.q_heads;
    if (key) head -= a.q_heads;
    const HeadsIn& hi = key ? a.k : a.q;
    const HeadsOut& ho = key ? a.k_out : a.q_out;
    const int64_t token = token0 + t;
    const T* in = static_cast<const T*>(hi.p) + token * hi.token + head * hi.head;
    out[u] = static_cast<T*>(ho.p) + token * ho.token + head * ho.head;
    if (item < p.turn_items) {
      const int e = item * VEC;
      kind[u] = 1;
      angle[u] = (int)t * p.pairs + (ADJACENT ? e / 2 : e);
      out[u] += e;
      x[u] = *reinterpret_cast<const V*>(in + e);
      if constexpr (kTwo) y[u] = *reinterpret_cast<const V*>(in + e + p.pairs);
    } else {
      const int e = a.rot_dim + (item - p.turn_items) * VEC;
      kind[u] = 2;
      out[u] += e;
      x[u] = *reinterpret_cast<const V*>(in + e);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (kind[u] == 0) continue;
    if (kind[u] == 1) {
      if constexpr (kTwo) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float2 cs = turns[angle[u] + i];
          const float p0 = Elem<DT>::get(x[u].v[i]), p1 = Elem<DT>::get(y[u].v[i]);
          x[u].v[i] = Elem<DT>::put(p0 * cs.x - p1 * cs.y);
          y[u].v[i] = Elem<DT>::put(p1 * cs.x + p0 * cs.y);
        }
        *reinterpret_cast<V*>(out[u] + p.pairs) = y[u];
      } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          const float2 cs = turns[angle[u] + i];
          const float p0 = Elem<DT>::get(x[u].v[2 * i]), p1 = Elem<DT>::get(x[u].v[2 * i + 1]);
          x[u].v[2 * i] = Elem<DT>::put(p0 * cs.x - p1 * cs.y);
          x[u].v[2 * i + 1] = Elem<DT>::put(p1 * cs.x + p0 * cs.y);
        }
      }
    }
    *reinterpret_cast<V*>(out[u]) = x[u];
  }
}

template <int DT, int VEC, bool ADJACENT, bool ALIGNED = true>
hipError_t launch_vec(const RopeArgs& a, hipStream_t stream) {
  const bool in_place = a.q_out.p == a.q.p && (a.k_heads == 0 || a.k_out.p == a.k.p);
  Plan p;
  p.pairs = a.rot_dim / 2;
  p.turn_items = (ADJACENT ? a.rot_dim : p.pairs) / VEC;
  p.head_items = p.turn_items + (in_place ? 0 : (a.head_dim - a.rot_dim) / VEC);
  p.token_items = (uint32_t)(a.q_heads + a.k_heads) * (uint32_t)p.head_items;
  p.items = a.tokens * (int64_t)p.token_items;
  p.by_token = FastDiv(p.token_items);
  p.by_head = FastDiv((uint32_t)p.head_items);
  // a run of n items that begins and ends inside a token touches at most this many tokens
  auto lds = [&](int64_t n) {
    return (size_t)std::min<int64_t>(a.tokens, (n - 2) / p.token_items + 2) * p.pairs * sizeof(float2);
  };
  const bool four = lds(4 * kThreads) <= kLdsMost;
  const int64_t n = four ? 4 * kThreads : kThreads, blocks = (p.items + n - 1) / n;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  if (four)
    rope_kernel<DT, VEC, ADJACENT, ALIGNED, 4><<<(unsigned)blocks, kThreads, lds(n), stream>>>(a, p);
  else
    rope_kernel<DT, VEC, ADJACENT, ALIGNED, 1><<<(unsigned)blocks, kThreads, lds(n), stream>>>(a, p);
  return hipGetLastError();
}

// the lowest set bit of everything that a vector has to divide, in elements
uint64_t spacing(const RopeArgs& a, int es) {
  uint64_t m = (uint64_t)a.rot_dim | (uint64_t)a.head_dim | 16u;
  if (!a.adjacent) m |= (uint64_t)a.rot_dim / 2;
  m |= (uint64_t)a.q.token | (uint64_t)a.q.head | (uint64_t)a.q_out.token | (uint64_t)a.q_out.head;
  m |= (reinterpret_cast<uintptr_t>(a.q.p) | reinterpret_cast<uintptr_t>(a.q_out.p)) / es;
  if (a.k_heads) {
    m |= (uint64_t)a.k.token | (uint64_t)a.k.head | (uint64_t)a.k_out.token | (uint64_t)a.k_out.head;
    m |= (reinterpret_cast<uintptr_t>(a.k.p) | reinterpret_cast<uintptr_t>(a.k_out.p)) / es;
  }
  return m & (~m + 1);
}

template <int DT, int ES, bool ADJACENT>
hipError_t launch_widest(const RopeArgs& a, hipStream_t stream) {
  const uint64_t by = spacing(a, ES);
  if constexpr (ES == 2) {
    if (by >= 8) return launch_vec<DT, 8, ADJACENT>(a, stream);
  }
  if (by >= 4) return launch_vec<DT, 4, ADJACENT>(a, stream);
  if (by >= 2) return launch_vec<DT, 2, ADJACENT>(a, stream);
  // neighbours turn together even where nothing lets them move together (head_dim and rot_dim are even)
  return launch_vec<DT, ADJACENT ? 2 : 1, ADJACENT, !ADJACENT>(a, stream);
}

template <int DT, int ES>
hipError_t launch_typed(const RopeArgs& a, hipStream_t stream) {
  return a.adjacent ? launch_widest<DT, ES, true>(a, stream) : launch_widest<DT, ES, false>(a, stream);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case 0: return launch_typed<0, 4>(a, stream);
    case 1: return launch_typed<1, 2>(a, stream);
    default: return launch_typed<2, 2>(a, stream);
  }
}

}  // namespace nvfp4
