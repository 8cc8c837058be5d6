// Rotary positions with several axes (nvfp4_rope): pair i of every head turns by
//   angle = positions[axis_i][token] * inv_freq_i,
//   (a, b) -> (a cos - b sin, b cos + a sin).
//
// The angle is held in 64 bits as a number of turns (right to 2^-51 of itself) and
// its whole part is dropped there.  What is left, at most half a turn, goes to the
// 32-bit sine and cosine of pi*x, and what its rounding to 32 bits drops, r < 2^-23,
// is added to first order: cos - r sin, sin + r cos.  So both are right to a few
// steps of their own size, next to their zeros too, and a position of a million
// loses nothing (without r they were off by up to 2^-23.3; it takes 0.01 of a decode
// step's 2.55 us, and nothing that shows of a prompt's 41).  An angle belongs to a
// token and a pair, not to a head, so a workgroup computes the angles of its tokens
// once, into LDS, and all heads of q and k use them.
//
// Bandwidth kernel: every element is read once and written once (8192 tokens, 28
// heads of 256 in bf16, 64 of them turning: 41 us, 5.7 TB/s, where a copy of that
// size reaches 5.5; 4099 tokens, 18 heads of 128 in f32: 13.8 us).  The loads are
// issued before the angles are computed, which hides them.  A workgroup owns a
// run of consecutive items of the flat list (token; turning or copied; head; item
// of the head), so that a wave's lanes do the same.  An item is two vectors of a
// head that turn together, or one vector past rot_dim that is copied (of heads that
// are not turned in place), each as wide as 16 bytes and the part of the head allow,
// at any alignment: a part's last vector ends where the part ends and shares elements
// with the one before (both store the same values).  In place, where nothing may be
// turned twice, a vector's width divides the part.
#include <algorithm>
#include <type_traits>

#include "nvfp4_device.h"
#include "kv_internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kMore = 2;  // items of a thread, where that gains
constexpr int64_t kInfinityCache = 256 << 20;
constexpr size_t kLdsMost = 32 * 1024;  // of angles in a workgroup, so that four fit a CU

struct Plan {
  int pairs;           // rot_dim / 2
  int turn_last, copy_last;  // where the last vector of a head's turning and copied part begins
  uint32_t turning;    // items of a token that turn; those that are copied follow them
  uint32_t copy_from;  // the first head that is copied
  uint32_t token_items;
  uint32_t items;
  FastDiv by_token, by_turn, by_copy, by_pair;  // items of a token, and of a head that turn and that are copied
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

// VEC elements, moved as one access; ALIGNED false: at element alignment
template <typename T, int VEC, bool ALIGNED>
struct alignas(ALIGNED ? sizeof(T) * VEC : sizeof(T)) Pack {
  T v[VEC];
};

// sixteen bytes at the alignment of a float32 or 16-bit element (a type's reduced alignment does not pass a template)
typedef uint32_t u32x4_by4_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_by2_t __attribute__((ext_vector_type(4), aligned(2)));

// Stores past the caches where they are as wide as that takes: the outputs of a prompt do not fit there, and
// leave the other halves of the lines being read in place (8192 tokens, 28 heads of 256: 70 -> 47 us).
template <typename V>
__device__ __forceinline__ void store(void* p, const V& v) {
  if constexpr (sizeof(V) != 16) {
    *reinterpret_cast<V*>(p) = v;
  } else {
    const u32x4_t w = __builtin_bit_cast(u32x4_t, v);
    if constexpr (alignof(V) == 16) __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(p));
    else if constexpr (alignof(V) == 4) __builtin_nontemporal_store(w, reinterpret_cast<u32x4_by4_t*>(p));
    else __builtin_nontemporal_store(w, reinterpret_cast<u32x4_by2_t*>(p));
  }
}

// VEC, COPY: elements of a turning and of a copied vector
template <int DT, int VEC, int COPY, bool ADJACENT, bool ALIGNED, int kUnroll>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, Plan p) {
  typedef typename Elem<DT>::type T;
  typedef Pack<T, VEC, ALIGNED> V;
  typedef Pack<T, COPY, ALIGNED> C;
  constexpr int kItems = kThreads * kUnroll;
  extern __shared__ float2 turns[];  // [token of this workgroup][pair] cosine and sine

  const uint32_t item0 = blockIdx.x * kItems;  // a launch has fewer than 2^29 items
  const uint32_t token0 = p.by_token.div(item0), skip = item0 - token0 * p.token_items;
  const int count = (int)min((uint32_t)kItems, p.items - item0);
  const int tokens = (int)(p.by_token.div(skip + count - 1)) + 1;

  V x[kUnroll], y[kUnroll];
  C z[kUnroll];
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
    const bool turn = in_token < p.turning;
    const uint32_t i = turn ? in_token : in_token - p.turning;
    uint32_t head = turn ? p.by_turn.div(i) : p.by_copy.div(i);
    const int item = (int)(i - head * (turn ? p.by_turn.d : p.by_copy.d));
    if (!turn) head += p.copy_from;
    const bool key = head >= (uint32_t)a.q_heads;
    if (key) head -= a.q_heads;
    // by value: a reference to either would be read from memory by each lane
    const HeadsIn hi = {key ? a.k.p : a.q.p, key ? a.k.token : a.q.token, key ? a.k.head : a.q.head};
    const HeadsOut ho = {key ? a.k_out.p : a.q_out.p, key ? a.k_out.token : a.q_out.token,
                         key ? a.k_out.head : a.q_out.head};
    const int64_t token = token0 + t;
    const int e = turn ? min(item * VEC, p.turn_last) : min(a.rot_dim + item * COPY, p.copy_last);
    const T* in = static_cast<const T*>(hi.p) + token * hi.token + head * hi.head + e;
    out[u] = static_cast<T*>(ho.p) + token * ho.token + head * ho.head + e;
    kind[u] = turn ? 1 : 2;
    angle[u] = (int)t * p.pairs + (ADJACENT ? e / 2 : e);
    if constexpr (COPY == VEC) {  // one load for both: a branch around it would wait for it
      x[u] = *reinterpret_cast<const V*>(in);
    } else {
      if (turn) x[u] = *reinterpret_cast<const V*>(in);
      else z[u] = *reinterpret_cast<const C*>(in);
    }
    if constexpr (kTwo) {
      if (turn) y[u] = *reinterpret_cast<const V*>(in + p.pairs);
    }
  }
  constexpr double kPerTurn = 0.15915494309189533576888;  // 1 / (2 pi)
  for (int i = threadIdx.x; i < tokens * p.pairs; i += kThreads) {
    const int t = (int)p.by_pair.div((uint32_t)i), pair = i - t * p.pairs;
    const int axis = min(max(a.axes[pair], 0), a.n_axes - 1);
    const double turn = (double)a.positions[axis * a.ld_pos + token0 + t] * ((double)a.inv_freq[pair] * kPerTurn);
    const double halves = (turn - rint(turn)) * 2.0;
    const float x = (float)halves, rest = (float)(halves - (double)x) * 3.14159265f;
    float s, c;
    sincospif(x, &s, &c);
    turns[i] = make_float2(c - s * rest, s + c * rest);
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (kind[u] == 1) {
      if constexpr (kTwo) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float2 cs = turns[angle[u] + i];
          const float p0 = Elem<DT>::get(x[u].v[i]), p1 = Elem<DT>::get(y[u].v[i]);
          x[u].v[i] = Elem<DT>::put(p0 * cs.x - p1 * cs.y);
          y[u].v[i] = Elem<DT>::put(p1 * cs.x + p0 * cs.y);
        }
        store<V>(out[u] + p.pairs, y[u]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          const float2 cs = turns[angle[u] + i];
          const float p0 = Elem<DT>::get(x[u].v[2 * i]), p1 = Elem<DT>::get(x[u].v[2 * i + 1]);
          x[u].v[2 * i] = Elem<DT>::put(p0 * cs.x - p1 * cs.y);
          x[u].v[2 * i + 1] = Elem<DT>::put(p1 * cs.x + p0 * cs.y);
        }
      }
      store<V>(out[u], x[u]);
    } else if (kind[u] == 2) {
      if constexpr (COPY == VEC) store<V>(out[u], x[u]);
      else store<C>(out[u], z[u]);
    }
  }
}

// whether some heads are turned in place, and what each of the others copies
bool some_in_place(const RopeArgs& a) { return rope_copied(a).count < a.q_heads + a.k_heads; }
int copied(const RopeArgs& a) { return rope_copied(a).count > 0 ? a.head_dim - a.rot_dim : 0; }

template <int DT, int VEC, int COPY, bool ADJACENT, bool ALIGNED>
hipError_t launch_vec(RopeArgs a, hipStream_t stream) {
  Plan p;
  p.pairs = a.rot_dim / 2;
  const uint32_t heads = (uint32_t)(a.q_heads + a.k_heads);
  const int turn = ADJACENT ? a.rot_dim : p.pairs, copy = copied(a);
  p.turn_last = turn - VEC;
  p.copy_last = a.head_dim - COPY;
  p.by_turn = FastDiv((uint32_t)(turn + VEC - 1) / VEC);
  p.by_copy = FastDiv((uint32_t)(copy + COPY - 1) / COPY);
  p.turning = heads * p.by_turn.d;
  p.token_items = p.turning + (uint32_t)rope_copied(a).count * p.by_copy.d;
  p.copy_from = (uint32_t)rope_copied(a).first;
  p.by_token = FastDiv(p.token_items);
  p.by_pair = FastDiv((uint32_t)p.pairs);
  // Two items to a thread gain where they leave every CU four workgroups, and while the call (read and written) is within
  // the Infinity Cache; beyond that they still do where items have one vector and whole 64-byte pieces.  Halves, which
  // have two vectors already, gain only beside a copied part, if that begins with a 64-byte piece.  One and two items, us
  // in a graph, operands of three calls in turn:
  //   tokens x heads x elements, turning         bytes  one / two    tokens x heads x elements, turning         bytes  one / two
  //   neighbours paired:
  //   4099 x 18 x 128, 64   bf16                 38 MB   9.3 / 8.2    1024 x 18 x 128, 64   bf16                 9 MB   4.0 / 4.5
  //   8192 x 28 x 256, 64   bf16                235     44.9 / 41.6   512 x 18 x 64, 64     f32                   5     3.4 / 3.8
  //   8192 x 28 x 128, 128  f32                 235     45.5 / 41.7   512 x 18 x 128, 48    f32                   9     4.1 / 4.4
  //   32768 x 28 x 256, 256 bf16                940      166 / 159    32768 x 28 x 256, 48  bf16                940      213 / 239
  //   4099 x 18 x 256, 48   bf16                 76     17.4 / 16.3
  //   halves:
  //   2048 x 28 x 256, 64   bf16                 59     12.4 / 11.5   1024 x 28 x 128, 64   bf16                 15     4.4 / 5.0
  //   8192 x 28 x 256, 64   bf16                235     43.2 / 42.3   32768 x 40 x 256, 64  bf16               1342      214 / 237
  //   8192 x 28 x 128, 64   bf16                117     21.9 / 21.3   8192 x 28 x 256, 128  f32                 470     79.1 / 84.4
  //   4099 x 18 x 256, 48   f32                 151     28.5 / 25.9   2048 x 28 x 128, 128  bf16                 29      7.0 / 7.4
  //   4099 x 18 x 128, 64   f32                  76     14.7 / 13.6   8192 x 28 x 128, 16   bf16                117     27.5 / 31.3
  constexpr int64_t ES = sizeof(typename Elem<DT>::type);
  const bool pieces = ALIGNED && (copy == 0 || a.rot_dim * ES % 64 == 0);
  for (int64_t left = a.tokens;;) {
    a.tokens = std::min(left, std::max<int64_t>(kMostWorkgroups * kThreads / p.token_items, 1));
    p.items = (uint32_t)(a.tokens * p.token_items);
    // a run of n items that begins and ends inside a token touches at most this many tokens
    auto lds = [&](int64_t n) {
      return (size_t)std::min<int64_t>(a.tokens, (n - 2) / p.token_items + 2) * p.pairs * sizeof(float2);
    };
    const bool cached = 2 * a.tokens * heads * a.head_dim * ES <= kInfinityCache;
    const bool gain = ADJACENT ? pieces || cached : copy > 0 && pieces && cached;
    const bool more = gain && lds(kMore * kThreads) <= kLdsMost &&
                      p.items >= (int64_t)device_cu_count() * 4 * kMore * kThreads;
    const uint32_t n = more ? kMore * kThreads : kThreads, blocks = (p.items + n - 1) / n;
    if constexpr (ADJACENT || ALIGNED) {
      if (more) rope_kernel<DT, VEC, COPY, ADJACENT, ALIGNED, kMore><<<blocks, kThreads, lds(n), stream>>>(a, p);
    }
    if (!more) rope_kernel<DT, VEC, COPY, ADJACENT, ALIGNED, 1><<<blocks, kThreads, lds(n), stream>>>(a, p);
    const hipError_t e = hipGetLastError();
    left -= a.tokens;
    if (e != hipSuccess || left == 0) return e;
    auto skip = [&](auto& x) {
      if (x.p) x.p = (decltype(x.p))((uintptr_t)x.p + (uintptr_t)(a.tokens * x.token * ES));
    };
    skip(a.q);
    skip(a.q_out);
    skip(a.k);
    skip(a.k_out);
    a.positions += a.tokens;
  }
}

template <int DT, bool ADJACENT>
hipError_t launch_widest(const RopeArgs& a, hipStream_t stream) {
  constexpr int ES = DT == 0 ? 4 : 2, kFull = 16 / ES;
  const int turn = ADJACENT ? a.rot_dim : a.rot_dim / 2, copy = copied(a);
  int vec = kFull;
  while (some_in_place(a) ? turn % vec != 0 : vec > turn) vec /= 2;
  const bool wide = copy == 0 || copy >= kFull;
  uint64_t at = (uint64_t)(turn | copy) * ES;  // its lowest set bit is that of all vectors' addresses
  for (int64_t s : {a.q.token, a.q.head, a.q_out.token, a.q_out.head}) at |= (uint64_t)s * ES;
  at |= reinterpret_cast<uintptr_t>(a.q.p) | reinterpret_cast<uintptr_t>(a.q_out.p);
  if (a.k_heads) {
    for (int64_t s : {a.k.token, a.k.head, a.k_out.token, a.k_out.head}) at |= (uint64_t)s * ES;
    at |= reinterpret_cast<uintptr_t>(a.k.p) | reinterpret_cast<uintptr_t>(a.k_out.p);
  }
  if (vec == kFull && wide && at % 16 == 0) return launch_vec<DT, kFull, kFull, ADJACENT, true>(a, stream);
  auto launch = [&](auto v) {
    constexpr int VEC = decltype(v)::value;
    return wide ? launch_vec<DT, VEC, kFull, ADJACENT, false>(a, stream)
                : launch_vec<DT, VEC, 1, ADJACENT, false>(a, stream);
  };
  if constexpr (ES == 2) {
    if (vec == 8) return launch(std::integral_constant<int, 8>());
  }
  if (vec == 4) return launch(std::integral_constant<int, 4>());
  if constexpr (!ADJACENT) {
    if (vec == 1) return launch(std::integral_constant<int, 1>());
  }
  return launch(std::integral_constant<int, 2>());  // neighbours always go together: rot_dim is even
}

template <int DT>
hipError_t launch_typed(const RopeArgs& a, hipStream_t stream) {
  return a.adjacent ? launch_widest<DT, true>(a, stream) : launch_widest<DT, false>(a, stream);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case 0: return launch_typed<0>(a, stream);
    case 1: return launch_typed<1>(a, stream);
    default: return launch_typed<2>(a, stream);
  }
}

}  // namespace nvfp4
