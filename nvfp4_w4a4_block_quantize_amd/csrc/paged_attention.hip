// Attention of one new token per sequence over a paged FP8 cache
// (nvfp4_paged_attention):
//   s_j = scale * q . k_j / k_scale,  out = sum_j softmax(s)_j v_j / v_scale.
//
// A cache byte that is read serves all G = q_heads / kv_heads queries of its head, or
// 16 or 32 of them (attention_rows_of_item), a wider group's bytes being read again
// for the rest: 4 operations a query for each pair of K and V bytes, far below what
// the matrix units do in the time that HBM takes to deliver them.  The kernel is built
// to keep loads in flight and little else: without its arithmetic it took 2% less.
// 64 contexts up to 16384 tokens, 24 heads of 256 on 4: 192 us for 1.17 GB, 6.1 TB/s (a
// streaming read reaches 7.1).  One of 131072: 53 us for 268 MB, of which first loads
// take 4 and the second kernel 5.
//
// Work.  Each (sequence, KV head) is an item of ceil(tokens / 128) units, and one
// more for what beginning and ending it costs.  The units of all items lie on
// one axis and the grid's workers take equal consecutive runs of it, whatever
// the lengths: a run covers the end of one item, whole items, and the beginning
// of another.  Whole items are finished in place.  Of the others each worker leaves
// a partial result (maximum, sum, unnormalised output; at most two of them), and a
// second, small kernel joins those.  Lengths are read on the device, so a captured
// graph follows them.  Runs are one to a resident workgroup: with two or four of
// them the ends are no more even (4 and 13% more for the 64 contexts).  Where items
// are short, each has a workgroup to itself instead, of more waves where it has the
// CU to itself, and nothing is joined (launch() says where).
//
// The workgroup's waves (four of them for a unit) take tiles of 32 tokens in turn and
// run on their own (maxima, sums and outputs of their own) until the item ends.
// Nothing passes through LDS or between lanes on the way of the data:
//  * S^T = K Q^T with v_mfma_16x16x32.  Lane (i = lane % 16, g = lane / 16) of
//    the K operand loads 16 consecutive bytes of one token's row, for two steps
//    of the product; Q is held in registers in the same order of d.  A load
//    should cover whole 128-byte lines, and neighbouring rows (a wave's loads are
//    then spread over the L2's channels), but the operand's rows are 16 with 64
//    bytes each.  So lanes i = 2 r and 2 r + 1 take the two halves of one token's
//    line, the operand meets the queries' first halves in one product and the
//    second halves in another, and a token's score is the sum of the first one's
//    even row and the second one's odd row (half of what the matrix unit does is
//    thrown away; it has the time).  Four products j = 0 .. 3 make a tile, of 8
//    neighbouring tokens each: row i is token 8 j + 4 (r % 2) + r / 2.  Where 64
//    bytes of a row remain (head_dim 64, 192), row i of the products j = 0, 1 is
//    token 16 j + 4 (i % 4) + i / 4.  Either way a lane's eight scores are those of
//    query i with the tokens g, 4 + g, .. 28 + g,
//  * which is just what O^T = V^T P^T wants of it as P^T operand.  For V^T the
//    lane loads D/16 bytes of those eight tokens' rows (four neighbouring rows a
//    load); after the exact conversion to fp16 one v_perm for two values turns
//    token pairs together.  Row i of the product for byte n is d = i D/16 + n.
//  * Eight neighbouring tokens lie in one page (page sizes are multiples of 8), so
//    a tile has four addresses, the same for all lanes: they are made from scalar
//    loads of the table, one tile ahead of the rows that they lead to.
//
// Softmax.  One pass: p = 2^(s' - m), s' = s log2(e), and m a running whole number that
// starts kShift below the first maximum and moves only when some score passes it by
// kShift + kSlack.  m cancels in the end and being whole, its changes scale by exact
// powers of two.  s' - m is rounded once; past kFar s' is rounded before, as it is for
// the maximum (else the largest score's p could be anything).  kShift puts p below
// 2^15, in fp16's upper range.  A probability meets its values as two fp16 parts and so
// is held to 2^-22 of itself, or to 2^-36 of the largest one where that is more.  With
// one part, outputs whose values cancel were off by many times their own rounding, bf16
// ones too (two tokens, 256 outputs: 10 to 20 times what is allowed); the second part
// takes 0.4 of 191.7 us (64 contexts up to 16384, 24 heads of 256 on 4) and 0.3 of 53.3
// (one of 131072).
#include <algorithm>
#include <type_traits>

#include "nvfp4_device.h"
#include "kv_internal.h"

namespace nvfp4 {
namespace {

constexpr int kTile = 32;                  // tokens of a wave's tile
constexpr int kUnitTiles = 4;
constexpr int kUnitTokens = kTile * kUnitTiles;  // the smallest unit
constexpr int kItemCost = 1;  // what beginning and ending an item costs, in units
constexpr float kNoMax = -3.402823466e38f;  // m before any score; finite, so that differences are numbers
constexpr float kShift = 12.0f, kSlack = 3.0f;
constexpr float kFar = 0x1p22f;  // of m, from where on a score's rounding to 32 bits is no small part of a power of two
constexpr float kLn2 = 0.69314718055994530942f;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// rows of a worker's partial results, and where they lie in the workspace
struct Partials {
  int4* split;   // items that several workers share: {sequence or -1, item of it, first worker, last worker},
                 // one entry for each item (by_item) or for each worker (the item that it leaves unfinished)
  float2* ml;    // [2 workers][rows] maximum and sum
  float* o;      // [2 workers][rows][D]
};

struct Params {
  PagedAttentionArgs a;
  FastDiv by_page;
  int group;      // query heads of a KV head
  int parts;      // items that a KV head's queries are split into
  int rows;       // query heads of an item
  int items;      // of a sequence: kv_heads * parts
  bool by_item;   // how `split` is indexed: by item where there are no more of them than workers
  bool whole;     // items are not split: each has a workgroup of its own
  int64_t page_bytes;
  Partials ws;
};

template <int DT>
struct OutType;
template <>
struct OutType<0> { typedef float type; };
template <>
struct OutType<1> { typedef __bf16 type; };
template <>
struct OutType<2> { typedef _Float16 type; };

// four outputs of one row
template <int DT>
__device__ __forceinline__ void store4(const PagedAttentionArgs& a, int seq, int head, int d, float4 v) {
  typedef typename OutType<DT>::type T;
  T* p = static_cast<T*>(a.out.p) + seq * a.out.token + head * a.out.head + d;
  struct alignas(4 * sizeof(T)) Four { T v[4]; };
  *reinterpret_cast<Four*>(p) = Four{{(T)v.x, (T)v.y, (T)v.z, (T)v.w}};
}

// {tokens, first seen token, where tiles begin, units} of a sequence of length `given`
__device__ __forceinline__ int4 span_of(const Params& p, int given) {
  const PagedAttentionArgs& a = p.a;
  const int len = min(max(given, 0), a.max_pages * a.page_size);
  const int start = a.window > 0 && a.window < len ? len - (int)a.window : 0;
  const int origin = start & ~7;  // groups of eight tokens share a page
  return make_int4(len, start, origin, (len - origin + kUnitTokens - 1) / kUnitTokens);
}

__device__ __forceinline__ int4 seq_span(const Params& p, int seq) { return span_of(p, p.a.seq_lens[seq]); }

// a sequence's length on the axis of work
__device__ __forceinline__ int64_t cost(const Params& p, int seq) {
  const int units = seq_span(p, seq).w;
  return units > 0 ? (int64_t)(units + kItemCost) * p.items : 0;
}

#if defined(__HIP_DEVICE_COMPILE__)

// a value that all lanes hold, known as such to the compiler (it came through LDS or a vector load)
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = uniform((int)(uint32_t)v), hi = uniform((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// eight matrix operands of a lane: E4M3 bytes as bf16 or fp16 (exact in both)
template <int DT>
__device__ __forceinline__ auto k_operand(uint32_t lo, uint32_t hi) {
  if constexpr (DT == 2) {
    half8_t r;
    const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
    r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
    return r;
  } else {
    bf16x8_t r;
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
    r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
    return r;
  }
}

__device__ __forceinline__ float4_t mfma(bf16x8_t a, bf16x8_t b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float4_t mfma(half8_t a, half8_t b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// a lane's query elements, the K operand's partners: one part in the 16-bit
// types; a float32 query is the exact sum of three bf16 parts, its upper, middle and
// lower eight bits (cut off, not rounded: the largest would become infinite)
template <int DT>
struct Query;
template <>
struct Query<0> {
  static constexpr int parts = 3;
  bf16x8_t v[3];
  __device__ __forceinline__ void load(const void* q, int64_t e) {
    const float* p = static_cast<const float*>(q) + e;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x = p[i];
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t top = __float_as_uint(x) & 0xFFFF0000u;
        v[k][i] = __builtin_bit_cast(__bf16, (uint16_t)(top >> 16));
        x -= __uint_as_float(top);
      }
    }
  }
};
template <>
struct Query<1> {
  static constexpr int parts = 1;
  bf16x8_t v[1];
  __device__ __forceinline__ void load(const void* q, int64_t e) {
    v[0] = *reinterpret_cast<const bf16x8_t*>(static_cast<const __bf16*>(q) + e);
  }
};
template <>
struct Query<2> {
  static constexpr int parts = 1;
  half8_t v[1];
  __device__ __forceinline__ void load(const void* q, int64_t e) {
    v[0] = *reinterpret_cast<const half8_t*>(static_cast<const _Float16*>(q) + e);
  }
};

template <int D>
struct Rows {  // a wave's tile of K and V as loaded
  static constexpr int kLines = D / 128, kRest = D % 128 / 64;  // of a row: whole lines, and whether half a one remains
  u32x4_t k[4][kLines > 0 ? kLines : 1], k_rest[2];
  uint32_t v[8][D / 64];
};

// Where a tile's four groups of eight tokens lie, the same for all lanes.
struct Place {
  int entry[4];  // of the table
  int off[4];    // tokens into the page
};

// at: byte offsets of the four groups in the cache, of this head
template <int D>
__device__ __forceinline__ void load_k(Rows<D>& r, const uint8_t* cache, const int64_t (&at)[4], int col, int grp) {
  const uint32_t line = ((col >> 1 & 1) * 4 + (col >> 2)) * D + (col & 1) * 64 + grp * 16;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int s = 0; s < Rows<D>::kLines; ++s)
      r.k[j][s] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(cache + at[j] + (line + s * 128)));
  if constexpr (Rows<D>::kRest) {
    const uint32_t rest = ((col & 1) * 4 + (col >> 2)) * D + (D - 64) + grp * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t second = at[2 * j + 1] - at[2 * j];  // rows 8 to 15 of the product lie in the next group
      r.k_rest[j] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_t*>(cache + at[2 * j] + (col & 2 ? second : 0) + rest));
    }
  }
}

template <int D>
__device__ __forceinline__ void load_v(Rows<D>& r, const uint8_t* cache, const int64_t (&at)[4], int col, int grp) {
  constexpr int W = D / 64;
  const uint32_t row = grp * D + col * (D / 16);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(cache + at[j >> 1] + (row + (j & 1) * 4 * D));
    if constexpr (W == 1) {
      r.v[j][0] = __builtin_nontemporal_load(src);
    } else if constexpr (W == 2) {
      const u32x2_t x = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(src));
      r.v[j][0] = x[0]; r.v[j][1] = x[1];
    } else if constexpr (W == 3) {
      r.v[j][0] = __builtin_nontemporal_load(src);
      r.v[j][1] = __builtin_nontemporal_load(src + 1);
      r.v[j][2] = __builtin_nontemporal_load(src + 2);
    } else {
      const u32x4_t x = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(src));
      r.v[j][0] = x[0]; r.v[j][1] = x[1]; r.v[j][2] = x[2]; r.v[j][3] = x[3];
    }
  }
}

#endif

// Workgroups that a CU holds (waves per SIMD), by what the registers and the LDS hold.
template <int DT, int D, int NQ>
constexpr int workers_per_cu() {
  if (NQ == 2) return D == 64 ? 3 : D == 128 ? 2 : 1;
  if (DT == 0) return D == 64 ? 3 : D == 128 ? 2 : 1;
  return D == 64 ? 4 : 2;
}

// Waves of a workgroup that has a CU to itself: four to each SIMD, or what its registers hold.
template <int DT, int D, int NQ>
constexpr int wide_waves() {
  const int held = workers_per_cu<DT, D, NQ>();
  return held >= 4 ? 16 : held >= 2 ? 8 : 4;
}

// NQ: 16-column tiles of queries (an item has at most 16 NQ query heads).  Workgroups of more than four waves are for
// items that are not split.
template <int DT, int D, int NQ, int kWaves>
__global__ __launch_bounds__(64 * kWaves, (kWaves == 4 ? workers_per_cu<DT, D, NQ>() : kWaves / 4)) void
paged_attention_kernel(Params p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kThreads = 64 * kWaves;
  const bool no_split = kWaves > 4 || p.whole;
  constexpr int KS = D / 64, ND = D / 16, VB = D / 16, VW = D / 64;
  constexpr int PP = 2;  // fp16 parts of a probability
  const PagedAttentionArgs& a = p.a;
  __shared__ __attribute__((aligned(16))) float lds_o[kWaves][16][D + 4];
  __shared__ float lds_m[kWaves][16], lds_l[kWaves][16];
  __shared__ int64_t lds_sum[kWaves + 1];
  __shared__ int64_t lds_first[2];
  __shared__ int lds_given;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int col = lane & 15, grp = lane >> 4;
  const int worker = blockIdx.x, n = a.n_seqs;

  int seq = 0;                        // where this worker's run begins:
  int64_t inside = 0, u = 0, u_end = 1;  // how far into the sequence, and where on the axis of work it begins and ends
  int64_t units = 1, workers = 1;
  int given = 0;  // the length of the run's first sequence
  int4 split = make_int4(-1, 0, 0, 0);

  // no token seen: zeros for the query heads h0 .. h1 - 1 of a sequence, by `count` threads of which this is the i-th
  auto clear = [&](int s, int h0, int h1, int i, int count) {
    for (int j = i; j < (h1 - h0) * (D / 4); j += count) {
      const int h = j / (D / 4);
      store4<DT>(a, s, h0 + h, (j - h * (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    if (a.lse)
      for (int h = h0 + i; h < h1; h += count) a.lse[(int64_t)s * a.q_heads + h] = -INFINITY;
  };
  // the same for all empty sequences: the grid's waves look for them, 64 at a time
  auto clear_empty = [&] {
    const int64_t waves = (int64_t)gridDim.x * kWaves;
    for (int64_t base = worker * kWaves + wave; base < n; base += 64 * waves) {
      const int64_t s = base + lane * waves;
      uint64_t empty = __ballot(s < n && seq_span(p, (int)min(s, (int64_t)n - 1)).w == 0);
      for (; empty; empty &= empty - 1) {
        const int e = (int)(base + __builtin_ctzll(empty) * waves);
        clear(e, 0, a.q_heads, lane, 64);
        if (p.by_item)
          for (int i = lane; i < p.items; i += 64) p.ws.split[e * p.items + i] = make_int4(-1, 0, 0, 0);
      }
    }
  };

  if (no_split) {  // one item
    seq = worker / p.items;
    inside = worker - seq * p.items;
    given = uniform(a.seq_lens[seq]);
    if (span_of(p, given).w == 0) {
      const int head = (int)inside / p.parts, first = head * p.group + ((int)inside - head * p.parts) * p.rows;
      clear(seq, first, min(first + p.rows, (head + 1) * p.group), tid, kThreads);
      return;
    }
  } else {
    // A prefix sum over the sequences' lengths on the axis, each thread summing a few neighbours.
    const int per = (n + kThreads - 1) / kThreads;
    int64_t mine = 0;
#pragma unroll 4
    for (int i = 0; i < per; ++i) {
      const int s = tid * per + i;
      mine += s < n ? cost(p, min(s, n - 1)) : 0;
    }
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up(upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 63) lds_sum[wave] = upto;
    __syncthreads();
    units = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) upto += units;
      units += lds_sum[w];
    }
    units = uniform(units);
    workers = min((int64_t)gridDim.x, units);
    if (worker >= workers) {
      if (!p.by_item && tid == 0) p.ws.split[worker] = split;
      clear_empty();
      return;
    }
    u = worker * units / workers;
    u_end = (worker + 1) * units / workers;
    if (mine > 0 && upto - mine <= u && u < upto) {
      int64_t at = upto - mine;
      int s = tid * per;
      for (int64_t c; at + (c = cost(p, s)) <= u; at += c) ++s;
      lds_first[0] = s;
      lds_first[1] = u - at;
      lds_given = a.seq_lens[s];
    }
    __syncthreads();
    seq = uniform((int)lds_first[0]);
    inside = uniform(lds_first[1]);
    given = uniform(lds_given);
  }

  bool first = true;
  while (u < u_end && seq < n) {
    const int4 span = span_of(p, first ? given : a.seq_lens[seq]);
    first = false;
    const int len = uniform(span.x), start = uniform(span.y), origin = uniform(span.z), per_item = uniform(span.w);
    if (per_item == 0) {  // the next one with units, of which there are some ahead
      uint64_t some = 0;
      for (++seq; seq < n; seq += 64) {
        some = __ballot(seq + lane < n && seq_span(p, min(seq + lane, n - 1)).w > 0);
        if (some) break;
      }
      seq += some ? __builtin_ctzll(some) : 0;
      continue;
    }
    // the run's part in this item
    const int length = no_split ? 1 : per_item + kItemCost;
    const int item = (int)((uint32_t)inside / (uint32_t)length), from = (int)inside - item * length;
    const int take = (int)min((int64_t)(length - from), u_end - u);
    const int unit0 = max(from - kItemCost, 0), unit1 = no_split ? per_item : from + take - kItemCost;
    const int64_t begin = u - from;
    u += take;
    inside += take;
    const int in = seq;
    if (inside == (int64_t)length * p.items) {
      inside = 0;
      ++seq;
    }
    if (unit1 <= unit0) continue;
    const int head = item / p.parts, q0 = (item - head * p.parts) * p.rows;
    const int rows = min(p.rows, p.group - q0);

    // scalar loads: nothing in this kernel writes to the table
    typedef const __attribute__((address_space(4))) int32_t* ConstInts;
    const ConstInts table = (ConstInts)(a.block_table + in * a.ld_table);
    auto find = [&](int tile) {
      Place w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t token = origin + tile * kTile + 8 * j, column = p.by_page.div(token);
        w.off[j] = token - column * a.page_size;
        // past the last token a tile may reach past the table's last column
        w.entry[j] = table[min(column, (uint32_t)a.max_pages - 1)];
      }
      return w;
    };
    auto place = [&](const Place& w, int64_t (&at)[4]) {  // and whether all its pages are the cache's
      bool good = true;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool ok = (uint32_t)w.entry[j] < (uint32_t)a.num_pages;
        good = good && ok;
        at[j] = (ok ? w.entry[j] : 0) * p.page_bytes + ((int64_t)head * a.page_size + w.off[j]) * D;
      }
      return good;
    };
    const int tiles = (len - origin + kTile - 1) / kTile;
    const int tile_end = min(unit1 * kUnitTiles, tiles);
    int tile = unit0 * kUnitTiles + wave;
    Place now = find(tile), next = find(tile + kWaves);

    Query<DT> q[NQ][2 * KS];
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      const int64_t e = in * a.q.token + (int64_t)(head * p.group + q0 + min(t * 16 + col, rows - 1)) * a.q.head;
#pragma unroll
      for (int s = 0; s < 2 * KS; ++s) q[t][s].load(a.q.p, e + (s >> 1) * 64 + grp * 16 + (s & 1) * 8);
    }
    float m[NQ], l[NQ];
    float4_t o[NQ][ND];
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      m[t] = kNoMax;
      l[t] = 0.f;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[t][i] = float4_t{0.f, 0.f, 0.f, 0.f};
    }

    if (tile < tile_end) {
      // the next tile's rows are under way before the present ones' results are used
      Rows<D> r;
      int64_t at[4];
      bool good = place(now, at);
      load_k(r, a.k_cache, at, col, grp);
      load_v(r, a.v_cache, at, col, grp);
      const double c64 = (double)a.softmax_scale * 1.44269504088896340736 / (double)*a.k_scale;
      // never 0, so that they leave the -infinity of tokens that are not seen (for which c_lo is not negative either)
      float c_hi = fmaxf((float)c64, 0x1p-149f), c_lo = 0.0f;
      if constexpr (DT == 0) {
        if ((double)c_hi > c64) c_hi = fmaxf(__uint_as_float(__float_as_uint(c_hi) - 1), 0x1p-149f);
        c_lo = fmaxf((float)(c64 - (double)c_hi), 0x1p-149f);
      }
      while (true) {
        const bool more = tile + kWaves < tile_end;

        float s[NQ][8];  // of this lane's eight tokens
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float4_t lo[NQ] = {}, hi[NQ] = {};
#pragma unroll
          for (int i = 0; i < 2 * Rows<D>::kLines; ++i) {
            const auto k = k_operand<DT>(r.k[j][i >> 1][2 * (i & 1)], r.k[j][i >> 1][2 * (i & 1) + 1]);
            const int piece = 4 * (i >> 1) + (i & 1);  // of the row's 16-byte pieces: this lane's in its half of the line
#pragma unroll
            for (int t = 0; t < NQ; ++t)
#pragma unroll
              for (int part = Query<DT>::parts - 1; part >= 0; --part) {
                lo[t] = mfma(k, q[t][piece].v[part], lo[t]);
                hi[t] = mfma(k, q[t][piece + 2].v[part], hi[t]);
              }
          }
#pragma unroll
          for (int t = 0; t < NQ; ++t) {
            s[t][2 * j] = lo[t][0] + hi[t][1];
            s[t][2 * j + 1] = lo[t][2] + hi[t][3];
          }
        }
        if constexpr (Rows<D>::kRest) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float4_t sum[NQ] = {};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const auto k = k_operand<DT>(r.k_rest[j][2 * i], r.k_rest[j][2 * i + 1]);
#pragma unroll
              for (int t = 0; t < NQ; ++t)
#pragma unroll
                for (int part = Query<DT>::parts - 1; part >= 0; --part)
                  sum[t] = mfma(k, q[t][2 * KS - 2 + i].v[part], sum[t]);
            }
#pragma unroll
            for (int t = 0; t < NQ; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[t][4 * j + i] += sum[t][i];
          }
        }
        const bool good_now = good;
        if (more) {
          good = place(next, at);
          load_k(r, a.k_cache, at, col, grp);
        }

        const bool whole = origin + tile * kTile >= start && origin + (tile + 1) * kTile <= len;
        uint32_t seen = 0xFF;  // of this lane's tokens
        if (!whole || !good_now) {
          const int token = origin + tile * kTile + grp;  // the first of this lane's eight
          seen = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if ((uint32_t)now.entry[j >> 1] < (uint32_t)a.num_pages && token + 4 * j >= start && token + 4 * j < len)
              seen |= 1u << j;
#pragma unroll
          for (int t = 0; t < NQ; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (!(seen >> j & 1)) s[t][j] = -INFINITY;
          // rows behind the last token hold anything, NaN among it
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int w = 0; w < VW; ++w) r.v[j][w] = seen >> j & 1 ? r.v[j][w] : 0u;
        }

        half8_t pr[NQ][PP];
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          float top = s[t][0];
#pragma unroll
          for (int j = 1; j < 8; ++j) top = fmaxf(top, s[t][j]);
          top *= c_hi;
          if (__any(top - m[t] > kShift + kSlack)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float whole_top = ceilf(top);
            float to = whole_top - kShift;
            if (whole_top - to > kShift) to = whole_top;  // past 2^26 steps are wider than that
            to = fmaxf(m[t], to);
            const float f = __builtin_amdgcn_exp2f(m[t] - to);
            m[t] = to;
            l[t] *= f;
#pragma unroll
            for (int i = 0; i < ND; ++i) o[t][i] *= f;
          }
          float y[8];
          if (__any(fabsf(m[t]) >= kFar && m[t] != kNoMax)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = s[t][j] * c_hi - m[t];
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              y[j] = fmaf(s[t][j], c_hi, -m[t]);
              if constexpr (DT == 0) y[j] = fmaf(s[t][j], c_lo, y[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float e = __builtin_amdgcn_exp2f(y[j]);
            l[t] += e;
            pr[t][0][j] = (_Float16)e;
            pr[t][1][j] = (_Float16)(e - (float)pr[t][0][j]);
          }
        }

#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[8], even[4], odd[4];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              x[j] = __builtin_bit_cast(uint32_t, h ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.v[j][w], 1.0f, true)
                                                    : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.v[j][w], 1.0f, false));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              even[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x05040100u);
              odd[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x07060302u);
            }
            const half8_t ve = __builtin_bit_cast(half8_t, u32x4_t{even[0], even[1], even[2], even[3]});
            const half8_t vo = __builtin_bit_cast(half8_t, u32x4_t{odd[0], odd[1], odd[2], odd[3]});
#pragma unroll
            for (int t = 0; t < NQ; ++t)
#pragma unroll
              for (int part = PP - 1; part >= 0; --part) {
                o[t][4 * w + 2 * h] = mfma(ve, pr[t][part], o[t][4 * w + 2 * h]);
                o[t][4 * w + 2 * h + 1] = mfma(vo, pr[t][part], o[t][4 * w + 2 * h + 1]);
              }
          }
        if (!more) break;
        load_v(r, a.v_cache, at, col, grp);
        tile += kWaves;
        now = next;
        next = find(tile + kWaves);
      }
    }

    // The waves' results into one, 16 query heads at a time.
    const float inv_vs = 1.0f / *a.v_scale;
    const bool ends = unit0 == 0 && unit1 == per_item;  // the whole item
    const int slot = 2 * worker + (unit0 == 0 ? 1 : 0);
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      if (t * 16 >= rows) break;
      float sum = l[t];
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      __syncthreads();  // the last results have been read
      if (grp == 0) {
        lds_m[wave][col] = m[t];
        lds_l[wave][col] = sum;
      }
      __syncthreads();
      float top = lds_m[0][col];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, lds_m[w][col]);
      const float f = __builtin_amdgcn_exp2f(m[t] - top);
      if (t * 16 + col < rows) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int i = 0; i < VB; i += 4)
            *reinterpret_cast<float4_t*>(&lds_o[wave][col][(4 * grp + r) * VB + i]) =
                float4_t{o[t][i][r], o[t][i + 1][r], o[t][i + 2][r], o[t][i + 3][r]} * f;
      }
      __syncthreads();
      const int here = min(16, rows - t * 16);
      for (int i = tid; i < here * (D / 4); i += kThreads) {
        const int row_ = i / (D / 4), d = (i - row_ * (D / 4)) * 4;
        float high = lds_m[0][row_], total = 0.f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) high = fmaxf(high, lds_m[w][row_]);
        float4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          total += lds_l[w][row_] * __builtin_amdgcn_exp2f(lds_m[w][row_] - high);
          v += *reinterpret_cast<const float4_t*>(&lds_o[w][row_][d]);
        }
        const int in_item = t * 16 + row_;
        if (ends) {
          const int h = head * p.group + q0 + in_item;
          const float by = total > 0.f ? inv_vs / total : 0.f;
          store4<DT>(a, in, h, d, make_float4(v[0] * by, v[1] * by, v[2] * by, v[3] * by));
          if (a.lse && d == 0)
            a.lse[(int64_t)in * a.q_heads + h] = total > 0.f ? (high + log2f(total)) * kLn2 : -INFINITY;
        } else {
          const int64_t at = (int64_t)slot * p.rows + in_item;
          *reinterpret_cast<float4_t*>(p.ws.o + at * D + d) = v;
          if (d == 0) p.ws.ml[at] = make_float2(high, total);
        }
      }
    }
    if (unit0 == 0 && !no_split) {
      // the item's last unit is that of the first worker whose run ends behind it
      if (!ends) split = make_int4(in, item, worker, (int)(((begin + length) * workers + units - 1) / units) - 1);
      if (p.by_item && tid == 0) p.ws.split[in * p.items + item] = split;
    }
  }
  if (no_split) return;
  if (!p.by_item && tid == 0) p.ws.split[worker] = split;
  clear_empty();
#endif
}

// Joins the partial results of a shared item: its first worker's second one and
// the first ones of the workers up to its last.  blockIdx.x is the entry of
// `split`, blockIdx.y a query head of the item and a slice of its outputs:
// `lanes` lanes, four outputs each.
constexpr int kJoinThreads = 256, kJoinWaves = kJoinThreads / 64;

template <int DT, int D>
__global__ __launch_bounds__(kJoinThreads) void paged_attention_join(Params p, int lanes) {
  const PagedAttentionArgs& a = p.a;
  extern __shared__ float weights[];  // [workers]
  __shared__ float4 lds_o[kJoinThreads];
  __shared__ float lds_r[2][kJoinWaves];
  const int4 split = p.ws.split[blockIdx.x];
  if (split.x < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slices = D / 4 / lanes, row = blockIdx.y / slices, slice = blockIdx.y - row * slices;
  const int seq = split.x, head = split.y / p.parts, q0 = (split.y - head * p.parts) * p.rows, worker = split.z;
  if (q0 + row >= p.group) return;
  const int count = split.w - worker + 1;
  auto at = [&](int i) { return (int64_t)(i == 0 ? 2 * worker + 1 : 2 * (worker + i)) * p.rows + row; };

  constexpr int kDeep = 16;  // loads of a lane in flight
  const int sets = kJoinThreads / lanes;  // partial results that are read side by side
  const int set = tid / lanes, in_set = tid - set * lanes, d = (slice * lanes + in_set) * 4;
  float4 x[kDeep];
  auto fetch = [&](int i) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (i + u * sets < count) x[u] = *reinterpret_cast<const float4*>(p.ws.o + at(i + u * sets) * D + d);
  };
  if (set < sets) fetch(set);  // needs no weights yet

  float top = kNoMax;
  for (int i = tid; i < count; i += kJoinThreads) top = fmaxf(top, p.ws.ml[at(i)].x);
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
  if (lane == 0) lds_r[0][wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) top = fmaxf(top, lds_r[0][w]);
  float total = 0.f;
  for (int i = tid; i < count; i += kJoinThreads) {
    const float2 ml = p.ws.ml[at(i)];
    const float f = exp2f(ml.x - top);
    weights[i] = f;
    total += ml.y * f;
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) total += __shfl_xor(total, s);
  if (lane == 0) lds_r[1][wave] = total;
  __syncthreads();
  total = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) total += lds_r[1][w];

  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (set < sets) {
    for (int i = set; i < count; i += sets * kDeep) {
      if (i != set) fetch(i);
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        if (i + u * sets >= count) break;
        const float f = weights[i + u * sets];
        v.x += x[u].x * f; v.y += x[u].y * f; v.z += x[u].z * f; v.w += x[u].w * f;
      }
    }
  }
  lds_o[tid] = v;
  __syncthreads();
  if (set == 0) {
    for (int s = 1; s < min(sets, count); ++s) {
      const float4 y = lds_o[s * lanes + tid];
      v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
    }
    const float by = total > 0.f ? 1.0f / *a.v_scale / total : 0.f;
    const int h = head * p.group + q0 + row;
    store4<DT>(a, seq, h, d, make_float4(v.x * by, v.y * by, v.z * by, v.w * by));
    if (a.lse && slice == 0 && tid == 0)
      a.lse[(int64_t)seq * a.q_heads + h] = total > 0.f ? (top + log2f(total)) * kLn2 : -INFINITY;
  }
}

template <int DT, int D, int NQ>
hipError_t launch(Params p, hipStream_t stream) {
  const PagedAttentionArgs& a = p.a;
  int64_t tokens = (int64_t)a.max_pages * a.page_size;  // of the longest item
  if (a.window > 0 && a.window < tokens) tokens = std::min(tokens, a.window + kUnitTokens);
  const int64_t units = (tokens + kUnitTokens - 1) / kUnitTokens, items = (int64_t)a.n_seqs * p.items;
  const int64_t cus = std::min(device_cu_count(), kMaxCus), resident = cus * workers_per_cu<DT, D, NQ>();
  // Unsplit, a call lasts as long as its longest item; split, as all tokens take on the resident workers, and some 8 us
  // more, for the scan of the lengths, the partial results and the second kernel.  With a CU to itself an item has more
  // waves, and takes 4 us and 0.7 for a unit of heads of 128 (0.5 with 64, 1.5 with 256).  Unsplit against split, in us:
  //   one to a CU, heads of 128:
  //     units of an item         3            9           12           17           15           19           32
  //     items                   16           32           64           64          128          128          256
  //                         6.2 / 10.3  10.5 / 11.2  13.4 / 14.5  16.2 / 15.0  15.9 / 17.8  19.0 / 18.1  32.8 / 34.9
  //   (heads of 64, 32 items of 6 and 16 units: 7.8 / 10.0 and 12.8 / 11.0; of 256, 64 of 6 and 128 of 13: 13.8 / 14.7
  //   and 23.3 / 21.5), and the same items in workgroups of four waves: 32 of 9 units 14.9, 64 of 5 units 9.8 for 7.7
  //   more than that, or too many registers for it:
  //     items, of what the CUs hold  512 of 512   1600 of 512   128 of 512   512 of 1024  512 of 512
  //     units                             9            17            9            17           63
  //                                  19.1 / 26.2  83.1 / 87.4  15.3 / 14.7  23.4 / 22.9  113 / 105
  constexpr int kWide = wide_waves<DT, D, NQ>();
  const bool wide = kWide > 4 && items <= cus;
  p.whole = items <= kMostWorkgroups && (wide ? units * std::max(D, 104) * cus <= 128 * (9 * cus + 23 * items)
                                              : units <= 6 || (units <= 20 && units * resident <= 20 * items));
  const int workers = (int)(p.whole ? items : std::min<int64_t>(resident, items * (units + kItemCost)));
  p.by_item = !p.whole && items <= workers;
  if (wide && p.whole)
    paged_attention_kernel<DT, D, NQ, kWide><<<workers, 64 * kWide, 0, stream>>>(p);
  else
    paged_attention_kernel<DT, D, NQ, 4><<<workers, 256, 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.whole) return e;
  // Few items are shared by many workers each: then slices of 64 outputs, to have more readers.
  const int entries = p.by_item ? (int)items : workers, slices = entries * p.rows <= 64 ? D / 64 : 1;
  paged_attention_join<DT, D><<<dim3(entries, p.rows * slices), kJoinThreads, workers * sizeof(float), stream>>>(
      p, D / 4 / slices);
  return hipGetLastError();
}

template <int DT, int D>
hipError_t launch_rows(const Params& p, hipStream_t stream) {
  if constexpr (DT != 0 && D <= 192) {
    if (p.rows > 16) return launch<DT, D, 2>(p, stream);
  }
  return launch<DT, D, 1>(p, stream);
}

template <int DT>
hipError_t launch_dim(const Params& p, hipStream_t stream) {
  switch (p.a.head_dim) {
    case 64: return launch_rows<DT, 64>(p, stream);
    case 128: return launch_rows<DT, 128>(p, stream);
    case 192: return launch_rows<DT, 192>(p, stream);
    default: return launch_rows<DT, 256>(p, stream);
  }
}

}  // namespace

hipError_t launch_paged_attention(const PagedAttentionArgs& a, hipStream_t stream) {
  Params p;
  p.a = a;
  p.by_page = FastDiv((uint32_t)a.page_size);
  p.group = a.q_heads / a.kv_heads;
  p.rows = attention_rows_of_item(p.group, a.dtype == 0, a.head_dim);
  p.parts = (p.group + p.rows - 1) / p.rows;
  p.items = a.kv_heads * p.parts;
  p.page_bytes = (int64_t)a.kv_heads * a.page_size * a.head_dim;
  char* w = static_cast<char*>(a.workspace);
  p.ws.o = reinterpret_cast<float*>(w);  // 16-byte aligned pieces first
  w += (int64_t)kMostWorkers * 2 * p.rows * 4 * a.head_dim;
  p.ws.split = reinterpret_cast<int4*>(w);
  w += kMostWorkers * 16;
  p.ws.ml = reinterpret_cast<float2*>(w);
  switch (a.dtype) {
    case 0: return launch_dim<0>(p, stream);
    case 1: return launch_dim<1>(p, stream);
    default: return launch_dim<2>(p, stream);
  }
}

}  // namespace nvfp4
