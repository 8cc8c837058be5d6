// The gated delta rule over ragged prompts (nvfp4_gated_delta_chunked).
//
//   S <- e^g S;  S <- S + k~ (beta (v - S^T k~))^T;  out = scale S^T q~
//
// In chunks of C = 64 tokens, with G_i the sum of g over the chunk's first i tokens, what
// the tokens write, V'_i = beta_i (v_i - S_i^T k~_i), solves a unit lower triangular
// system, and everything else is products:
//
//   A_ij = beta_i e^(G_i - G_j) k~_i . k~_j  (j < i),  T = (1 + A)^-1
//   X    = beta (V - e^G K~ S),  V' = T X
//   out  = scale (e^G Q~ S + P V'),  P_ij = e^(G_i - G_j) q~_i . k~_j  (j <= i)
//   S   <- e^(G_C) S + (e^(G_C - G) K~)^T V'
//
// Three kernels.  The first normalises keys and queries and leaves their products, which a
// key head's value heads share.  The second has a wave for each chunk and value head, all
// independent, and leaves T, P and the gates in the workspace.  The third, the chain, walks
// the chunks of a sequence with 16 columns of the state in a wave's registers: columns never
// meet, and the matrix unit's results lie as its next operands want them, so S, X and V' pass
// through neither LDS nor other lanes.  Where columns are too few to fill the card, sequences
// are taken in parts at once, as a part does one linear map to the state it is given.
//
// In us (bf16 and fp16, heads of 128; keys, solve, chain; the whole call as a graph):
//   8192 tokens of 48 heads     21, 39, ends 154 + join 20 + parts 141; 336
//   12 prompts, 26518 tokens    57, 128, 463; 616
//   16411 tokens of 6 heads     9, 16, ends 51 + join 44 + parts 48; 158
// The solve's stores bound it (25 KB a chunk and head: 4 TB/s).  The chain's chunk takes a
// wave some 2100 cycles of the matrix unit; with 8 waves LDS (6300) and issue (5800) bound it,
// 10400 cycles a chunk, with one wave a SIMD what a product waits for the one before, 6000.
//
// Precision.  Operands are fp16 parts, sums fp32.  A row of keys or queries is scaled by a
// power of two to a length in [16, 32): 16-bit inputs fit one part but for 2^-29 of that
// length (half of fp16's last step, 2^-25, of 2^4); float32 takes two.  |T| and |P| are at
// most 1 and scaled by 2^14; a column of S, and with it X and V', is scaled by a power of two
// that follows it and the values, so that their largest M is from 2^5 to 2^9: each is cut into
// two parts, off by 2^-22 of the element or 2^-25, which is 2^-30 of M, and 2^-29 where V'
// has been taken by a key's norm.  Of products of two cut operands the low parts' is dropped
// (2^-22 again).  Against 64 bits, relative lengths, beside products in fp32: outputs 0.95 to
// 1.11 times as far off (float32, 2.1e-7 to 3.4e-7); states of 16-bit inputs 0.94 to 1.13
// times, of float32 inputs 1.1 to 2.1 times (2.3e-7 and 1.1e-7 under strong decay).
#include <algorithm>

#include "gdn_device.h"

namespace nvfp4 {
namespace {

constexpr int kC = kDeltaChunk;
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kBlock = 1024;  // an operand of 16 x 32 fp16 elements: 16 bytes a lane
constexpr int kTies = 6;      // blocks of 16 x 32 that meet the lower triangle of 64 x 64
constexpr int kPAt = kTies * 2 * kBlock, kGatesAt = 2 * kPAt;
constexpr float kUp = 16384.0f, kDown = 1.0f / 16384.0f;  // 2^14
constexpr int kLength = 4;                                // rows of keys and queries have lengths from 2^4 to 2^5
constexpr float kLong = 1 << kLength;

// per token of a chunk, after T and P
enum { kBeta, kGainK, kUntil, kGainQ, kDecay, kGates };
static_assert(kGatesAt + kGates * kC * 4 <= kDeltaTieBytes, "the workspace's entry holds it");

constexpr int tie(int mt, int s) { return mt < 2 ? mt : 2 * mt - 2 + s; }  // of rows 16 mt.., columns 32 s..

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float4_t mfma(half8_t a, half8_t b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// eight floats as fp16 parts, the second what the first leaves
struct Parts {
  half8_t hi, lo;
};
__device__ __forceinline__ half8_t halves(const float (&x)[8]) {
  half8_t y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const half2_t p = __builtin_convertvector(float2_t{x[2 * i], x[2 * i + 1]}, half2_t);
    y[2 * i] = p[0];
    y[2 * i + 1] = p[1];
  }
  return y;
}
__device__ __forceinline__ Parts cut(const float (&x)[8]) {
  Parts p;
  p.hi = halves(x);
  // x - hi as one multiply-add that takes the half as it lies (v_fma_mix_f32), which the compiler makes of a factor that
  // it does not know
  float less;
  asm("s_mov_b32 %0, -1.0" : "=s"(less));
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = __builtin_fmaf((float)p.hi[i], less, x[i]);
  p.lo = halves(rest);
  return p;
}
__device__ __forceinline__ Parts cut(float4_t a, float4_t b) {
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return cut(x);
}

// ---------------------------------------------------------------- a chunk's ties

// A block of 16 x 16 floats in LDS: where four of a row lie.  Lanes that take one column of rows 4 g + r, or four elements of
// every row, meet distinct banks; 16 floats between blocks part those that the diagonals' lanes read together (against rows
// 20 floats apart, with which two workgroups fit a CU and not three: 8192 tokens of 48 heads 42.0 -> 37.4 us, 12 ragged
// prompts 147 -> 134).
constexpr int kSquare = 16 * 16 + 16;
__device__ __forceinline__ int cell(int row, int quad) { return ((row & 3) * 4 + (row >> 2)) * 16 + 4 * (quad ^ (row & 3)); }
constexpr int square(int j, int i) { return i * (i + 1) / 2 + j; }  // of block column j, block row i

struct SolveLds {
  float a[10 * kSquare];  // A^T by blocks: row j, column i; then the inverse's
  double log_decay[kC];
  float beta[kC];
};

// Rows of q or k as operands: lane (g, m) holds elements 32 s + 8 g.. of row m, a power of two times the input; what that
// times `norm` is, has length 1.
template <int DT, int DK>
struct Row {
  static constexpr int kSteps = DK / 32, kParts = DT == 0 ? 2 : 1;
  half8_t part[kParts][kSteps];
  float norm;
  __device__ __forceinline__ void load(const HeadsIn& x, int64_t token, int head, int g, bool there, float eps) {
    Elements<DT, 8> e[kSteps];
    const int64_t at = token * x.token + head * x.head + 8 * g;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      e[s].load(x.p, at + 32 * s);
      if (!there) e[s].zero();
    }
    float top = 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(e[s].get(i)));
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    int up = -__builtin_amdgcn_frexp_expf(top);  // the largest into [1/2, 1), so that squares neither overflow nor vanish
    float squares = 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __builtin_amdgcn_ldexpf(e[s].get(i), up);
        squares = __builtin_fmaf(y, y, squares);
      }
    squares += __shfl_xor(squares, 16);
    squares += __shfl_xor(squares, 32);
    const int more_up = kLength + 1 - ((__builtin_amdgcn_frexp_expf(squares) + 1) >> 1);
    up += more_up;
    squares = __builtin_amdgcn_ldexpf(squares, 2 * more_up);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_ldexpf(e[s].get(i), up);
      if constexpr (kParts == 2) {
        const Parts p = cut(y);
        part[0][s] = p.hi;
        part[1][s] = p.lo;
      } else {
        part[0][s] = halves(y);
      }
    }
    norm = norm_of(squares, up, eps);
  }
  __device__ __forceinline__ void store(uint8_t* image, int mt, int lane) const {
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        *reinterpret_cast<half8_t*>(image + ((p * 4 + mt) * kSteps + s) * kBlock + lane * 16) = part[p][s];
  }
  __device__ __forceinline__ void read(const uint8_t* image, int mt, int lane) {
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        part[p][s] = *reinterpret_cast<const half8_t*>(image + ((p * 4 + mt) * kSteps + s) * kBlock + lane * 16);
  }
};

// rows of a times rows of b: lane (g, n) has rows 4 g.. of a against row n of b
template <int DT, int DK>
__device__ __forceinline__ float4_t dots(const Row<DT, DK>& a, const Row<DT, DK>& b) {
  float4_t c = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
    c = mfma(a.part[0][s], b.part[0][s], c);
    if constexpr (DT == 0) {
      c = mfma(a.part[0][s], b.part[1][s], c);
      c = mfma(a.part[1][s], b.part[0][s], c);
    }
  }
  return c;
}

// the chunk of place c: its sequence and rows; false if no sequence has it
struct Place {
  int r, slot;
  int64_t begin, end;
};
__device__ __forceinline__ bool find_place(const DeltaArgs& a, int64_t c, Place& p) {
  int low = 0, high = a.n_seqs;  // the last sequence whose first place is at most c
  while (high - low > 1) {
    const int mid = low + (high - low) / 2;
    if (start_of(a.token_starts, mid, a.tokens) / kC + mid <= c) low = mid; else high = mid;
  }
  const int64_t start = start_of(a.token_starts, low, a.tokens);
  const int64_t at = c - (start / kC + low);
  p.r = low;
  p.begin = start + at * kC;
  p.end = start_of(a.token_starts, low + 1, a.tokens);
  p.slot = a.slots[low];
  return at >= 0 && p.begin < p.end && slot_ok(p.slot, a.num_slots);
}

// c - a b, of 16 x 16 blocks in fp32: a from LDS by rows, b and c as the matrix unit leaves results.  Step r of four takes
// the products' elements 4 g + r, which are register r of b.
__device__ __forceinline__ float4_t less_product(const float* a, float4_t b, float4_t c, int g, int n) {
  const float4_t row = *reinterpret_cast<const float4_t*>(a + cell(n, g));
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(-row[r], b[r], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ void store_block(float* to, float4_t x, int g, int n) {
#pragma unroll
  for (int r = 0; r < 4; ++r) to[cell(4 * g + r, n >> 2) + (n & 3)] = x[r];
}
__device__ __forceinline__ float4_t load_block(const float* from, int g, int n) {
  float4_t x;
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = from[cell(4 * g + r, n >> 2) + (n & 3)];
  return x;
}

// rows 16 mt.. of T or P, transposed as the matrix unit leaves them (block j: columns 16 j..), into operands
__device__ __forceinline__ void store_ties(uint8_t* to, int mt, const float4_t (&block)[4], int lane) {
  const float4_t none = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s <= mt / 2; ++s) {
    const Parts p = cut(block[2 * s] * kUp, 2 * s + 1 <= mt ? block[2 * s + 1] * kUp : none);
    *reinterpret_cast<half8_t*>(to + (2 * tie(mt, s)) * kBlock + lane * 16) = p.hi;
    *reinterpret_cast<half8_t*>(to + (2 * tie(mt, s) + 1) * kBlock + lane * 16) = p.lo;
  }
}

// Sequences in the order of their lengths, the longest first, so that the last workgroups of the chain have the least to do
// (12 prompts up to 4096 tokens of 48 heads, in the order they are given: 682 us and not 608).
constexpr int kMostOrdered = 512;
__device__ __forceinline__ void find_order(const DeltaArgs& a, int32_t* order) {
  __shared__ int32_t lens[kMostOrdered];
  const int r = threadIdx.x;
  if (r < a.n_seqs) lens[r] = (int32_t)(start_of(a.token_starts, r + 1, a.tokens) - start_of(a.token_starts, r, a.tokens));
  __syncthreads();
  if (r >= a.n_seqs) return;
  const int32_t own = lens[r];
  int before = 0;
  for (int i = 0; i < a.n_seqs; ++i) before += lens[i] > own || (lens[i] == own && i < r);
  order[before] = r;
}

// An entry of a chunk and key head: operands of keys and of queries, the rows' norms, and the products k~_i . k~_j and
// q~_i . k~_j that its value heads share, by blocks j <= i as the matrix unit leaves them (lane (g, n): j = 4 g.., i = n).
template <int DT, int DK>
struct KeyEntry {
  static constexpr int64_t kBytes = delta_key_bytes(DK, DT), kImage = 2 * kC * DK * (DT == 0 ? 2 : 1), kNorms = 2 * kImage;
  static constexpr int64_t kDots = kNorms + 2 * kC * 4;
  static_assert(kDots + 20 * kBlock <= kBytes, "the workspace's entry holds it");
};

// Keys and queries of a chunk and key head: eight waves take 16 rows each, then every eighth of the products' 20 blocks.
template <int DT, int DK>
__global__ __launch_bounds__(512) void gated_delta_keys_kernel(DeltaArgs a, FastDiv by_heads, int64_t first_place, int32_t* order) {
  using E = KeyEntry<DT, DK>;
  __shared__ __attribute__((aligned(16))) uint8_t images[2 * E::kImage];
  __shared__ float norms[2 * kC];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  const uint32_t of_launch = by_heads.div(blockIdx.x);
  const int kh = (int)(blockIdx.x - of_launch * by_heads.d);
  const int64_t place = first_place + of_launch;
  if (order && place == 0 && kh == 0) find_order(a, order);
  Place at;
  if (!find_place(a, place, at)) return;
  const int rows = (int)std::min<int64_t>(kC, at.end - at.begin);
  const bool of_q = wave >= 4;
  const int mt = wave & 3, row = 16 * mt + n;
  uint8_t* entry = static_cast<uint8_t*>(a.workspace) + place * delta_chunk_bytes(a.k_heads, a.v_heads, DK, DT) + kh * E::kBytes;
  Row<DT, DK> x;
  x.load(of_q ? a.q : a.k, at.begin + std::min(row, rows - 1), kh, g, row < rows, a.eps);
  x.store(entry + (of_q ? E::kImage : 0), mt, lane);
  x.store(images + (of_q ? E::kImage : 0), mt, lane);
  if (g == 0) {
    norms[(of_q ? kC : 0) + row] = x.norm;
    reinterpret_cast<float*>(entry + E::kNorms)[(of_q ? kC : 0) + row] = x.norm;
  }
  __syncthreads();
  for (int t = wave; t < 20; t += 8) {
    const int q = t >= 10, of = t - 10 * q, bi = (of >= 1) + (of >= 3) + (of >= 6), bj = of - square(0, bi);
    Row<DT, DK> y;
    x.read(images, bj, lane);
    y.read(images + q * E::kImage, bi, lane);
    const float4_t of_rows = *reinterpret_cast<const float4_t*>(norms + 16 * bj + 4 * g);
    *reinterpret_cast<float4_t*>(entry + E::kDots + t * kBlock + lane * 16) = dots(x, y) * (of_rows * norms[q * kC + 16 * bi + n]);
  }
}

template <int DT, int DK>
__global__ __launch_bounds__(kThreads) void gated_delta_solve_kernel(DeltaArgs a, FastDiv by_group, FastDiv by_blocks,
                                                                     int64_t first_place) {
  using E = KeyEntry<DT, DK>;
  __shared__ SolveLds all[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  const uint32_t of_launch = by_blocks.div(blockIdx.x);
  const int h = (int)(blockIdx.x - of_launch * by_blocks.d) * kWaves + wave;
  const int64_t place = first_place + of_launch;
  Place at;
  if (h >= a.v_heads || !find_place(a, place, at)) return;  // whole waves: the kernel has no barrier
  const int kh = (int)by_group.div((uint32_t)h);
  const int rows = (int)std::min<int64_t>(kC, at.end - at.begin);
  SolveLds& lds = all[wave];
  uint8_t* base = static_cast<uint8_t*>(a.workspace) + place * delta_chunk_bytes(a.k_heads, a.v_heads, DK, DT);
  const uint8_t* entry = base + kh * E::kBytes;
  const float* norms = reinterpret_cast<const float*>(entry + E::kNorms);
  uint8_t* ties = base + a.k_heads * E::kBytes + (int64_t)h * kDeltaTieBytes;

  float4_t dot[20];
#pragma unroll
  for (int t = 0; t < 20; ++t) dot[t] = *reinterpret_cast<const float4_t*>(entry + E::kDots + t * kBlock + lane * 16);
  const float k_norm = norms[lane], q_norm = norms[kC + lane];

  // gates of token `lane`: the sum of log2 decays in 64 bits, since only differences count
  const int64_t token = at.begin + std::min(lane, rows - 1);
  const float decay = -expf(a.a_log[h]) * softplus(element<DT>(a.a, token * a.a_token + h) + a.dt_bias[h]);
  const float beta = lane < rows ? sigmoid<true>(element<DT>(a.b, token * a.b_token + h)) : 0.0f;
  // at 2^-256 nothing is left in fp32; less would cost the sums of later tokens their last bits.  A NaN stays one, for the
  // chunk's outputs and the state behind it to show.
  double log_decay = lane < rows ? (double)decay * 1.4426950408889634 : 0.0;
  if (log_decay < -256.0) log_decay = -256.0;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double before = __shfl_up(log_decay, d);
    if (lane >= d) log_decay += before;
  }
  const double whole = __shfl(log_decay, 63);
  lds.log_decay[lane] = log_decay;
  lds.beta[lane] = beta;
  wave_sync();

  // e^(G_i - G_j) of this lane's elements of block (j, i): column i = 16 bi + n, rows j = 16 bj + 4 g + r
  auto ratio = [&](int bj, int bi) {
    const double of_i = lds.log_decay[16 * bi + n];
    float4_t x;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float d = (float)(of_i - lds.log_decay[16 * bj + 4 * g + r]);
      x[r] = bj < bi || 4 * g + r <= n ? __builtin_amdgcn_exp2f(d) : 0.0f;
    }
    return x;
  };

  // P by rows of blocks, and A^T
#pragma unroll
  for (int bi = 0; bi < 4; ++bi) {
    const float strength = lds.beta[16 * bi + n];
    float4_t p[4];
#pragma unroll
    for (int bj = 0; bj <= bi; ++bj) {
      const float4_t e = ratio(bj, bi);
      p[bj] = e * dot[10 + square(bj, bi)];
      float4_t x = e * strength * dot[square(bj, bi)];
      if (bj == bi) {
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = 4 * g + r < n ? x[r] : 0.0f;
      }
      store_block(lds.a + square(bj, bi) * kSquare, x, g, n);
    }
    store_ties(ties + kPAt, bi, p, lane);
  }
  wave_sync();

  // T of the diagonal blocks by substitution: lane (b, c) has column c of block b, and takes column j of A once x_j is known
  {
    float* block = lds.a + square(g, g) * kSquare;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == n ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < 15; ++j) {
#pragma unroll
      for (int i4 = (j + 1) / 4; i4 < 4; ++i4) {
        const float4_t col = *reinterpret_cast<const float4_t*>(block + cell(j, i4));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * i4 + i > j) x[4 * i4 + i] = __builtin_fmaf(-col[i], x[j], x[4 * i4 + i]);
      }
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4_t*>(block + cell(n, i)) = float4_t{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    wave_sync();
  }
  // U = T^T by blocks: [U0 U01; 0 U1] has U01 = -U0 A01^T U1, first of 16 x 16, then of 32 x 32
  const float4_t none = {0, 0, 0, 0};
  auto of = [&](int j, int i) { return lds.a + square(j, i) * kSquare; };
  float4_t u[4][4];
#pragma unroll
  for (int b = 0; b < 4; ++b) u[b][b] = load_block(of(b, b), g, n);
#pragma unroll
  for (int b = 0; b < 4; b += 2) {
    const float4_t x = less_product(of(b, b + 1), u[b + 1][b + 1], none, g, n);
    u[b][b + 1] = -less_product(of(b, b), x, none, g, n);
  }
  wave_sync();
  store_block(of(0, 1), u[0][1], g, n);
  wave_sync();
#pragma unroll
  for (int i = 2; i < 4; ++i) {
    float4_t x[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      x[j] = less_product(of(j, 2), u[2][i], none, g, n);
      if (i == 3) x[j] = less_product(of(j, 3), u[3][3], x[j], g, n);
    }
    u[1][i] = -less_product(of(1, 1), x[1], none, g, n);
    u[0][i] = -less_product(of(0, 1), x[1], less_product(of(0, 0), x[0], none, g, n), g, n);
  }
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const float4_t rows_of[4] = {u[0][mt], mt >= 1 ? u[1][mt] : none, mt >= 2 ? u[2][mt] : none, mt >= 3 ? u[3][mt] : none};
    store_ties(ties, mt, rows_of, lane);
  }

  float* gates = reinterpret_cast<float*>(ties + kGatesAt);
  const float since = __builtin_amdgcn_exp2f((float)log_decay);
  gates[kBeta * kC + lane] = beta;
  gates[kGainK * kC + lane] = beta * since * k_norm * (1.0f / kLong);
  gates[kUntil * kC + lane] = __builtin_amdgcn_exp2f((float)(whole - log_decay)) * k_norm * kLong;
  gates[kGainQ * kC + lane] = since * q_norm * (kUp / kLong);
  gates[kDecay * kC + lane] = __builtin_amdgcn_exp2f((float)whole);
}

// -------------------------------------------------------------- the states' chain

// What a launch does: whole sequences; the ends of their parts (of a part's state, started from zeros but for the first
// part, and of the identity: a part takes any state S to `turn` S + `end`); or the parts themselves, from known states.
enum { kWhole, kEnds, kPart };

struct PartArgs {
  int parts;           // of a sequence, at most
  float *first, *turn;  // [sequence][v_heads][parts]: states that parts start from [head_k][head_v], what they do [head_k][head_k]
};

// the chunks of a part, equal in number but for the last part's
struct Part {
  int64_t low, high;  // of the sequence's chunks; none if not low < high
  bool last;
};
__device__ __forceinline__ int64_t chunks_of_part(int64_t chunks, int parts) {
  return std::max<int64_t>((chunks + parts - 1) / parts, kDeltaPartChunks);
}
__device__ __forceinline__ Part find_part(int64_t chunks, int parts, int part) {
  const int64_t each = chunks_of_part(chunks, parts), high = (part + 1) * each;
  return {part * each, std::min(high, chunks), high >= chunks};
}

typedef short short4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4_t lds_short4_t;

// Four rows of 16 16-bit elements that a group of 16 lanes points at, four elements a lane; lane n gets column n.
__device__ __forceinline__ short4_t read_columns(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)p);
}

// WAVES of a workgroup hold 16 columns each, LOADERS more move data for them.  A stage is keys, T, gates, values, queries, P:
// of the ends of parts, all but the last two.
template <int DT, int DK, int MODE, int WAVES, int LOADERS>
struct Chain {
  static constexpr int kParts = DT == 0 ? 2 : 1, kSteps = DK / 32, kTiles = DK / 16;
  static constexpr int kCols = 16 * WAVES;                    // of a workgroup
  static constexpr int kThreads = 64 * (WAVES + LOADERS);
  static constexpr int kKeys = kParts * 4 * kSteps * kBlock;  // bytes of K; Q follows
  static constexpr int kRow = kCols * element_size(DT);       // of V, then of the outputs
  static constexpr int kTurnAt = kKeys, kGatesIn = kTurnAt + kPAt, kValuesAt = kGatesIn + 2 * kBlock;
  static constexpr int kQueriesAt = kValuesAt + kC * kRow, kInnerAt = kQueriesAt + kKeys;
  static constexpr int kStage = MODE == kEnds ? kQueriesAt : kInnerAt + kPAt;
  static constexpr int kStages = 2 * kStage <= (160 << 10) ? 2 : 1;
  static_assert(kStages * kStage <= (160 << 10), "the stages fit LDS");
  // Where byte `x` of a row of V lies in it: rows of 128 bytes or more would meet in the same banks.
  static __device__ __forceinline__ int turned(int row, int x) { return kRow >= 128 ? x ^ (((row ^ (row >> 2)) & 3) << 5) : x; }
};

#if defined(__HIP_DEVICE_COMPILE__)
// From memory to LDS past the registers, 16 bytes a lane to byte lds + 16 lane.  M0 is set in the same block, one wait
// state before the loads read it; an instruction's offset counts on both sides.  M0 is a reserved register, which a block
// cannot name as changed: nothing else in these kernels uses it.
__device__ __forceinline__ void to_lds4(uint32_t lds, const void* base, uint32_t offset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "global_load_lds_dwordx4 %1, %2 offset:1024\n\t"
      "global_load_lds_dwordx4 %1, %2 offset:2048\n\t"
      "global_load_lds_dwordx4 %1, %2 offset:3*1024" ::"s"(lds), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void to_lds2(uint32_t lds, const void* base, uint32_t offset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "global_load_lds_dwordx4 %1, %2 offset:1024" ::"s"(lds), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void to_lds(uint32_t lds, const void* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}
#endif

// the largest of the four lanes that share a column
__device__ __forceinline__ float of_column(float x) {
  const auto rows = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(rows[0]), __uint_as_float(rows[1]));
  const auto pairs = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(pairs[0]), __uint_as_float(pairs[1]));
}

template <int DT, int DK, int MODE, int WAVES, int LOADERS>
__global__ __launch_bounds__(64 * (WAVES + LOADERS))
    __attribute__((amdgpu_waves_per_eu(WAVES + LOADERS > 4 ? 2 : 1))) void gated_delta_chain_kernel(
        DeltaArgs a, PartArgs parts, const int32_t* order, FastDiv by_seq, FastDiv by_key_heads, FastDiv by_parts, uint32_t slices,
        uint32_t first, uint32_t pairs) {
#if defined(__HIP_DEVICE_COMPILE__)
  using L = Chain<DT, DK, MODE, WAVES, LOADERS>;
  constexpr int kSize = element_size(DT);
  __shared__ __attribute__((aligned(1024))) uint8_t stage[L::kStages * L::kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;

  // Workgroups go to the XCDs in turn: those of one sequence and head (and part), which read the same ties, and where there
  // are 8 key heads (or a multiple) those of one key head lie on one XCD, 8 apart.  Parts are dealt one by one, so that few
  // heads reach every XCD (6 heads in 32 parts: 184 us, and 200 with a head on one XCD).
  const uint32_t at = first + blockIdx.x, eight = at >> 3;
  const uint32_t octet = eight / slices, unit_of_work = octet * 8 + (at & 7);
  const uint32_t pair = MODE == kWhole ? unit_of_work : by_parts.div(unit_of_work);
  if (pair >= pairs) return;
  const uint32_t turn_of_seq = by_seq.div(pair), in_seq = pair - turn_of_seq * by_seq.d;
  const uint32_t r = order ? (uint32_t)order[turn_of_seq] : turn_of_seq;
  const uint32_t of_group = by_key_heads.div(in_seq);
  const int kh = (int)(in_seq - of_group * by_key_heads.d), h = kh * (a.v_heads / a.k_heads) + (int)of_group;
  const int slot = a.slots[r];
  const int64_t from_start = start_of(a.token_starts, (int)r, a.tokens), end = start_of(a.token_starts, (int)r + 1, a.tokens);
  if (!slot_ok(slot, a.num_slots) || from_start >= end) return;
  const int part = MODE == kWhole ? 0 : (int)(unit_of_work - pair * by_parts.d);
  Part of_chunks = {0, (end - from_start + kC - 1) / kC, true};
  if (MODE != kWhole) of_chunks = find_part(of_chunks.high, parts.parts, part);
  if (of_chunks.low >= of_chunks.high || (MODE == kEnds && of_chunks.last)) return;
  // of the ends, slices behind the values' are columns of the identity
  int group_column = (int)(eight - octet * slices) * L::kCols;
  const bool unit = MODE == kEnds && group_column >= a.head_v;
  if (unit) {
    if (part == 0) return;
    group_column -= a.head_v;
  }
  const int64_t chunks = of_chunks.high - of_chunks.low, start = from_start + of_chunks.low * kC;
  const int64_t chunk_bytes = delta_chunk_bytes(a.k_heads, a.v_heads, DK, DT);
  const uint8_t* from = static_cast<const uint8_t*>(a.workspace) + (from_start / kC + r + of_chunks.low) * chunk_bytes;
  const int64_t keys_at = kh * delta_key_bytes(DK, DT),
                ties_at = a.k_heads * delta_key_bytes(DK, DT) + (int64_t)h * kDeltaTieBytes;
  const char* values = static_cast<const char*>(a.v.p) + (h * a.v.head + group_column) * kSize;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)stage;

  // Moving data is kOf waves' work, this one's share is `share`: the loaders' where there are any, else each wave's.  A
  // wave's rows of values are its own here: it fills them again as soon as it has read the outputs in them.
  constexpr int kOf = LOADERS ? LOADERS : WAVES;
  const int share = LOADERS ? wave - WAVES : wave;
  constexpr int kLanes = L::kRow / 16, kRows = 64 / kLanes, kMoves = kC / kOf / kRows;  // of a row, rows of a move
  auto moved_row = [&](int i) { return share * (kC / kOf) + i * kRows + lane / kLanes; };
  // A chunk on its way into a stage: values,
  auto issue_values = [&](int64_t c, int to) {
    if (unit) return;
#pragma unroll
    for (int i = 0; i < kMoves; ++i) {
      const int row = moved_row(i);
      const int64_t token = std::min(start + c * kC + row, end - 1);
      to_lds(lds0 + to * L::kStage + L::kValuesAt + (share * (kC / kOf) + i * kRows) * L::kRow,
             values + token * a.v.token * kSize + L::turned(row, lane % kLanes * 16));
    }
  };
  // and turns of 4 blocks of keys, T, queries and P, kOf of them at a time; the gates go with the first
  constexpr int kKeyTurns = L::kKeys / (4 * kBlock), kTieTurns = kPAt / (4 * kBlock);
  constexpr int kAll = (MODE == kEnds ? 1 : 2) * (kKeyTurns + kTieTurns), kTurns = (kAll + kOf - 1) / kOf;
  auto issue_turn = [&](int64_t c, int to, int i) {
    const uint32_t lds = lds0 + to * L::kStage;
    const uint8_t* base = from + c * chunk_bytes;
    if (i == 0 && share == kOf - 1) to_lds2(lds + L::kGatesIn, base + ties_at + kGatesAt, lane * 16);
    int turn = i * kOf + share;
    if (turn >= kAll) return;
    const bool second = turn >= kKeyTurns + kTieTurns;  // queries and P
    if (second) turn -= kKeyTurns + kTieTurns;
    const bool tie = turn >= kKeyTurns;
    const int64_t in = (tie ? ties_at + (second ? kPAt : 0) - L::kKeys : keys_at + (second ? L::kKeys : 0)) + turn * 4 * kBlock;
    to_lds4(lds + (second ? L::kQueriesAt : 0) + turn * 4 * kBlock, base + in, lane * 16);
  };
  auto issue = [&](int64_t c, int to) {
    issue_values(c, to);
#pragma unroll
    for (int i = 0; i < kTurns; ++i) issue_turn(c, to, i);
  };
  // outputs of a chunk from its stage
  auto put_out = [&](int64_t c, int from_stage) {
    if (MODE == kEnds) return;
    const uint8_t* outs = stage + from_stage * L::kStage + L::kValuesAt + share * (kC / kOf) * L::kRow;
    char* to = static_cast<char*>(a.out.p) + (h * a.out.head + group_column) * kSize;
    u32x4_t held[kMoves];
#pragma unroll
    for (int i = 0; i < kMoves; ++i) held[i] = *reinterpret_cast<const u32x4_t*>(outs + i * kBlock + lane * 16);
#pragma unroll
    for (int i = 0; i < kMoves; ++i) {
      const int row = moved_row(i);
      const int64_t token = start + c * kC + row;
      if (token < end)
        *reinterpret_cast<u32x4_t*>(to + token * a.out.token * kSize + L::turned(row, lane % kLanes * 16)) = held[i];
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read, before it is filled again
  };
  auto meet = [&] {  // everyone's loads are there and LDS accesses done
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // between two chunks: the last one's outputs leave and the next one's operands come
  auto move = [&](int64_t c, int now) {
    if (L::kStages == 1) return;
    if (c > 0) put_out(c - 1, now ^ 1);
    if (c + 1 >= chunks) return;
    if (LOADERS) issue(c + 1, now ^ 1);
    else issue_values(c + 1, now ^ 1);
  };
  // with one stage: between the chunks, which all wait for
  auto change = [&](int64_t c) {
    if (L::kStages == 2 || c + 1 == chunks) return;
    if (!LOADERS || wave >= WAVES) {
      put_out(c, 0);
      issue(c + 1, 0);
    }
    meet();
  };

  if (LOADERS && wave >= WAVES) {
    issue(0, 0);
    meet();
    for (int64_t c = 0; c < chunks; ++c) {
      move(c, (int)(c & 1));
      meet();
      change(c);
    }
    put_out(chunks - 1, L::kStages == 2 ? (int)((chunks - 1) & 1) : 0);
    return;
  }
  if (!LOADERS) issue(0, 0);
  // The state: tile 2 s + t, register q of lane (g, n) is row 32 s + 8 g + 4 t + q, column n, so that two tiles are the
  // eight elements of an operand that meet elements 32 s + 8 g.. of a row of K or Q.
  float4_t s[L::kTiles];
  int scaled = kLength;  // the state is s 2^(scaled - 4), values are taken times 2^-scaled
  const int col = group_column + 16 * wave + n;
  const int64_t of_slot = ((int64_t)slot * a.v_heads + h) * DK * a.head_v;
  const int64_t of_parts = ((int64_t)r * a.v_heads + h) * parts.parts + part;
  {
    const float* begin = MODE == kPart ? parts.first + of_parts * DK * a.head_v : a.state + of_slot;
    const bool carried = MODE == kPart || (part == 0 && (!a.cached_lens || a.cached_lens[r] > 0));
#pragma unroll
    for (int t = 0; t < L::kTiles; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 32 * (t / 2) + 8 * g + 4 * (t & 1) + q;
        s[t][q] = carried ? begin[(int64_t)row * a.head_v + col] : unit && row == col ? 1.0f : 0.0f;
      }
  }
  meet();

  for (int64_t c = 0; c < chunks; ++c) {
    const int now = L::kStages == 2 ? (int)(c & 1) : 0;
    uint8_t* here = stage + now * L::kStage;
    const float* gates = reinterpret_cast<const float*>(here + L::kGatesIn);
    uint8_t* rows = here + L::kValuesAt;  // of values, then of outputs
    // byte x of this wave's columns in row 16 mt + 4 g + i
    auto place = [&](int mt, int i, int x) {
      return rows + (4 * g + i) * L::kRow + L::turned(4 * g + i, 16 * wave * kSize + x) + 16 * mt * L::kRow;
    };
    auto key = [&](int of_q, int part, int mt, int st) {
      return *reinterpret_cast<const half8_t*>(here + (of_q ? L::kQueriesAt : 0) + ((part * 4 + mt) * L::kSteps + st) * kBlock + lane * 16);
    };
    auto tied = [&](int at, int mt, int st, int part) {
      return *reinterpret_cast<const half8_t*>(here + at + (2 * tie(mt, st) + part) * kBlock + lane * 16);
    };
    auto gate = [&](int which, int mt) { return *reinterpret_cast<const float4_t*>(gates + which * kC + 16 * mt + 4 * g); };

    // Operands are read a step before they are needed: few waves hide little of what LDS takes.
    constexpr int kOfQ = MODE == kEnds ? 1 : 2;
    half8_t keys[2][kOfQ][4][L::kParts];
    auto read_keys = [&](int st) {
#pragma unroll
      for (int of_q = 0; of_q < kOfQ; ++of_q)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int p = 0; p < L::kParts; ++p) keys[st & 1][of_q][mt][p] = key(of_q, p, mt, st);
    };
    float4_t beta[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) beta[mt] = gate(kBeta, mt);
    float4_t x[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      if (unit) {
        x[mt] = float4_t{0, 0, 0, 0};
      } else if constexpr (DT == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[mt][i] = *reinterpret_cast<const float*>(place(mt, i, 4 * n));
      } else {
        const short4_t e = read_columns(place(mt, n / 4, (n % 4) * 8));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (DT == 1)
            x[mt][q] = __uint_as_float((uint32_t)(uint16_t)e[q] << 16);
          else
            x[mt][q] = (float)__builtin_bit_cast(_Float16, (short)e[q]);
        }
      }
    }
    read_keys(0);
    if (!LOADERS) move(c, now);
    __builtin_amdgcn_sched_barrier(0);

    // What a column's tokens bring, beta v, and its power of two, with M the largest of that and of the state's elements: M
    // goes to 2^7..2^8 when it has left 2^5..2^9.  The state's length is at most sqrt(128) M and grows by M a token, so that
    // X and V' stay below 75 M < 2^16; |S| 2^4 is below 2^13; half of a part's last step is 2^-30 of M at most.
    {
      float top = 0.0f, high = 0.0f;
#pragma unroll
      for (int t = 0; t < L::kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(s[t][i]));
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        x[mt] *= beta[mt];
#pragma unroll
        for (int i = 0; i < 4; ++i) high = fmaxf(high, fabsf(x[mt][i]));
      }
      const float both = of_column(fmaxf(top * (1.0f / kLong), __builtin_amdgcn_ldexpf(high, -scaled)));
      if (__any(c == 0 || both > 512.0f || (both < 32.0f && both > 0.0f && scaled > -150))) {
        const float of_s = of_column(top), of_x = of_column(high);
        constexpr int kNone = -100000;
        const int of_state = of_s > 0.0f ? __builtin_amdgcn_frexp_expf(of_s) + scaled - kLength : kNone;
        const int of_values = of_x > 0.0f ? __builtin_amdgcn_frexp_expf(of_x) : kNone;
        const int most = std::max(of_state, of_values), by_now = most - scaled;
        if (most != kNone && (by_now > 9 || by_now < 6)) {
          const int next = std::max(most - 8, -150), by = scaled - next;
          scaled = next;
#pragma unroll
          for (int t = 0; t < L::kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[t][i] = __builtin_amdgcn_ldexpf(s[t][i], by);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);

    // K S and Q S
    const float4_t none = {0, 0, 0, 0};
    float4_t y[4], o[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) y[mt] = o[mt] = none;
    half8_t turn[kTies][2];
    auto read_ties = [&](half8_t (&to)[kTies][2], int at, int st) {
#pragma unroll
      for (int mt = 2 * st; mt < 4; ++mt)
#pragma unroll
        for (int p = 0; p < 2; ++p) to[tie(mt, st)][p] = tied(at, mt, st, p);
    };
    float4_t gain[4];
    Parts b[2], d;
    b[0] = cut(s[0], s[1]);
#pragma unroll
    for (int st = 0; st < L::kSteps; ++st) {
      if (st + 1 < L::kSteps) read_keys(st + 1);
      if (st + 1 == L::kSteps) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) gain[mt] = gate(kGainK, mt);
        read_ties(turn, L::kTurnAt, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 1 + L::kParts; ++i)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          const int part = i == 2 ? L::kParts - 1 : 0;
          const half8_t of_s = i == 1 ? b[st & 1].lo : b[st & 1].hi;
          y[mt] = mfma(keys[st & 1][0][mt][part], of_s, y[mt]);
          if (MODE != kEnds) o[mt] = mfma(keys[st & 1][kOfQ - 1][mt][part], of_s, o[mt]);
        }
      if (st + 1 < L::kSteps) b[(st + 1) & 1] = cut(s[2 * st + 2], s[2 * st + 3]);
      // The next chunk's loads in between: all at once, at the chunk's begin, a wave waits until its queue takes them (the
      // chain of 12 prompts 466 us and not 449, the ends of 31 parts of 6 heads 74 and not 70).
      if (!LOADERS && L::kStages == 2 && c + 1 < chunks) {
#pragma unroll
        for (int i = st; i < kTurns; i += L::kSteps) issue_turn(c + 1, now ^ 1, i);
      }
    }
    __builtin_amdgcn_sched_barrier(0);

    // X
    const float whole = gates[kDecay * kC];
    float4_t gain_q[4], until[4];
    read_ties(turn, L::kTurnAt, 1);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      until[mt] = gate(kUntil, mt);
      if (MODE != kEnds) gain_q[mt] = gate(kGainQ, mt);
    }
#pragma unroll
    for (int st = 0; st < 2; ++st) {
#pragma unroll
      for (int mt = 2 * st; mt < 2 * st + 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[mt][i] = __builtin_fmaf(-gain[mt][i], y[mt][i], __builtin_amdgcn_ldexpf(x[mt][i], -scaled));
      b[st] = cut(x[2 * st], x[2 * st + 1]);
    }
    half8_t turned[L::kTiles][L::kParts], inner[kTies][2];  // rows of K^T; P
    auto read_turned = [&](int st) {
#pragma unroll
      for (int t = 0; t < L::kTiles; ++t)
#pragma unroll
        for (int p = 0; p < L::kParts; ++p) {
          short4_t e[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)  // tokens 32 st + 16 j + 4 g.., rows of this tile
            e[j] = read_columns(here + ((p * 4 + 2 * st + j) * L::kSteps + t / 2) * kBlock +
                                ((n % 4) * 16 + 4 * g + n / 4) * 16 + 8 * (t & 1));
          turned[t][p] = __builtin_bit_cast(half8_t, __builtin_shufflevector(e[0], e[1], 0, 1, 2, 3, 4, 5, 6, 7));
        }
    };
    read_turned(0);
    __builtin_amdgcn_sched_barrier(0);

    // V' = T X; the state's decay among it
    float4_t z[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) z[mt] = none;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int mt = 2 * half; mt < 2 * half + 2; ++mt)
          z[mt] = mfma(turn[tie(mt, 0)][i == 2], i == 1 ? b[0].lo : b[0].hi, z[mt]);
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int mt = 2; mt < 4; ++mt) z[mt] = mfma(turn[tie(mt, 1)][i == 2], i == 1 ? b[1].lo : b[1].hi, z[mt]);
#pragma unroll
    for (int t = 0; t < L::kTiles; ++t) s[t] *= whole;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
      if (MODE != kEnds) o[mt] *= gain_q[mt];

    // K^T V' onto the decayed state, P V' onto Q S
    auto cut_values = [&](int st) {
      const float4_t v0 = z[2 * st] * kDown, v1 = z[2 * st + 1] * kDown;
      d = cut(v0 * until[2 * st], v1 * until[2 * st + 1]);
      if (MODE != kEnds) b[st] = cut(v0, v1);
    };
    cut_values(0);
    if (MODE != kEnds) read_ties(inner, L::kInnerAt, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
#pragma unroll
      for (int i = 0; i < 1 + L::kParts; ++i)
#pragma unroll
        for (int t = 0; t < L::kTiles; ++t)
          s[t] = mfma(turned[t][i == 2 ? L::kParts - 1 : 0], i == 1 ? d.lo : d.hi, s[t]);
      if (st == 0) {
        cut_values(1);
        read_turned(1);
      }
#pragma unroll
      for (int i = 0; i < (MODE == kEnds ? 0 : 3); ++i)
#pragma unroll
        for (int mt = 2 * st; mt < 4; ++mt)
          o[mt] = mfma(inner[tie(mt, st)][i == 2], i == 1 ? b[st].lo : b[st].hi, o[mt]);
      if (MODE != kEnds && st == 0) read_ties(inner, L::kInnerAt, 1);
    }

    // outputs, to where this wave's values were
    if (MODE != kEnds) {
      const float back = __builtin_amdgcn_ldexpf(a.scale, scaled - 14);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float z0 = o[mt][i] * back, z1 = o[mt][i + 1] * back;
          if constexpr (DT == 0) {
            *reinterpret_cast<float*>(place(mt, i, 4 * n)) = z0;
            *reinterpret_cast<float*>(place(mt, i + 1, 4 * n)) = z1;
          } else {
            const uint32_t both = pack2<DT>(z0, z1);
            *reinterpret_cast<uint16_t*>(place(mt, i, 2 * n)) = (uint16_t)both;
            *reinterpret_cast<uint16_t*>(place(mt, i + 1, 2 * n)) = (uint16_t)(both >> 16);
          }
        }
      }
    }
    meet();
    change(c);
  }
  if (!LOADERS) put_out(chunks - 1, L::kStages == 2 ? (int)((chunks - 1) & 1) : 0);

  if (MODE == kPart && !of_chunks.last) return;
  float* to = a.state_out + of_slot;  // of the ends: where the next part starts, or what this one does
  if (MODE == kEnds) to = unit ? parts.turn + of_parts * DK * DK : parts.first + (of_parts + 1) * DK * a.head_v;
  const int64_t pitch = unit ? DK : a.head_v;
#pragma unroll
  for (int t = 0; t < L::kTiles; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        to[(int64_t)(32 * (t / 2) + 8 * g + 4 * (t & 1) + q) * pitch + col] =
            __builtin_amdgcn_ldexpf(s[t][q], scaled - kLength);
#endif
}

// The states that parts start from: S_0 as it is given, S_1 the first part's end, S_(p+1) = end_p + turn_p S_p.  A
// workgroup has 16 columns of a sequence and head, each of its waves 16 rows; products in fp32, a state passes through LDS
// in the order in which the matrix unit takes it (step r of four: elements 4 g + r of 16).
template <int DK>
__global__ __launch_bounds__(4 * DK) void gated_delta_join_kernel(DeltaArgs a, PartArgs parts, uint32_t slices) {
  constexpr int kTiles = DK / 16;
  __shared__ float4_t state[2][kTiles][64];
  const int lane = threadIdx.x & 63, tile = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  // columns of one sequence and head lie on one XCD, 8 apart, whose L2 then fetches `turn` once for them
  const uint32_t eight = blockIdx.x >> 3, octet = eight / slices;
  const int64_t pair = octet * 8 + (blockIdx.x & 7), r = pair / a.v_heads;
  if (r >= a.n_seqs) return;
  const int col = (int)(eight - octet * slices) * 16 + n;
  const int h = (int)(pair - r * a.v_heads);
  const int slot = a.slots[r];
  const int64_t start = start_of(a.token_starts, (int)r, a.tokens), end = start_of(a.token_starts, (int)r + 1, a.tokens);
  if (!slot_ok(slot, a.num_slots) || start >= end) return;
  const int64_t chunks = (end - start + kC - 1) / kC, each = chunks_of_part(chunks, parts.parts);
  const int count = (int)((chunks + each - 1) / each);
  const bool carried = !a.cached_lens || a.cached_lens[r] > 0;
  const int64_t of_state = (int64_t)DK * a.head_v, own = (int64_t)(16 * tile + 4 * g) * a.head_v + col;
  const float* given = a.state + ((int64_t)slot * a.v_heads + h) * of_state + own;
  float* first = parts.first + pair * parts.parts * of_state + own;
  const float* turn = parts.turn + pair * parts.parts * DK * DK + (16 * tile + n) * DK + 4 * g;
#pragma unroll
  for (int q = 0; q < 4; ++q) first[q * a.head_v] = carried ? given[q * a.head_v] : 0.0f;
  // ends and rows are asked for a part ahead
  float4_t row[2][kTiles], end_of[2];
  auto ask = [&](int p, int at) {
    if (p >= count) return;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) row[at][t] = *reinterpret_cast<const float4_t*>(turn + (int64_t)(p - 1) * DK * DK + 16 * t);
#pragma unroll
    for (int q = 0; q < 4; ++q) end_of[at][q] = first[p * of_state + q * a.head_v];
  };
  if (count < 2) return;
  float4_t one;
#pragma unroll
  for (int q = 0; q < 4; ++q) one[q] = first[of_state + q * a.head_v];
  ask(2, 0);
  state[0][tile][lane] = one;
  auto join = [&](int p, int at) {
    ask(p + 1, at ^ 1);
    // The last state is there.  Only LDS is waited for: what is asked for stays under way.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    float4_t b[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) b[t] = state[at][t][lane];
    float4_t s = end_of[at];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) s = __builtin_amdgcn_mfma_f32_16x16x4f32(row[at][t][q], b[t][q], s, 0, 0, 0);
    state[at ^ 1][tile][lane] = s;
#pragma unroll
    for (int q = 0; q < 4; ++q) first[p * of_state + q * a.head_v] = s[q];
  };
  for (int p = 2; p < count; p += 2) {
    join(p, 0);
    if (p + 1 < count) join(p + 1, 1);
  }
}

// `launch(first place, places)` for all places of chunks, so many at a time
template <typename F>
hipError_t for_places(const DeltaArgs& a, int64_t workgroups_of_place, F launch) {
  const int64_t places = delta_chunk_places(a.tokens, a.n_seqs), most = std::max<int64_t>(kMostWorkgroups / workgroups_of_place, 1);
  for (int64_t first = 0; first < places; first += most) {
    launch(first, (uint32_t)std::min(most, places - first));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int DK, int MODE, int WAVES, int LOADERS>
hipError_t launch_chain(const DeltaArgs& a, const PartArgs& parts, const int32_t* order, hipStream_t stream) {
  using L = Chain<DT, DK, MODE, WAVES, LOADERS>;
  const uint32_t slices = (uint32_t)((a.head_v + (MODE == kEnds ? DK : 0)) / L::kCols);
  const int of_parts = MODE == kWhole ? 1 : MODE == kEnds ? parts.parts - 1 : parts.parts;
  const FastDiv by_seq((uint32_t)a.v_heads), by_key_heads((uint32_t)a.k_heads), by_parts((uint32_t)of_parts);
  const int64_t pairs = (int64_t)a.n_seqs * a.v_heads, all = (pairs * of_parts + 7) / 8 * 8 * slices;
  for (int64_t first = 0; first < all; first += kMostWorkgroups) {
    const uint32_t grid = (uint32_t)std::min<int64_t>(kMostWorkgroups, all - first);
    gated_delta_chain_kernel<DT, DK, MODE, WAVES, LOADERS><<<grid, L::kThreads, 0, stream>>>(
        a, parts, order, by_seq, by_key_heads, by_parts, slices, (uint32_t)first, (uint32_t)pairs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Columns of a workgroup of the chain: 32, with two waves besides that move its data, while a CU then has one workgroup at
// most; 64 while that still holds, 128 above it (float32's stage holds 64).  8192 tokens, heads of 128, in us for 32, 64 and
// 128:  32 heads 344, 405, 583   64 heads 369, 435, 609   72 heads 668, 442, 617   128 heads 715, 508, 664
// 192 heads 1059, 895, 733   12 prompts of 48 heads 974, 690, 618.  float32: 64 heads 772, 863   96 heads 1439, 903
bool wide(const DeltaArgs& a, int64_t states) { return a.head_v % 128 == 0 && states * a.head_v > 64 * device_cu_count(); }

template <int DT, int DK>
hipError_t launch_parts(const DeltaArgs& a, int count, hipStream_t stream) {
  PartArgs parts = {count, nullptr, nullptr};
  const int64_t pairs = (int64_t)a.n_seqs * a.v_heads;
  parts.first = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) +
                                         delta_chunk_places(a.tokens, a.n_seqs) * delta_chunk_bytes(a.k_heads, a.v_heads, DK, DT));
  parts.turn = parts.first + pairs * count * DK * a.head_v;
  hipError_t e = launch_chain<DT, DK, kEnds, 4, 0>(a, parts, nullptr, stream);
  if (e != hipSuccess) return e;
  const uint32_t slices = (uint32_t)(a.head_v / 16);
  // a call in parts has at most 2^15 columns
  gated_delta_join_kernel<DK><<<(uint32_t)((pairs + 7) / 8 * 8 * slices), 4 * DK, 0, stream>>>(a, parts, slices);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if constexpr (DT != 0) {
    if (wide(a, pairs * count)) return launch_chain<DT, DK, kPart, 8, 0>(a, parts, nullptr, stream);
  }
  return launch_chain<DT, DK, kPart, 4, 0>(a, parts, nullptr, stream);
}

template <int DT, int DK>
hipError_t launch_sized(const DeltaArgs& a, hipStream_t stream) {
  const uint32_t k_heads = (uint32_t)a.k_heads, blocks = (uint32_t)((a.v_heads + kWaves - 1) / kWaves);
  const FastDiv by_heads(k_heads), by_group((uint32_t)(a.v_heads / a.k_heads)), by_blocks(blocks);
  // behind the chunks; parts, which calls of few sequences have, would lie there too
  int32_t* order = nullptr;
  const int64_t parts = delta_parts(a.tokens, a.n_seqs, a.v_heads, a.head_v);
  if (parts == 0 && a.n_seqs > 1 && a.n_seqs <= kMostOrdered)
    order = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(a.workspace) +
                                       delta_chunk_places(a.tokens, a.n_seqs) * delta_chunk_bytes(a.k_heads, a.v_heads, DK, DT));
  hipError_t e = for_places(a, k_heads, [&](int64_t first, uint32_t places) {
    gated_delta_keys_kernel<DT, DK><<<places * k_heads, 512, 0, stream>>>(a, by_heads, first, order);
  });
  if (e != hipSuccess) return e;
  e = for_places(a, blocks, [&](int64_t first, uint32_t places) {
    gated_delta_solve_kernel<DT, DK><<<places * blocks, kThreads, 0, stream>>>(a, by_group, by_blocks, first);
  });
  if (e != hipSuccess) return e;
  if (parts) return launch_parts<DT, DK>(a, (int)parts, stream);
  const int64_t pairs = (int64_t)a.n_seqs * a.v_heads;
  if (pairs * a.head_v <= 32 * device_cu_count()) return launch_chain<DT, DK, kWhole, 2, 2>(a, {}, order, stream);
  if constexpr (DT != 0) {
    if (wide(a, pairs)) return launch_chain<DT, DK, kWhole, 8, 0>(a, {}, order, stream);
  }
  return launch_chain<DT, DK, kWhole, 4, 0>(a, {}, order, stream);
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
