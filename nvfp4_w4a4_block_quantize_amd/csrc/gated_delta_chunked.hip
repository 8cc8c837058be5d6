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
// Three kernels.  The first normalises keys and queries.  The second has a wave for each
// chunk and value head, all independent, and leaves T, P and the gates in the workspace.
// The third walks the chunks of a sequence with 16 columns of the state in a wave's registers:
// columns never meet, and the matrix unit's results lie as its next operands want them,
// so S, X and V' pass through neither LDS nor other lanes.
//
// Precision.  Operands are fp16 parts, sums fp32.  A row of keys or queries is scaled by a
// power of two to a length in [16, 32): 16-bit inputs fit one part but for what lies 2^-30
// below that length; float32 takes two.  |T| and |P| are at most 1 and scaled by 2^14;
// a column of S, and with it X and V', is scaled by a power of two that follows it and the
// values: each is cut into two parts, 2^-22 of the element or 2^-31 of the column's largest.
// Of products of two cut operands the low parts' is dropped (2^-22 again).
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
enum { kBeta, kGainK, kUntil, kGainQ, kWhole, kGates };
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

constexpr int kPitch = 20;  // floats of a row of 16 in LDS: rows that lanes read side by side meet distinct banks
constexpr int kSquare = 16 * kPitch;
constexpr int square(int j, int i) { return i * (i + 1) / 2 + j; }  // of block column j, block row i

struct SolveLds {
  float a[10 * kSquare];  // A^T by blocks: row j, column i; then the inverse's
  double log_decay[kC];
  float beta[kC], k_norm[kC];
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
    // 1 / sqrt(|x|^2 + eps), of x scaled: where eps is then infinite, x is nothing beside it
    const float more = __builtin_amdgcn_ldexpf(eps, 2 * up), all = squares + more;
    norm = more > 3e38f ? __builtin_amdgcn_ldexpf(1.0f / sqrtf(eps), -up) : 1.0f / sqrtf(all);
    if (squares == 0.0f) norm = 0.0f;  // at most 2^-4 then, whatever eps is
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
  const float4_t row = *reinterpret_cast<const float4_t*>(a + n * kPitch + 4 * g);
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(-row[r], b[r], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ void store_block(float* to, float4_t x, int g, int n) {
#pragma unroll
  for (int r = 0; r < 4; ++r) to[(4 * g + r) * kPitch + n] = x[r];
}
__device__ __forceinline__ float4_t load_block(const float* from, int g, int n) {
  float4_t x;
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = from[(4 * g + r) * kPitch + n];
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

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

// Keys and queries of a chunk and key head: eight waves take 16 rows each.
template <int DT, int DK>
__global__ __launch_bounds__(512) void gated_delta_keys_kernel(DeltaArgs a, FastDiv by_heads, int64_t first_place) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  const uint32_t of_launch = by_heads.div(blockIdx.x);
  const int kh = (int)(blockIdx.x - of_launch * by_heads.d);
  const int64_t place = first_place + of_launch;
  Place at;
  if (!find_place(a, place, at)) return;
  const int rows = (int)std::min<int64_t>(kC, at.end - at.begin);
  const bool of_q = wave >= 4;
  const int mt = wave & 3, row = 16 * mt + n;
  constexpr int64_t kBytes = delta_key_bytes(DK, DT), kImage = (kBytes - 1024) / 2;
  uint8_t* keys = static_cast<uint8_t*>(a.workspace) + place * delta_chunk_bytes(a.k_heads, a.v_heads, DK, DT) + kh * kBytes;
  Row<DT, DK> x;
  x.load(of_q ? a.q : a.k, at.begin + std::min(row, rows - 1), kh, g, row < rows, a.eps);
  x.store(keys + (of_q ? kImage : 0), mt, lane);
  if (g == 0) reinterpret_cast<float*>(keys + 2 * kImage)[(of_q ? kC : 0) + row] = x.norm;
}

template <int DT, int DK>
__global__ __launch_bounds__(kThreads) void gated_delta_solve_kernel(DeltaArgs a, FastDiv by_group, FastDiv by_blocks,
                                                                     int64_t first_place) {
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
  constexpr int64_t kBytes = delta_key_bytes(DK, DT), kImage = (kBytes - 1024) / 2;
  uint8_t* base = static_cast<uint8_t*>(a.workspace) + place * delta_chunk_bytes(a.k_heads, a.v_heads, DK, DT);
  const uint8_t* keys = base + kh * kBytes;
  const float* norms = reinterpret_cast<const float*>(keys + 2 * kImage);
  uint8_t* ties = base + a.k_heads * kBytes + (int64_t)h * kDeltaTieBytes;

  Row<DT, DK> k[4];
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) k[mt].read(keys, mt, lane);
  const float k_norm = norms[lane], q_norm = norms[kC + lane];

  // gates of token `lane`: the sum of log2 decays in 64 bits, since only differences count
  const int64_t token = at.begin + std::min(lane, rows - 1);
  const float decay = -expf(a.a_log[h]) * softplus(element<DT>(a.a, token * a.a_token + h) + a.dt_bias[h]);
  const float beta = lane < rows ? sigmoid<true>(element<DT>(a.b, token * a.b_token + h)) : 0.0f;
  double log_decay = lane < rows ? (double)decay * 1.4426950408889634 : 0.0;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double before = __shfl_up(log_decay, d);
    if (lane >= d) log_decay += before;
  }
  const double whole = __shfl(log_decay, 63);
  lds.log_decay[lane] = log_decay;
  lds.beta[lane] = beta * k_norm;
  lds.k_norm[lane] = k_norm;
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
  auto of_rows = [&](const float* x, int bj) { return *reinterpret_cast<const float4_t*>(x + 16 * bj + 4 * g); };

  // P by rows of blocks, and A^T
#pragma unroll
  for (int bi = 0; bi < 4; ++bi) {
    Row<DT, DK> q;
    q.read(keys + kImage, bi, lane);
    const float strength = lds.beta[16 * bi + n], of_q = __shfl(q_norm, 16 * bi + n);
    float4_t p[4];
#pragma unroll
    for (int bj = 0; bj <= bi; ++bj) {
      const float4_t e = ratio(bj, bi) * of_rows(lds.k_norm, bj);
      p[bj] = e * of_q * dots(k[bj], q);
      float4_t x = e * strength * dots(k[bj], k[bi]);
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
        const float4_t col = *reinterpret_cast<const float4_t*>(block + j * kPitch + 4 * i4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * i4 + i > j) x[4 * i4 + i] = __builtin_fmaf(-col[i], x[j], x[4 * i4 + i]);
      }
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4_t*>(block + n * kPitch + 4 * i) = float4_t{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
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
  gates[kWhole * kC + lane] = __builtin_amdgcn_exp2f((float)whole);
}

// -------------------------------------------------------------- the states' chain

typedef short short4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4_t lds_short4_t;

// Four rows of 16 16-bit elements that a group of 16 lanes points at, four elements a lane; lane n gets column n.
__device__ __forceinline__ short4_t read_columns(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)p);
}

// WAVES of a workgroup hold columns, LOADERS more move data for them
template <int DT, int DK, int WAVES, int LOADERS>
struct Chain {
  static constexpr int kParts = DT == 0 ? 2 : 1, kSteps = DK / 32, kTiles = DK / 16;
  static constexpr int kCols = 16 * WAVES;                    // of a workgroup
  static constexpr int kThreads = 64 * (WAVES + LOADERS);
  static constexpr int kKeys = kParts * 4 * kSteps * kBlock;  // bytes of K; Q follows
  static constexpr int kRow = 16 * element_size(DT), kValues = kC * kRow;  // a wave's columns of V, then of the outputs
  static constexpr int kTiesAt = 2 * kKeys, kValuesAt = kTiesAt + kDeltaTieBytes;
  static constexpr int kStage = kValuesAt + WAVES * kValues;
  static constexpr int kStages = 2 * kStage <= (160 << 10) ? 2 : 1;
  static_assert(kStages * kStage <= (160 << 10), "the stages fit LDS");
};

#if defined(__HIP_DEVICE_COMPILE__)
// From memory to LDS past the registers, 16 bytes a lane to byte lds + 16 lane.  M0 is set in the same block, one wait
// state before the loads read it; an instruction's offset counts on both sides.
__device__ __forceinline__ void to_lds4(uint32_t lds, const void* base, uint32_t offset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "global_load_lds_dwordx4 %1, %2 offset:1024\n\t"
      "global_load_lds_dwordx4 %1, %2 offset:2048\n\t"
      "global_load_lds_dwordx4 %1, %2 offset:3072" ::"s"(lds), "v"(offset), "s"(base) : "memory");
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

template <int DT, int DK, int WAVES, int LOADERS>
__global__ __launch_bounds__(64 * (WAVES + LOADERS), (WAVES + LOADERS + 3) / 4) void gated_delta_chain_kernel(
    DeltaArgs a, FastDiv by_seq, FastDiv by_key_heads, uint32_t slices, uint32_t first, uint32_t pairs) {
#if defined(__HIP_DEVICE_COMPILE__)
  using L = Chain<DT, DK, WAVES, LOADERS>;
  constexpr int kSize = element_size(DT);
  __shared__ __attribute__((aligned(1024))) uint8_t stage[L::kStages * L::kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;

  // Workgroups go to the XCDs in turn: those of one sequence and head, which read the same ties, and where there are 8 key
  // heads (or a multiple) those of one key head lie on one XCD, 8 apart.
  const uint32_t at = first + blockIdx.x, eight = at >> 3;
  const uint32_t octet = eight / slices, pair = octet * 8 + (at & 7);
  if (pair >= pairs) return;
  const int group_column = (int)(eight - octet * slices) * L::kCols;
  const uint32_t r = by_seq.div(pair), in_seq = pair - r * by_seq.d;
  const uint32_t of_group = by_key_heads.div(in_seq);
  const int kh = (int)(in_seq - of_group * by_key_heads.d), h = kh * (a.v_heads / a.k_heads) + (int)of_group;
  const int slot = a.slots[r];
  const int64_t start = start_of(a.token_starts, (int)r, a.tokens), end = start_of(a.token_starts, (int)r + 1, a.tokens);
  if (!slot_ok(slot, a.num_slots) || start >= end) return;
  const int64_t chunks = (end - start + kC - 1) / kC;
  const int64_t chunk_bytes = delta_chunk_bytes(a.k_heads, a.v_heads, DK, DT);
  const uint8_t* from = static_cast<const uint8_t*>(a.workspace) + (start / kC + r) * chunk_bytes;
  const int64_t keys_at = kh * delta_key_bytes(DK, DT),
                ties_at = a.k_heads * delta_key_bytes(DK, DT) + (int64_t)h * kDeltaTieBytes;
  const char* values = static_cast<const char*>(a.v.p) + (h * a.v.head + group_column) * kSize;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)stage;

  // Moving data is `of` waves' work, this one's share is `share`: the loaders' where there are any, else each wave's, and
  // then its columns are its own, so that it may fill them again as soon as it has read them.
  constexpr int kOf = LOADERS ? LOADERS : WAVES;
  const int share = LOADERS ? wave - WAVES : wave;
  constexpr int kLanes = L::kRow / 16, kRows = 64 / kLanes, kMoves = kC / kRows;  // of a row, rows of a move
  // a chunk on its way into a stage: turns of 4 blocks of keys and queries, then of T and P, the gates, and values
  auto issue = [&](int64_t c, int to) {
    const uint32_t lds = lds0 + to * L::kStage;
    const uint8_t* base = from + c * chunk_bytes;
    constexpr int kTurns = 2 * L::kKeys / (4 * kBlock), kAll = kTurns + kGatesAt / (4 * kBlock);
#pragma unroll
    for (int w = 0; w < WAVES / kOf; ++w) {
      const int of = share + w * kOf;
#pragma unroll
      for (int i = 0; i < kMoves; ++i) {
        const int64_t token = std::min(start + c * kC + i * kRows + lane / kLanes, end - 1);
        to_lds(lds + L::kValuesAt + of * L::kValues + i * kBlock,
               values + token * a.v.token * kSize + of * L::kRow + lane % kLanes * 16);
      }
    }
#pragma unroll
    for (int i = 0; i < (kAll + kOf - 1) / kOf; ++i) {
      const int turn = i * kOf + share;
      if (turn >= kAll) break;
      const bool tie = turn >= kTurns;
      to_lds4(lds + turn * 4 * kBlock, base + (tie ? ties_at - L::kTiesAt : keys_at) + turn * 4 * kBlock, lane * 16);
    }
    if (share == kOf - 1) to_lds2(lds + L::kTiesAt + kGatesAt, base + ties_at + kGatesAt, lane * 16);
  };
  // outputs of a chunk from its stage
  auto put_out = [&](int64_t c, int from_stage) {
    const int64_t token = start + c * kC + lane / kLanes;
    char* to = static_cast<char*>(a.out.p) + (token * a.out.token + h * a.out.head + group_column) * kSize + lane % kLanes * 16;
    u32x4_t held[WAVES / kOf][kMoves];
#pragma unroll
    for (int w = 0; w < WAVES / kOf; ++w)
#pragma unroll
      for (int i = 0; i < kMoves; ++i)
        held[w][i] = *reinterpret_cast<const u32x4_t*>(stage + from_stage * L::kStage + L::kValuesAt + (share + w * kOf) * L::kValues +
                                                       i * kBlock + lane * 16);
#pragma unroll
    for (int w = 0; w < WAVES / kOf; ++w)
#pragma unroll
      for (int i = 0; i < kMoves; ++i)
        if (token + i * kRows < end)
          *reinterpret_cast<u32x4_t*>(to + i * kRows * a.out.token * kSize + (share + w * kOf) * L::kRow) = held[w][i];
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
    if (c + 1 < chunks) issue(c + 1, now ^ 1);
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
  const int64_t state = ((int64_t)slot * a.v_heads + h) * DK * a.head_v + group_column + 16 * wave + n;
  const bool carried = !a.cached_lens || a.cached_lens[r] > 0;
#pragma unroll
  for (int t = 0; t < L::kTiles; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      s[t][q] = carried ? a.state[state + (int64_t)(32 * (t / 2) + 8 * g + 4 * (t & 1) + q) * a.head_v] : 0.0f;
  meet();

  for (int64_t c = 0; c < chunks; ++c) {
    const int now = L::kStages == 2 ? (int)(c & 1) : 0;
    uint8_t* here = stage + now * L::kStage;
    const uint8_t* ties = here + L::kTiesAt;
    const float* gates = reinterpret_cast<const float*>(ties + kGatesAt);
    uint8_t* mine = here + L::kValuesAt + wave * L::kValues;
    auto key = [&](int of_q, int part, int mt, int st) {
      return *reinterpret_cast<const half8_t*>(here + of_q * L::kKeys + ((part * 4 + mt) * L::kSteps + st) * kBlock + lane * 16);
    };
    auto tied = [&](int at, int mt, int st, int part) {
      return *reinterpret_cast<const half8_t*>(ties + at + (2 * tie(mt, st) + part) * kBlock + lane * 16);
    };
    auto gate = [&](int which, int mt) { return *reinterpret_cast<const float4_t*>(gates + which * kC + 16 * mt + 4 * g); };

    float4_t x[4], beta[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      beta[mt] = gate(kBeta, mt);
      if constexpr (DT == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[mt][i] = *reinterpret_cast<const float*>(mine + (16 * mt + 4 * g + i) * L::kRow + 4 * n);
      } else {
        const short4_t e = read_columns(mine + (16 * mt + 4 * g + n / 4) * L::kRow + (n % 4) * 8);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (DT == 1)
            x[mt][q] = __uint_as_float((uint32_t)(uint16_t)e[q] << 16);
          else
            x[mt][q] = (float)__builtin_bit_cast(_Float16, (short)e[q]);
        }
      }
    }
    // Operands are read a step before they are needed: at most two waves a SIMD hide little of what LDS takes.
    half8_t keys[2][4][L::kParts];
    auto read_keys = [&](int of_q, int st) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int p = 0; p < L::kParts; ++p) keys[st & 1][mt][p] = key(of_q, p, mt, st % L::kSteps);
    };
    read_keys(0, 0);
    if (!LOADERS) move(c, now);
    __builtin_amdgcn_sched_barrier(0);

    // What a column's tokens bring, beta v, and its power of two, with M the largest of that and of the state's elements: M
    // goes to 2^7..2^8 when it has left 2^5..2^9.  The state's length is at most sqrt(128) M and grows by M a token, so that
    // X and V' stay below 75 M < 2^16; |S| 2^4 is below 2^13; a part's last bit lies 2^31 below M.
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
      const float both = fmaxf(top * (1.0f / kLong), __builtin_amdgcn_ldexpf(high, -scaled));
      if (__any(c == 0 || both > 512.0f || (both < 32.0f && both > 0.0f && scaled > -150))) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        high = fmaxf(high, __shfl_xor(high, 16));
        high = fmaxf(high, __shfl_xor(high, 32));
        constexpr int kNone = -100000;
        const int of_state = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) + scaled - kLength : kNone;
        const int of_values = high > 0.0f ? __builtin_amdgcn_frexp_expf(high) : kNone;
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

    // K S
    const float4_t none = {0, 0, 0, 0};
    float4_t y[4] = {none, none, none, none}, o[4] = {none, none, none, none};
    Parts of_s[L::kSteps];
    float4_t gain[4], gain_q[4];
    of_s[0] = cut(s[0], s[1]);
#pragma unroll
    for (int st = 0; st < L::kSteps; ++st) {
      if (st + 1 < L::kSteps) {
        read_keys(0, st + 1);
      } else {
        read_keys(1, L::kSteps);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) gain[mt] = gate(kGainK, mt);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 1 + L::kParts; ++i)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
          y[mt] = mfma(keys[st & 1][mt][i == 2 ? L::kParts - 1 : 0], i == 1 ? of_s[st].lo : of_s[st].hi, y[mt]);
      if (st + 1 < L::kSteps) of_s[st + 1] = cut(s[2 * st + 2], s[2 * st + 3]);
    }

    // Q S, which nothing waits for, among the arithmetic of X
    half8_t turn[kTies][2];
    auto read_ties = [&](half8_t (&to)[kTies][2], int at, int st) {
#pragma unroll
      for (int mt = 2 * st; mt < 4; ++mt)
#pragma unroll
        for (int p = 0; p < 2; ++p) to[tie(mt, st)][p] = tied(at, mt, st, p);
    };
    Parts b[2], d[2];
#pragma unroll
    for (int st = 0; st < L::kSteps; ++st) {
      if (st + 1 < L::kSteps) read_keys(1, st + 1 + L::kSteps);
      else read_ties(turn, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 1 + L::kParts; ++i)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
          o[mt] = mfma(keys[st & 1][mt][i == 2 ? L::kParts - 1 : 0], i == 1 ? of_s[st].lo : of_s[st].hi, o[mt]);
      // a share of X in each step
#pragma unroll
      for (int mt = 4 * st / L::kSteps; mt < 4 * (st + 1) / L::kSteps; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[mt][i] = __builtin_fmaf(-gain[mt][i], y[mt][i], __builtin_amdgcn_ldexpf(x[mt][i], -scaled));
      if (st == L::kSteps / 2) b[0] = cut(x[0], x[1]);
    }
    b[1] = cut(x[2], x[3]);

    // V' = T X; the state's decay among it
    const float whole = gates[kWhole * kC];
    float4_t until[4], z[4] = {none, none, none, none};
    half8_t turned[L::kTiles][L::kParts], inner[kTies][2];  // rows of K^T; P
    auto read_turned = [&](int st) {
#pragma unroll
      for (int t = 0; t < L::kTiles; ++t)
#pragma unroll
        for (int p = 0; p < L::kParts; ++p) {
          short4_t e[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)  // tokens 32 st + 16 j + 4 g.., rows of this tile
            e[j] = read_columns(here + ((p * 4 + 2 * st + j) * L::kSteps + t / 2) * kBlock + ((n % 4) * 16 + 4 * g + n / 4) * 16 +
                                8 * (t & 1));
          turned[t][p] = __builtin_bit_cast(half8_t, __builtin_shufflevector(e[0], e[1], 0, 1, 2, 3, 4, 5, 6, 7));
        }
    };
    read_ties(turn, 0, 1);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      until[mt] = gate(kUntil, mt);
      gain_q[mt] = gate(kGainQ, mt);
    }
    read_turned(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int mt = 2 * half; mt < 2 * half + 2; ++mt) z[mt] = mfma(turn[tie(mt, 0)][i == 2], i == 1 ? b[0].lo : b[0].hi, z[mt]);
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int mt = 2; mt < 4; ++mt) z[mt] = mfma(turn[tie(mt, 1)][i == 2], i == 1 ? b[1].lo : b[1].hi, z[mt]);
#pragma unroll
    for (int t = 0; t < L::kTiles; ++t) s[t] *= whole;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) o[mt] *= gain_q[mt];

    // K^T V' onto the decayed state, P V' onto Q S
    auto cut_values = [&](int st) {
      const float4_t v0 = z[2 * st] * kDown, v1 = z[2 * st + 1] * kDown;
      d[st] = cut(v0 * until[2 * st], v1 * until[2 * st + 1]);
      b[st] = cut(v0, v1);
    };
    cut_values(0);
    read_ties(inner, kPAt, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
#pragma unroll
      for (int i = 0; i < 1 + L::kParts; ++i)
#pragma unroll
        for (int t = 0; t < L::kTiles; ++t) s[t] = mfma(turned[t][i == 2 ? L::kParts - 1 : 0], i == 1 ? d[st].lo : d[st].hi, s[t]);
      if (st == 0) cut_values(1);
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int mt = 2 * st; mt < 4; ++mt)
          o[mt] = mfma(inner[tie(mt, st)][i == 2], i == 1 ? b[st].lo : b[st].hi, o[mt]);
      if (st == 0) {
        read_turned(1);
        read_ties(inner, kPAt, 1);
      }
    }

    // outputs, to where this wave's values were
    const float back = __builtin_amdgcn_ldexpf(a.scale, scaled - 14);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      uint8_t* row = mine + (16 * mt + 4 * g) * L::kRow + n * kSize;
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float z0 = o[mt][i] * back, z1 = o[mt][i + 1] * back;
        if constexpr (DT == 0) {
          *reinterpret_cast<float*>(row + i * L::kRow) = z0;
          *reinterpret_cast<float*>(row + (i + 1) * L::kRow) = z1;
        } else {
          const uint32_t both = pack2<DT>(z0, z1);
          *reinterpret_cast<uint16_t*>(row + i * L::kRow) = (uint16_t)both;
          *reinterpret_cast<uint16_t*>(row + (i + 1) * L::kRow) = (uint16_t)(both >> 16);
        }
      }
    }
    meet();
    change(c);
  }
  if (!LOADERS) put_out(chunks - 1, L::kStages == 2 ? (int)((chunks - 1) & 1) : 0);

#pragma unroll
  for (int t = 0; t < L::kTiles; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      a.state_out[state + (int64_t)(32 * (t / 2) + 8 * g + 4 * (t & 1) + q) * a.head_v] =
          __builtin_amdgcn_ldexpf(s[t][q], scaled - kLength);
#endif
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

template <int DT, int DK, int WAVES, int LOADERS>
hipError_t launch_chain(const DeltaArgs& a, hipStream_t stream) {
  using L = Chain<DT, DK, WAVES, LOADERS>;
  const uint32_t slices = (uint32_t)(a.head_v / L::kCols);
  const FastDiv by_seq((uint32_t)a.v_heads), by_key_heads((uint32_t)a.k_heads);
  const int64_t pairs = (int64_t)a.n_seqs * a.v_heads, all = (pairs + 7) / 8 * 8 * slices;
  for (int64_t first = 0; first < all; first += kMostWorkgroups) {
    const uint32_t grid = (uint32_t)std::min<int64_t>(kMostWorkgroups, all - first);
    gated_delta_chain_kernel<DT, DK, WAVES, LOADERS>
        <<<grid, L::kThreads, 0, stream>>>(a, by_seq, by_key_heads, slices, (uint32_t)first, (uint32_t)pairs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int DK>
hipError_t launch_sized(const DeltaArgs& a, hipStream_t stream) {
  const uint32_t k_heads = (uint32_t)a.k_heads, blocks = (uint32_t)((a.v_heads + kWaves - 1) / kWaves);
  const FastDiv by_heads(k_heads), by_group((uint32_t)(a.v_heads / a.k_heads)), by_blocks(blocks);
  hipError_t e = for_places(a, k_heads, [&](int64_t first, uint32_t places) {
    gated_delta_keys_kernel<DT, DK><<<places * k_heads, 512, 0, stream>>>(a, by_heads, first);
  });
  if (e != hipSuccess) return e;
  e = for_places(a, blocks, [&](int64_t first, uint32_t places) {
    gated_delta_solve_kernel<DT, DK><<<places * blocks, kThreads, 0, stream>>>(a, by_group, by_blocks, first);
  });
  if (e != hipSuccess) return e;
  const int64_t columns = (int64_t)a.n_seqs * a.v_heads * a.head_v;
  if (columns <= 32 * device_cu_count()) return launch_chain<DT, DK, 2, 2>(a, stream);
  if constexpr (DT != 0) {
    if (a.head_v % 128 == 0) return launch_chain<DT, DK, 8, 0>(a, stream);
  }
  return launch_chain<DT, DK, 4, 0>(a, stream);
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
