// K and V rows to E4M3 bytes in cache pages (nvfp4_kv_cache_write).
//
// Per element the rule of the dense quantiser: y = fp32(x * s), clamped to
// [-448, 448], v_cvt_pk_fp8_f32 (nearest even; checked on every fp32 input by
// conformance_cvt).  The row of one token and head goes to
//   cache[page][head][offset][:], slot = page * page_size + offset,
// head_dim consecutive bytes.
//
// Bandwidth kernel: 2 B read and 1 B written per bf16 element (32768 tokens, 4
// heads of 256 in rows of 14336: 38 us, 5.3 TB/s).  One thread takes 16
// consecutive elements (8 where head_dim is no multiple of 16) and stores 16
// bytes at once.  More pieces a thread were no faster on long prompts and slower
// on short calls (32 tokens, 4 heads of 256: 2.3 us, 3.2 with four pieces).
// What goes past the caches, in us a call:           32768 x 8 x 128   5003 x 8 x
//                                                    bf16       f32    128, f16
//   loads (rows too many to be there)                37.5       83     8.6
//   stores                                           41.5       62     6.6
//   both                                             40.1       81     8.0
//   neither                                          42.3       65     6.8
// (a lane's four float32 loads share their lines).  So many rows of a 16-bit type
// are loaded past them, and all others are stored past them.
//
// Where that many rows are strided, K's and V's of a token lie in one projection's
// row, and workgroups take them in turns of kRun: 38 us with 64 or 256, 41 with 1024,
// 45 with all of K first (the same 32768 tokens in rows of 14336).  Dense rows gain
// nothing (36.3 and 35.9 us for 32768 tokens of 8 x 128) and take K first.
#include "nvfp4_device.h"
#include "kv_internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kRun = 256;
constexpr int64_t kManyElements = 1 << 24;  // of K: 64 MiB with V, a quarter of the Infinity Cache

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// E elements from 16-byte loads (PAST: past the caches)
template <int DT, int E, bool PAST>
struct Raw {
  static constexpr int kLoads = E * (DT == 0 ? 4 : 2) / 16;
  u32x4_t w[kLoads];
  __device__ __forceinline__ void load(const void* x, int64_t elem) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(x) + elem * (DT == 0 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kLoads; ++i) w[i] = PAST ? __builtin_nontemporal_load(p + i) : p[i];
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == 0) {
      return __uint_as_float(w[i >> 2][i & 3]);
    } else {
      const uint32_t v = w[i >> 3][(i & 7) >> 1];
      if constexpr (DT == 1) return __uint_as_float(i & 1 ? v & 0xFFFF0000u : v << 16);
      const uint16_t h = (uint16_t)(i & 1 ? v >> 16 : v & 0xFFFFu);
      _Float16 f;
      __builtin_memcpy(&f, &h, 2);
      return (float)f;
    }
  }
};

__device__ __forceinline__ uint32_t e4m3x4(float y0, float y1, float y2, float y3) {
  auto clamp = [](float y) { return __builtin_amdgcn_fmed3f(y, -448.0f, 448.0f); };
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(clamp(y0), clamp(y1), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp(y2), clamp(y3), lo, true);
}

template <int DT, int E, bool PAST>
__global__ __launch_bounds__(kThreads) void kv_cache_write_kernel(CacheWriteArgs a, FastDiv by_row, FastDiv by_head,
                                                                  FastDiv by_page, FastDiv by_run, uint32_t chunks) {
  const uint32_t turn = PAST ? by_run.div(blockIdx.x) : blockIdx.y;
  const uint32_t block = PAST ? (turn >> 1) * by_run.d + blockIdx.x - turn * by_run.d : blockIdx.x;
  const bool value = turn & 1;  // K, then V
  const HeadsIn in = value ? a.v : a.k;
  const float s = value ? *a.v_scale : *a.k_scale;
  const uint32_t at = block * kThreads + threadIdx.x;  // a launch has at most 2^28 chunks, and a row 2^23
  const uint32_t t = by_row.div(at), in_row = at - t * by_row.d;
  const uint32_t head = by_head.div(in_row), chunk = in_row - head * by_head.d;
  // no branch before the store, which would wait for what it asks (39.4 us for 37.2, 32768 tokens of 8 x 128)
  const bool inside = at < chunks;
  const int64_t token = inside ? t : 0;
  const int slot = a.slot_map[token];  // asked for before the elements: loads return in order
  Raw<DT, E, PAST> raw;
  raw.load(in.p, token * in.token + head * in.head + chunk * E);
  const bool there = slot >= 0 && slot < a.num_pages * a.page_size;
  const uint32_t page = by_page.div((uint32_t)slot & 0x7FFFFFFFu), off = (uint32_t)slot - page * by_page.d;
  uint8_t* out = (value ? a.v_cache : a.k_cache) +
                 (((int64_t)page * a.kv_heads + head) * a.page_size + off) * a.head_dim + chunk * E;
  uint32_t w[E / 4];
#pragma unroll
  for (int i = 0; i < E / 4; ++i)
    w[i] = e4m3x4(raw.get(4 * i) * s, raw.get(4 * i + 1) * s, raw.get(4 * i + 2) * s, raw.get(4 * i + 3) * s);
  if (!there || !inside) return;
  if constexpr (E == 8)
    *reinterpret_cast<u32x2_t*>(out) = u32x2_t{w[0], w[1]};
  else if constexpr (PAST)
    *reinterpret_cast<u32x4_t*>(out) = u32x4_t{w[0], w[1], w[2], w[3]};
  else
    __builtin_nontemporal_store(u32x4_t{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4_t*>(out));
}

template <int DT, int E, bool PAST>
hipError_t launch_chunks(CacheWriteArgs a, hipStream_t stream) {
  const uint32_t of_head = (uint32_t)(a.head_dim / E), of_row = (uint32_t)a.kv_heads * of_head;
  const bool strided = a.k.token != (int64_t)a.kv_heads * a.head_dim;
  for (int64_t left = a.tokens;;) {
    a.tokens = std::min(left, std::max<int64_t>(kMostWorkgroups * kThreads / of_row, 1));
    const uint32_t chunks = (uint32_t)(a.tokens * of_row), all = (chunks + kThreads - 1) / kThreads;
    const uint32_t run = PAST && strided && all > kRun ? kRun : all;
    const dim3 grid = PAST ? dim3((all + run - 1) / run * run * 2) : dim3(all, 2);
    kv_cache_write_kernel<DT, E, PAST><<<grid, kThreads, 0, stream>>>(
        a, FastDiv(of_row), FastDiv(of_head), FastDiv((uint32_t)a.page_size), FastDiv(run), chunks);
    const hipError_t e = hipGetLastError();
    left -= a.tokens;
    if (e != hipSuccess || left == 0) return e;
    auto behind = [&](HeadsIn x) { return static_cast<const char*>(x.p) + a.tokens * x.token * (DT == 0 ? 4 : 2); };
    a.k.p = behind(a.k);
    a.v.p = behind(a.v);
    a.slot_map += a.tokens;
  }
}

template <int DT>
hipError_t launch_typed(const CacheWriteArgs& a, hipStream_t stream) {
  if (a.head_dim % 16 != 0) return launch_chunks<DT, 8, false>(a, stream);
  if constexpr (DT != 0) {
    if (a.tokens * a.kv_heads * a.head_dim >= kManyElements) return launch_chunks<DT, 16, true>(a, stream);
  }
  return launch_chunks<DT, 16, false>(a, stream);
}

}  // namespace

hipError_t launch_kv_cache_write(const CacheWriteArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case 0: return launch_typed<0>(a, stream);
    case 1: return launch_typed<1>(a, stream);
    default: return launch_typed<2>(a, stream);
  }
}

}  // namespace nvfp4
