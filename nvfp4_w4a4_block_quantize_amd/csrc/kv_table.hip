// Block tables and slot maps from request lengths (nvfp4_kv_block_table).
//
// With c cached and n new tokens of a request and pages of P tokens:
//   held = ceil(c/P), all = ceil((c+n)/P), need = all - held fresh pages;
//   upto_r = used + sum_{i<=r} need_i picks them from the free list in order;
//   slot(t) = page(pos / P) * P + pos % P for the new token at position pos.
//
// A workgroup of 1024 threads scans the requests, one to a thread or, where there are
// more of them, four neighbours (4000 requests of 200 tokens: 3.8 us less than in four
// rounds of one), with running sums of tokens and pages (64-bit: neither sum is
// bounded by 32 bits before the limits are applied).  The tokens are then spread
// over threads, up to four consecutive ones each: a thread finds its request by
// bisection in the starts and walks on from there.  The thread whose token opens a
// page also enters it in the block table, so fresh pages cost no pass of their own
// and nobody reads an entry that this call writes.
//
// Latency decides, so there is one launch where that is less: up to kInLds
// requests, every workgroup makes the sums for itself, keeps what it needs of them
// in LDS and spreads its tokens; the first one writes them down (1000 requests,
// 150 thousand tokens: 6.7 us, 11.5 with a second kernel that spreads them; 96
// requests, 1.6 million: 13.3 and 10.6).  In place (seq_lens is cached_lens, or
// free_used_out is free_used) that holds for a single workgroup only, since the
// others could find lengths that the first one has moved on already.
//
// A decode step's requests bring one token each.  Where the slot map has room for
// kOwn tokens of each at most, and none brings more, threads place their requests'
// tokens themselves, with the page that a token continues already loaded while the
// sums are made (256 requests: 4.4 us, 5.5 by bisection).  More requests than
// threads are placed faster by many workgroups (4096 requests: 10.2 and 9.9 us).
// What is left is latency: a launch, the lengths, the sums, a page and the stores,
// one after another.
#include <algorithm>
#include <type_traits>

#include "kv_internal.h"

namespace nvfp4 {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kScanWaves = kScanThreads / 64;
constexpr int kSpreadThreads = 256;
constexpr int kSpreadLds = 1024;    // requests that a workgroup of the second launch keeps in LDS
constexpr int kPerThread = 4;       // tokens at most, one 16-byte store
constexpr int kInLds = 4096;        // requests whose sums a workgroup keeps in LDS
constexpr int kMany = kInLds / kScanThreads;  // neighbouring requests of a thread, where there are more than threads
constexpr int kOwn = 8;             // tokens of a request, at most one fresh page among them
constexpr int kOneWorkgroup = 8192; // slots that a single workgroup fills in less time than a second launch takes
constexpr int kOneLaunch = 1 << 19; // slots up to which making the sums again in every workgroup takes less

// What spreading the tokens needs of the requests' sums: in LDS, or as they were written down.
struct LdsSums {
  const int32_t *starts, *first, *cached;
  __device__ __forceinline__ int start(int r) const { return starts[r]; }
  __device__ __forceinline__ int first_page(int r) const { return first[r]; }
  __device__ __forceinline__ int cached_len(int r) const { return cached[r]; }
};
struct WrittenSums {
  const int32_t *starts, *first, *seq_lens, *new_lens;
  __device__ __forceinline__ int start(int r) const { return starts[r]; }
  __device__ __forceinline__ int first_page(int r) const { return first[r]; }
  // of a served request, whose seq_lens counts its new tokens already
  __device__ __forceinline__ int cached_len(int r) const { return seq_lens[r] - new_lens[r]; }
};

struct Sums {
  int64_t tokens, pages;
};

__device__ __forceinline__ Sums operator+(Sums x, Sums y) { return {x.tokens + y.tokens, x.pages + y.pages}; }

__device__ __forceinline__ Sums shifted(Sums x, int d, int width) {
  return {__shfl_up(x.tokens, d, width), __shfl_up(x.pages, d, width)};
}

// inclusive prefix sums over the workgroup; `total` is the sum of all
__device__ __forceinline__ Sums block_scan(Sums v, Sums* wave_sums, Sums& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const Sums o = shifted(v, d, 64);
    if (lane >= d) v = v + o;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 63) wave_sums[wave] = v;
  __syncthreads();
  const int in_row = lane & (kScanWaves - 1);
  Sums sums = wave_sums[in_row];
#pragma unroll
  for (int d = 1; d < kScanWaves; d <<= 1) {
    const Sums o = shifted(sums, d, kScanWaves);
    if (in_row >= d) sums = sums + o;
  }
  total = {__shfl(sums.tokens, kScanWaves - 1), __shfl(sums.pages, kScanWaves - 1)};
  const int before = max(wave - 1, 0);
  const Sums b = {__shfl(sums.tokens, before), __shfl(sums.pages, before)};
  return wave > 0 ? v + b : v;
}

// slots of P tokens from t0
template <int P, typename Sums>
__device__ __forceinline__ void spread(const BlockTableArgs& a, FastDiv by_page, const Sums& sums, int t0) {
  int32_t slot[P];
  // the last request that begins at or before t0; n_seqs: behind the last token
  int lo = 0, hi = a.n_seqs + 1;
  while (lo < hi) {
    const int mid = (int)(((uint32_t)lo + (uint32_t)hi) >> 1);
    if (sums.start(mid) <= t0) lo = mid + 1;
    else hi = mid;
  }
  int r = lo - 1, loaded = -1, first = 0, cached = 0, held = 0, begin = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int t = t0 + i;
    while (r < a.n_seqs && sums.start(r + 1) <= t) ++r;
    slot[i] = -1;
    if (r >= a.n_seqs || t >= a.max_tokens) continue;
    if (r != loaded) {
      loaded = r;
      first = sums.first_page(r);
      begin = sums.start(r);
      if (first >= 0) {
        cached = sums.cached_len(r);
        held = (int)by_page.div((uint32_t)(cached + a.page_size - 1));
      }
    }
    if (first < 0) continue;
    const int pos = cached + (t - begin);
    const int col = (int)by_page.div((uint32_t)pos), off = pos - col * a.page_size;
    int page;
    if (col < held) {
      page = a.block_table[(int64_t)r * a.ld_table + col];
    } else {
      page = a.free_pages[first + (col - held)];
      if (off == 0) a.block_table[(int64_t)r * a.ld_table + col] = page;
    }
    const int64_t s = (int64_t)page * a.page_size + off;
    if (page >= 0 && s <= INT32_MAX) slot[i] = (int32_t)s;
  }
  int32_t* out = a.slot_map + t0;
  if constexpr (P == 4) {
    if (a.max_tokens - t0 >= P && (reinterpret_cast<uintptr_t>(out) & 15) == 0) {
      *reinterpret_cast<int4*>(out) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (i < a.max_tokens - t0) out[i] = slot[i];
}

// ONE: the only launch, of one or more workgroups.  OWN: the first of them places its threads' short requests right away.
// PER: neighbouring requests of a thread in a round.  P: neighbouring tokens of a thread
template <bool ONE, bool OWN, int PER, int P>
__global__ __launch_bounds__(kScanThreads) void kv_table_scan(BlockTableArgs a, FastDiv by_page) {
  __shared__ Sums sums[kScanWaves];
  __shared__ int32_t lds_starts[ONE ? kInLds + 1 : 1], lds_first[ONE ? kInLds : 1], lds_cached[ONE ? kInLds : 1];
  __shared__ unsigned long long taken;
  __shared__ int lds_many;  // whether some request brings more than kOwn tokens
  const bool writes = !ONE || blockIdx.x == 0;
  if (threadIdx.x == 0) {
    taken = 0;
    lds_many = !OWN;
  }
  const int64_t used = max(0, *a.free_used);
  const uint32_t up = (uint32_t)a.page_size - 1;
  Sums done = {0, 0};
  for (int64_t base = 0; base < a.n_seqs; base += kScanThreads * PER) {
    const int64_t r0 = base + threadIdx.x * PER;
    int cached[PER], news[PER], pages[PER];  // pages: the one that the first new token continues
    Sums mine = {0, 0};
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const bool in = r0 + k < a.n_seqs;
      cached[k] = in ? a.cached_lens[r0 + k] : 0;
      news[k] = in ? a.new_lens[r0 + k] : 0;
    }
    const int64_t limit = (int64_t)a.max_pages * a.page_size;
    auto valid = [&](int k) {
      return r0 + k < a.n_seqs && cached[k] >= 0 && news[k] >= 0 && (int64_t)cached[k] + news[k] <= limit;
    };
    auto pages_held = [&](int k) { return valid(k) ? by_page.div((uint32_t)cached[k] + up) : 0u; };
    // A request past the slot map's end is followed by such only, so that its pages, which are counted here though it
    // cannot have them, change nothing for those that fit.
    auto pages_needed = [&](int k) -> int64_t {
      return valid(k) ? by_page.div((uint32_t)cached[k] + (uint32_t)news[k] + up) - pages_held(k) : 0;
    };
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const uint32_t held = pages_held(k);
      pages[k] = -1;
      if constexpr (OWN) {
        if (writes && news[k] > 0 && held > 0) pages[k] = a.block_table[(r0 + k) * a.ld_table + held - 1];
      }
      mine = mine + Sums{max(news[k], 0), pages_needed(k)};
    }
    Sums sum;
    const Sums upto_mine = block_scan(mine, sums, sum);
    Sums to = {done.tokens + upto_mine.tokens - mine.tokens, done.pages + upto_mine.pages - mine.pages};
    done = done + sum;
    int64_t got = -1;  // pages gone with this thread's last request that gets any
    int32_t start[PER], first[PER], fresh[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t need = pages_needed(k), start_all = to.tokens, first_all = used + to.pages;
      to = to + Sums{max(news[k], 0), need};
      const bool served = valid(k) && to.tokens <= a.max_tokens && (need == 0 || used + to.pages <= a.n_free);
      start[k] = (int32_t)min(start_all, (int64_t)a.max_tokens);
      first[k] = served ? (int32_t)min(first_all, (int64_t)a.n_free) : -1;
      fresh[k] = -1;
      if (served && need > 0) {
        got = to.pages;
        if constexpr (OWN) {
          if (writes && news[k] <= kOwn) fresh[k] = a.free_pages[first[k]];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t r = r0 + k;
      if (r >= a.n_seqs) break;
      if (writes) {
        a.token_starts[r] = start[k];
        a.seq_lens[r] = first[k] >= 0 ? cached[k] + news[k] : cached[k];
        a.first_pages[r] = first[k];
      }
      if constexpr (ONE) {
        lds_starts[r] = start[k];
        lds_first[r] = first[k];
        lds_cached[r] = cached[k];
      }
      if constexpr (OWN) {
        if (news[k] > kOwn) {
          lds_many = 1;
        } else if (writes && news[k] > 0) {
          const int64_t held = pages_held(k), own = held * a.page_size;  // positions that held pages have
          if (first[k] >= 0 && pages_needed(k) > 0) a.block_table[r * a.ld_table + held] = fresh[k];
          for (int i = 0; i < news[k] && start[k] + i < a.max_tokens; ++i) {
            const int64_t pos = (int64_t)cached[k] + i, off = pos - (pos < own ? own - a.page_size : own);
            const int p = pos < own ? pages[k] : fresh[k];
            const int64_t slot = (int64_t)p * a.page_size + off;
            a.slot_map[start[k] + i] = first[k] >= 0 && p >= 0 && slot <= INT32_MAX ? (int32_t)slot : -1;
          }
        }
      }
    }
    // whoever gets pages comes before whoever does not: the last of them says how many are gone
    const uint64_t some = __ballot(got >= 0);
    if (some && (int)(threadIdx.x & 63) == 63 - __builtin_clzll(some))
      atomicMax(&taken, (unsigned long long)got);
  }
  __syncthreads();
  const int last = (int)min(done.tokens, (int64_t)a.max_tokens);
  if (writes && threadIdx.x == 0) {
    a.token_starts[a.n_seqs] = last;
    *a.free_used_out = (int32_t)(used + (int64_t)taken);
  }
  if constexpr (ONE) {
    if (OWN && !lds_many) {
      if (writes)
        for (int64_t t = (int64_t)last + threadIdx.x; t < a.max_tokens; t += kScanThreads) a.slot_map[t] = -1;
      return;
    }
    if (threadIdx.x == 0) lds_starts[a.n_seqs] = last;
    __syncthreads();
    const LdsSums all{lds_starts, lds_first, lds_cached};
    for (int64_t t0 = ((int64_t)blockIdx.x * kScanThreads + threadIdx.x) * P; t0 < a.max_tokens;
         t0 += (int64_t)gridDim.x * kScanThreads * P)
      spread<P>(a, by_page, all, (int)t0);
  }
}

// LDS: what is needed of the requests is loaded at once, not one dependent load after another
template <bool LDS>
__global__ __launch_bounds__(kSpreadThreads) void kv_table_spread(BlockTableArgs a, FastDiv by_page) {
  const WrittenSums all{a.token_starts, a.first_pages, a.seq_lens, a.new_lens};
  const int64_t t0 = ((int64_t)blockIdx.x * kSpreadThreads + threadIdx.x) * kPerThread;
  if constexpr (LDS) {
    __shared__ int32_t starts[kSpreadLds + 1], first[kSpreadLds], cached[kSpreadLds];
    for (int r = threadIdx.x; r <= a.n_seqs; r += kSpreadThreads) {
      starts[r] = all.start(r);
      if (r < a.n_seqs) {
        first[r] = all.first_page(r);
        cached[r] = all.cached_len(r);
      }
    }
    __syncthreads();
    if (t0 < a.max_tokens) spread<kPerThread>(a, by_page, LdsSums{starts, first, cached}, (int)t0);
  } else {
    if (t0 < a.max_tokens) spread<kPerThread>(a, by_page, all, (int)t0);
  }
}

}  // namespace

hipError_t launch_kv_block_table(const BlockTableArgs& a, hipStream_t stream) {
  const FastDiv by_page((uint32_t)a.page_size);
  const bool in_place = a.seq_lens == a.cached_lens || a.free_used_out == a.free_used;
  if (a.n_seqs <= kInLds && a.max_tokens <= (in_place ? kOneWorkgroup : kOneLaunch)) {
    // as few tokens to a thread as leave no more workgroups than CUs (1000 requests, 150 thousand tokens: 6.7 us with one
    // token, 7.3 with two, 8.6 with four; 4000 requests, 400 thousand tokens: 18, 11 and 12)
    const int most = in_place ? 1 : device_cu_count(), work = (a.max_tokens + kScanThreads - 1) / kScanThreads;
    auto launch = [&](auto own, auto per, auto p) {
      constexpr int P = decltype(p)::value;
      kv_table_scan<true, decltype(own)::value, decltype(per)::value, P>
          <<<in_place ? 1 : (work + P - 1) / P, kScanThreads, 0, stream>>>(a, by_page);
      return hipGetLastError();
    };
    auto spread_over = [&](auto own, auto per) {
      if (work <= most) return launch(own, per, std::integral_constant<int, 1>());
      if (work <= 2 * most) return launch(own, per, std::integral_constant<int, 2>());
      return launch(own, per, std::integral_constant<int, kPerThread>());
    };
    if (a.n_seqs > kScanThreads) return spread_over(std::false_type(), std::integral_constant<int, kMany>());
    if (a.max_tokens > kOwn * a.n_seqs) return spread_over(std::false_type(), std::integral_constant<int, 1>());
    return spread_over(std::true_type(), std::integral_constant<int, 1>());
  }
  if (a.n_seqs <= kScanThreads) kv_table_scan<false, false, 1, 1><<<1, kScanThreads, 0, stream>>>(a, by_page);
  else kv_table_scan<false, false, kMany, 1><<<1, kScanThreads, 0, stream>>>(a, by_page);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t per_block = (int64_t)kSpreadThreads * kPerThread;
  const int64_t blocks = ((int64_t)a.max_tokens + per_block - 1) / per_block;
  if (a.n_seqs <= kSpreadLds) kv_table_spread<true><<<(unsigned)blocks, kSpreadThreads, 0, stream>>>(a, by_page);
  else kv_table_spread<false><<<(unsigned)blocks, kSpreadThreads, 0, stream>>>(a, by_page);
  return hipGetLastError();
}

}  // namespace nvfp4
