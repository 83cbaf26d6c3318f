// Bounds of the keys of a page, and the choice of pages by them, for gfx950.
//
// Mathematics.  With lo and hi the lowest and highest value of each column of a
// page's keys, no key k of the page has a larger q k than
//     sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// and the sum of that over the query heads of a key head needs the heads' sums
// of max(q_d, 0) and min(q_d, 0) only: one row of products for all of them.
// A choice jumps where two scores cross, so scores are kept in fp64 all the way:
// the heads' sums of bf16 or fp32 queries are off by 2^-53 of them at most for each
// addition, and so is a score for each of its 2 D.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kv_tiles.h"

namespace tms {
namespace {

// The values of a 16-byte word as floats.
template <int DT>
struct Word {
  static constexpr int N = DT == 0 ? 4 : 8;
  static __device__ inline void unpack(u32x4 w, float (&x)[N]) {
    if constexpr (DT == 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
  }
  static __device__ inline u32x4 pack(const float (&x)[N]) {  // of values that have this type
    if constexpr (DT == 0) {
      return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    } else {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(x[2 * e]) >> 16 | (__float_as_uint(x[2 * e + 1]) & 0xffff0000u);
      return w;
    }
  }
};

// Lower and higher of two values; NaN where one is.
__device__ inline float lower(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ inline float higher(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// A wavefront takes the keys of one page, key head and layer: a lane the same
// columns of every RPI-th row.
//
// Bound by memory: 5 prompts of 1801 to 4100 tokens behind 0 to 1000, 8 key heads of
// 128, 8 layers (249 MB of keys and bounds) 47 us, 5.3 TB/s of the 6.1 that a
// plain read reaches.  A token each of 64 sequences, of which one in 64 fills a
// page, 4.4 us: the chain length, page number, keys.
template <int DT, int D>
__global__ __launch_bounds__(kBlock) void bounds_kernel(KvCache c, KvBounds b, int steps) {
  using W = Word<DT>;
  constexpr int CH = D / W::N, RPI = kWave / CH, kLoads = 8;  // words of a row, rows of a load
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int layer = blockIdx.z, h = blockIdx.y * kWaves + wave;
  const int s = blockIdx.x / steps;
  const int len = c.length[s], all = min(c.held[s], c.max_pages);
  if (h >= c.kv_heads || c.status[s] != TMS_OK || len <= 0) return;
  const int whole = min(len >> c.page_shift, all);
  const int n = b.n_new ? min(max(b.n_new[s], 0), len) : len;
  for (int j = ((len - n) >> c.page_shift) + blockIdx.x % steps; j < whole; j += steps) {
    const int page = c.table[int64_t(s) * c.max_pages + j];
    if (page < 0 || page >= c.pages) continue;
    const int64_t slot = (int64_t(layer) * c.pages + page) * c.kv_heads + h;
    const u32x4* keys = static_cast<const u32x4*>(c.kv) + (slot + (int64_t(layer) * c.pages + page) * c.kv_heads) * c.page_tokens * CH;
    float lo[W::N], hi[W::N];
    for (int r0 = 0; r0 < c.page_tokens; r0 += RPI * kLoads) {
      u32x4 w[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i)  // rows past the page's end: its last ones again
        w[i] = keys[min(r0 + i * RPI, c.page_tokens - RPI) * CH + lane];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        float x[W::N];
        W::unpack(w[i], x);
#pragma unroll
        for (int e = 0; e < W::N; ++e) {
          lo[e] = r0 || i ? lower(lo[e], x[e]) : x[e];
          hi[e] = r0 || i ? higher(hi[e], x[e]) : x[e];
        }
      }
    }
#pragma unroll
    for (int step = CH; step < kWave; step *= 2)
#pragma unroll
      for (int e = 0; e < W::N; ++e) {
        lo[e] = lower(lo[e], __shfl_xor(lo[e], step));
        hi[e] = higher(hi[e], __shfl_xor(hi[e], step));
      }
    u32x4* to = static_cast<u32x4*>(b.bounds) + slot * 2 * CH;
    if (lane < CH) to[lane] = W::pack(lo), to[CH + lane] = W::pack(hi);
  }
}

// ---------------------------------------------------------------- choice --

constexpr int kThreads = 512, kSelectWaves = kThreads / kWave;
constexpr int kHeld = 4096;   // keys that LDS holds: three workgroups on a compute unit, beside the bins
constexpr int kBins = 2048;
// Few lists are cut, as a workgroup reads 43 GB/s: 8 lists of 1875 pages in one
// piece 33 us, in pieces of 64 pages 16.  Many fill the chip by themselves, and the
// last piece's wait for the others costs more than it saves: 512 lists of up to 937
// pages 22 us in one piece, for 1024 and 2048 workgroups 26 and 33.
constexpr int kCutPages = 64;  // pages of a workgroup at least, where a list has several
constexpr int kLists = kWorkCounts / 4, kGroups = 512;  // lists that are cut (a counter each), workgroups then

// A score as an integer that orders as the score does, NaN above all.
constexpr uint64_t kAlways = 0xfff0000000000000ull;  // of infinity, and of the first and last pages
__device__ inline uint64_t order(double x) {
  if (x != x) return ~uint64_t(0);
  if (x == 0.) x = 0.;  // -0 and 0 are equal
  const uint64_t u = __double_as_longlong(x);
  return u >> 63 ? ~u : u | uint64_t(1) << 63;
}

// Of `Count` values of each of Lanes lanes the sums over the lanes, one of them
// in a lane: value lane % Count.  Each step halves the values that a lane has.
template <int Count, int Lanes>
__device__ inline double lane_sums(double (&v)[Count]) {
  const int lane = threadIdx.x % kWave;
  int step = 1;
#pragma unroll
  for (int n = Count; n > 1; n /= 2, step *= 2) {
    const bool odd = lane & step;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const double keep = odd ? v[2 * i + 1] : v[2 * i], give = odd ? v[2 * i] : v[2 * i + 1];
      v[i] = keep + __shfl_xor(give, step);
    }
  }
  double x = v[0];
#pragma unroll
  for (; step < Lanes; step *= 2) x += __shfl_xor(x, step);
  return x;
}

// Combines each lane's value with those of the lanes before it: the last lane
// has all of them.  from_lane gives 0 where there is none.
template <class F>
__device__ inline void along_lanes(F&& f) {
  f([](int x) { return from_lane<0x111, 0xf>(x); });  // 1, 2, 4 and 8 lanes down in rows of 16
  f([](int x) { return from_lane<0x112, 0xf>(x); });
  f([](int x) { return from_lane<0x114, 0xf>(x); });
  f([](int x) { return from_lane<0x118, 0xf>(x); });
  f([](int x) { return from_lane<0x142, 0xa>(x); });  // row 0 to row 1, row 2 to row 3
  f([](int x) { return from_lane<0x143, 0xc>(x); });  // lane 31 to rows 2 and 3
}

// Exclusive sums over the workgroup's threads; `sums` is free again behind the
// next barrier.
__device__ inline int thread_prefix(int mine, int* sums, int* total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int incl = mine;
  along_lanes([&](auto from) __attribute__((always_inline)) { incl += from(incl); });
  if (lane == kWave - 1) sums[wave] = incl;
  __syncthreads();
  int before = incl - mine;
  *total = 0;
  for (int w = 0; w < kSelectWaves; ++w) {
    if (w < wave) before += sums[w];
    *total += sums[w];
  }
  return before;
}

// A workgroup takes the pages of one token and key head, or one of up to `most`
// parts of them; the last of these to arrive chooses.
//
// Scores: the lanes share a page's 2 D bounds (or several pages', where they
// fit), and every lane keeps its columns' factors; the loads of the next pages
// are in flight during the sums.  Choice: the keys' range, from the lowest to the
// highest finite one, is cut into kBins bins, and the bin with the k-th highest
// again, until all of a bin are taken or it is one value.
//
// A call of few pages takes 8 us: offsets, table, bounds, sums, range, two rounds of
// bins and the output, one behind the other.  64 tokens behind 100 to 60000 rows, 8
// key heads of 128, 22 us, where their 43 MB would take 7: the longest lists' 937
// pages of 512 bytes, one workgroup each, end last.  Twice the loads in flight are
// slower (22 -> 30: registers).
template <int DT, int D>
__global__ __launch_bounds__(kThreads, 6) void select_kernel(KvCache c, KvSelect a, int most) {
  using W = Word<DT>;
  constexpr int CH = D / W::N, Two = 2 * CH;                       // words of the bounds of a page
  constexpr int Lanes = Two < kWave ? Two : kWave, Each = Two / Lanes, Pages = kWave / Lanes;
  constexpr int U = Each == 1 ? 4 : 2;                             // loads in flight of a lane, of pages
  __shared__ uint64_t held[kHeld];
  __shared__ uint32_t bins[kBins];
  __shared__ int sums[kSelectWaves], sums2[kSelectWaves];
  __shared__ uint32_t range[2];
  __shared__ int found, last_s, bin_s[3];
  const int cut = blockIdx.x % most, h = blockIdx.x / most % c.kv_heads, t = blockIdx.x / most / c.kv_heads;
  const int tid = threadIdx.x, wave = uniform(tid / kWave), lane = tid % kWave;
  for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
  if (tid == 0) found = -1, range[0] = range[1] = 0;
  __syncthreads();
  for (int s = tid; s < c.seqs; s += kThreads)
    if (a.a.start[s] <= t && t < a.a.start[s + 1]) found = s;
  __syncthreads();
  const int s = uniform(found);
  if (s < 0) return;  // a token of nobody: its list stays as it is
  const Seq q = sequence(c, a.a, s, 1, 1);
  const int whole = q.bad ? 0 : uniform(q.len) >> c.page_shift;
  int32_t* out = a.chosen + (int64_t(t) * c.kv_heads + h) * a.k;
  if (whole <= a.k) {  // all of them
    if (cut == 0)
      for (int i = tid; i < a.k; i += kThreads) out[i] = i < whole ? i : -1;
    return;
  }
  // pages [first, end) are chosen by their scores, the others always
  const int first = min(a.first, whole), end = max(whole - a.last, first);
  const int cuts = max(1, min(most, (end - first) / kCutPages));
  if (cut >= cuts) return;
  const int each = (((end - first + cuts - 1) / cuts) + 15) & ~15;
  const int from = min(first + cut * each, end), to = min(from + each, end);
  double* scores = static_cast<double*>(a.work) + (int64_t(t) * c.kv_heads + h) * c.max_pages;
  const bool in_lds = cuts == 1 && end - first <= kHeld;
  {
    const int group = a.a.q_heads / c.kv_heads, word = lane % Lanes;
    const float sign = a.a.scale < 0.f ? -1.f : 1.f;
    double f[Each][W::N];
#pragma unroll
    for (int i = 0; i < Each; ++i)
#pragma unroll
      for (int e = 0; e < W::N; ++e) f[i][e] = 0.;
    for (int g = 0; g < group; ++g) {
      const int64_t at = int64_t(t) * a.a.ldq + int64_t(h * group + g) * D;
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.a.q) + at * (DT == 0 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < Each; ++i) {
        float x[W::N];
        const int w = word + i * Lanes;
        W::unpack(p[w % CH], x);
#pragma unroll
        for (int e = 0; e < W::N; ++e) {
          const float y = a.a.scale == 0.f ? 0.f : x[e] * sign;
          f[i][e] += y != y ? y : w < CH ? fminf(y, 0.f) : fmaxf(y, 0.f);
        }
      }
    }
    const u32x4* bounds = static_cast<const u32x4*>(a.bounds) + (int64_t(a.a.layer) * c.pages * c.kv_heads + h) * Two;
    const int32_t* table = c.table + int64_t(s) * c.max_pages;
    constexpr int Step = U * Pages * kSelectWaves;  // pages of an iteration of the workgroup
    int page[U];
    u32x4 w[U][Each];
    auto look = [&](int j0) {
#pragma unroll
      for (int u = 0; u < U; ++u) page[u] = table[max(min(j0 + u * Pages + lane / Lanes, to - 1), 0)];
    };
    auto load = [&]() {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const u32x4* p = bounds + int64_t(max(0, min(page[u], c.pages - 1))) * c.kv_heads * Two + word;
#pragma unroll
        for (int i = 0; i < Each; ++i) w[u][i] = p[i * Lanes];
      }
    };
    int j0 = from + wave * U * Pages;
    if (j0 < to) {
      look(j0);
      load();
      look(j0 + Step);
    }
    for (; j0 < to; j0 += Step) {
      double sum[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        sum[u] = 0.;
#pragma unroll
        for (int i = 0; i < Each; ++i) {
          float x[W::N];
          W::unpack(w[u][i], x);
#pragma unroll
          for (int e = 0; e < W::N; ++e) sum[u] = fma(f[i][e], double(x[e]), sum[u]);
        }
      }
      load();
      look(j0 + 2 * Step);
      const double x = lane_sums<U, Lanes>(sum);
      const int j = j0 + word * Pages + lane / Lanes;
      if (word < U && j < to) {
        if (in_lds) held[j - first] = order(x);
        else if (cuts == 1) scores[j] = x;
        else __hip_atomic_store(reinterpret_cast<uint64_t*>(scores) + j, __double_as_longlong(x), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }
  const uint64_t* kept = reinterpret_cast<const uint64_t*>(scores);
  if (cuts > 1) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the scores are written
    __syncthreads();
    uint32_t* arrived = static_cast<uint32_t*>(c.work) + blockIdx.x / most;
    if (tid == 0) {
      last_s = atomicAdd(arrived, 1u) == uint32_t(cuts - 1);
      if (last_s) *arrived = 0;
    }
    __syncthreads();
    if (!last_s) return;
  }
  auto score = [&](int j) {
    return __longlong_as_double(cuts == 1 ? kept[j] : __hip_atomic_load(kept + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  };
  const int n = end - first;
  const bool fits = n <= kHeld;
  if (fits && !in_lds)
    for (int i = tid; i < n; i += kThreads) held[i] = order(score(first + i));
  __syncthreads();
  auto key = [&](int i) { return fits ? held[i] : order(score(first + i)); };
  // the range of the keys, of their upper 32 bits
  {
    uint32_t low = 0, high = 0;  // of the complements, for the lowest
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t x = key(i) >> 32;
      low = max(low, ~x), high = max(high, x);
    }
    along_lanes([&](auto from) __attribute__((always_inline)) {
      low = max(low, uint32_t(from(low))), high = max(high, uint32_t(from(high)));
    });
    if (lane == kWave - 1) atomicMax(&range[0], low), atomicMax(&range[1], high);
    __syncthreads();
  }
  // need: how many of the n are taken; a NaN comes before the pages that are
  // always chosen, which may be more than k
  const int always = whole - n;
  int need = a.k - always;
  uint64_t low = uint64_t(~range[0]) << 32, border = 0;
  const uint64_t high = uint64_t(range[1]) << 32 | 0xffffffffu;
  const bool plain = need > 0 && high < kAlways;
  int at = 0, always_taken = always;  // taken of the pages at the border, and of those always chosen
  if (need > 0 || high >= kAlways) {
    if (!plain) {
      // NaN first, then the always chosen and infinite ones by their place: the
      // number of NaN, and of infinite scores
      int nan = 0, inf = 0, all;
      for (int i = tid; i < n; i += kThreads) nan += key(i) > kAlways, inf += key(i) == kAlways;
      thread_prefix(nan, sums, &all);
      nan = all;
      thread_prefix(inf, sums2, &all);
      inf = all;
      __syncthreads();
      if (nan >= a.k) {  // of NaN only, the lowest
        border = ~uint64_t(0), at = a.k, always_taken = 0;
        need = 0;
      } else if (nan + inf + always >= a.k) {  // the border is among the infinite ones, by place
        border = kAlways, at = a.k - nan, always_taken = -1;
        need = 0;
      }
    }
    if (need > 0) {
      int left = need, span = 64 - __clzll((long long)((high - low) | 1));
      // keys in [low, low + 2^span) are looked at, `left` of them are taken
      for (;;) {
        const int shift = max(span - 11, 0);
        for (int i = tid; i < n; i += kThreads) {
          const uint64_t x = key(i) - low;  // below low: a large number
          if (key(i) >= low && (span >= 64 || x >> span == 0)) atomicAdd(&bins[x >> shift], 1u);
        }
        __syncthreads();
        // the bin with the `left`-th highest key: thread t has the bins from the
        // (4 t)-th highest on
        constexpr int Own = kBins / kThreads;
        int mine = 0, total;
        uint32_t b[Own];
#pragma unroll
        for (int i = 0; i < Own; ++i) b[i] = bins[kBins - 1 - (tid * Own + i)], mine += b[i];
        int before = thread_prefix(mine, sums, &total);
        if (before < left && before + mine >= left) {
#pragma unroll
          for (int i = 0; i < Own; ++i) {
            if (before < left && before + int(b[i]) >= left) bin_s[0] = kBins - 1 - (tid * Own + i), bin_s[1] = left - before, bin_s[2] = b[i];
            before += b[i];
          }
        }
        __syncthreads();
        low += uint64_t(bin_s[0]) << shift;
        left = bin_s[1];
        const bool done = shift == 0 || bin_s[2] == left;
        __syncthreads();
        if (done) {
          // all keys of the bin are taken, or `left` of equal ones
          if (shift == 0) border = low, at = left;
          else border = low - 1, at = 0;
          break;
        }
        span = shift;
        for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
        __syncthreads();
      }
    }
  } else {  // only of those that are always chosen: the lowest k
    border = ~uint64_t(0), at = 0, always_taken = a.k;
  }
  // ascending: a thread takes a run of pages; the ones at the border by place
  const bool by_place = always_taken < 0;  // the always chosen are at the border too
  const int run = (whole + kThreads - 1) / kThreads, r0 = min(tid * run, whole), r1 = min(r0 + run, whole);
  auto kind = [&](int j) {  // 2 taken, 1 at the border
    if (j < first || j >= end) return by_place ? 1 : 3;
    const uint64_t x = key(j - first);
    return x > border ? 2 : x == border && at > 0 ? 1 : 0;
  };
  int taken = 0, equal = 0, always_here = 0, all;
  for (int j = r0; j < r1; ++j) {
    const int x = kind(j);
    taken += x == 2, equal += x == 1, always_here += x == 3;
  }
  int e = 0, w = always_here;
  __syncthreads();
  if (at > 0 || always_taken != always) {  // by place
    const int before = thread_prefix(equal, sums, &all);
    e = min(max(at - before, 0), equal);
    const int always_before = thread_prefix(always_here, sums2, &all);
    w = min(max(always_taken - always_before, 0), always_here);
    __syncthreads();
  }
  int place = thread_prefix(taken + e + w, sums, &all);
  for (int j = r0; j < r1; ++j) {
    const int x = kind(j);
    if (x == 2 || (x == 1 && e-- > 0) || (x == 3 && w-- > 0)) out[place++] = j;
  }
}

template <int DT, int D>
hipError_t bounds(const KvCache& c, const KvBounds& b, hipStream_t s) {
  // pages that a sequence's new rows can make whole
  const int64_t most = b.n_new ? std::min<int64_t>((b.max_new >> c.page_shift) + 1, c.max_pages) : c.max_pages;
  const int64_t steps = std::min<int64_t>(most, std::max<int64_t>(1, (int64_t(1) << 22) / c.seqs));
  bounds_kernel<DT, D><<<dim3(unsigned(steps * c.seqs), (c.kv_heads + kWaves - 1) / kWaves, c.layers), kBlock, 0, s>>>(c, b, int(steps));
  return hipGetLastError();
}

template <int DT, int D>
hipError_t select(const KvCache& c, const KvSelect& a, hipStream_t s) {
  // long contexts of few tokens: a list by several workgroups
  const int64_t lists = int64_t(a.a.T) * c.kv_heads;
  const int most = lists > kLists ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(c.max_pages / kCutPages, kGroups / lists)));
  if (lists * most >= (int64_t(1) << 32) / kThreads) return hipErrorInvalidValue;
  select_kernel<DT, D><<<unsigned(lists * most), kThreads, 0, s>>>(c, a, most);
  return hipGetLastError();
}

}  // namespace

int64_t kv_select_work_bytes(const KvCache& c, int32_t T) { return int64_t(T) * c.kv_heads * c.max_pages * 8; }

hipError_t launch_kv_bounds(const KvCache& c, const KvBounds& b, hipStream_t s) {
  if (c.dtype == TMS_F32) return c.head_dim == 64 ? bounds<0, 64>(c, b, s) : c.head_dim == 128 ? bounds<0, 128>(c, b, s) : bounds<0, 256>(c, b, s);
  return c.head_dim == 64 ? bounds<1, 64>(c, b, s) : c.head_dim == 128 ? bounds<1, 128>(c, b, s) : bounds<1, 256>(c, b, s);
}

hipError_t launch_kv_select(const KvCache& c, const KvSelect& a, hipStream_t s) {
  if (c.dtype == TMS_F32) return c.head_dim == 64 ? select<0, 64>(c, a, s) : c.head_dim == 128 ? select<0, 128>(c, a, s) : select<0, 256>(c, a, s);
  return c.head_dim == 64 ? select<1, 64>(c, a, s) : c.head_dim == 128 ? select<1, 128>(c, a, s) : select<1, 256>(c, a, s);
}

}  // namespace tms
