// Bounds of the keys of a page, and the choice of pages by them, for gfx950.
//
// Mathematics.  With lo and hi the lowest and highest value of each column of a
// page's keys, no key k of the page has a larger q k than
//     sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// and the sum of that over the query heads of a key head needs the heads' sums
// of max(q_d, 0) and min(q_d, 0) only: one row of products for all of them.
// A choice jumps where two scores cross, so scores are not rounded on the way:
// products of bf16 and of fp32 are exact in fp64, where they are added.
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

// Sequence of token t, and what its list is chosen from: of `whole` pages the
// ones in [first, end) by their scores, the others always.
struct Range {
  int s, whole, first, end;
};

// All threads; ends with a barrier.
__device__ inline Range range_of(const KvCache& c, const KvSelect& a, int t) {
  __shared__ int found;
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  for (int s = threadIdx.x; s < c.seqs; s += blockDim.x)
    if (a.a.start[s] <= t && t < a.a.start[s + 1]) found = s;
  __syncthreads();
  Range r{uniform(found), 0, 0, 0};
  if (r.s < 0) return r;
  const Seq q = sequence(c, a.a, r.s, 1, 1);
  r.whole = q.bad ? 0 : uniform(q.len) >> c.page_shift;
  r.first = min(a.first, r.whole), r.end = max(r.whole - a.last, r.first);
  return r;
}

// Scores of a token and key head, [T][kv_heads][max_pages] in fp64.
__device__ inline double* scores(const KvCache& c, const KvSelect& a, int t, int h) {
  return static_cast<double*>(a.work) + (int64_t(t) * c.kv_heads + h) * c.max_pages;
}

// A wavefront takes pages of one token and key head: the lanes share a page's
// 2 D bounds (or several pages', where they fit).
template <int DT, int D>
__global__ __launch_bounds__(kBlock) void score_kernel(KvCache c, KvSelect a, int cuts) {
  using W = Word<DT>;
  constexpr int CH = D / W::N, Two = 2 * CH;                       // words of the bounds of a page
  constexpr int Lanes = Two < kWave ? Two : kWave, Each = Two / Lanes, Pages = kWave / Lanes;
  const int cut = blockIdx.x % cuts, h = blockIdx.x / cuts % c.kv_heads, t = blockIdx.x / cuts / c.kv_heads;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const Range r = range_of(c, a, t);
  if (r.s < 0 || r.whole <= a.k) return;
  const int group = a.a.q_heads / c.kv_heads, word = lane % Lanes;
  const float sign = a.a.scale < 0.f ? -1.f : a.a.scale == 0.f ? 0.f : 1.f;
  double f[Each][W::N];
#pragma unroll
  for (int i = 0; i < Each; ++i)
#pragma unroll
    for (int e = 0; e < W::N; ++e) f[i][e] = 0.;
  for (int g = 0; g < group; ++g) {
    const int64_t at = int64_t(t) * a.a.ldq + int64_t(h * group + g) * D;
    const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.a.q) + at * (DT == 0 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < Each; ++i) {
      float x[W::N];
      const int w = word + i * Lanes;
      W::unpack(q[w % CH], x);
#pragma unroll
      for (int e = 0; e < W::N; ++e) {
        const float y = sign == 0.f ? 0.f : x[e] * sign;
        f[i][e] += y != y ? y : w < CH ? fminf(y, 0.f) : fmaxf(y, 0.f);
      }
    }
  }
  const u32x4* bounds = static_cast<const u32x4*>(a.bounds) + (int64_t(a.a.layer) * c.pages * c.kv_heads + h) * Two;
  const int32_t* table = c.table + int64_t(r.s) * c.max_pages;
  double* out = scores(c, a, t, h);
  const int stride = cuts * kWaves * Pages;
  for (int j0 = r.first + (cut * kWaves + wave) * Pages; j0 < r.end; j0 += stride) {
    const int j = min(j0 + lane / Lanes, r.end - 1), page = max(0, min(table[j], c.pages - 1));
    const u32x4* p = bounds + int64_t(page) * c.kv_heads * Two + word;
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < Each; ++i) {
      float x[W::N];
      W::unpack(p[i * Lanes], x);
#pragma unroll
      for (int e = 0; e < W::N; ++e) sum = fma(f[i][e], double(x[e]), sum);
    }
#pragma unroll
    for (int step = 1; step < Lanes; step *= 2) sum += __shfl_xor(sum, step);
    if (word == 0) out[j] = sum;
  }
}

// A score as an integer that orders as the score does, NaN above all.
__device__ inline uint64_t order(double x) {
  if (x != x) return ~uint64_t(0);
  if (x == 0.) x = 0.;  // -0 and 0 are equal
  const uint64_t u = __double_as_longlong(x);
  return u >> 63 ? ~u : u | uint64_t(1) << 63;
}

constexpr int kPick = 256, kBins = 256;

// Workgroup of one token and key head: its list.  The pages above a border are
// taken, and of those at it the lowest: the border is found digit by digit.
__global__ __launch_bounds__(kPick) void pick_kernel(KvCache c, KvSelect a) {
  __shared__ uint32_t bins[kBins];
  __shared__ int sums[kPick / kWave];
  __shared__ uint64_t border_s;
  __shared__ int need_s;
  const int h = blockIdx.x % c.kv_heads, t = blockIdx.x / c.kv_heads, tid = threadIdx.x;
  const Range r = range_of(c, a, t);
  if (r.s < 0) return;
  int32_t* out = a.chosen + (int64_t(t) * c.kv_heads + h) * a.k;
  if (r.whole <= a.k) {
    for (int i = tid; i < a.k; i += kPick) out[i] = i < r.whole ? i : -1;
    return;
  }
  const double* in = scores(c, a, t, h);
  constexpr uint64_t kAlways = 0xfff0000000000000ull;  // order(infinity)
  auto key = [&](int j) { return j < r.first || j >= r.end ? kAlways : order(in[j]); };
  // border: the k-th highest key.  Keys whose digits above `shift` are prefix's
  // are looked at
  uint64_t prefix = 0;
  int need = a.k;  // how many of them are taken
  for (int shift = 56;; shift -= 8) {
    bins[tid] = 0;
    __syncthreads();
    for (int j = tid; j < r.whole; j += kPick) {
      const uint64_t x = key(j);
      if (shift == 56 || x >> (shift + 8) == prefix) atomicAdd(&bins[x >> shift & 255], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      int left = need, d = kBins - 1;
      for (; left > int(bins[d]); --d) left -= bins[d];
      border_s = d, need_s = left;
    }
    __syncthreads();
    prefix = prefix << 8 | border_s;
    need = need_s;
    __syncthreads();
    if (shift == 0) break;
  }
  // in ascending order: a page is taken above the border, or at it among the first `need`
  int before = 0, equal_before = 0;  // taken, and at the border
  for (int j0 = 0; j0 < r.whole; j0 += kPick) {
    const int j = j0 + tid, lane = tid % kWave, wave = tid / kWave;
    const uint64_t x = j < r.whole ? key(j) : 0;
    const bool equal = j < r.whole && x == prefix;
    auto rank = [&](bool on, int& total) {
      const uint64_t all = __ballot(on);
      __syncthreads();
      if (lane == 0) sums[wave] = __popcll(all);
      __syncthreads();
      int n = __popcll(all & ((uint64_t(1) << lane) - 1));
      total = 0;
      for (int w = 0; w < kPick / kWave; ++w) {
        if (w < wave) n += sums[w];
        total += sums[w];
      }
      return n;
    };
    int equals, takes;
    const int at_border = equal_before + rank(equal, equals);
    const bool take = j < r.whole && (x > prefix || (equal && at_border < need));
    const int place = before + rank(take, takes);
    if (take) out[place] = j;
    before += takes, equal_before += equals;
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
  const int64_t lists = int64_t(a.a.T) * c.kv_heads;
  const int cuts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(c.max_pages / 32, 1024 / lists)));
  if (lists * cuts >= (int64_t(1) << 32) / kBlock) return hipErrorInvalidValue;
  score_kernel<DT, D><<<unsigned(lists * cuts), kBlock, 0, s>>>(c, a, cuts);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  pick_kernel<<<unsigned(lists), kPick, 0, s>>>(c, a);
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
