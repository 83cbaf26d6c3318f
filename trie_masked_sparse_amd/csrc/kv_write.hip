// Norm of queries and keys for each head, rotation, and the keys and values
// into their pages, for gfx950.
//
// Every value is read once and written once, so memory bounds it: a wavefront
// takes one token and a few of its heads, a lane 16 bytes of a head, and
// nothing but the sum of squares (over a head's lanes) and the rotation's
// partner values (one exchange between lanes) leaves the registers.  The
// angles depend on the token and on the lane's place in the head only, so they
// are computed once for all heads of the wavefront, reduced to a turn in fp64:
// pos * inv_freq passes 10^5 and its fp32 product would be off by 10^-2.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kv_cache.h"
#include "tms.h"

namespace tms {
namespace {

constexpr int kWave = 64;

__device__ inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two floats rounded to nearest even into one word of bf16.
__device__ inline uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}

template <int DT>
struct Chunk;  // the values of 16 bytes
template <>
struct Chunk<0> {
  static constexpr int N = 4;
  static __device__ inline void unpack(const uint4& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y), x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
  }
  static __device__ inline uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Chunk<1> {
  static constexpr int N = 8;
  static __device__ inline void unpack(const uint4& r, float (&x)[8]) {
    x[0] = bf16_lo(r.x), x[1] = bf16_hi(r.x), x[2] = bf16_lo(r.y), x[3] = bf16_hi(r.y);
    x[4] = bf16_lo(r.z), x[5] = bf16_hi(r.z), x[6] = bf16_lo(r.w), x[7] = bf16_hi(r.w);
  }
  static __device__ inline uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
};

// What a token's row depends on: its sequence s, the number of offsets
// start[1..seqs] at or below t (seqs where there is none), and that sequence's
// first token and the one past its last, committed and held rows and status.  A small write is a chain of
// memory latencies, so every lane reads all of that of one sequence at once
// (only with more than 64 sequences, at most 4096, after a read of the
// blocks of 64).  Forks, drafts written into 8 layers and commits of 256
// sequences: 204 -> 200 us.
struct Place {
  int s, begin, end, length, held, status;
};
__device__ inline Place place_of(const KvCache& c, const int32_t* __restrict__ start, int t, int lane) {
  int block = 0;
  if (c.seqs > kWave) {
    const int coarse = (lane + 1) * kWave;  // last offset of block `lane`
    block = __popcll(__ballot(coarse <= c.seqs && start[min(coarse, c.seqs)] <= t));
  }
  const int mine = min(block * kWave + lane, c.seqs - 1);
  const int end = start[mine + 1], begin = start[mine], length = c.length[mine], held = c.held[mine], status = c.status[mine];
  const int n = __popcll(__ballot(block * kWave + lane < c.seqs && end <= t)), at = min(n, kWave - 1);
  return Place{block * kWave + n, __builtin_amdgcn_readlane(begin, at), __builtin_amdgcn_readlane(end, at),
               __builtin_amdgcn_readlane(length, at), __builtin_amdgcn_readlane(held, at),
               __builtin_amdgcn_readlane(status, at)};
}

// Heads that a wavefront has in flight: 64 / LPR of them to a load, kBatch
// loads before the first is used.
constexpr int kBatch = 4;

// DT: 0 fp32, 1 bf16.  LPR: lanes of a head.  One wavefront: token t, the
// groups of 64 / LPR heads g0, g0 + step, ...; heads are the queries', then
// the keys', then the values'.
// 12220 tokens of 32 query and 8 key heads of 128 in bf16: 74.8 us, 4.02 TB/s of
// the 4.93 that a plain copy reaches; 64 tokens 4.6 us, the chain of reads that
// ends in the row's page.
template <int DT, int LPR>
__global__ __launch_bounds__(256) void write_kernel(KvCache c, KvWrite a, int waves_per_token) {
  constexpr int N = Chunk<DT>::N, D = LPR * N, RPW = kWave / LPR;
  const int lane = threadIdx.x % kWave, wave = blockIdx.x * (256 / kWave) + threadIdx.x / kWave;
  const int t = __builtin_amdgcn_readfirstlane(wave / waves_per_token);
  if (t >= a.T) return;
  const int g0 = __builtin_amdgcn_readfirstlane(wave % waves_per_token) * RPW, step = waves_per_token * RPW;
  const int col = lane % LPR, sub = lane / LPR;  // chunk of the head, head of the group
  const int heads = a.q_heads + 2 * c.kv_heads, k_end = a.q_heads + c.kv_heads;
  const uint4* q = static_cast<const uint4*>(a.q) + int64_t(t) * (a.ldq / N) + col;
  const uint4* k = static_cast<const uint4*>(a.k) + int64_t(t) * (a.ldk / N) + col;
  const uint4* v = static_cast<const uint4*>(a.v) + int64_t(t) * (a.ldv / N) + col;
  auto load = [&](int h) {
    return h < a.q_heads ? q[h * LPR] : h < k_end ? k[(h - a.q_heads) * LPR] : v[(min(h, heads - 1) - k_end) * LPR];
  };
  const int groups = (heads - g0 + step - 1) / step;
  const bool rows = g0 + (groups - 1) * step + RPW - 1 >= a.q_heads;  // keys or values among them
  Place at{};
  if (rows) at = place_of(c, a.start, t, lane);
  uint4 raw[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u)
    if (g0 + u * step < heads) raw[u] = load(g0 + u * step + sub);
  // the angles of the lane's values: bf16 results leave no trace of the
  // hardware's sine (about 2^-20 off); fp32 ones take the library's
  const int first = col * N;
  const bool rotate = first < 2 * a.n_freq;
  float cs[N], sn[N];
  if (rotate && g0 < k_end) {
    const double pos = a.pos[t] * 0.15915494309189533577;  // in turns for a frequency of 1
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = first + i, f = a.interleaved ? e / 2 : (e < a.n_freq ? e : e - a.n_freq);
      double turn = pos * static_cast<double>(a.inv_freq[f]);
      turn -= rint(turn);
      if constexpr (DT == 1) {
        sn[i] = __builtin_amdgcn_sinf(static_cast<float>(turn));
        cs[i] = __builtin_amdgcn_cosf(static_cast<float>(turn));
      } else {
        sincospif(2.f * static_cast<float>(turn), &sn[i], &cs[i]);
      }
    }
  }
  // Where the token's keys and values go; null where they may not.  A sequence
  // is refused as a whole: wavefronts that read its status before and after one
  // of them sets it all decide alike.
  uint4* kv_row = nullptr;
  if (rows && at.s < c.seqs && at.status == TMS_OK) {
    const int64_t row = int64_t(at.length) + (t - at.begin), end = int64_t(at.length) + (min(at.end, a.T) - at.begin);
    if (t >= at.begin && end <= int64_t(min(at.held, c.max_pages)) << c.page_shift) {
      const int32_t* pages = c.table + int64_t(at.s) * c.max_pages;
      const int32_t p = pages[row >> c.page_shift];
      // the page that the committed rows end in may be others' too (a fork
      // without a reserve); the ones behind it never are
      const int32_t first = at.length & (c.page_tokens - 1) ? pages[at.length >> c.page_shift] : -1;
      const bool shared = first >= 0 && first < c.pages && c.refs[first] > 1;
      if (p >= 0 && p < c.pages && !shared)
        kv_row = static_cast<uint4*>(c.kv) +
                 ((int64_t(a.layer) * c.pages + p) * 2 * c.kv_heads * c.page_tokens + (row & (c.page_tokens - 1))) * LPR +
                 col;
    }
    if (!kv_row && lane == 0) c.status[at.s] = TMS_ERR_INVALID_ARG;
  }
  auto finish = [&](int h, uint4 r) {
    if (h >= heads) return;  // whole heads: the lanes that exchange values leave together
    const bool is_q = h < a.q_heads;
    if (h < k_end) {
      const void* weight = is_q ? a.q_weight : a.k_weight;
      float x[N];
      Chunk<DT>::unpack(r, x);
      if (weight) {
        float ss = 0.f, w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int d = 1; d < LPR; d *= 2) ss += __shfl_xor(ss, d);
        const float inv = 1.f / sqrtf(ss / D + a.eps);
        Chunk<DT>::unpack(static_cast<const uint4*>(weight)[col], w);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = x[i] * inv * w[i];
      }
      if (a.n_freq) {
        if (a.interleaved) {
          if (rotate) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
              const float lo = x[i], hi = x[i + 1];
              x[i] = lo * cs[i] - hi * sn[i];
              x[i + 1] = hi * cs[i] + lo * sn[i];
            }
          }
        } else {
          const int half = a.n_freq / N, lower = first < a.n_freq;
          const int other = lane + (rotate ? (lower ? half : -half) : 0);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float y = __shfl(x[i], other);
            if (rotate) x[i] = lower ? x[i] * cs[i] - y * sn[i] : x[i] * cs[i] + y * sn[i];
          }
        }
      }
      r = Chunk<DT>::pack(x);
    }
    if (is_q) static_cast<uint4*>(a.q_out)[(int64_t(t) * a.q_heads + h) * LPR + col] = r;
    else if (kv_row) kv_row[int64_t(h - a.q_heads) * c.page_tokens * LPR] = r;  // keys, then values of a page
  };
  for (int g = g0; g < heads; g += kBatch * step) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (g + u * step < heads) finish(g + u * step + sub, raw[u]);
    if (g + kBatch * step >= heads) break;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (g + (kBatch + u) * step < heads) raw[u] = load(g + (kBatch + u) * step + sub);
  }
}

template <int DT>
hipError_t launch(const KvCache& c, const KvWrite& a, hipStream_t s) {
  const int lpr = c.head_dim / Chunk<DT>::N, rpw = kWave / lpr;
  const int groups = (a.q_heads + 2 * c.kv_heads + rpw - 1) / rpw;
  // all loads of a wavefront at once; more wavefronts while they do not fill
  // the chip (4096: four on a SIMD)
  int64_t per = (groups + kBatch - 1) / kBatch;
  if (per * a.T < 4096) per = std::min<int64_t>(groups, (4096 + a.T - 1) / a.T);
  const int64_t grid = (int64_t(a.T) * per + 3) / 4;
  if (grid > (int64_t(1) << 24) - 1) return hipErrorInvalidValue;
  auto run = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), 256, 0, s>>>(c, a, static_cast<int>(per));
    return hipGetLastError();
  };
  switch (lpr) {
    case 8: return run(write_kernel<DT, 8>);
    case 16: return run(write_kernel<DT, 16>);
    case 32: return run(write_kernel<DT, 32>);
    default: return run(write_kernel<DT, 64>);
  }
}

}  // namespace

hipError_t launch_kv_write(const KvCache& c, const KvWrite& a, hipStream_t s) {
  return c.dtype == TMS_F32 ? launch<0>(c, a, s) : launch<1>(c, a, s);
}

}  // namespace tms
