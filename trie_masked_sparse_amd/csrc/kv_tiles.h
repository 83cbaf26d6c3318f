// Device helpers that the attention kernels over the paged cache share: matrix
// operands, copies into LDS, who sees which new row, values that are not finite,
// parts of a row that are joined.
#pragma once
#include <hip/hip_runtime.h>

#include "kv_cache.h"
#include "tms.h"

namespace tms {
namespace {

constexpr int kWave = 64, kWaves = 4, kBlock = kWave * kWaves;
constexpr int kTree = 1024, kTreeWords = kTree / 32 + 1;  // drafts of a tree; words of 32 keys they may touch
constexpr int kMixedWords = kTreeWords + 2;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef const __attribute__((address_space(3))) u32x4* lds_u32x4;
typedef const __attribute__((address_space(4))) int32_t* const_i32;  // read through the scalar cache

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Workgroup barrier that orders LDS only: global loads stay in flight across it.
__device__ inline void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A value that is the same in all lanes, in scalar registers.
__device__ inline int64_t uniform(int64_t x) {
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
  return static_cast<int64_t>(uint64_t(hi) << 32 | uint32_t(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x))));
}
__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// 16 bytes for each lane from address `from` + `offset` (per lane) to LDS: lane i's go
// to byte `to` + 16 i.  The compiler does not see the copy: wait_copies, then
// a barrier, before LDS is read.
__device__ inline void copy_to_lds(int64_t from, int offset, int to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(uniform(to)), "v"(offset),
               "s"(uniform(from))
               : "memory", "m0");
}
// All copies but the last N of this wavefront are in LDS.
template <int N>
__device__ inline void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The value of a lane before this one (DPP control), 0 where there is none.
template <int Control, int Rows>
__device__ inline int from_lane(int x) {
  return __builtin_amdgcn_update_dpp(0, x, Control, Rows, 0xf, false);
}

// Maximum and sum over the 4 lanes of a query row (lane % 16).
__device__ inline float row_max(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ inline float row_sum(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ inline uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}

// 8 weights cut to bf16, and what that leaves of them, rounded: together within
// 2^-15 of each.  Of a weight that is not 0 both are above 0 (2^-24 of it is
// added for that), so an infinite value times them is infinite.
__device__ inline void split_bf16(const float (&x)[8], u32x4* high, u32x4* low) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __float_as_uint(x[2 * i]), b = __float_as_uint(x[2 * i + 1]) & 0xffff0000u;
    (*high)[i] = b | a >> 16;
    (*low)[i] = pack_bf16(fmaf(x[2 * i], 0x1p-24f, x[2 * i] - __uint_as_float(a & 0xffff0000u)),
                          fmaf(x[2 * i + 1], 0x1p-24f, x[2 * i + 1] - __uint_as_float(b)));
  }
}

// 4 values at element i of an output.
template <int DT>
__device__ inline void store4(void* out, int64_t i, f32x4 x) {
  if constexpr (DT == 1)
    *reinterpret_cast<u32x2*>(static_cast<char*>(out) + i * 2) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
  else
    *reinterpret_cast<f32x4*>(static_cast<char*>(out) + i * 4) = x;
}

// a / b of values that are not negative: the division of 64-bit integers is some 150
// instructions, and stands several times in the start of a workgroup.
__device__ inline int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

struct Seq {
  int begin, n, len, rows_tiles, key_tiles;  // tokens, committed rows; key_tiles 1 where bad
  int bad;                                   // the outputs are NaN
};

// Rows of a sequence at most: row numbers are 32 bits, and the kernels count on
// from the last one to the end of its row tile (256) and of the key tiles that
// copies are planned for (four of 64).
constexpr int64_t kMostRows = (int64_t(1) << 31) - 1024;

__device__ inline Seq sequence(const KvCache& c, const KvAttention& a, int s, int rows, int keys) {
  Seq q{};
  q.begin = a.start[s];
  const int end = a.start[s + 1];
  q.n = end - q.begin;
  if (q.begin < 0 || end > a.T || q.n <= 0) q.n = 0;
  q.len = c.length[s];
  const int64_t all = int64_t(q.len) + q.n;
  q.bad = c.status[s] != TMS_OK || q.n > a.max_new || q.len < 0 ||
          all > min(int64_t(min(c.held[s], c.max_pages)) << c.page_shift, kMostRows);
  const int64_t r = int64_t(q.n) * (a.q_heads / c.kv_heads);
  q.rows_tiles = static_cast<int>((r + rows - 1) / rows);
  q.key_tiles = q.bad ? 1 : static_cast<int>((all + keys - 1) / keys);
  return q;
}

__device__ inline Seq uniform(const Seq& q) {
  return Seq{uniform(q.begin), uniform(q.n), uniform(q.len), uniform(q.rows_tiles), uniform(q.key_tiles), uniform(q.bad)};
}

// Drafts of the tokens tok0 .. tok1 of a sequence: for each one bit a key from
// key (len & ~31) on, set for committed rows and for the drafts on its walk to
// the root.  Ends with a barrier.
// words: of a token, at least (drafts + 31) / 32 + 1.
template <int Threads>
__device__ inline void walk_tree(const KvAttention& a, const Seq& q, int tok0, int tok1, int32_t* par, uint32_t* seen,
                                 int words) {
  const int tid = threadIdx.x, low = q.len & 31;
  for (int i = tid; i < q.n; i += Threads) par[i] = a.parent[q.begin + i];
  for (int i = tid; i < (tok1 - tok0 + 1) * words; i += Threads) seen[i] = i % words ? 0 : (1u << low) - 1;
  __syncthreads();
  if (tid <= tok1 - tok0)
    for (int j = tok0 + tid; j >= 0;) {
      const int bit = low + j, p = par[j];
      seen[tid * words + (bit >> 5)] |= 1u << (bit & 31);
      j = p < j ? p : -1;
    }
  __syncthreads();
}

// New rows of a segment that some of its query rows see and others do not: keys
// first .. first + count - 1, the last of them also because its copies fill up
// its tile, which no row sees.  A value there that is not finite would reach all
// rows of a product, as 0 x inf or 0 x NaN.  So a segment whose outputs are not
// all finite is worked through once more: such values are looked for, taken out
// of the tiles in LDS, and added to the rows that see them at the end (looking
// for them in every segment before its first tile took 4 % of a prompt's time).
// bits: one bit a key from key (first & ~31) on, set where a row has such a
// value (also for the copies of the last row that fill up its tile).
struct Mixed {
  int first, count;
  uint32_t* bits;

  __device__ uint32_t word(int at) const {  // of the keys at .. at + 31, at a multiple of 32
    const int i = (at - (first & ~31)) >> 5;
    return i >= 0 && i < kMixedWords ? bits[i] : 0u;
  }
};
__device__ inline Mixed mixed_rows(const KvAttention& a, const Seq& q, int tok0, int tok1, uint32_t* bits) {
  return a.parent ? Mixed{q.len, q.n, bits} : Mixed{q.len + tok0, tok1 - tok0 + 1, bits};
}

// 0, or NaN where a value is not finite.
template <typename V, int N>
__device__ inline float zero_or_nan(const V (&x)[N], float z = 0.f) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < int(sizeof(V) / 4); ++e) z = fmaf(x[i][e], 0.f, z);
  return z;
}

// The values of a 16-byte word that are not finite, or the ones that are; 0 in
// the others' places.
template <int DT>
__device__ inline uint32_t keep_finite(uint32_t w, bool finite) {
  if constexpr (DT == 0) return ((w & 0x7f800000u) != 0x7f800000u) == finite ? w : 0u;
  const uint32_t low = ((w & 0x7f80u) != 0x7f80u) == finite ? 0xffffu : 0u;
  return w & (low | (((w & 0x7f800000u) != 0x7f800000u) == finite ? 0xffff0000u : 0u));
}
template <int DT>
__device__ inline u32x4 keep_finite(u32x4 w, bool finite) {
  return u32x4{keep_finite<DT>(w[0], finite), keep_finite<DT>(w[1], finite), keep_finite<DT>(w[2], finite),
               keep_finite<DT>(w[3], finite)};
}

// The values from column `at` (a multiple of 4) on of a V row that are not finite.
template <int DT>
__device__ inline f32x4 odd_values(const u32x4* row, int at) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(row) + (DT == 0 ? at : at / 2);
  f32x4 x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (DT == 0) x[e] = __uint_as_float(keep_finite<DT>(w[e], false));
    else x[e] = __uint_as_float(e % 2 ? keep_finite<DT>(w[e / 2], false) & 0xffff0000u : keep_finite<DT>(w[e / 2], false) << 16);
  }
  return x;
}

// Page of a key: from a table of the keys' pages, or as a function says.
__device__ inline int key_page(const KvCache& c, const int32_t* table, int key) {
  return max(0, min(table[key >> c.page_shift], c.pages - 1));
}
template <class PageAt>
__device__ inline int key_page(const KvCache&, const PageAt& page_at, int key) {
  return page_at(key);
}

// Address of the V row of a key.
template <class Table>
__device__ inline const u32x4* value_row(const KvCache& c, const Table& table, const u32x4* values, int64_t page_stride,
                                         int ch, int row) {
  const int page = key_page(c, table, row);
  return values + page * page_stride + int64_t(row & (c.page_tokens - 1)) * ch;
}

// Sets m.bits; whether any is set.  Ends with a barrier.
template <int Threads, int DT, int D, class Table>
__device__ inline bool find_nonfinite(const KvCache& c, const Table& table, const u32x4* values, int64_t page_stride,
                                      const Mixed& m) {
  constexpr int CH = D * (DT == 0 ? 4 : 2) / 16, kFill = 63;
  const int tid = threadIdx.x, lane = tid % kWave;
  for (int i = tid; i < kMixedWords; i += Threads) m.bits[i] = 0;
  __syncthreads();
  for (int i = tid; i < m.count * CH; i += Threads) {
    const int row = m.first + i / CH;
    const u32x4 w = value_row(c, table, values, page_stride, CH, row)[i % CH], odd = keep_finite<DT>(w, false);
    if (odd[0] | odd[1] | odd[2] | odd[3]) {
      const int last = i / CH + 1 == m.count ? row + kFill : row;
      for (int r = row; r <= last; ++r) atomicOr(&m.bits[(r - (m.first & ~31)) >> 5], 1u << (r & 31));
    }
  }
  __syncthreads();
  return __any(lane < kMixedWords && m.bits[min(lane, kMixedWords - 1)] != 0);
}

// Keys first .. first+31 (first a multiple of 32 in the tree's region) that
// token tok sees, one bit each.
__device__ inline uint32_t sees(const KvAttention& a, const Seq& q, int tok, int tok0, int first, const uint32_t* seen,
                                int words) {
  if (a.parent) return seen[max(tok - tok0, 0) * words + ((first - (q.len & ~31)) >> 5)];
  const int count = q.len + tok + 1 - first;
  return count >= 32 ? ~0u : (1u << max(count, 0)) - 1;
}

// Parts that another workgroup of the same launch reads go past the XCD's L2,
// by device-scope accesses: a fence would write back and drop all of it
// (measured: 64 ragged sequences 53 -> 188 us).
template <bool Shared, typename T>
__device__ inline T part_load(const T* p) {
  if constexpr (!Shared) {
    return *p;
  } else if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __hip_atomic_load(reinterpret_cast<const uint32_t*>(p), __ATOMIC_RELAXED,
                                                   __HIP_MEMORY_SCOPE_AGENT));
  } else {
    uint64_t w[2];
    for (int i = 0; i < 2; ++i)
      w[i] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p) + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    T x;
    __builtin_memcpy(&x, w, 16);
    return x;
  }
}
template <bool Shared>
__device__ inline void part_store(float* p, float x) {
  if constexpr (Shared)
    __hip_atomic_store(reinterpret_cast<uint32_t*>(p), __float_as_uint(x), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  else
    *p = x;
}
template <bool Shared>
__device__ inline void part_store(f32x4* p, f32x4 x) {
  if constexpr (Shared) {
    uint64_t w[2];
    __builtin_memcpy(w, &x, 16);
    for (int i = 0; i < 2; ++i)
      __hip_atomic_store(reinterpret_cast<uint64_t*>(p) + i, w[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  } else {
    *p = x;
  }
}

// Weight 2^x of a part (or half) of a row's keys beside the others.  Never 0: a
// draft's infinite value stays infinite however little its part weighs, and
// finite ones do not notice 2^-126.
__device__ inline float part_weight(float x) { return fmaxf(exp2_fast(x), 0x1p-126f); }

// Geometry of a wavefront's key tile by type.
template <int DT, int D>
struct Tile;
template <int D>
struct Tile<1, D> {                      // bf16
  static constexpr int Keys = 32, Sub = 2;  // two 16-key halves
  static constexpr uint32_t Mask = ~0u;     // of a word of 32 keys
  static constexpr int Loads = D / 32;      // 16-byte words of a key for each lane
  static constexpr int Chunks = D / 8;      // 16-byte words of a row
  // place of word c of key r in the LDS tile: the transposing read takes 2
  // words of 8 keys at once, from different banks.  Of the cycles that LDS works
  // 32 % are conflicts all the same (64 ragged tokens); it works 7 % of the time.
  static __device__ inline int at(int r, int c) {
    const int f = D == 64 ? (r & 6) | (r >> 3 & 1) : (r & 7) << 1 | (r >> 3 & 1);
    return r * Chunks + (c ^ f);
  }
};
template <int D>
struct Tile<0, D> {                      // fp32
  static constexpr int Keys = 16, Sub = 1;
  static constexpr uint32_t Mask = 0xffffu;
  static constexpr int Loads = D / 16;
  static constexpr int Chunks = D / 4;
  static __device__ inline int at(int r, int c) { return r * Chunks + (c ^ (r & 15)); }
};

}  // namespace
}  // namespace tms
