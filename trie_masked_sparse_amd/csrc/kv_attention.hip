// Attention of new tokens (one, a tree of drafts, a whole prompt) over the
// paged key/value cache, for gfx950.
//
// Mathematics.  The query rows of a sequence that share a key head are taken
// together (row = token * group + query head of the group).  With c = |scale|
// log2(e) and the sign of the scale moved into q, a row's weights are
// exp2(c s - m), s = q k; m (the running maximum of c s), l (the sum of the
// weights) and the output are kept in fp32 and rescaled when m grows; parts of
// a row's keys are joined by the same rule.
//
// Layout of the products.  S^T = K Q^T comes out of the matrix cores with a
// query row in each lane (lane % 16) and 4 adjacent keys in its registers,
// which is the operand layout that O^T = V^T P^T wants for P^T: the weights go
// from one product into the next without leaving the lane, and a row's
// maximum, sum and rescaling factor are one register of its lanes.  V^T comes
// from a row-major tile in LDS: bf16 through the transposing read (4 keys of
// one column to a lane), fp32 through one word per key.
#include <hip/hip_runtime.h>

#include "kv_cache.h"
#include "tms.h"

namespace tms {
namespace {

constexpr int kWave = 64, kWaves = 4, kBlock = kWave * kWaves;
constexpr int kTree = 1024, kTreeWords = kTree / 32 + 1;  // drafts of a tree; words of 32 keys they may touch

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

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

// ------------------------------------------------------------------ plan --

// What a launch works on.  A segment is the row tile of one key head of one
// sequence; its keys are cut into tiles.  All tiles in the order (sequence,
// key head, row tile, key tile) are dealt to the workgroups in equal
// contiguous shares, so ragged batches and long contexts balance by
// themselves; a segment that does not lie in one share is joined by
// combine_kernel.
struct Seq {
  int begin, n, len, rows_tiles, key_tiles;  // tokens, committed rows; key_tiles 1 where bad
  bool bad;                                  // the outputs are NaN
};

__device__ inline Seq sequence(const KvCache& c, const KvAttention& a, int s, int rows, int keys) {
  Seq q{};
  q.begin = a.start[s];
  const int end = a.start[s + 1];
  q.n = end - q.begin;
  if (q.begin < 0 || end > a.T || q.n <= 0) q.n = 0;
  q.len = c.length[s];
  const int64_t all = int64_t(q.len) + q.n;
  q.bad = c.status[s] != TMS_OK || q.n > a.max_new || q.len < 0 ||
          all > int64_t(min(c.held[s], c.max_pages)) << c.page_shift;
  const int64_t r = int64_t(q.n) * (a.q_heads / c.kv_heads);
  q.rows_tiles = static_cast<int>((r + rows - 1) / rows);
  q.key_tiles = q.bad ? 1 : static_cast<int>((all + keys - 1) / keys);
  return q;
}

__device__ inline int64_t tiles_of(const KvCache& c, const Seq& q) {
  return int64_t(q.rows_tiles) * q.key_tiles * c.kv_heads;
}

// A segment that several workgroups share, written by the one it starts in.
struct Join {
  int32_t s, h, rt, last;  // last: the last workgroup that holds a part (-1: nothing to join)
};

// Work memory: Join [shares], then for every share two parts (its first and
// its last segment) of kRows rows: maximum and sum of every row, then the
// unnormalised outputs in the lanes' order.
__host__ __device__ inline int64_t round256(int64_t x) { return (x + 255) & ~int64_t(255); }
__host__ __device__ inline int64_t part_floats(int rows, int dim) { return int64_t(rows) * (dim + 2); }

constexpr int kShares = 512;
constexpr int64_t kPartFloats = 64 * (128 + 2) > 32 * (256 + 2) ? 64 * (128 + 2) : 32 * (256 + 2);

__device__ inline Join* joins(const KvCache& c) { return static_cast<Join*>(c.work); }
__device__ inline float* part(const KvCache& c, int share, int which, int64_t floats) {
  return reinterpret_cast<float*>(static_cast<char*>(c.work) + round256(kShares * int64_t(sizeof(Join)))) +
         (2 * int64_t(share) + which) * floats;
}

// First tile of a share of the `total` tiles, and the share that a tile is in.
__device__ inline int64_t share_begin(int64_t total, int shares, int w) { return total * w / shares; }
__device__ inline int share_of(int64_t total, int shares, int64_t tile) {
  int w = static_cast<int>(tile * shares / total);
  while (w + 1 < shares && share_begin(total, shares, w + 1) <= tile) ++w;
  return w;
}

// ------------------------------------------------- few rows: token, drafts --

// Geometry of a wavefront's key tile by type.
template <int DT, int D>
struct Tile;
template <int D>
struct Tile<1, D> {                      // bf16
  static constexpr int Keys = 32, Sub = 2;  // two 16-key halves
  static constexpr int Loads = D / 32;      // 16-byte words of a key for each lane
  static constexpr int Chunks = D / 8;      // 16-byte words of a row
  // place of word c of key r in the LDS tile: the transposing read takes 2
  // words of 8 keys at once and the write 1 word of 8 keys, without conflicts
  static __device__ inline int at(int r, int c) {
    const int f = D == 64 ? (r & 6) | (r >> 3 & 1) : (r & 7) << 1 | (r >> 3 & 1);
    return r * Chunks + (c ^ f);
  }
};
template <int D>
struct Tile<0, D> {                      // fp32
  static constexpr int Keys = 16, Sub = 1;
  static constexpr int Loads = D / 16;
  static constexpr int Chunks = D / 4;
  static __device__ inline int at(int r, int c) { return r * Chunks + (c ^ (r & 15)); }
};

// Workgroup of 4 wavefronts over the segments of its share.  Each wavefront
// holds all rows of the segment and takes every 4th key tile: K straight into
// registers, V through its own part of LDS, no barrier among them; the next
// tile's loads are in flight during the softmax and the second product.
template <int DT, int D, int MT>
__global__ __launch_bounds__(kBlock) void few_rows_kernel(KvCache c, KvAttention a, int shares) {
  using T = Tile<DT, D>;
  constexpr int M = 16 * MT, KW = T::Keys, DB = D / 16, L = T::Loads;
  constexpr int kVWords = KW * T::Chunks;                  // 16-byte words of a V tile
  constexpr int kLds = kWaves * kVWords > kWaves * M * D / 4 ? kWaves * kVWords : kWaves * M * D / 4;
  __shared__ u32x4 lds[kLds];
  __shared__ float stat[kWaves][2][M];
  __shared__ uint32_t seen[M][kTreeWords];
  __shared__ int32_t par[kTree];
  __shared__ int64_t scan[kWaves];
  __shared__ int found_s;
  __shared__ int64_t found_base;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
  const int col = lane % 16, g = lane / 16;
  const int group = a.q_heads / c.kv_heads;
  // a scale of 0 clears q instead: a masked score stays -inf
  const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
  const uint32_t flip = a.scale < 0.f ? (DT == 0 ? 0x80000000u : 0x80008000u) : 0u, on = a.scale == 0.f ? 0u : ~0u;

  // share: prefix sums of the sequences' tiles
  int64_t mine = 0, total = 0, before = 0;
  const int each = (c.seqs + kBlock - 1) / kBlock;
  for (int i = 0; i < each; ++i) {
    const int s = tid * each + i;
    if (s < c.seqs) mine += tiles_of(c, sequence(c, a, s, M, KW));
  }
  {
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const int64_t o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == kWave - 1) scan[wave] = incl;
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) {
      if (i < wave) before += scan[i];
      total += scan[i];
    }
    before += incl - mine;
  }
  // at least one tile for every wavefront
  shares = static_cast<int>(max(int64_t(1), min(int64_t(shares), total / kWaves)));
  const int me = blockIdx.x;
  if (tid == 0) joins(c)[me] = Join{0, 0, 0, -1};
  if (me >= shares || total == 0) return;
  int64_t lo = share_begin(total, shares, me);
  const int64_t hi = share_begin(total, shares, me + 1);
  if (lo >= before && lo < before + mine) {
    int64_t base = before;
    for (int s = tid * each;; ++s) {
      const int64_t t = tiles_of(c, sequence(c, a, s, M, KW));
      if (lo < base + t) {
        found_s = s;
        found_base = base;
        break;
      }
      base += t;
    }
  }
  __syncthreads();
  int s = found_s;
  int64_t base = found_base;
  Seq q = sequence(c, a, s, M, KW);

  while (lo < hi) {
    while (lo >= base + tiles_of(c, q)) {
      base += tiles_of(c, q);
      q = sequence(c, a, ++s, M, KW);
    }
    const int64_t off = lo - base;
    const int seg = static_cast<int>(off / q.key_tiles), kt0 = static_cast<int>(off % q.key_tiles);
    const int h = seg / q.rows_tiles, rt = seg % q.rows_tiles;
    const int kt1 = static_cast<int>(min(int64_t(q.key_tiles), kt0 + hi - lo));
    const int rows = q.n * group;  // of the sequence and key head
    const int all = q.len + q.n;
    // the queries: B operand, row = lane % 16
    u32x4 qr[MT][L];
    int tok[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = rt * M + m * 16 + col;
      tok[m] = r < rows ? r / group : -1;
      const int64_t at = int64_t(q.begin + max(tok[m], 0)) * a.ldq + int64_t(h * group + (r < rows ? r % group : 0)) * D;
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + at * (DT == 0 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < L; ++i) {
        qr[m][i] = (p[i * 4 + g] ^ flip) & on;
      }
    }
    const int tok0 = rt * M / group, tok1 = min(q.n - 1, (rt * M + M - 1) / group);  // tokens of the tile
    const int limit = a.parent ? all : q.len + tok1 + 1;                             // keys that any row sees
    const int end = min(kt1, (limit + KW - 1) / KW);
    const int base32 = q.len & ~31;  // key of bit 0 of the words of `seen`
    if (a.parent && !q.bad && end * KW > q.len) {
      // who sees whom: for each token of the tile one bit a key from base32
      // on, set for committed rows and for the drafts on its walk to the root
      for (int i = tid; i < q.n; i += kBlock) par[i] = a.parent[q.begin + i];
      for (int i = tid; i < (tok1 - tok0 + 1) * kTreeWords; i += kBlock)
        seen[i / kTreeWords][i % kTreeWords] = i % kTreeWords ? 0 : (1u << (q.len - base32)) - 1;
      __syncthreads();
      if (tid <= tok1 - tok0)
        for (int j = tok0 + tid; j >= 0;) {
          const int bit = q.len - base32 + j, p = par[j];
          seen[tid][bit >> 5] |= 1u << (bit & 31);
          j = p < j ? p : -1;
        }
      __syncthreads();
    }

    f32x4 o[MT][DB];
    float mx[MT], sum[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mx[m] = -INFINITY, sum[m] = 0.f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int32_t* table = c.table + int64_t(s) * c.max_pages;
    const int64_t head_stride = int64_t(c.page_tokens) * T::Chunks;  // 16-byte words
    const u32x4* kv = static_cast<const u32x4*>(c.kv) +
                      (int64_t(a.layer) * c.pages * 2 * c.kv_heads + h) * head_stride;
    const int64_t v_off = c.kv_heads * head_stride, page_stride = 2 * v_off;
    u32x4* vt = lds + wave * kVWords;
    u32x4 kr[T::Sub][L], vr[T::Sub][L];
    // keys past the end are read from the last row: in bounds, and masked
    auto page_at = [&](int kt, int i) {
      const int32_t p = table[min(kt * KW + i * 16 + col, all - 1) >> c.page_shift];
      return max(0, min(p, c.pages - 1));
    };
    int32_t pg[T::Sub];
    auto load = [&](int kt) {
#pragma unroll
      for (int i = 0; i < T::Sub; ++i) {
        const int r = min(kt * KW + i * 16 + col, all - 1);
        const u32x4* p = kv + pg[i] * page_stride + int64_t(r & (c.page_tokens - 1)) * T::Chunks + g;
#pragma unroll
        for (int j = 0; j < L; ++j) kr[i][j] = p[j * 4];
#pragma unroll
        for (int j = 0; j < L; ++j) vr[i][j] = p[v_off + j * 4];
      }
    };
    int kt = kt0 + wave;
    if (!q.bad && kt < end) {
#pragma unroll
      for (int i = 0; i < T::Sub; ++i) pg[i] = page_at(kt, i);
      load(kt);
#pragma unroll
      for (int i = 0; i < T::Sub; ++i) pg[i] = page_at(min(kt + kWaves, end - 1), i);
    }
    for (; !q.bad && kt < end; kt += kWaves) {
      // V to LDS, S^T from the registers
#pragma unroll
      for (int i = 0; i < T::Sub; ++i)
#pragma unroll
        for (int j = 0; j < L; ++j) vt[T::at(i * 16 + col, j * 4 + g)] = vr[i][j];
      f32x4 sc[MT][T::Sub];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < T::Sub; ++i) {
          f32x4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < L; ++j) {
            if constexpr (DT == 1) {
              x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kr[i][j]),
                                                          __builtin_bit_cast(bf16x8, qr[m][j]), x, 0, 0, 0);
            } else {
              const f32x4 k4 = __builtin_bit_cast(f32x4, kr[i][j]), q4 = __builtin_bit_cast(f32x4, qr[m][j]);
#pragma unroll
              for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_16x16x4f32(k4[e], q4[e], x, 0, 0, 0);
            }
          }
          sc[m][i] = x;
        }
      if (kt + kWaves < end) {
        load(kt + kWaves);
#pragma unroll
        for (int i = 0; i < T::Sub; ++i) pg[i] = page_at(min(kt + 2 * kWaves, end - 1), i);
      }
      if ((kt + 1) * KW > q.len) {  // new rows among the keys: who sees them
        const int first = kt * KW, at = first & 31;  // key and bit of the tile's first key
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int count = q.len + tok[m] + 1 - (first & ~31);  // causal: keys seen from the word's first on
          uint32_t word = count >= 32 ? ~0u : (1u << max(count, 0)) - 1;
          if (a.parent) word = seen[max(tok[m] - tok0, 0)][(first - base32) >> 5];
          word >>= at + 4 * g;
#pragma unroll
          for (int i = 0; i < T::Sub; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[m][i][e] = word >> (16 * i + e) & 1 ? sc[m][i][e] : -INFINITY;
        }
      }
      u32x4 pw[MT];  // bf16 weights, the keys of both halves in the order of V below
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float top = sc[m][0][0];
#pragma unroll
        for (int i = 0; i < T::Sub; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[m][i][e]);
        top = row_max(top) * scale;
        if (top > mx[m]) {
          const float turn = exp2_fast(mx[m] - top);  // 0 for the first tile
          mx[m] = top;
          sum[m] *= turn;
#pragma unroll
          for (int d = 0; d < DB; ++d) o[m][d] *= turn;
        }
        const float at = mx[m] == -INFINITY ? 0.f : mx[m];
#pragma unroll
        for (int i = 0; i < T::Sub; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[m][i][e] = exp2_fast(fmaf(sc[m][i][e], scale, -at));
            sum[m] += sc[m][i][e];
          }
        if constexpr (DT == 1)
          pw[m] = u32x4{pack_bf16(sc[m][0][0], sc[m][0][1]), pack_bf16(sc[m][0][2], sc[m][0][3]),
                        pack_bf16(sc[m][1][0], sc[m][1][1]), pack_bf16(sc[m][1][2], sc[m][1][3])};
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        if constexpr (DT == 1) {
          // 4 keys of column 16 d + lane % 16, from both halves
          const int r = 4 * g + col / 4, half = col % 4 / 2;
          const char* p0 = reinterpret_cast<const char*>(vt + T::at(r, 2 * d + half)) + col % 2 * 8;
          const char* p1 = reinterpret_cast<const char*>(vt + T::at(16 + r, 2 * d + half)) + col % 2 * 8;
          const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p0));
          const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p1));
          const short v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
          bf16x8 va;
          __builtin_memcpy(&va, v, 16);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            o[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, __builtin_bit_cast(bf16x8, pw[m]), o[m][d], 0, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = reinterpret_cast<const float*>(vt + T::at(4 * g + e, 4 * d + col / 4))[col % 4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
              o[m][d] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, sc[m][0][e], o[m][d], 0, 0, 0);
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }

    // the four wavefronts' parts joined; wavefront w ends with a quarter of
    // the columns
    __syncthreads();
    f32x4* buf = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      sum[m] = row_sum(sum[m]);
      if (g == 0) stat[wave][0][m * 16 + col] = mx[m], stat[wave][1][m * 16 + col] = sum[m];
#pragma unroll
      for (int d = 0; d < DB; ++d) buf[((wave * MT + m) * DB + d) * kWave + lane] = o[m][d];
    }
    __syncthreads();
    constexpr int Q = DB / kWaves;
    const bool whole = kt0 == 0 && kt1 == q.key_tiles;
    float* to = part(c, me, kt0 == 0, part_floats(M, D));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float top = -INFINITY, weight[kWaves], l = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat[w][0][m * 16 + col]);
      const float at = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        weight[w] = exp2_fast(stat[w][0][m * 16 + col] - at);
        l += weight[w] * stat[w][1][m * 16 + col];
      }
      if (!whole && wave == 0 && g == 0) to[m * 16 + col] = top, to[M + m * 16 + col] = l;
      const int r = rt * M + m * 16 + col;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int d = wave * Q + i;
        f32x4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) x += buf[((w * MT + m) * DB + d) * kWave + lane] * weight[w];
        if (!whole) {
          reinterpret_cast<f32x4*>(to + 2 * M)[(m * DB + d) * kWave + lane] = x;
        } else if (r < rows) {
          if (q.bad) x = f32x4{NAN, NAN, NAN, NAN}, l = 1.f;
          const int64_t at_out = (int64_t(q.begin + r / group) * a.q_heads + h * group + r % group) * D + 16 * d + 4 * g;
          x *= 1.f / l;
          if constexpr (DT == 1) {
            *reinterpret_cast<u32x2*>(static_cast<char*>(a.out) + at_out * 2) =
                u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
          } else {
            *reinterpret_cast<f32x4*>(static_cast<char*>(a.out) + at_out * 4) = x;
          }
        }
      }
    }
    if (kt0 == 0 && !whole && tid == 0)
      joins(c)[me] = Join{s, h, rt, share_of(total, shares, lo + q.key_tiles - 1)};
    __syncthreads();
    lo += kt1 - kt0;
  }
}

// Joins the parts of a segment that starts in share blockIdx.x and ends in a
// later one.  blockIdx.y: 16 of its rows.
template <int DT, int D>
__global__ __launch_bounds__(kBlock) void combine_kernel(KvCache c, KvAttention a, int M) {
  constexpr int DB = D / 16, Q = DB / kWaves;
  const Join j = joins(c)[blockIdx.x];
  if (j.last < 0) return;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, col = lane % 16, g = lane / 16, m = blockIdx.y;
  const int group = a.q_heads / c.kv_heads, begin = a.start[j.s], rows = (a.start[j.s + 1] - begin) * group;
  const int64_t floats = part_floats(M, D);
  f32x4 x[Q] = {};
  float top = -INFINITY, l = 0.f;
  for (int w = blockIdx.x; w <= j.last; ++w) {
    const float* p = part(c, w, w == static_cast<int>(blockIdx.x), floats);
    const float t = p[m * 16 + col], k = p[M + m * 16 + col];
    const float next = fmaxf(top, t), at = next == -INFINITY ? 0.f : next;
    const float old = exp2_fast(top - at), now = exp2_fast(t - at);
    top = next;
    l = l * old + k * now;
#pragma unroll
    for (int i = 0; i < Q; ++i)
      x[i] = x[i] * old + reinterpret_cast<const f32x4*>(p + 2 * M)[(m * DB + wave * Q + i) * kWave + lane] * now;
  }
  const int r = j.rt * M + m * 16 + col;
  if (r >= rows) return;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int64_t at = (int64_t(begin + r / group) * a.q_heads + j.h * group + r % group) * D + 16 * (wave * Q + i) + 4 * g;
    x[i] *= 1.f / l;
    if constexpr (DT == 1) {
      *reinterpret_cast<u32x2*>(static_cast<char*>(a.out) + at * 2) =
          u32x2{pack_bf16(x[i][0], x[i][1]), pack_bf16(x[i][2], x[i][3])};
    } else {
      *reinterpret_cast<f32x4*>(static_cast<char*>(a.out) + at * 4) = x[i];
    }
  }
}

template <int DT, int D, int MT>
hipError_t few_rows(const KvCache& c, const KvAttention& a, hipStream_t s) {
  few_rows_kernel<DT, D, MT><<<kShares, kBlock, 0, s>>>(c, a, kShares);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  combine_kernel<DT, D><<<dim3(kShares, MT), kBlock, 0, s>>>(c, a, 16 * MT);
  return hipGetLastError();
}

template <int DT, int D>
hipError_t launch(const KvCache& c, const KvAttention& a, hipStream_t s) {
  const int64_t rows = int64_t(a.max_new) * (a.q_heads / c.kv_heads);
  constexpr int kMost = DT == 1 ? (D == 256 ? 2 : 4) : (D == 256 ? 1 : 2);
  if constexpr (kMost >= 4)
    if (rows > 32) return few_rows<DT, D, 4>(c, a, s);
  if constexpr (kMost >= 2)
    if (rows > 16) return few_rows<DT, D, 2>(c, a, s);
  return few_rows<DT, D, 1>(c, a, s);
}

template <int DT>
hipError_t launch(const KvCache& c, const KvAttention& a, hipStream_t s) {
  if (c.head_dim == 64) return launch<DT, 64>(c, a, s);
  if (c.head_dim == 128) return launch<DT, 128>(c, a, s);
  return launch<DT, 256>(c, a, s);
}

}  // namespace

int64_t kv_attention_work_bytes(const KvCache&) {
  return round256(kShares * int64_t(sizeof(Join))) + 2 * kShares * kPartFloats * 4;
}

hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, hipStream_t s) {
  return c.dtype == TMS_F32 ? launch<0>(c, a, s) : launch<1>(c, a, s);
}

}  // namespace tms
