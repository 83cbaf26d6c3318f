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

#include <algorithm>
#include <type_traits>

#include "kv_tiles.h"

namespace tms {
namespace {

constexpr int kAhead = 3;  // products of 32 rows that the reads of LDS run ahead

// ------------------------------------------------------------------ plan --

// What a launch works on.  A segment is the row tile of one key head of one
// sequence; its keys are cut into tiles.  All tiles in the order (sequence,
// key head, row tile, key tile) are dealt to the workgroups in equal
// contiguous shares, so ragged batches and long contexts balance by
// themselves; the parts of a segment that does not lie in one share are joined
// by the last of its workgroups (few rows; up to 64 with few parts) or by
// combine_kernel (more rows, whose parts are too large for one workgroup).
// Where no segment is much longer than a share, a workgroup takes a whole one
// instead.

// Key tiles that row tile rt works on: all, or the ones up to its last token
// (causal; at most one more at the end of the sequence).
template <int M, int KT>
__device__ inline int tiles_of(const KvAttention& a, const Seq& q, int rt, int group) {
  if (a.parent || q.bad) return q.key_tiles;
  return (q.len + (rt * M + M - 1) / group + KT) / KT;
}

// Units of work.  Of a segment: its key tiles and kOpen more.  A segment's start
// (queries, page numbers, the first keys, the join of the wavefronts) is a
// chain of memory latencies that a share pays for each of its segments:
// without kOpen a share of many short contexts takes several times as long as
// one of a long context.  Causal row tiles are taken in pairs, a long one and a
// short one, whose sum is the same for all up to the rounding of two tiles.
constexpr int kOpen = 4;

// The least units of a share, and the tiles that take as long as the join of a
// part.  Few rows: one tile for each wavefront (8 units: one sequence of 517
// tokens of 8 key heads 12 -> 15 us), and 0.4 of a tile to a part, which one
// workgroup joins (without that rule 36000 keys of 2 heads took 45 us, with it
// 22; 8000 keys of 8 heads 35 and 23).  Many rows: parts are joined by
// many workgroups, so only the start of a segment counts (1, 2 and 5 units:
// 1000 keys of 8 heads and 30 drafts 16.8, 16.6 and 20.4 us; 10000 of 2 heads
// and 18 drafts 17.9, 15.6 and 17.9).
constexpr int kLeastFew = kWaves, kLeastMany = 2;
constexpr float kJoinFew = 0.4f, kJoinMany = 0.f;

// Whole segments instead of shares, chosen by the kernel: where the longest
// takes no more than a share and the writing and joining of its parts,
// kApart units for each row of a workgroup and part (three prompts of 610 to
// 1125 tokens of 16 query heads 49 -> 44 us, two of 1000 of 32 59 -> 45, 64 trees of
// 50 to 64 drafts behind 1000 tokens 97 -> 78; four times that 36 -> 45 us for
// two prompts of 374 to 618 with heads of 256).  Kernels that memory bounds (up
// to 64 rows) lose less by a long segment, as the others' bandwidth goes to it:
// 1.5 shares (5 to 31 drafts behind 64 contexts of 1201 to 2500 tokens 114 -> 99
// us, tokens of 16 rows behind 64 of 3000 to 5000 196 -> 188).
constexpr float kScaleMemory = 1.5f, kApart = 9.f / 256;
enum { kWhole = 0, kSplit, kEither };

template <int M, int KT>
__device__ inline int units_each(const KvAttention& a, const Seq& q, int group, bool* pairs) {
  *pairs = !a.parent && !q.bad && q.rows_tiles > 1;
  if (!*pairs) return q.key_tiles + kOpen;
  return tiles_of<M, KT>(a, q, 0, group) + tiles_of<M, KT>(a, q, q.rows_tiles - 1, group) + 2 + 2 * kOpen;
}

// Of a sequence; whole segments where they are not split.
template <int M, int KT>
__device__ inline int64_t units_of(const KvCache& c, const KvAttention& a, const Seq& q, bool split) {
  if (!split) return int64_t(q.rows_tiles) * c.kv_heads;
  bool pairs;
  const int each = units_each<M, KT>(a, q, a.q_heads / c.kv_heads, &pairs);
  return int64_t(pairs ? (q.rows_tiles + 1) / 2 : q.rows_tiles) * each * c.kv_heads;
}

// The segment at unit lo of sequence q (whose first unit is base), as far as
// the share goes: key tiles kt0 .. kt1 - 1 of `tiles`; first and last are the
// units of the segment's first and last tile.  lo moves past it.
struct Segment {
  int h, rt, kt0, kt1, tiles;
  int64_t first, last;
};

template <int M, int KT>
__device__ inline bool next_segment(const KvCache& c, const KvAttention& a, const Seq& q, bool split, int64_t base,
                                    int64_t hi, int64_t& lo, Segment* g) {
  if (!split) {  // heads of a row tile next to each other (each on its own XCD's cache), long rows first
    const int off = static_cast<int>(lo - base);
    g->h = off % c.kv_heads, g->rt = q.rows_tiles - 1 - off / c.kv_heads;
    g->tiles = q.key_tiles, g->kt0 = 0, g->kt1 = q.key_tiles;
    g->first = g->last = 0;
    ++lo;
    return true;
  }
  const int group = a.q_heads / c.kv_heads;
  bool pairs;
  const int each = units_each<M, KT>(a, q, group, &pairs);
  const int count = pairs ? (q.rows_tiles + 1) / 2 : q.rows_tiles;  // of a head
  const int64_t past = quotient(lo - base, each);
  const int at = static_cast<int>(past);
  int u = static_cast<int>(lo - base - past * each);
  const int64_t next = lo - u + each;
  g->h = at / count, g->rt = at % count;
  int units = each;
  if (pairs) {
    const int other = g->rt;
    g->rt = q.rows_tiles - 1 - other;
    units = kOpen + tiles_of<M, KT>(a, q, g->rt, group);
    if (u >= units) {  // past the long one
      u -= units;
      units = other < g->rt ? kOpen + tiles_of<M, KT>(a, q, other, group) : 0;
      g->rt = other;
      if (u >= units) {
        lo = next;
        return false;
      }
    }
  }
  const int end = static_cast<int>(min(int64_t(units), u + hi - lo));
  g->tiles = units - kOpen;
  g->last = lo + units - u - 1;
  g->first = g->last - g->tiles + 1;
  lo += end - u;
  if (end <= kOpen) return false;  // the share ends before the segment's first tile
  g->kt0 = max(u - kOpen, 0), g->kt1 = end - kOpen;
  return true;
}

// A segment that several workgroups share, written by the one it starts in.
struct Join {
  int32_t s, h, rt, last;  // last: the last workgroup that holds a part (-1: nothing to join)
};

// Work memory: a count of the parts that have arrived for every share in which
// a segment starts (zero between calls), Join [shares], then for every share
// two parts (its first and
// its last segment) of kRows rows: maximum and sum of every row, then the
// unnormalised outputs in the lanes' order.
__host__ __device__ inline int64_t round256(int64_t x) { return (x + 255) & ~int64_t(255); }
__host__ __device__ inline int64_t part_floats(int rows, int dim) { return int64_t(rows) * (dim + 2); }

constexpr int kShares = 512;  // few rows: two workgroups for each compute unit
constexpr int kManyShares = 256;
static_assert(kShares * 4 <= kWorkCounts, "a counter for each share");

__device__ inline uint32_t* arrived(const KvCache& c) { return static_cast<uint32_t*>(c.work); }
__device__ inline Join* joins(const KvCache& c) {
  return reinterpret_cast<Join*>(static_cast<char*>(c.work) + kWorkCounts);
}
__device__ inline float* part(const KvCache& c, int share, int which, int64_t floats) {
  return reinterpret_cast<float*>(static_cast<char*>(c.work) + kWorkCounts + round256(kShares * int64_t(sizeof(Join)))) +
         (2 * int64_t(share) + which) * floats;
}

// First unit of a share of the `total` units, and the share that a unit is in:
// the first total % shares of them have one unit more.
__device__ inline int64_t share_begin(int64_t total, int shares, int w) {
  const int64_t each = quotient(total, shares);
  return w * each + min(int64_t(w), total - each * shares);
}
__device__ inline int share_of(int64_t total, int shares, int64_t unit) {
  const int64_t each = quotient(total, shares), longer = total - each * shares, past = unit - longer * (each + 1);
  return static_cast<int>(past < 0 ? quotient(unit, each + 1) : longer + quotient(past, each));
}

__device__ inline int64_t read_lane(int64_t x, int lane) {
  const uint64_t low = uint32_t(__builtin_amdgcn_readlane(int(x), lane)), high = uint32_t(__builtin_amdgcn_readlane(int(x >> 32), lane));
  return int64_t(high << 32 | low);
}

// The share [*lo, *hi) of this workgroup among all units, the sequence *s that
// it starts in (*q) and that sequence's first unit *base: a prefix sum over the
// sequences.  shares is cut so that a share has at least `least` units, and
// sqrt(`join` n) for the n tiles of the longest segment: the time of a
// share's tiles and the time to join a segment's parts are the same then,
// if a part takes as long to join as `join` tiles.  With split = kEither it
// becomes kWhole, and a
// workgroup takes a whole segment, where the longest one, or all of them
// with the last ones to be started, end within `scale` shares and `more` units
// (writing and joining parts is saved), or no segment is longer than three
// quarters of a share.
// Returns whether there is work.
template <int M, int KW, int W>
__device__ inline bool my_share(const KvCache& c, const KvAttention& a, int& split, bool mark, int& shares, int least, float join,
                                float scale, float more, int64_t* lo, int64_t* hi, int* s_out, Seq* q_out, int64_t* base_out, int64_t* total_out) {
  __shared__ int64_t scan[W];
  __shared__ int segments[W], longest[W], latest[W], found[7];
  __shared__ int64_t found_base;
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
  int64_t mine = 0, total = 0, before = 0;
  int tiles = 0, tail = 0, my_count = 0, count = 0, count_before = 0;
  // up to 64 sequences: every wavefront has them all, and none waits for another
  const bool alone = c.seqs <= kWave;
  const int each = alone ? 1 : (c.seqs + W * kWave - 1) / (W * kWave), place = alone ? lane : tid * each;
  Seq q{};  // the thread's last sequence; its only one where each is 1
  for (int i = 0; i < each; ++i) {
    const int s = place + i;
    if (s < c.seqs) {
      q = sequence(c, a, s, M, KW);
      mine += units_of<M, KW>(c, a, q, kSplit);
      my_count += static_cast<int>(units_of<M, KW>(c, a, q, kWhole));
      if (q.n) {
        tiles = max(tiles, q.key_tiles);
        if (split == kEither && int(gridDim.x) > shares) tail = max(tail, tiles_of<M, KW>(a, q, 0, a.q_heads / c.kv_heads));
      }
    }
  }
  int64_t incl = mine;
  int incl_count = my_count;
  auto step = [&](auto from) __attribute__((always_inline)) {
    const uint64_t low = uint32_t(from(int(incl))), high = uint32_t(from(int(incl >> 32)));
    incl += int64_t(high << 32 | low), incl_count += from(incl_count);
    tiles = max(tiles, from(tiles)), tail = max(tail, from(tail));
  };
  step([](int x) { return from_lane<0x111, 0xf>(x); });  // 1, 2, 4 and 8 lanes down in rows of 16
  step([](int x) { return from_lane<0x112, 0xf>(x); });
  step([](int x) { return from_lane<0x114, 0xf>(x); });
  step([](int x) { return from_lane<0x118, 0xf>(x); });
  step([](int x) { return from_lane<0x142, 0xa>(x); });  // row 0 to row 1, row 2 to row 3
  step([](int x) { return from_lane<0x143, 0xc>(x); });  // lane 31 to rows 2 and 3
  constexpr int kLast = kWave - 1;
  if (alone) {
    total = read_lane(incl, kLast), count = __builtin_amdgcn_readlane(incl_count, kLast);
    tiles = __builtin_amdgcn_readlane(tiles, kLast), tail = __builtin_amdgcn_readlane(tail, kLast);
  } else {
    if (lane == kLast) scan[wave] = incl, segments[wave] = incl_count, longest[wave] = tiles, latest[wave] = tail;
    __syncthreads();
    for (int i = 0; i < W; ++i) {
      if (i < wave) before += scan[i], count_before += segments[i];
      total += scan[i], count += segments[i];
      tiles = max(tiles, longest[i]), tail = max(tail, latest[i]);
    }
  }
  before += incl - mine;
  total = uniform(total), count = uniform(count), tiles = uniform(tiles), tail = uniform(tail);
  if (split == kEither) {
    const float share = static_cast<float>(total) / shares;
    const float whole = fmaxf(tiles + kOpen, count <= shares ? 0.f : share + tail + kOpen);
    if (count <= int(gridDim.x) && (whole <= scale * share + more * (shares + min(count, shares)) / shares || 1.33f * tiles <= share))
      split = kWhole;
  }
  if (split == kWhole) {
    before = count_before + incl_count - my_count, mine = my_count, total = count;
  }
  least = uniform(max(least, static_cast<int>(sqrtf(join * tiles))));
  if (split) shares = static_cast<int>(max(int64_t(1), min(int64_t(shares), total / least)));
  const int me = blockIdx.x;
  if (mark && tid == 0) joins(c)[me] = Join{0, 0, 0, -1};
  *lo = split ? share_begin(total, shares, me) : me;
  *hi = split ? share_begin(total, shares, me + 1) : me + 1;
  if (me >= (split ? shares : total) || total == 0) return false;
  *total_out = total;
  const bool here = *lo >= before && *lo < before + mine;
  if (alone) {
    const int from = __builtin_ctzll(__ballot(here));
    auto word = [&](int x) { return __builtin_amdgcn_readlane(x, from); };
    *s_out = from;
    *q_out = Seq{word(q.begin), word(q.n), word(q.len), word(q.rows_tiles), word(q.key_tiles), word(q.bad)};
    *base_out = read_lane(before, from);
    return true;
  }
  if (here) {
    int64_t base = before;
    int s = place;
    for (; each > 1; ++s) {
      q = sequence(c, a, s, M, KW);
      const int64_t t = units_of<M, KW>(c, a, q, split);
      if (*lo < base + t) break;
      base += t;
    }
    const int words[7] = {s, q.begin, q.n, q.len, q.rows_tiles, q.key_tiles, q.bad};
#pragma unroll
    for (int i = 0; i < 7; ++i) found[i] = words[i];
    found_base = base;
  }
  __syncthreads();
  *s_out = uniform(found[0]);
  *q_out = Seq{uniform(found[1]), uniform(found[2]), uniform(found[3]), uniform(found[4]), uniform(found[5]),
               uniform(found[6])};
  *base_out = uniform(found_base);
  return true;
}

// Row and column of value 4 i of a part's outputs: the lanes' order of the
// 16-row (few rows) and of the 32-row products (many rows).
template <int D>
__device__ inline void part_place(int i, int wide, int* row, int* column) {
  const int lane = i % kWave, block = i / kWave;
  if (wide) {
    *row = block / (D / 8) * 32 + lane % 32;
    *column = block % (D / 8) * 8 + lane / 32 * 4;
  } else {
    *row = block / (D / 16) * 16 + lane % 16;
    *column = block % (D / 16) * 16 + lane / 16 * 4;
  }
}

// Whether this workgroup is the last of the shares first .. last of a segment to
// have written its part.
__device__ inline bool last_to_arrive(const KvCache& c, int first, int last) {
  __shared__ uint32_t arrivals;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the part is written
  __syncthreads();
  if (threadIdx.x == 0) {
    arrivals = atomicAdd(&arrived(c)[first], 1u);
    if (arrivals == uint32_t(last - first)) arrived(c)[first] = 0;
  }
  __syncthreads();
  return arrivals == uint32_t(last - first);
}

struct Sum {
  float top = -INFINITY, l = 0.f;
  f32x4 x{0.f, 0.f, 0.f, 0.f};
};

// Values 4 i .. 4 i + 3, of row `row`, of a segment of M rows that starts in
// share `first`: the parts in the shares w .. last joined, in that order.
template <int D, bool Shared>
__device__ inline Sum sum_parts(const KvCache& c, int first, int w, int last, int M, int row, int i) {
  const int64_t floats = part_floats(M, D);
  Sum s;
  constexpr int kParts = Shared ? 12 : 8;  // in flight
  for (; w <= last; w += kParts) {
    float t[kParts], k[kParts];
    f32x4 y[kParts];
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
      t[u] = -INFINITY, k[u] = 0.f, y[u] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (w + u <= last) {
        const float* p = part(c, w + u, w + u == first, floats);
        t[u] = part_load<Shared>(p + row), k[u] = part_load<Shared>(p + M + row);
        y[u] = part_load<Shared>(reinterpret_cast<const f32x4*>(p + 2 * M) + i);
      }
    }
    float next = s.top;
#pragma unroll
    for (int u = 0; u < kParts; ++u) next = fmaxf(next, t[u]);
    const float at = next == -INFINITY ? 0.f : next, old = part_weight(s.top - at);
    s.top = next;
    s.l *= old, s.x *= old;
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
      const float now = part_weight(t[u] - at);
      s.l += k[u] * now;
      s.x += y[u] * now;
    }
  }
  return s;
}

template <int DT, int D>
__device__ inline void store_joined(const KvAttention& a, const KvCache& c, const Join& j, int M, int row, int column,
                                    const Sum& s) {
  const int group = a.q_heads / c.kv_heads, begin = a.start[j.s], rows = (a.start[j.s + 1] - begin) * group;
  const int r = j.rt * M + row;
  if (row < M && r < rows)
    store4<DT>(a.out, (int64_t(begin + r / group) * a.q_heads + j.h * group + r % group) * D + column, s.x * (1.f / s.l));
}

// Values 4 i .. 4 i + 3 of the output of a segment whose parts are in the
// shares first .. j.last.
template <int DT, int D, bool Shared>
__device__ inline void join_parts(const KvCache& c, const KvAttention& a, const Join& j, int first, int M, int wide, int i) {
  int row, column;
  part_place<D>(i, wide, &row, &column);
  if (row < M) store_joined<DT, D>(a, c, j, M, row, column, sum_parts<D, Shared>(c, first, first, j.last, M, row, i));
}

// ------------------------------------------------- few rows: token, drafts --

// Workgroup of 4 wavefronts over the segments of its share.  Each wavefront
// holds all rows of the segment and takes every 4th key tile: K straight into
// registers, V through its own part of LDS, no barrier among them; the next
// tile's loads are in flight during the softmax and the second product.
//
// Up to 16 rows fill half of a matrix product and read K and V once, so memory
// bounds them: 8 sequences of 40000 to 60000 tokens (32 query, 8 key heads of
// 128, bf16) 299 us, 5.5 TB/s of 6.1 that a plain read reaches.  64 of 0 to 8191
// tokens take 50.5 us, 3.6 TB/s, where a plain read would take 30: about 8 of the
// 20 are the start of a workgroup (dependent reads: offsets, page numbers, first
// keys); a share has about 26 units there, six or seven tiles of a wavefront,
// and begins that chain again for each of its segments.  One sequence of 517
// tokens 12 us, nothing but that chain and the join.  fp32 takes 32
// rows to a workgroup where there are more than 16, which halves the reads of K
// and V: two prompts of 2000 to 3000 tokens 825 us, 43 % of the rate of a plain
// product (the reads of V by single words bound it).
template <int DT, int D, int MT>
__global__ __launch_bounds__(kBlock) void few_rows_kernel(KvCache c, KvAttention a, int shares, int split) {
  using T = Tile<DT, D>;
  constexpr int M = 16 * MT, KW = T::Keys, DB = D / 16, L = T::Loads;
  constexpr int kVWords = KW * T::Chunks;                  // 16-byte words of a V tile
  constexpr int kLds = kWaves * kVWords > kWaves * M * D / 4 ? kWaves * kVWords : kWaves * M * D / 4;
  __shared__ u32x4 lds[kLds];
  __shared__ float stat[kWaves][2][M];
  __shared__ uint32_t seen[M * kTreeWords];
  __shared__ int32_t par[kTree];
  __shared__ uint32_t nonfinite[kMixedWords];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
  const int col = lane % 16, g = lane / 16;
  const int group = a.q_heads / c.kv_heads;
  // a scale of 0 clears q instead: a masked score stays -inf
  const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
  const uint32_t flip = a.scale < 0.f ? (DT == 0 ? 0x80000000u : 0x80008000u) : 0u, on = a.scale == 0.f ? 0u : ~0u;

  int64_t lo, hi, base, total;
  int s;
  Seq q;
  if (!my_share<M, KW, kWaves>(c, a, split, false, shares, kLeastFew, kJoinFew, kScaleMemory, M * kApart, &lo, &hi, &s, &q, &base, &total)) return;
  const int me = blockIdx.x;

  int again = 0;  // the segment is worked on for the second time
  while (lo < hi) {
    const int64_t lo_here = lo;
    while (lo >= base + units_of<M, KW>(c, a, q, split)) {
      base += units_of<M, KW>(c, a, q, split);
      q = uniform(sequence(c, a, ++s, M, KW));
    }
    Segment sg;
    if (!next_segment<M, KW>(c, a, q, split, base, hi, lo, &sg)) continue;
    const int h = sg.h, rt = sg.rt, kt0 = sg.kt0, kt1 = sg.kt1;
    const int rows = q.n * group;  // of the sequence and key head
    const int all = q.len + q.n;
    const int tok0 = rt * M / group, tok1 = min(q.n - 1, (rt * M + M - 1) / group);  // tokens of the tile
    const int limit = a.parent ? all : q.len + tok1 + 1;                             // keys that any row sees
    const int end = q.bad ? 0 : min(kt1, (limit + KW - 1) / KW);
    const int32_t* table = c.table + int64_t(s) * c.max_pages;
    const int64_t head_stride = int64_t(c.page_tokens) * T::Chunks;  // 16-byte words
    const u32x4* kv = static_cast<const u32x4*>(c.kv) +
                      (int64_t(a.layer) * c.pages * 2 * c.kv_heads + h) * head_stride;
    const int64_t v_off = c.kv_heads * head_stride, page_stride = 2 * v_off;
    // keys past the last one to be used are read from that one: in bounds, and masked
    auto page_at = [&](int kt, int i) {
      const int32_t p = table[min(kt * KW + i * 16 + col, limit - 1) >> c.page_shift];
      return max(0, min(p, c.pages - 1));
    };
    int kt = kt0 + wave;
    int32_t pg[T::Sub];
    if (kt < end)
#pragma unroll
      for (int i = 0; i < T::Sub; ++i) pg[i] = page_at(kt, i);
    // the queries: B operand, row = lane % 16; asked for before the first keys,
    // used after them
    u32x4 qr[MT][L];
    int tok[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = rt * M + m * 16 + col;
      tok[m] = r < rows ? r / group : -1;
      const int64_t at = int64_t(q.begin + max(tok[m], 0)) * a.ldq + int64_t(h * group + (r < rows ? r % group : 0)) * D;
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + at * (DT == 0 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < L; ++i) qr[m][i] = p[i * 4 + g];
    }
    u32x4* vt = lds + wave * kVWords;
    u32x4 kr[T::Sub][L], vr[T::Sub][L];
    auto load = [&](int kt) {
#pragma unroll
      for (int i = 0; i < T::Sub; ++i) {
        const int r = min(kt * KW + i * 16 + col, limit - 1);
        const u32x4* p = kv + pg[i] * page_stride + int64_t(r & (c.page_tokens - 1)) * T::Chunks + g;
#pragma unroll
        for (int j = 0; j < L; ++j) kr[i][j] = p[j * 4];
#pragma unroll
        for (int j = 0; j < L; ++j) vr[i][j] = p[v_off + j * 4];
      }
    };
    if (kt < end) {
      load(kt);
#pragma unroll
      for (int i = 0; i < T::Sub; ++i) pg[i] = page_at(min(kt + kWaves, end - 1), i);
    }
    if (a.parent && !q.bad && end * KW > q.len) walk_tree<kBlock>(a, q, tok0, tok1, par, seen, kTreeWords);
    const Mixed mixed = mixed_rows(a, q, tok0, tok1, nonfinite);
    bool odd = false;
    if (again)
      odd = find_nonfinite<kBlock, DT, D>(c, table, kv + v_off, page_stride, mixed);
    f32x4 o[MT][DB];
    float mx[MT], sum[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mx[m] = -INFINITY, sum[m] = 0.f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < L; ++i) qr[m][i] = (qr[m][i] ^ flip) & on;
    }
    for (; kt < end; kt += kWaves) {
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
          const uint32_t word = sees(a, q, tok[m], tok0, first & ~31, seen, kTreeWords) >> (at + 4 * g);
#pragma unroll
          for (int i = 0; i < T::Sub; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[m][i][e] = word >> (16 * i + e) & 1 ? sc[m][i][e] : -INFINITY;
        }
      }
      // Weights in two parts of bf16, the keys of both halves in the order of V
      // below: 16 bits of each take one product more, up to 1 % here (256 tokens
      // behind 10 to 4000 keys 147.3 -> 148.2 us, 64 behind 1000 48.3 -> 48.8, 8
      // behind 40000 to 60000 298 -> 299).
      u32x4 pw[MT], pl[MT];
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
          split_bf16({sc[m][0][0], sc[m][0][1], sc[m][0][2], sc[m][0][3], sc[m][1][0], sc[m][1][1], sc[m][1][2], sc[m][1][3]},
                     &pw[m], &pl[m]);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (odd) {
        for (uint32_t word = mixed.word(kt * KW & ~31) >> (kt * KW & 31) & T::Mask; word; word &= word - 1) {
          const int r = __builtin_ctz(word);
          for (int i = lane; i < T::Chunks; i += kWave) vt[r * T::Chunks + i] = keep_finite<DT>(vt[r * T::Chunks + i], true);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        if constexpr (DT == 1) {
          // 4 keys of column 16 d + lane % 16, from both halves
          const int r = 4 * g + col / 4, half = col % 4 / 2;
          const char* p0 = reinterpret_cast<const char*>(vt + T::at(r, 2 * d + half)) + col % 2 * 8;
          const char* p1 = reinterpret_cast<const char*>(vt + T::at(16 + r, 2 * d + half)) + col % 2 * 8;
          const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p0));
          const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p1));
          const bf16x8 va = __builtin_bit_cast(bf16x8, s16x8(__builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7)));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            o[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, __builtin_bit_cast(bf16x8, pl[m]), o[m][d], 0, 0, 0);
            o[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, __builtin_bit_cast(bf16x8, pw[m]), o[m][d], 0, 0, 0);
          }
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

    float z = 0.f;
    if (!again && !q.bad && end * KW > mixed.first)
#pragma unroll
      for (int m = 0; m < MT; ++m) z = zero_or_nan(o[m], z);
    // every wavefront is done with its tiles
    if (__syncthreads_or(z != z)) {
      again = 1, lo = lo_here;
      continue;
    }
    again = 0;
    // the four wavefronts' parts joined; wavefront w ends with a quarter of
    // the columns
    f32x4* buf = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      sum[m] = row_sum(sum[m]);
      if (g == 0) stat[wave][0][m * 16 + col] = mx[m], stat[wave][1][m * 16 + col] = sum[m];
#pragma unroll
      for (int d = 0; d < DB; ++d) buf[((wave * MT + m) * DB + d) * kWave + lane] = o[m][d];
    }
    if (odd)  // every wavefront for the tiles that it had
      for (kt = kt0 + wave; kt < end; kt += kWaves)
        for (uint32_t word = mixed.word(kt * KW & ~31) >> (kt * KW & 31) & T::Mask; word; word &= word - 1) {
          const int row = kt * KW + __builtin_ctz(word);
          if (row >= limit) break;
          const u32x4* p = value_row(c, table, kv + v_off, page_stride, T::Chunks, row);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (sees(a, q, tok[m], tok0, row & ~31, seen, kTreeWords) >> (row & 31) & 1)
#pragma unroll 1
              for (int d = 0; d < DB; ++d)
                buf[((wave * MT + m) * DB + d) * kWave + lane] += odd_values<DT>(p, 16 * d + 4 * g);
        }
    __syncthreads();
    constexpr int Q = DB / kWaves;
    const bool whole = kt0 == 0 && kt1 == sg.tiles;
    float* to = part(c, me, kt0 == 0, part_floats(M, D));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float top = -INFINITY, weight[kWaves], l = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat[w][0][m * 16 + col]);
      const float at = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        weight[w] = part_weight(stat[w][0][m * 16 + col] - at);
        l += weight[w] * stat[w][1][m * 16 + col];
      }
      if (!whole && wave == 0 && g == 0) part_store<true>(to + m * 16 + col, top), part_store<true>(to + M + m * 16 + col, l);
      const int r = rt * M + m * 16 + col;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int d = wave * Q + i;
        f32x4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) x += buf[((w * MT + m) * DB + d) * kWave + lane] * weight[w];
        if (!whole) {
          part_store<true>(reinterpret_cast<f32x4*>(to + 2 * M) + (m * DB + d) * kWave + lane, x);
        } else if (r < rows) {
          if (q.bad) x = f32x4{NAN, NAN, NAN, NAN}, l = 1.f;
          const int64_t at_out = (int64_t(q.begin + r / group) * a.q_heads + h * group + r % group) * D + 16 * d + 4 * g;
          store4<DT>(a.out, at_out, x * (1.f / l));
        }
      }
    }
    if (!whole) {
      // the last share to arrive joins the parts, in their order: every share
      // from the one with the segment's first tile to the one with its last
      // has a part
      const int first = share_of(total, shares, sg.first), end_share = share_of(total, shares, sg.last);
      if (last_to_arrive(c, first, end_share)) {
        for (int i = tid; i < M * D / 4; i += kBlock)
          join_parts<DT, D, true>(c, a, Join{s, h, rt, end_share}, first, M, 0, i);
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------ many rows: drafts, whole prompts --

// Words of the table of drafts that a workgroup of 32 RW rows has, and of a
// token's row in it: a tree fits in one row tile below 8 x 32 rows; there, the
// rows are of at most 128 tokens with two query heads or more to a key head
// (any tree), and of 256 with one (trees of up to 512 drafts).  Trees that do
// not fit these take 128 rows with the whole table (AnyTree).
template <int RW, bool AnyTree>
constexpr int kSeen = AnyTree ? 32 * RW * kTreeWords : RW == 8 ? 256 * 17 : 32 * RW * (RW + 1);
template <int RW, bool AnyTree>
int tree_words(int group) {
  return AnyTree ? kTreeWords : RW < 8 ? RW + 1 : group > 1 ? kTreeWords : 17;
}

// Workgroup of RW x KS wavefronts over a segment (whole prompts: the heaviest
// first) or over a share of the key tiles (drafts over a long context).  A
// wavefront holds 32 rows and takes 1 / KS of the keys of every tile; the tiles
// of K and V are in LDS, two buffers each.
//
// A tile is two phases: the products (scores of this tile, output of the one
// before) and the softmax with the copies of later tiles into LDS.  With 8
// wavefronts, two on a SIMD, the second four run one phase behind: while one
// wavefront of a SIMD feeds the matrix cores the other has the vector units.
//
// Bound by the matrix cores and the vector units in turns (a 64-key tile of 256
// rows: 2304 cycles of products, 256 of them for the row sums, about 4000 in
// all: the time of the two adds up more than it overlaps).  32 query, 8 key heads
// of 128: three prompts of 2300 to 4097 tokens 320 us (929 TFLOP/s; the matrix
// cores busy 51 % of the cycles, the vector units issuing other work 37 %), one
// of 16000 tokens 1110 TFLOP/s (a plain product of 16384^3: 1340), 63 drafts over
// two contexts of 90000 to 120000 253 us (857 TFLOP/s).  Fewer rows are bound by
// memory: 5 to 31 drafts behind 64 contexts of 1201 to 2500 tokens 96.5 us, 4.7
// TB/s.  Heads of 256 have one wavefront on a SIMD and nothing beside its
// softmax: two prompts of 2000 to 3000 tokens of 8 query, 2 key heads 128 us, 417
// TFLOP/s.  K and V go straight into LDS: through registers 463 us for the
// prompts.
template <int D, int RW, int KS, bool AnyTree>
__global__ __launch_bounds__(RW * KS * kWave, D == 256 ? 1 : 2) void many_rows_kernel(KvCache c, KvAttention a, int shares, int split, int words, int join) {
  constexpr int W = RW * KS, M = 32 * RW, CH = D / 8, KK = D / 16, DB = D / 32, Threads = W * kWave;
  constexpr bool Behind = W == 8, Fine = KS == 2;
  constexpr int KT = 64, TileWords = KT * CH;       // keys of a tile, its 16-byte words
  constexpr int NB = KT / 32 / KS;                  // 32-key blocks of a tile for each wavefront
  constexpr int Ahead = Behind ? 2 : 1;             // tiles that the copies run ahead
  constexpr int Bufs = Behind ? Ahead + 2 : Ahead + 1;
  constexpr int RPI = kWave / CH, P = KT / RPI / W;  // rows of a copying instruction, instructions of a wavefront
  // K tiles, then V tiles; the outputs of the second half of the keys at the end
  __shared__ u32x4 tiles[2 * Bufs * TileWords];
  __shared__ float stat[KS == 2 ? 2 * M : 1];
  __shared__ uint32_t seen[kSeen<RW, AnyTree>];
  __shared__ int32_t par[AnyTree || RW == 8 ? kTree : M];
  __shared__ uint32_t nonfinite[kMixedWords];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
  const int rw = wave % RW, ks = wave / RW, col = lane % 32, hi2 = lane / 32;
  const bool behind = Behind && wave >= 4;
  const int group = a.q_heads / c.kv_heads;
  const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
  const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u, on = a.scale == 0.f ? 0u : ~0u;
  const int tiles_at = static_cast<int>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)tiles));
  // places in LDS: K is read 16 bytes of 16 rows at a time, V 64 bytes of 4, each
  // from 64 different banks (but K of 64-value heads, where pairs of rows meet: an
  // order without that was 3 % slower)
  constexpr int Mask = (CH < 16 ? CH : 16) - 1, VShift = D == 64 ? 1 : 2;
  auto k_at = [](int r, int ch) { return r * CH + (ch ^ (r & Mask)); };
  auto v_at = [](int r, int ch) { return r * CH + (ch ^ (r << VShift & Mask)); };

  int64_t lo, hi, base, total;
  int s;
  Seq q;
  if (!my_share<M, KT, W>(c, a, split, !join && int(blockIdx.x) < shares, shares, kLeastMany, kJoinMany, KS == 2 ? kScaleMemory : 1.f, M * kApart, &lo, &hi, &s, &q, &base, &total)) return;
  int again = 0;  // the segment is worked on for the second time
  while (lo < hi) {
    const int64_t lo_here = lo;
    while (lo >= base + units_of<M, KT>(c, a, q, split)) {
      base += units_of<M, KT>(c, a, q, split);
      q = uniform(sequence(c, a, ++s, M, KT));
    }
    Segment sg;
    if (!next_segment<M, KT>(c, a, q, split, base, hi, lo, &sg)) continue;
    const int h = uniform(sg.h), rt = uniform(sg.rt), kt0 = uniform(sg.kt0), kt1 = uniform(sg.kt1);
    const int rows = q.n * group, all = q.len + q.n;
    const int r = rt * M + rw * 32 + col, tok = r < rows ? r / group : -1;
    u32x4 qr[KK];  // asked for here, used after the first copies are
    {
      const int64_t at = int64_t(q.begin + max(tok, 0)) * a.ldq + int64_t(h * group + (r < rows ? r % group : 0)) * D;
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + at * 2);
#pragma unroll
      for (int i = 0; i < KK; ++i) qr[i] = p[2 * i + hi2];
    }
    const int tok0 = rt * M / group, tok1 = min(q.n - 1, (rt * M + M - 1) / group);  // of the workgroup
    const int limit = a.parent ? all : q.len + tok1 + 1;
    const int end = q.bad ? kt0 : min(kt1, (limit + KT - 1) / KT);
    // keys that all rows of the wavefront see
    const int clear = uniform(a.parent ? q.len : q.len + min((rt * M + rw * 32) / group, q.n - 1) + 1);

    const f32x16 zero = {};
    f32x16 o[DB], sc[NB], total_w;  // total_w: a row's sum of weights, in every register
    float mx = -INFINITY;
    const bf16x8 ones = {1, 1, 1, 1, 1, 1, 1, 1};
#pragma unroll
    for (int e = 0; e < 16; ++e) total_w[e] = 0.f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
    const int32_t* table = c.table + int64_t(uniform(s)) * c.max_pages;
    const int64_t head_stride = int64_t(c.page_tokens) * CH;  // 16-byte words
    const u32x4* kv = static_cast<const u32x4*>(c.kv) + (int64_t(a.layer) * c.pages * 2 * c.kv_heads + h) * head_stride;
    const int64_t v_off = c.kv_heads * head_stride, page_stride = 2 * v_off;
    // Copies from the cache straight into LDS, 1 KB an instruction: rows r0 ..
    // r0 + RPI - 1 of a tile, in one page (a page has at least 8 rows).  LDS
    // fills in the lanes' order, so the lanes take the words in the order that
    // k_at and v_at have them.  Rows past the last one to be used are filled
    // with that one: in bounds, and masked or never used.
    const int final_row = uniform(max(min(limit, end * KT) - 1, 0));
    const int my_row = lane / CH, k_ch = lane % CH ^ ((wave * RPI + my_row) & Mask),
              v_ch = lane % CH ^ ((wave * RPI + my_row) << VShift & Mask);
    // Step x copies K of tile x + 1 + Ahead and V of tile x + Ahead; a tile's
    // page numbers are asked for one step before its K, its addresses are kept
    // for its V.
    const const_i32 pages = (const_i32)(table);
    const uint32_t page_words = 2 * c.kv_heads * c.page_tokens * CH;
    int next_page[P], row_at[P];
    int64_t from[P];  // addresses
    auto look = [&](int kt, int i) __attribute__((always_inline)) {
      next_page[i] = pages[uint32_t(min(kt * KT + (i * W + wave) * RPI, final_row)) >> c.page_shift];
    };
    auto find = [&](int kt, int i) __attribute__((always_inline)) {
      const int r0 = kt * KT + (i * W + wave) * RPI, first = min(r0, final_row & ~(RPI - 1));
      const uint32_t page = uniform(max(0, min(next_page[i], c.pages - 1)));
      from[i] = uniform(reinterpret_cast<int64_t>(kv) +
                        (int64_t(uint64_t(page) * page_words) + uint32_t(first & (c.page_tokens - 1)) * CH) * 16);
      row_at[i] = (min(r0 + my_row, final_row) - first) * (CH * 16);
    };
    auto copy = [&](int64_t off, int ch, int step, int to, int i) __attribute__((always_inline)) {
      copy_to_lds(from[i] + off, row_at[i] + (ch ^ (i * W * RPI * step & Mask)) * 16,
                  tiles_at + to * (TileWords * 16) + (i * W + wave) * (kWave * 16));
    };
    // buffers of the V tile and of the K tile of the next step
    int to_v = 0, to_k = 1;
    auto ask = [&](int x, int piece) __attribute__((always_inline)) {
      const int i = piece % P;
      if (piece < P) {
        copy(v_off * 16, v_ch, 1 << VShift, Bufs + to_v, i);
      } else {
        find(x + 1 + Ahead, i);
        copy(0, k_ch, 1, to_k, i);
        look(x + 2 + Ahead, i);
      }
      if (piece == 2 * P - 1) {
        to_v = to_v + 1 == Bufs ? 0 : to_v + 1;
        to_k = to_k + 1 == Bufs ? 0 : to_k + 1;
      }
    };
    // words of LDS that the products read.  V^T: lane (d = lane % 32 of the
    // block, keys 4 hi2 .. +3 of two groups of 8) as the weights have them
    const int vrow = 4 * hi2 + lane % 16 / 4, vch = 2 * (lane % 32 / 16) + lane % 4 / 2, vb = lane % 2 * 8;
    int k_at_lds[KK], v_at_lds[DB];
#pragma unroll
    for (int j = 0; j < KK; ++j) k_at_lds[j] = tiles_at + k_at(ks * NB * 32 + col, 2 * j + hi2) * 16;
#pragma unroll
    for (int d = 0; d < DB; ++d)
      v_at_lds[d] = tiles_at + (Bufs * TileWords + v_at(ks * NB * 32 + vrow, 4 * d + vch)) * 16 + vb;
    // operands of the products: K of 32 rows, V of 16 keys, from LDS byte `at` on
    auto k_words = [&](int at) __attribute__((always_inline)) { return __builtin_bit_cast(bf16x8, *(lds_u32x4)(at)); };
    auto v_words = [&](int at) __attribute__((always_inline)) {
      const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at));
      const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at + 8 * CH * 16));
      return __builtin_bit_cast(bf16x8, s16x8(__builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7)));
    };
    const Mixed mixed = mixed_rows(a, q, tok0, tok1, nonfinite);
    int odd = 0;
    if (kt0 < end) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        look(kt0, i);
        find(kt0, i);
        copy(0, k_ch, 1, 0, i);
        look(kt0 + 1, i);
      }
#pragma unroll
      for (int x = -Ahead; x < 0; ++x)
#pragma unroll
        for (int i = 0; i < 2 * P; ++i) ask(kt0 + x, i);
      // the tree is walked while the first copies are on their way
      if (a.parent && end * KT > q.len) walk_tree<Threads>(a, q, tok0, tok1, par, seen, words);
      if (again)
        odd = uniform(find_nonfinite<Threads, 1, D>(c, table, kv + v_off, page_stride, mixed));
#pragma unroll
      for (int i = 0; i < KK; ++i) qr[i] = (qr[i] ^ flip) & on;
      wait_copies<2 * P * Ahead>();
      lds_barrier();
      if (behind) lds_barrier();
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < KK; ++j)
          sc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k_words(k_at_lds[j] + i * 32 * CH * 16), __builtin_bit_cast(bf16x8, qr[j]), j ? sc[i] : zero, 0, 0, 0);
      if (behind) wait_copies<2 * P * (Ahead - 1)>();  // K of tile kt0 + 1, V of tile kt0
      lds_barrier();
    }
    // a tile: softmax, output, the scores of the next tile (past the last one:
    // not used)
    int v_buf = 0, k_buf = 1;
    for (int kt = kt0; kt < end; ++kt) {
      if ((kt + 1) * KT > clear) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int first = kt * KT + 32 * (ks * NB + i);
          uint32_t word = first < q.len ? ~0u : 0u;
          if (!a.parent || (first + 32 > q.len && first < all)) word = sees(a, q, tok, tok0, first, seen, words);
          word >>= 4 * hi2;
#pragma unroll
          for (int e = 0; e < 16; ++e) sc[i][e] = word >> (8 * (e / 4) + e % 4) & 1 ? sc[i][e] : -INFINITY;
        }
      }
      float top = sc[0][0];
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[i][e]);
      {
        auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
        top = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])) * scale;
      }
      // the maximum is moved only when a row has outgrown it by 2^8: weights
      // stay below 256, and most tiles need no rescaling
      if (__any(top > mx + 8.f)) {
        const float next = fmaxf(mx, top), turn = next == -INFINITY ? 1.f : exp2_fast(mx - next);
        mx = next;
        total_w *= turn;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] *= turn;
      }
      const float at = mx == -INFINITY ? 0.f : mx;
      // the weights, and between them the copies of a step: all at once they
      // would wait for each other's way to LDS.  Up to 64 rows they keep 16 bits,
      // in two parts (15 to 20 drafts behind 64 contexts of 1201 to 2500 tokens 98 ->
      // 102 us, 5 to 31 95.1 -> 96.5); more rows are bound by the products, so theirs are
      // rounded to bf16, as the values that they weigh are (in two parts three
      // prompts of 2300 to 4097 tokens 322 -> 474 us, 63 drafts behind 90000 to
      // 120000 keys 253 -> 358).
      u32x4 pw[2 * NB], pl[2 * NB];
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] = exp2_fast(fmaf(sc[j / 2][j % 2 * 8 + e], scale, -at));
        }
        if constexpr (Fine) split_bf16(w, &pw[j], &pl[j]);
        else pw[j] = u32x4{pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])};
#pragma unroll
        for (int i = j * P / NB; i < (j + 1) * P / NB; ++i) ask(kt, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      // the weights are finished before the barrier: behind it the other
      // wavefront of the SIMD has the vector units
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) asm volatile("" : "+v"(pw[j]));
      // K of tile kt + 1 and V of tile kt are there, of all wavefronts behind the barrier
      if (!behind) wait_copies<2 * P * Ahead>();
      lds_barrier();
      // O^T += V^T P^T, then the scores of the next tile.  The operands come
      // from LDS kAhead products before their use; the order is fixed here
      // because the compiler's own puts every read next to its product
      constexpr int PV = DB * 2 * NB, QK = NB * KK;
      if (odd) {  // the wavefronts write the same
        for (int i = 0; i < NB; ++i) {
          const int block = ks * NB + i;
          for (uint32_t word = mixed.word(kt * KT + 32 * block); word; word &= word - 1) {
            u32x4* p = tiles + (Bufs + v_buf) * TileWords + (32 * block + __builtin_ctz(word)) * CH;
            if (lane < CH) p[lane] = keep_finite<1>(p[lane], true);
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      int k_now[KK], v_now[DB];
#pragma unroll
      for (int j = 0; j < KK; ++j) k_now[j] = k_at_lds[j] + k_buf * (TileWords * 16);
#pragma unroll
      for (int d = 0; d < DB; ++d) v_now[d] = v_at_lds[d] + v_buf * (TileWords * 16);
#pragma unroll
      for (int j = 0; j < KK; ++j) asm volatile("" : "+v"(k_now[j]));
#pragma unroll
      for (int d = 0; d < DB; ++d) asm volatile("" : "+v"(v_now[d]));
      v_buf = k_buf, k_buf = k_buf + 1 == Bufs ? 0 : k_buf + 1;
      auto fetch = [&](int i) __attribute__((always_inline)) {
        if (i < PV) return v_words(v_now[i % DB] + i / DB * (16 * CH * 16));
        return k_words(k_now[(i - PV) / NB] + (i - PV) % NB * (32 * CH * 16));
      };
      bf16x8 f[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i] = fetch(i);
#pragma unroll
      for (int i = 0; i < PV + QK; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if (i < PV) {
          const int j = i / DB, d = i % DB;
          if constexpr (Fine) {
            if (d == 0) total_w = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ones, __builtin_bit_cast(bf16x8, pl[j]), total_w, 0, 0, 0);
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % kAhead], __builtin_bit_cast(bf16x8, pl[j]), o[d], 0, 0, 0);
          }
          if (d == 0) total_w = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ones, __builtin_bit_cast(bf16x8, pw[j]), total_w, 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % kAhead], __builtin_bit_cast(bf16x8, pw[j]), o[d], 0, 0, 0);
        } else {
          const int j = (i - PV) / NB, k = (i - PV) % NB;
          sc[k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % kAhead], __builtin_bit_cast(bf16x8, qr[j]), j ? sc[k] : zero, 0, 0, 0);
        }
        if (i + kAhead < PV + QK) f[i % kAhead] = fetch(i + kAhead);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (behind) wait_copies<2 * P * (Ahead - 1)>();  // K of tile kt + 2, V of tile kt + 1
      lds_barrier();
    }
    if (kt0 < end) {  // the copies asked for past the end, before LDS is used for anything else
      wait_copies<0>();
      if (Behind && !behind) lds_barrier();
      lds_barrier();
    }
    if (!again && kt0 < end && end * KT > mixed.first) {
      const float z = zero_or_nan(o);
      if (__syncthreads_or(z != z)) {
        again = 1, lo = uniform(lo_here);
        continue;
      }
    }
    again = 0;
    float sum = total_w[0];
    if constexpr (KS == 2) {  // the two halves of the keys joined
      static_assert(KS == 1 || RW * DB * 4 * kWave <= 2 * Bufs * TileWords, "the outputs of one half fit the tiles");
      f32x4* buf = reinterpret_cast<f32x4*>(tiles);
      if (ks == 1) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            buf[((rw * DB + d) * 4 + j) * kWave + lane] =
                f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
        if (hi2 == 0) stat[rw * 64 + col] = mx, stat[rw * 64 + 32 + col] = sum;
      }
      lds_barrier();
      if (ks == 0) {
        const float m1 = stat[rw * 64 + col], top = fmaxf(mx, m1), at = top == -INFINITY ? 0.f : top;
        const float mine = part_weight(mx - at), other = part_weight(m1 - at);
        mx = top;
        sum = sum * mine + stat[rw * 64 + 32 + col] * other;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 y = buf[((rw * DB + d) * 4 + j) * kWave + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][4 * j + e] = o[d][4 * j + e] * mine + y[e] * other;
          }
      }
      lds_barrier();
    }
    const bool whole = kt0 == 0 && kt1 == sg.tiles;
    if (ks != 0) {
      // the other half has its outputs
    } else if (whole) {
      if (r < rows) {
        const float inv = 1.f / sum;
        const int64_t at = (int64_t(q.begin + tok) * a.q_heads + h * group + r % group) * D + 4 * hi2;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 x{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
            store4<1>(a.out, at + 32 * d + 8 * j, q.bad ? f32x4{NAN, NAN, NAN, NAN} : x * inv);
          }
      }
    } else {
      float* to = part(c, blockIdx.x, kt0 == 0, part_floats(M, D));
      auto write = [&](auto shared) __attribute__((always_inline)) {
        constexpr bool Shared = decltype(shared)::value;
        if (hi2 == 0) part_store<Shared>(to + rw * 32 + col, mx), part_store<Shared>(to + M + rw * 32 + col, sum);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            part_store<Shared>(reinterpret_cast<f32x4*>(to + 2 * M) + ((rw * DB + d) * 4 + j) * kWave + lane,
                               f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]});
      };
      if (KS == 2 && join) write(std::true_type());
      else write(std::false_type());
      if (kt0 == 0 && tid == 0 && !join) joins(c)[blockIdx.x] = Join{s, h, rt, share_of(total, shares, sg.last)};
    }
    if (odd && ks == 0 && r < rows)  // to the values that this lane has just stored
      for (int at = kt0 * KT; at < end * KT; at += 32)
        for (uint32_t word = mixed.word(at); word; word &= word - 1) {
          const int row = at + __builtin_ctz(word);
          if (row >= limit) break;
          if (!(sees(a, q, tok, tok0, at, seen, words) >> (row & 31) & 1)) continue;
          const u32x4* p = value_row(c, table, kv + v_off, page_stride, CH, row);
#pragma unroll 1
          for (int d = 0; d < 4 * DB; ++d) {
            const f32x4 x = odd_values<1>(p, 8 * d + 4 * hi2);
            if (whole) {
              const int64_t out = (int64_t(q.begin + tok) * a.q_heads + h * group + r % group) * D + 8 * d + 4 * hi2;
              const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const char*>(a.out) + out * 2);
              store4<1>(a.out, out, x + f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u),
                                              __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xffff0000u)});
            } else {
              f32x4* to = reinterpret_cast<f32x4*>(part(c, blockIdx.x, kt0 == 0, part_floats(M, D)) + 2 * M) + (rw * DB * 4 + d) * kWave + lane;
              if (KS == 2 && join) part_store<true>(to, part_load<true>(to) + x);
              else *to += x;
            }
          }
        }
    if (odd) lds_barrier();  // the next segment's tree comes after the last use of this one's
    if constexpr (KS == 2)
      if (join && !whole) {
        const int first = share_of(total, shares, sg.first), last = share_of(total, shares, sg.last);
        if (last_to_arrive(c, first, last)) {
          for (int i = tid; i < M * D / 4; i += Threads) join_parts<1, D, true>(c, a, Join{s, h, rt, last}, first, M, 1, i);
        }
        lds_barrier();
      }
  }
}

// Joins the parts of the segment blockIdx.x of those that several shares have;
// they are found by the shares in which one starts.  A thread takes 4 values of
// a row; with few segments (long contexts of few heads: many parts each), G
// threads take them, each a run of the parts: the join is bound by the loads'
// latency (calls of 18 drafts over 10000 keys of 2 heads 47 -> 16 us, of 30
// over 30000 of one head 123 -> 31).
template <int D, int G>
__global__ __launch_bounds__(256) void combine_kernel(KvCache c, KvAttention a, int shares, int M) {
  const int tid = threadIdx.x;
  int first = blockIdx.x;
  if (int(gridDim.x) < shares) {
    __shared__ int count[4], start;
    int before = blockIdx.x;  // segments to go
    if (tid == 0) start = -1;
    __syncthreads();
    for (int base = 0; base < shares; base += 256) {
      const bool here = base + tid < shares && joins(c)[min(base + tid, shares - 1)].last >= 0;
      const uint64_t all = __ballot(here);
      if (tid % kWave == 0) count[tid / kWave] = __popcll(all);
      __syncthreads();
      int rank = __popcll(all & ((uint64_t(1) << tid % kWave) - 1)), sum = 0;
      for (int i = 0; i < 4; ++i) {
        if (i < tid / kWave) rank += count[i];
        sum += count[i];
      }
      if (here && rank == before) start = base + tid;
      before -= sum;
      __syncthreads();
    }
    first = start;
    if (first < 0) return;
  }
  const Join j = joins(c)[first];
  if (j.last < 0) return;
  if constexpr (G == 1) {
    for (int i = blockIdx.y * 256 + tid; i < M * D / 4; i += gridDim.y * 256) join_parts<1, D, false>(c, a, j, first, M, 1, i);
  } else {
    __shared__ float stat[2][256];
    __shared__ f32x4 values[256];
    const int parts = j.last - first + 1, each = (parts + G - 1) / G, g = tid / (256 / G);
    const int i = blockIdx.y * (256 / G) + tid % (256 / G);
    int row, column;
    part_place<D>(i, 1, &row, &column);
    Sum sum;
    if (row < M) sum = sum_parts<D, false>(c, first, first + g * each, min(j.last, first + (g + 1) * each - 1), M, row, i);
    stat[0][tid] = sum.top, stat[1][tid] = sum.l, values[tid] = sum.x;
    __syncthreads();
    if (g == 0 && row < M) {
      float top = sum.top;
      for (int o = 1; o < G; ++o) top = fmaxf(top, stat[0][tid + o * (256 / G)]);
      const float at = top == -INFINITY ? 0.f : top;
      Sum all{top, 0.f, f32x4{0.f, 0.f, 0.f, 0.f}};
      for (int o = 0; o < G; ++o) {
        const float now = part_weight(stat[0][tid + o * (256 / G)] - at);
        all.l += stat[1][tid + o * (256 / G)] * now, all.x += values[tid + o * (256 / G)] * now;
      }
      store_joined<1, D>(a, c, j, M, row, column, all);
    }
  }
}

// Row tiles of all sequences and key heads, at most.
int64_t segments_of(const KvCache& c, const KvAttention& a, int rows) {
  return (int64_t(a.T) * (a.q_heads / c.kv_heads) / rows + c.seqs) * c.kv_heads;
}

template <int DT, int D, int MT>
hipError_t few_rows(const KvCache& c, const KvAttention& a, hipStream_t s) {
  const int64_t segments = segments_of(c, a, 16 * MT);
  if (segments >= (int64_t(1) << 32) / kBlock) return hipErrorInvalidValue;
  // more segments than shares: whole ones of prompts only (the contexts of
  // tokens and drafts differ)
  const bool prompts = !a.parent && a.max_new * (a.q_heads / c.kv_heads) > 16 * MT;
  few_rows_kernel<DT, D, MT><<<prompts ? int(std::max<int64_t>(segments, kShares)) : kShares, kBlock, 0, s>>>(c, a, kShares, kEither);
  return hipGetLastError();
}

template <int D, int RW, int KS, bool AnyTree = false>
hipError_t many_rows(const KvCache& c, const KvAttention& a, hipStream_t s) {
  constexpr int M = 32 * RW, Threads = RW * KS * kWave;
  const int64_t segments = segments_of(c, a, M);
  if (segments >= (int64_t(1) << 32) / Threads) return hipErrorInvalidValue;
  // workgroups that the chip holds at once
  constexpr int kFit = Threads == 512 || D == 256 || AnyTree ? kManyShares : 2 * kManyShares;
  const int64_t group = a.q_heads / c.kv_heads, longest = ((int64_t(c.max_pages) << c.page_shift) + 63) / 64;
  // prompts that are whole segments by my_share's last rule, however long their
  // contexts are: T tokens of `seqs` sequences have at least these units (the
  // launch that would join parts is saved, 3 to 5 us)
  const double units = (double(a.T) * a.T * group / (2.0 * 64 * c.seqs) + double(kOpen) * a.T * group) / M * c.kv_heads;
  const int split = a.parent || 1.34 * longest * kFit > units ? kEither : kWhole;
  const int joined = static_cast<int>(std::min<int64_t>(segments, kFit));  // at most: one starts in a share
  // small parts, and few of a segment: joined by the last of its workgroups (5 to
  // 31 drafts behind 64 contexts of 1201 to 2500 tokens 98 -> 96 us; 8 drafts behind 8
  // of 20000 to 30000, with 8 parts of a segment, 162 -> 165)
  const int join = KS == 2 && 2 * joined > kFit;
  many_rows_kernel<D, RW, KS, AnyTree><<<int(std::max<int64_t>(segments, kFit)), Threads, 0, s>>>(c, a, kFit, split, tree_words<RW, AnyTree>(group), join);
  if (hipError_t e = hipGetLastError(); e != hipSuccess || split == kWhole || join) return e;
  // few segments have many parts; else as many workgroups as are quickly gone
  // where there is nothing to join
  if (8 * joined <= kFit) combine_kernel<D, 8><<<dim3(joined, M * D / 4 / 32), 256, 0, s>>>(c, a, kFit, M);
  else combine_kernel<D, 1><<<dim3(joined, std::max(1, std::min(4096 / joined, M * D / 4 / 256))), 256, 0, s>>>(c, a, kFit, M);
  return hipGetLastError();
}

template <int DT, int D>
hipError_t launch(const KvCache& c, const KvAttention& a, hipStream_t s) {
  const int64_t group = a.q_heads / c.kv_heads, rows = a.max_new * group;
  if (rows <= 16) return few_rows<DT, D, 1>(c, a, s);
  if constexpr (DT == 0) {
    if constexpr (D == 256) return few_rows<DT, D, 1>(c, a, s);
    else return few_rows<DT, D, 2>(c, a, s);
  } else if constexpr (D == 256) {
    return rows > 64 ? many_rows<D, 4, 1, true>(c, a, s) : many_rows<D, 2, 2>(c, a, s);
  } else {
    if (a.parent && a.max_new > 512 && group == 1) return many_rows<D, 4, 1, true>(c, a, s);  // the table of drafts
    // 256 rows a workgroup have the faster loop (16 x 1000 tokens of 32 query
    // heads 249 against 256 us, one of 512 tokens behind 30000 255 against 285),
    // two workgroups of 128 rows overlap their starts and ends, which are most
    // of a short prompt (64 x 300 tokens of 16 query heads 98 against 120 us,
    // 32 x 600 117 against 137)
    const bool short_prompts = !a.parent && a.T * group < 4096ll * c.seqs && segments_of(c, a, 256) >= 2 * kManyShares;
    if (rows > 128 && !short_prompts) return many_rows<D, 8, 1>(c, a, s);
    if (rows > 64) return many_rows<D, 4, 1>(c, a, s);
    return rows > 32 ? many_rows<D, 2, 2>(c, a, s) : many_rows<D, 1, 2>(c, a, s);
  }
}

template <int DT>
hipError_t launch(const KvCache& c, const KvAttention& a, hipStream_t s) {
  if (c.head_dim == 64) return launch<DT, 64>(c, a, s);
  if (c.head_dim == 128) return launch<DT, 128>(c, a, s);
  return launch<DT, 256>(c, a, s);
}

}  // namespace

int64_t kv_attention_work_bytes(const KvCache& c) {
  // two parts of a share: at most 128 rows in each of kShares, or 256 in each of
  // half as many; heads of 256: 128 in each of kManyShares
  return kWorkCounts + round256(kShares * int64_t(sizeof(Join))) +
         2 * 4 * (c.head_dim == 256 ? kManyShares : kShares) * part_floats(128, c.head_dim);
}

hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, hipStream_t s) {
  return c.dtype == TMS_F32 ? launch<0>(c, a, s) : launch<1>(c, a, s);
}

}  // namespace tms
