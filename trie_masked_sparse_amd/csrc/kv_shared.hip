// Attention of a batch whose sequences hold the same pages: each page is read
// once for the query rows of all of them, for gfx950.
//
// Mathematics.  A row's keys are cut into runs: runs of pages that several
// sequences hold at the same places, and what a sequence has for itself.  With
// m the maximum of a run's scores (times log2(e)), l the sum of the weights
// relative to it and o their sum of values,
//     m = max m_i,  l = sum_i l_i 2^(m_i - m),  out = sum_i o_i 2^(m_i - m) / l.
// A node is a run of pages with the query rows of the sequences that hold it.
//
// Work memory ("plan"), made by plan_kernel from the cache's tables and used
// for every layer: see Plan.
#include <algorithm>
#include <climits>

#include "kv_many.h"

namespace tms {
namespace {

constexpr int kLevels = 3;      // nodes of a sequence beside its own
constexpr int kSeqs = 4096;     // sequences of a cache, at most
constexpr int kPlan = 1024, kPlanWaves = kPlan / kWave;
constexpr int kSlots = 512;     // workgroups that a launch should have
constexpr int kTile = 64;       // keys that the plan counts in
constexpr int kSmall = 16;      // rows of a small node
constexpr int kMagic = 0x73686172;

// Sequences of more rows of a key head than this read their pages for
// themselves: the products bound them, and many rows share a page's read already.
constexpr int kMostRowsShared = 128;

// A node pays where the keys that are not read again (its keys, times the
// readers that it saves) are more than these and what its rows' parts cost: a
// part is written and read, 8 bytes a value, a key 2 values of the cache's type.
constexpr int kLeastSaved = 256;
__device__ inline bool pays(int64_t keys, int64_t readers, int64_t rows, int dtype) {
  return keys * readers >= kLeastSaved + (dtype == 0 ? 2 : 4) * rows;
}

constexpr int kRounds = 8;

// Key tiles of a chunk, at least.
constexpr int kLeastTiles = 4;

struct Head {
  int32_t magic, T, q_heads, units, nodes, rows, pad[2];
};

struct PlanSeq {
  int32_t begin, n, len, levels;               // tokens, committed rows; nodes (-1: its outputs are NaN)
  int32_t node[kLevels + 1], at[kLevels + 1];  // nodes, and where its tokens are among a node's
};

struct Node {
  int32_t seq, key0, keys;   // the sequence whose table has the pages; first row, rows
  int32_t tokens, list;      // query tokens; their place in the list, -1: begin ..
  int32_t begin, n, len;     // of one sequence's own: its new tokens, committed rows from key0 on
  int32_t unit, chunks, tiles, rows;  // first unit, chunks of `tiles` key tiles, rows of a row tile
  int64_t part;              // first row of its parts
};

// Places in the plan.  M: rows of a tile of nodes that are not small.
struct Layout {
  int64_t seqs, nodes, units, tokens, owner, stats, values, bytes;
  int32_t most_nodes, most_units;
  int64_t most_rows;
};

int64_t up(int64_t x) { return (x + 255) & ~int64_t(255); }

Layout layout(const KvCache& c, int32_t T, int32_t q_heads, int M) {
  Layout y{};
  const int64_t group = q_heads / c.kv_heads, n = std::min<int64_t>(c.seqs, T);
  y.most_nodes = static_cast<int32_t>(n + kLevels * (n / 2));
  // a node's row tiles, each cut at most as often as fills the chip
  const int64_t tiles = (kLevels + 1) * (int64_t(T) * group / std::max(M, kSmall)) + y.most_nodes;
  y.most_units = static_cast<int32_t>(tiles + kSlots / c.kv_heads + 1);
  y.most_rows = (kLevels + 1) * int64_t(T) * q_heads + (kSlots + c.kv_heads) * int64_t(M);
  y.seqs = up(sizeof(Head));
  y.nodes = up(y.seqs + c.seqs * int64_t(sizeof(PlanSeq)));
  y.units = up(y.nodes + y.most_nodes * int64_t(sizeof(Node)));
  y.tokens = up(y.units + y.most_units * int64_t(4));
  y.owner = up(y.tokens + kLevels * int64_t(T) * 4);
  y.stats = up(y.owner + int64_t(T) * 4);
  y.values = up(y.stats + y.most_rows * 8);
  y.bytes = up(y.values + y.most_rows * c.head_dim * 4);
  return y;
}

struct Plan {
  char* at;
  Layout y;
  __device__ Head* head() const { return reinterpret_cast<Head*>(at); }
  __device__ PlanSeq* seqs() const { return reinterpret_cast<PlanSeq*>(at + y.seqs); }
  __device__ Node* nodes() const { return reinterpret_cast<Node*>(at + y.nodes); }
  __device__ int32_t* units() const { return reinterpret_cast<int32_t*>(at + y.units); }    // node of every unit
  __device__ int32_t* tokens() const { return reinterpret_cast<int32_t*>(at + y.tokens); }  // of the nodes, a list for each level
  __device__ int32_t* owner() const { return reinterpret_cast<int32_t*>(at + y.owner); }    // sequence of every token, -1
  __host__ __device__ Parts parts() const {
    return Parts{reinterpret_cast<float*>(at + y.values), reinterpret_cast<float2*>(at + y.stats)};
  }
};

// Pages that the sequences first, first + step, ... (kTogether of them) have in
// common with their leaders, from their next pages on, where redo says so; by one
// wavefront.
constexpr int kTogether = 4;
template <class Redo>
__device__ inline void common(const KvCache& c, int n, int first, int step, const int* lead, const int* pos, const int* whole,
                              int* same, Redo redo) {
  constexpr int kLoads = 6;
  const int lane = threadIdx.x % kWave;
  int at[kTogether], most[kTogether];
  const int32_t *x[kTogether], *y[kTogether];
  bool left = false;
#pragma unroll
  for (int i = 0; i < kTogether; ++i) {
    const int s = min(first + i * step, n - 1), t = uniform(lead[s]);
    at[i] = most[i] = 0;
    x[i] = c.table + int64_t(s) * c.max_pages, y[i] = c.table + int64_t(t) * c.max_pages;
    if (first + i * step >= n || !redo(s)) continue;
    if (lane == 0) same[s] = 0;
    if (t == s) continue;
    at[i] = uniform(pos[s]), most[i] = uniform(min(whole[s], whole[t]));
    left |= at[i] < most[i];
  }
  while (left) {
    int a[kTogether][kLoads], b[kTogether][kLoads];
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
      if (at[i] < most[i])
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int j = min(at[i] + u * kWave + lane, most[i] - 1);
          a[i][u] = x[i][j], b[i][u] = y[i][j];
        }
    left = false;
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      if (at[i] >= most[i]) continue;
      const int s = first + i * step;
      int end = -1;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const uint64_t differ = __ballot(a[i][u] != b[i][u] || at[i] + u * kWave + lane >= most[i]);
        if (differ && end < 0) end = min(at[i] + u * kWave + __builtin_ctzll(differ), most[i]);
      }
      at[i] += kLoads * kWave;
      if (end < 0 && at[i] >= most[i]) end = most[i];
      if (end >= 0) {
        if (lane == 0) same[s] = end - pos[s];
        at[i] = most[i];
      } else {
        left = true;
      }
    }
  }
}

// Sums over the workgroup's threads before this one, and of all; `sums` is free
// again behind the next barrier.
template <typename T>
__device__ inline T threads_before(T mine, T* sums, T* total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  T incl = mine;
#pragma unroll
  for (int step = 1; step < kWave; step *= 2) {
    const T x = __shfl_up(incl, step);
    if (lane >= step) incl += x;
  }
  if (lane == kWave - 1) sums[wave] = incl;
  __syncthreads();
  T before = incl - mine;
  *total = 0;
  for (int w = 0; w < kPlanWaves; ++w) {
    if (w < wave) before += sums[w];
    *total += sums[w];
  }
  return before;
}

// One workgroup.  In every round, sequences that have the same next page form a
// group; its first sequence is the leader.  The pages that the whole group has
// make a node, if that pays: without it, every branch of the group (sequences
// that have the same page behind them) would read them.  Else every branch is
// a group, and the cut that saves most reads (pages in common with the leader,
// times the sequences that have them but one) makes a node.  The sequences of a
// node go on behind it in the next round.  Pages are compared one by one, so a
// table that no fork has made is planned rightly too.
//
// Bound by latency: a dozen reads of global memory one after the other, and the
// walks of every sequence over all, which are shared by the threads that are to
// spare, 4 sequences a step.
__global__ __launch_bounds__(kPlan) void plan_kernel(KvCache c, KvAttention a, Plan plan, int M) {
  // of every sequence: its next page's number, then the leader of the node that
  // it is in; its group's leader; pages that it is past; pages in common with
  // the leader; tokens (0: none to plan); whole pages of committed rows.  Of a
  // leader: pages of its node; the fewest that one of its group has in common;
  // branches and tokens of its group
  __shared__ int next[kSeqs], lead[kSeqs], pos[kSeqs], same[kSeqs], count[kSeqs], whole[kSeqs], cut[kSeqs];
  __shared__ union {
    unsigned long long best[kSeqs];
    struct {
      int fewest[kSeqs], branches[kSeqs];
    } of;
  } lds;
  __shared__ int nodes_s, list_s, big_s;
  __shared__ int64_t sums[3][kPlanWaves];
  __shared__ int sums32[kPlanWaves];
  constexpr int kEach = kSeqs / kPlan;
  const int tid = threadIdx.x, wave = uniform(tid / kWave), lane = tid % kWave, n = c.seqs, group = a.q_heads / c.kv_heads;
  const int n4 = (n + 3) / 4;
  int parts = 1;  // threads of a sequence, adjacent lanes
  while (parts < kWave && 2 * parts * n <= kPlan) parts *= 2;
  const int first = tid / parts, share = tid % parts;
  auto each_seq = [&](auto f) __attribute__((always_inline)) {  // f(i, s), of every sequence of this thread
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (first + i * kPlan < n) f(i, first + i * kPlan);
  };
  auto all_of = [&](int x, auto join) __attribute__((always_inline)) {  // over the threads of a sequence
    for (int step = 1; step < parts; step *= 2) x = join(x, __shfl_xor(x, step));
    return x;
  };
  auto plus = [](int x, int y) { return x + y; };
  auto fours = [](const int* x, int j) { return reinterpret_cast<const int4*>(x)[j]; };
  a.max_new = INT_MAX;
  if (tid == 0) nodes_s = list_s = big_s = 0;
  for (int i = tid; i < a.T; i += kPlan) plan.owner()[i] = -1;
  if (tid < n4 * 4 - n) {  // so that sequences are taken 4 at a time
    next[n + tid] = INT_MAX, count[n + tid] = 0, lead[n + tid] = pos[n + tid] = same[n + tid] = -1;
  }
  PlanSeq mine[kEach];
  int64_t tokens = 0, all_tokens;
  each_seq([&](int i, int s) __attribute__((always_inline)) {
    const Seq q = sequence(c, a, s, 1, 1);
    const bool on = q.n && !q.bad;
    mine[i].begin = q.begin, mine[i].n = q.n, mine[i].len = q.len, mine[i].levels = on ? 0 : -1;
    if (share == 0) {
      count[s] = on ? q.n : 0, pos[s] = 0;
      whole[s] = on && int64_t(q.n) * group <= kMostRowsShared ? q.len >> c.page_shift : 0;
      same[s] = q.begin, lead[s] = q.n;
      tokens += on ? q.n : 0;
    }
  });
  // tokens that two sequences claim (start not ascending) would not fit the lists
  threads_before(tokens, sums[0], &all_tokens);
  if (all_tokens > a.T) {
    if (tid == 0) *plan.head() = Head{};
    return;
  }
  for (int s = wave; s < n; s += kPlanWaves)
    for (int i = lane; i < lead[s]; i += kWave) plan.owner()[same[s] + i] = s;
  for (int round = 0; round < kRounds; ++round) {
    __syncthreads();
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      if (share) return;
      next[s] = pos[s] < whole[s] && mine[i].levels < kLevels ? c.table[int64_t(s) * c.max_pages + pos[s]] : -1;
      lds.of.fewest[s] = INT_MAX, lds.of.branches[s] = 0, cut[s] = 0;
    });
    __syncthreads();
    // the first sequence with the same x and the same y
    auto first_like = [&](int s, const int* x, const int* y) __attribute__((always_inline)) {
      const int u = x[s], v = y[s];
      int t = s;
      if (u >= 0)
        for (int j = share; j * 4 < s; j += parts) {
          const int4 p = fours(x, j), q = fours(y, j);
          const int hit = p.x == u && q.x == v ? 0 : p.y == u && q.y == v ? 1 : p.z == u && q.z == v ? 2 : p.w == u && q.w == v ? 3 : 4;
          if (hit < 4) {
            t = min(4 * j + hit, s);
            break;
          }
        }
      return all_of(t, [](int x, int y) { return min(x, y); });
    };
    bool groups = false;
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      const int t = first_like(s, next, pos);
      if (share == 0) lead[s] = t;
      groups |= t != s;
    });
    if (!__syncthreads_or(groups)) break;
    for (int s = wave; s < n; s += kTogether * kPlanWaves) common(c, n, s, kPlanWaves, lead, pos, whole, same, [](int) { return true; });
    __syncthreads();
    each_seq([&](int, int s) __attribute__((always_inline)) {
      if (share == 0 && lead[s] != s) atomicMin(&lds.of.fewest[lead[s]], same[s]);
    });
    __syncthreads();
    each_seq([&](int, int s) __attribute__((always_inline)) {  // the page behind what all have
      if (share) return;
      const int d = lds.of.fewest[lead[s]], p = pos[s] + d;
      next[s] = d < INT_MAX && p < whole[s] ? c.table[int64_t(s) * c.max_pages + p] : -1;
    });
    __syncthreads();
    int branch[kEach];
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      branch[i] = first_like(s, next, lead);
      if (share == 0 && branch[i] == s) atomicAdd(&lds.of.branches[lead[s]], 1);
    });
    __syncthreads();
    bool any = false, redo = false;
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      const int l = lead[s], d = lds.of.fewest[l];
      if (d == INT_MAX) return;  // alone
      int tokens = 0;
      for (int j = share; j < n4; j += parts) {
        const int4 x = fours(lead, j), k = fours(count, j);
        tokens += (x.x == l ? k.x : 0) + (x.y == l ? k.y : 0) + (x.z == l ? k.z : 0) + (x.w == l ? k.w : 0);
      }
      tokens = all_of(tokens, plus);
      const bool all = d > 0 && pays(int64_t(d) << c.page_shift, lds.of.branches[l] - 1, int64_t(tokens) * group, c.dtype);
      if (all && share == 0 && s == l) cut[s] = d;
      if (all) branch[i] = -1;  // in the node of the whole group
    });
    __syncthreads();
    // groups that have no node: their branches
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      const bool other = branch[i] >= 0 && lds.of.fewest[lead[s]] < INT_MAX && branch[i] != lead[s];
      if (share == 0) next[s] = other;
      redo |= other;
      if (share == 0 && other) lead[s] = branch[i];
    });
    if (__syncthreads_or(redo)) {
      for (int s = wave; s < n; s += kTogether * kPlanWaves)
        common(c, n, s, kPlanWaves, lead, pos, whole, same, [&](int s) { return uniform(next[s]) != 0; });
      __syncthreads();
    }
    each_seq([&](int, int s) __attribute__((always_inline)) {
      if (share == 0) lds.best[s] = 0;
    });
    __syncthreads();
    unsigned long long saved[kEach];
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      saved[i] = 0;
      const int l = lead[s], d = same[s];
      if (l == s || cut[l] > 0 || d == 0) return;
      int m = 0, tokens = 0;  // of those that have d pages in common with the leader
      for (int j = l / 4 + share; j < n4; j += parts) {
        const int4 y = fours(lead, j), z = fours(same, j), k = fours(count, j);
        auto one = [&](int y, int z, int k) {
          const bool on = y == l && z >= d;
          m += on, tokens += on ? k : 0;
        };
        one(y.x, z.x, k.x), one(y.y, z.y, k.y), one(y.z, z.z, k.z), one(y.w, z.w, k.w);
      }
      m = all_of(m, plus), tokens = all_of(tokens, plus) + count[l];
      if (pays(int64_t(d) << c.page_shift, m, int64_t(tokens) * group, c.dtype)) saved[i] = static_cast<unsigned long long>(d) * m;
      if (share == 0 && saved[i]) atomicMax(&lds.best[l], saved[i]);
    });
    __syncthreads();
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      if (share == 0 && saved[i] && saved[i] == lds.best[lead[s]]) atomicMax(&cut[lead[s]], same[s]);
    });
    __syncthreads();
    each_seq([&](int, int s) __attribute__((always_inline)) {
      const int d = cut[lead[s]];
      any |= d > 0;
      if (share == 0) next[s] = d > 0 && (lead[s] == s || same[s] >= d) ? lead[s] : INT_MAX;
    });
    if (!__syncthreads_or(any)) break;
    const int first_node = nodes_s, first_token = list_s;
    __syncthreads();
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      const int l = next[s];
      if (l == INT_MAX) return;
      // the lists of a round: nodes in the order of their leaders, tokens in the
      // order of their sequences
      int node = 0, list = 0, at = 0, of_node = 0;
      for (int j = share; j < n4; j += parts) {
        const int4 x = fours(next, j), k = fours(count, j);
        auto one = [&](int t, int y, int z) {
          node += y == t && t < l;
          list += y < l ? z : 0;
          of_node += y == l ? z : 0;
          at += y == l && t < s ? z : 0;
        };
        one(4 * j, x.x, k.x), one(4 * j + 1, x.y, k.y), one(4 * j + 2, x.z, k.z), one(4 * j + 3, x.w, k.w);
      }
      node = first_node + all_of(node, plus), list = first_token + all_of(list, plus);
      of_node = all_of(of_node, plus), at = all_of(at, plus);
      PlanSeq& p = mine[i];
      for (int u = share; u < count[s]; u += parts) plan.tokens()[list + at + u] = p.begin + u;
#pragma unroll
      for (int v = 0; v < kLevels; ++v)
        if (p.levels == v) p.node[v] = node, p.at[v] = at;
      ++p.levels;
      if (s == l && share == 0) {
        Node x{};
        x.seq = s, x.key0 = pos[s] << c.page_shift, x.keys = cut[s] << c.page_shift;
        x.tokens = of_node, x.list = list;
        plan.nodes()[node] = x;
        atomicAdd(&nodes_s, 1), atomicAdd(&list_s, of_node);
      }
    });
    __syncthreads();
    each_seq([&](int, int s) __attribute__((always_inline)) {
      if (share == 0 && next[s] != INT_MAX) pos[s] += cut[next[s]];
    });
  }
  __syncthreads();
  // what every sequence has for itself
  int nodes = nodes_s;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (i * kPlan >= n) continue;
    const int s = first + i * kPlan;
    const bool on = share == 0 && s < n && count[s] > 0;
    int total;
    const int node = nodes + threads_before(int(on), sums32, &total);
    nodes += total;
    __syncthreads();
    if (s >= n || share) continue;
    PlanSeq& p = mine[i];
    if (on) {
      Node x{};
      x.seq = s, x.key0 = pos[s] << c.page_shift;
      x.len = p.len - x.key0, x.n = p.n, x.keys = x.len + x.n, x.begin = p.begin;
      x.tokens = p.n, x.list = -1;
      plan.nodes()[node] = x;
#pragma unroll
      for (int v = 0; v <= kLevels; ++v)
        if (p.levels == v) p.node[v] = node, p.at[v] = 0;
      ++p.levels;
    }
    plan.seqs()[s] = p;
  }
  __syncthreads();
  // chunks of the keys, equal for all, so that there is a workgroup for each slot
  const int each = (nodes + kPlan - 1) / kPlan, from = min(tid * each, nodes), to = min(from + each, nodes);
  struct Size {
    int rows, row_tiles, key_tiles;
  };
  auto size = [&](const Node& x) {
    const int64_t rows = int64_t(x.tokens) * group;
    const int of = rows <= kSmall ? kSmall : M;
    return Size{of, static_cast<int>((rows + of - 1) / of), (x.keys + kTile - 1) / kTile};
  };
  int64_t work = 0, total;
  for (int i = from; i < to; ++i) {
    const Size z = size(plan.nodes()[i]);
    work += int64_t(z.row_tiles) * z.key_tiles;
  }
  threads_before(work, sums[0], &total);
  const int64_t tiles = max(int64_t(kLeastTiles), (total * c.kv_heads + kSlots - 1) / kSlots);
  auto chunks = [&](const Size& z) { return static_cast<int>((z.key_tiles + tiles - 1) / tiles); };
  int64_t units = 0, rows = 0, all_units, all_rows;
  for (int i = from; i < to; ++i) {
    const Node& x = plan.nodes()[i];
    const Size z = size(x);
    units += int64_t(z.row_tiles) * chunks(z), rows += int64_t(x.tokens) * a.q_heads * chunks(z);
  }
  units = threads_before(units, sums[1], &all_units), rows = threads_before(rows, sums[2], &all_rows);
  const bool fits = all_units <= plan.y.most_units && all_rows <= plan.y.most_rows;
  for (int i = from; fits && i < to; ++i) {
    Node& x = plan.nodes()[i];
    const Size z = size(x);
    x.chunks = chunks(z), x.tiles = static_cast<int>(min(tiles, int64_t(z.key_tiles))), x.rows = z.rows;
    x.unit = static_cast<int>(units), x.part = rows;
    const int count_here = z.row_tiles * x.chunks;
    if (count_here <= 2) {
      for (int u = 0; u < count_here; ++u) plan.units()[units + u] = i;
    } else {  // many: by all threads
      const int at = atomicAdd(&big_s, 1);
      if (at < kSeqs) next[at] = i, lead[at] = static_cast<int>(units), pos[at] = count_here;
      else
        for (int u = 0; u < count_here; ++u) plan.units()[units + u] = i;
    }
    units += z.row_tiles * x.chunks, rows += int64_t(x.tokens) * a.q_heads * x.chunks;
  }
  __syncthreads();
  const int big = min(big_s, kSeqs);
  for (int b = wave; b < big; b += kPlanWaves)
    for (int u = lane; u < pos[b]; u += kWave) plan.units()[lead[b] + u] = next[b];
  if (tid == 0) *plan.head() = Head{fits ? kMagic : 0, a.T, a.q_heads, fits ? int(all_units) : 0, nodes, M, {}};
}

// Whether the plan is one for this call.
__device__ inline bool planned(const Plan& plan, const KvAttention& a, int M) {
  const Head* h = plan.head();
  return h->magic == kMagic && h->T == a.T && h->q_heads == a.q_heads && h->rows == M;
}

// First part row of row tile rt, chunk k of a node and key head: a chunk's parts
// are the tile's rows for head 0, then for head 1, ...
__device__ inline int64_t part_row(const KvCache& c, const Node& x, int group, int rt, int k, int h) {
  const int64_t all = int64_t(x.tokens) * group, first = int64_t(rt) * x.rows, rows = min(int64_t(x.rows), all - first);
  return x.part + c.kv_heads * (first * x.chunks + k * rows) + h * rows;
}

// What a node that is not small is worked on by.
enum { kFew16 = 0, kFew32, kMany64, kMany128 };
constexpr int rows_of(int shape) { return shape == kFew16 ? 16 : shape == kFew32 ? 32 : shape == kMany64 ? 64 : 128; }

template <int DT, int D, int Shape>
struct Body {
  using Type = FewRows<DT, D, Shape == kFew32 ? 2 : 1>;
};
template <int D>
struct Body<1, D, kMany64> {
  using Type = ManyRows<D, 2, 2>;
};
template <int D>
struct Body<1, D, kMany128> {
  using Type = ManyRows<D, 4, 1>;
};

// A unit of the plan (row tile and chunk of a node) and a key head.
template <int DT, int D, int Shape>
__global__ __launch_bounds__(kBlock, D == 256 ? 1 : 2) void nodes_kernel(KvCache c, KvAttention a, Plan plan) {
  using Small = FewRows<DT, D, 1>;
  using Large = typename Body<DT, D, Shape>::Type;
  __shared__ union {
    typename Small::Lds small;
    typename Large::Lds large;
  } lds;
  const int h = blockIdx.x % c.kv_heads, unit = blockIdx.x / c.kv_heads;
  if (!planned(plan, a, rows_of(Shape)) || unit >= plan.head()->units) return;
  const Node& at = plan.nodes()[plan.units()[unit]];
  Node x;
  x.seq = uniform(at.seq), x.key0 = uniform(at.key0), x.keys = uniform(at.keys), x.tokens = uniform(at.tokens);
  x.list = uniform(at.list), x.begin = uniform(at.begin), x.n = uniform(at.n), x.len = uniform(at.len);
  x.unit = uniform(at.unit), x.chunks = uniform(at.chunks), x.tiles = uniform(at.tiles), x.rows = uniform(at.rows);
  x.part = uniform(at.part);
  const int group = a.q_heads / c.kv_heads, all = x.tokens * group;
  const int rt = (unit - x.unit) / x.chunks, k = (unit - x.unit) % x.chunks, row0 = rt * x.rows, rows = min(x.rows, all - row0);
  const int32_t* table = c.table + int64_t(x.seq) * c.max_pages + (x.key0 >> c.page_shift);
  const int32_t* list = plan.tokens() + max(x.list, 0);
  const bool own = x.list < 0;  // keys of one sequence, its new rows among them
  if (own && x.n > a.max_new) return;
  FewTile t{};
  t.h = h;
  if (own) {
    t.q.begin = x.begin, t.q.n = x.n, t.q.len = x.len;
    t.tok0 = row0 / group, t.tok1 = (row0 + rows - 1) / group;
    t.limit = a.parent ? x.keys : x.len + t.tok1 + 1;
  } else {  // all rows see all keys
    a.parent = nullptr;
    t.q.len = t.limit = x.keys;
    t.tok0 = t.tok1 = -1;
  }
  auto query = [&](int r) {
    const int row = row0 + min(r, rows - 1), i = row / group;
    const int token = own ? x.begin + i : list[i];
    return int64_t(token) * a.ldq + int64_t(h * group + row % group) * D;
  };
  auto token = [&](int r) { return own && r < rows ? (row0 + r) / group : -1; };
  const Parts parts = plan.parts();
  const int64_t part = part_row(c, x, group, rt, k, h);
  auto emit = [&](int r, int column, f32x4 v, float top, float l) {
    if (r >= rows) return;
    *reinterpret_cast<f32x4*>(parts.values + (part + r) * D + column) = v;
    if (column == 0) parts.stats[part + r] = float2{top, l};
  };
  auto tiles = [&](int keys) {  // key tiles of this many keys
    t.kt0 = k * x.tiles * (kTile / keys);
    t.kt1 = min(t.kt0 + x.tiles * (kTile / keys), (x.keys + keys - 1) / keys);
  };
  auto page_at = [&](int key) { return max(0, min(table[key >> c.page_shift], c.pages - 1)); };
  if (Shape == kFew16 || x.rows == kSmall) {
    tiles(Small::KW);
    Small::run(c, a, lds.small, t, page_at, query, token, emit);
  } else if constexpr (Shape == kFew32) {
    tiles(Large::KW);
    Large::run(c, a, lds.large, t, page_at, query, token, emit);
  } else if constexpr (Shape >= kMany64) {
    tiles(Large::KT);
    Large::run(c, a, lds.large, t, table, query, token, emit);
  }
}

// The parts of a token and query head over all its nodes: D / 4 threads to a row.
template <int DT, int D>
__global__ __launch_bounds__(kBlock) void join_nodes_kernel(KvCache c, KvAttention a, Plan plan, int M) {
  const int64_t row = int64_t(blockIdx.x) * (kBlock * 4 / D) + threadIdx.x / (D / 4);
  if (row >= int64_t(a.T) * a.q_heads) return;
  const int column = threadIdx.x % (D / 4) * 4, t = static_cast<int>(row / a.q_heads), head = static_cast<int>(row % a.q_heads);
  const int group = a.q_heads / c.kv_heads, h = head / group;
  f32x4 x{NAN, NAN, NAN, NAN};
  if (planned(plan, a, M)) {
    const int s = plan.owner()[t];
    if (s < 0) return;  // a token of nobody: its outputs stay as they are
    const PlanSeq& p = plan.seqs()[s];
    // what the plan was made from
    if (p.levels > 0 && c.status[s] == TMS_OK && p.len == c.length[s] && p.begin == a.start[s] && p.n <= a.max_new) {
      PartSum sum;
      for (int i = 0; i < p.levels; ++i) {
        const Node& node = plan.nodes()[p.node[i]];
        const int r = (p.at[i] + t - p.begin) * group + head % group, rt = r / node.rows;
        const int64_t first = part_row(c, node, group, rt, 0, h) + r % node.rows;
        const int64_t step = part_row(c, node, group, rt, 1, h) + r % node.rows - first;
        sum.add<D>(plan.parts(), node.chunks, column, [&](int k) { return first + k * step; });
      }
      x = sum.x * (1.f / sum.l);
    }
  }
  store4<DT>(a.out, row * D + column, x);
}

int shape(const KvCache& c, int32_t T, int32_t q_heads) {
  const int64_t rows = int64_t(T) * (q_heads / c.kv_heads);  // of a node, at most
  if (rows <= 16) return kFew16;
  if (c.dtype == TMS_F32) return c.head_dim < 256 ? kFew32 : kFew16;
  return rows <= 32 && c.head_dim < 256 ? kFew32 : rows <= 64 ? kMany64 : kMany128;
}

template <int DT, int D, int Shape>
hipError_t launch(const KvCache& c, const KvAttention& a, const Plan& plan, hipStream_t s) {
  const int64_t blocks = int64_t(plan.y.most_units) * c.kv_heads, rows = int64_t(a.T) * a.q_heads;
  constexpr int kRows = kBlock * 4 / D;
  if (blocks >= (int64_t(1) << 32) / kBlock || rows >= (int64_t(1) << 32) / kBlock) return hipErrorInvalidValue;
  nodes_kernel<DT, D, Shape><<<unsigned(blocks), kBlock, 0, s>>>(c, a, plan);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  join_nodes_kernel<DT, D><<<unsigned((rows + kRows - 1) / kRows), kBlock, 0, s>>>(c, a, plan, rows_of(Shape));
  return hipGetLastError();
}

template <int DT, int D>
hipError_t launch(const KvCache& c, const KvAttention& a, const Plan& plan, int shape, hipStream_t s) {
  if (shape == kFew16) return launch<DT, D, kFew16>(c, a, plan, s);
  if constexpr (DT == 1) {
    if (shape == kMany64) return launch<DT, D, kMany64>(c, a, plan, s);
    if (shape == kMany128) return launch<DT, D, kMany128>(c, a, plan, s);
  }
  if constexpr (D < 256) return launch<DT, D, kFew32>(c, a, plan, s);
  return hipErrorInvalidValue;
}

Plan plan_of(const KvCache& c, const KvShared& sh, int shape) {
  return Plan{static_cast<char*>(sh.plan), layout(c, sh.a.T, sh.a.q_heads, rows_of(shape))};
}

}  // namespace

int64_t kv_share_bytes(const KvCache& c, int32_t T, int32_t q_heads) {
  return layout(c, T, q_heads, rows_of(shape(c, T, q_heads))).bytes;
}

hipError_t launch_kv_share(const KvCache& c, const KvShared& sh, hipStream_t s) {
  const int x = shape(c, sh.a.T, sh.a.q_heads);
  plan_kernel<<<1, kPlan, 0, s>>>(c, sh.a, plan_of(c, sh, x), rows_of(x));
  return hipGetLastError();
}

hipError_t launch_kv_attention_shared(const KvCache& c, const KvShared& sh, hipStream_t s) {
  // where every sequence has many rows there is nothing to share
  if (int64_t(sh.a.max_new) * (sh.a.q_heads / c.kv_heads) > kMostRowsShared) return launch_kv_attention(c, sh.a, s);
  const int x = shape(c, sh.a.T, sh.a.q_heads);
  const Plan plan = plan_of(c, sh, x);
  if (c.dtype == TMS_F32) {
    if (c.head_dim == 64) return launch<0, 64>(c, sh.a, plan, x, s);
    return c.head_dim == 128 ? launch<0, 128>(c, sh.a, plan, x, s) : launch<0, 256>(c, sh.a, plan, x, s);
  }
  if (c.head_dim == 64) return launch<1, 64>(c, sh.a, plan, x, s);
  return c.head_dim == 128 ? launch<1, 128>(c, sh.a, plan, x, s) : launch<1, 256>(c, sh.a, plan, x, s);
}

}  // namespace tms
