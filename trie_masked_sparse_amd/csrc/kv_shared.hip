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
//
// Measured, a layer (us, MI355X; 32 query and 8 key heads of 128, bf16, pages of
// 64; four batches of other inputs in turn): 64 tokens behind one prompt of 9000
// rows and up to 400 of their own 45, where kv_attention takes 265; 256 behind four
// prompts of 9000 to 24000 that share 2048 rows and up to 1000 of their own 229
// (2222).  The plan adds 12 to 34 once for all layers, so four sequences of 150 rows
// are quicker without (14 and 10).
#include <algorithm>
#include <climits>

#include "kv_many.h"
#include "kv_plan.h"

namespace tms {
namespace {

constexpr int kSeqs = 4096;  // sequences of a cache, at most
constexpr int kPlan = 1024, kPlanWaves = kPlan / kWave;
constexpr int kMagic = 0x73686172;

// Sequences of more rows of a key head than this read their pages for
// themselves: the products bound them, and many rows share a page's read already
// (5 to 31 drafts of 64 sequences behind prompts of 1201 to 2500 tokens: 2 rows a
// draft, heads of 128 79 us alone, 57 shared; 4 rows, heads of 256 88 and 120).
__host__ __device__ inline int most_rows_shared(const KvCache& c) { return c.head_dim == 256 ? 64 : 128; }

// A node pays where the keys that are not read again (its keys, times the
// readers that it saves) are more than these and what its rows' parts cost: a
// part is written and read, 8 bytes a value, a key 2 values of the cache's type.
constexpr int kLeastSaved = 256;
__device__ inline bool pays(int64_t keys, int64_t readers, int64_t rows, int dtype) {
  return keys * readers >= kLeastSaved + (dtype == 0 ? 2 : 4) * rows;
}

constexpr int kRounds = 16;  // branchings of the trie that are looked at, one behind the other

struct Plan {
  char* at;
  Layout y;
  __device__ Head* head() const { return reinterpret_cast<Head*>(at); }
  __device__ PlanSeq* seqs() const { return reinterpret_cast<PlanSeq*>(at + y.seqs); }
  __device__ Meet* meets() const { return reinterpret_cast<Meet*>(at + y.meets); }
  __device__ Node* nodes() const { return reinterpret_cast<Node*>(at + y.nodes); }
  __device__ Unit* units() const { return reinterpret_cast<Unit*>(at + y.units); }
  __device__ int32_t* tokens() const { return reinterpret_cast<int32_t*>(at + y.tokens); }  // of the nodes, a list for each level
  __device__ int32_t* owner() const { return reinterpret_cast<int32_t*>(at + y.owner); }    // sequence of every token, -1
  __host__ __device__ Parts parts() const {
    return Parts{reinterpret_cast<float*>(at + y.values), reinterpret_cast<float2*>(at + y.stats)};
  }
};

// Whole pages of committed rows of a sequence that may be shared.
__device__ inline int shared_pages(const KvCache& c, const KvAttention& a, const Seq& q) {
  return q.n && !q.bad && int64_t(q.n) * (a.q_heads / c.kv_heads) <= most_rows_shared(c) ? q.len >> c.page_shift : 0;
}

// Meet of sequence s, by one wavefront; whole(t): shared_pages of a sequence.  A
// sequence that has more pages in common than the best so far has the same page
// behind these, which is looked for first; pages are then compared one by one,
// so a table that no fork has made is planned rightly too.
template <class Whole>
__device__ inline Meet meet(const KvCache& c, int s, Whole whole) {
  constexpr int kLoads = 4;
  const int lane = threadIdx.x % kWave, mine = uniform(whole(s));
  const int32_t* x = c.table + int64_t(s) * c.max_pages;
  Meet best{s, 0};
  for (int t0 = 0; t0 < s && best.pages < mine;) {
    const int page = uniform(x[best.pages]);
    // (a page that no other sequence holds is not looked for)
    if (page < 0 || page >= c.pages || uniform(c.refs[page]) < 2) break;
    int t = s;
    for (; t0 < s && t == s; t0 += kWave) {
      const int u = t0 + lane;
      const bool hit = u < s && whole(min(u, s)) > best.pages && c.table[int64_t(min(u, s)) * c.max_pages + best.pages] == page;
      const uint64_t hits = __ballot(hit);
      if (hits) t = t0 + __builtin_ctzll(hits);
    }
    if (t == s) break;
    t0 = t + 1;
    const int most = min(mine, uniform(whole(t)));
    const int32_t* y = c.table + int64_t(t) * c.max_pages;
    int end = most;
    for (int j0 = 0; j0 < most && end == most; j0 += kLoads * kWave) {
      int p[kLoads], q[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int j = min(j0 + u * kWave + lane, most - 1);
        p[u] = x[j], q[u] = y[j];
      }
#pragma unroll
      for (int u = kLoads - 1; u >= 0; --u) {
        const uint64_t differ = __ballot(p[u] != q[u]);
        if (differ) end = min(j0 + u * kWave + __builtin_ctzll(differ), most);
      }
    }
    if (end > best.pages) best = Meet{t, end};
  }
  return best;
}

// A wavefront for each sequence.  Bound by latency, 0.7 us a read: a sequence's
// pages, the others' at one place, one other's pages, behind one another.  64
// sequences 6 to 7 us, 256 of four prompts 8.
__global__ __launch_bounds__(kWave) void meet_kernel(KvCache c, KvAttention a, Plan plan) {
  a.max_new = INT_MAX;
  const Meet m = meet(c, blockIdx.x, [&](int t) { return shared_pages(c, a, sequence(c, a, t, 1, 1)); });
  if (threadIdx.x == 0) plan.meets()[blockIdx.x] = m;
}

// Sums over the workgroup's threads before this one, and of all, of N values;
// `sums` is free again behind the next barrier.
template <int N, typename T>
__device__ inline void threads_before(T (&x)[N], T (*sums)[kPlanWaves], T (&total)[N]) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  T incl[N];
#pragma unroll
  for (int i = 0; i < N; ++i) incl[i] = x[i];
#pragma unroll
  for (int step = 1; step < kWave; step *= 2) {
    T y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = __shfl_up(incl[i], step);
#pragma unroll
    for (int i = 0; i < N; ++i) incl[i] += lane >= step ? y[i] : 0;
  }
  if (lane == kWave - 1)
#pragma unroll
    for (int i = 0; i < N; ++i) sums[i][wave] = incl[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = incl[i] - x[i], total[i] = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
      if (w < wave) x[i] += sums[i][w];
      total[i] += sums[i][w];
    }
  }
}

// Sum of the lanes' values up to and including this one's.
__device__ inline int lanes_up_to(int x) {
  x += from_lane<0x111, 0xf>(x);  // 1, 2, 4 and 8 lanes down in rows of 16
  x += from_lane<0x112, 0xf>(x);
  x += from_lane<0x114, 0xf>(x);
  x += from_lane<0x118, 0xf>(x);
  x += from_lane<0x142, 0xa>(x);  // row 0 to row 1, row 2 to row 3
  x += from_lane<0x143, 0xc>(x);  // lane 31 to rows 2 and 3
  return x;
}

// Calls f(value, lanes that have it), a value after the other, for the lanes
// where `on`; all lanes of the wavefront are active.
template <class F>
__device__ inline void each_value(bool on, int value, F f) {
  for (uint64_t left = __ballot(on); left;) {
    const int v = __builtin_amdgcn_readlane(value, __builtin_ctzll(left));
    const uint64_t same = __ballot(on && value == v);
    f(v, same);
    left &= ~same;
  }
}

// First part row of row tile rt, chunk k of a node's key head: a chunk's parts
// are the tile's rows for head 0, then for head 1, ...
__device__ inline int64_t part_row(int64_t part, int kv_heads, int all, int M, int chunks, int rt, int k, int h) {
  const int64_t first = int64_t(rt) * M, rows = min(int64_t(M), all - first);
  return part + kv_heads * (first * chunks + k * rows) + h * rows;
}

// Unit i of a node: heads next to each other, then the chunks of a row tile.
__device__ inline Unit unit_of(const KvCache& c, const Node& x, int group, int heads, int i) {
  const int h = i % heads * (c.kv_heads / heads), k = i / heads % x.chunks, rt = i / heads / x.chunks;
  Unit u{};
  u.seq = x.seq, u.key0 = x.key0, u.keys = x.keys, u.list = x.list, u.begin = x.begin, u.n = x.n, u.len = x.len;
  u.all = x.tokens * group, u.row0 = rt * x.rows, u.rows = min(x.rows, u.all - u.row0), u.h = h, u.M = x.rows;
  u.tile0 = k * x.tiles, u.tile1 = u.tile0 + x.tiles;
  u.part = part_row(x.part, c.kv_heads, u.all, x.rows, x.chunks, rt, k, h);
  return u;
}

// One workgroup.  In every round a group are the sequences that go through one
// place of the trie; its first is the leader.  The pages that the whole group
// has in common, from where its sequences read, make a node, if that pays:
// without it every branch of the group (sequences that have the next page in
// common too) would read them.  Behind them every branch is a group.
//
// Bound by latency: reads of global memory one after the other, barriers, and the
// code itself, which is fetched for the first time in every call (kEach 4, for all
// caches, is four times as much: 64 sequences 34 us where kEach 1 took 27 then).
// 4 sequences 13 us, 64 behind one prompt 15, 64 behind four that branch 20, 256 30.
constexpr int kMeetHere = 16;  // sequences whose meets are found here: a launch less
template <int kEach>
__global__ __launch_bounds__(kPlan) void plan_kernel(KvCache c, KvAttention a, Plan plan, int M, int heads) {
  constexpr int kMost = kEach * kPlan;  // sequences
  // of every sequence: the first of its group; tokens (0: none to share); its Meet.
  // Of a leader: the fewest pages that one of its group has in common with it, the
  // others' tokens, branches; its node's number and list
  __shared__ union {
    struct {
      int lead[kMost], with[kMost], pages[kMost], fewest[kMost], of_group[kMost], branches[kMost], place[kMost], whole[kMost];
    } s;
    int first_unit[2 * kMost];  // of every node, when the others are done with
  } lds;
  auto &lead = lds.s.lead, &with = lds.s.with, &pages = lds.s.pages, &fewest = lds.s.fewest, &of_group = lds.s.of_group,
       &branches = lds.s.branches, &place = lds.s.place, &whole = lds.s.whole;
  __shared__ uint16_t count[kMost];
  __shared__ int nodes_s, list_s;
  __shared__ int64_t sums[3][kPlanWaves];
  __shared__ int sums32[1][kPlanWaves];
  const int tid = threadIdx.x, wave = uniform(tid / kWave), lane = tid % kWave, n = c.seqs, group = a.q_heads / c.kv_heads;
  auto each_seq = [&](auto f) __attribute__((always_inline)) {  // f(i, s), of every sequence of this thread
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (tid + i * kPlan < n) f(i, tid + i * kPlan);
  };
  // the same, by whole wavefronts: on, whether there is such a sequence (s is the last one where not)
  auto each_lane = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (wave * kWave + i * kPlan < n) f(i, min(tid + i * kPlan, n - 1), tid + i * kPlan < n);
  };
  a.max_new = INT_MAX;
  if (tid == 0) nodes_s = list_s = 0;
  for (int i = tid; i < a.T; i += kPlan) plan.owner()[i] = -1;
  PlanSeq mine[kEach];
  int64_t tokens[1] = {0}, all_tokens[1];
  each_seq([&](int i, int s) __attribute__((always_inline)) {
    const Seq q = sequence(c, a, s, 1, 1);
    const bool on = q.n && !q.bad;
    mine[i].begin = q.begin, mine[i].n = q.n, mine[i].len = q.len, mine[i].levels = on ? 0 : -1;
    whole[s] = shared_pages(c, a, q);
    count[s] = whole[s] ? q.n : 0;
    if (n > kMeetHere) {
      const Meet m = plan.meets()[s];
      with[s] = m.with, pages[s] = m.pages;
    }
    fewest[s] = q.begin, lead[s] = q.n;
    tokens[0] += on ? q.n : 0;
  });
  // tokens that two sequences claim (start not ascending) would not fit the lists
  threads_before(tokens, sums, all_tokens);
  if (all_tokens[0] > a.T) {
    if (tid == 0) *plan.head() = Head{};
    return;
  }
  for (int s = wave; s < n; s += kPlanWaves)
    for (int i = lane; i < lead[s]; i += kWave) plan.owner()[fewest[s] + i] = s;
  if (n <= kMeetHere && wave < n) {
    const Meet m = meet(c, wave, [&](int t) { return whole[t]; });
    if (lane == 0) with[wave] = m.with, pages[wave] = m.pages;
  }
  // the first sequence that goes through the place behind `depth` pages of
  // sequence s, and the pages that s has in common with it
  auto first_at = [&](int s, int depth, int* in_common) __attribute__((always_inline)) {
    int m = INT_MAX, v = s;
    for (int p = pages[v]; p > depth; p = pages[v]) m = min(m, p), v = with[v];
    *in_common = m;
    return v;
  };
  int depth[kEach], pos[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) depth[i] = pos[i] = 0;
  for (int round = 0; round < kRounds; ++round) {
    __syncthreads();
    int in_common[kEach];
    bool groups = false;
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      lead[s] = whole[s] && mine[i].levels < kLevels ? first_at(s, depth[i], &in_common[i]) : s;
      groups |= lead[s] != s;
      fewest[s] = INT_MAX, of_group[s] = branches[s] = 0;
    });
    if (!__syncthreads_or(groups)) break;
    each_lane([&](int i, int s, bool here) __attribute__((always_inline)) {
      const int l = lead[s];
      each_value(here && l != s, l, [&](int v, uint64_t lanes) {
        const bool on = lanes >> lane & 1;
        int least = on ? in_common[i] : INT_MAX;
        const int tokens = __builtin_amdgcn_readlane(lanes_up_to(on ? count[s] : 0), kWave - 1);
        for (int step = 1; step < kWave; step *= 2) least = min(least, __shfl_xor(least, step));
        if (lane == __builtin_ctzll(lanes)) atomicAdd(&of_group[v], tokens), atomicMin(&fewest[v], least);
      });
    });
    __syncthreads();
    each_lane([&](int i, int s, bool here) __attribute__((always_inline)) {
      const int l = lead[s], d = fewest[l];
      int unused;
      each_value(here && d < INT_MAX && first_at(s, d, &unused) == s, l, [&](int v, uint64_t lanes) {
        if (lane == __builtin_ctzll(lanes)) atomicAdd(&branches[v], __popcll(lanes));
      });
    });
    __syncthreads();
    bool any = false;
    int level_pages[kEach];
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      const int l = lead[s], d = fewest[l];
      level_pages[i] = 0;
      if (d == INT_MAX) return;  // alone
      if (pays(int64_t(d - pos[i]) << c.page_shift, branches[l] - 1, int64_t(of_group[l] + count[l]) * group, c.dtype)) {
        level_pages[i] = d - pos[i];
        any = true;
      }
      depth[i] = d;
    });
    if (!__syncthreads_or(any)) continue;
    // the lists of a round: nodes in the order of their leaders, tokens in the
    // order of their sequences: by one wavefront, 64 sequences a step
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      of_group[s] = 0;
      if (level_pages[i] == 0) lead[s] = -1;  // no node
    });
    __syncthreads();
    if (wave == 0) {
      for (int s0 = 0; s0 < n; s0 += kWave) {
        const int s = min(s0 + lane, n - 1), l = lead[s], k = count[s];
        each_value(s0 + lane < n && l >= 0, l, [&](int v, uint64_t lanes) {
          const bool on = lanes >> lane & 1;
          const int up = lanes_up_to(on ? k : 0), before = of_group[v];
          if (on) fewest[s] = before + up - k;  // place among the node's tokens
          if (lane == 0) of_group[v] = before + __builtin_amdgcn_readlane(up, kWave - 1);
        });
      }
      int node = nodes_s, list = list_s;
      for (int s0 = 0; s0 < n; s0 += kWave) {
        const int s = min(s0 + lane, n - 1);
        const bool on = s0 + lane < n && lead[s] == s;
        const uint64_t leaders = __ballot(on);
        const int tokens = on ? of_group[s] : 0, up = lanes_up_to(tokens);
        if (on) branches[s] = node + __popcll(leaders & ((uint64_t(1) << lane) - 1)), place[s] = list + up - tokens;  // node, its list
        node += __popcll(leaders), list += __builtin_amdgcn_readlane(up, kWave - 1);
      }
      if (lane == 0) nodes_s = node, list_s = list;
    }
    __syncthreads();
    each_seq([&](int i, int s) __attribute__((always_inline)) {
      const int l = lead[s];
      if (l < 0) return;
      const int node = branches[l], list = place[l], at = fewest[s];
      PlanSeq& p = mine[i];
      for (int u = 0; u < count[s]; ++u) plan.tokens()[list + at + u] = p.begin + u;
#pragma unroll
      for (int v = 0; v < kLevels; ++v)
        if (p.levels == v) p.of[v].node = node, p.of[v].at = at;
      ++p.levels;
      if (s == l) {
        Node x{};
        x.seq = s, x.key0 = pos[i] << c.page_shift, x.keys = level_pages[i] << c.page_shift;
        x.tokens = of_group[s], x.list = list;
        plan.nodes()[node] = x;
      }
      pos[i] += level_pages[i];
    });
  }
  __syncthreads();
  // what every sequence has for itself
  int nodes = nodes_s;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (i * kPlan >= n) continue;
    const int s = tid + i * kPlan;
    const bool on = s < n && mine[i].levels >= 0;
    int before[1] = {int(on)}, total[1];
    threads_before(before, sums32, total);
    const int node = nodes + before[0];
    nodes += total[0];
    __syncthreads();
    if (s >= n) continue;
    PlanSeq& p = mine[i];
    if (on) {
      Node x{};
      x.seq = s, x.key0 = pos[i] << c.page_shift;
      x.len = p.len - x.key0, x.n = p.n, x.keys = x.len + x.n, x.begin = p.begin;
      x.tokens = p.n, x.list = -1;
      plan.nodes()[node] = x;
#pragma unroll
      for (int v = 0; v <= kLevels; ++v)
        if (p.levels == v) p.of[v].node = node, p.of[v].at = 0;
      ++p.levels;
    }
  }
  __syncthreads();
  const int each = (nodes + kPlan - 1) / kPlan, from = min(tid * each, nodes), to = min(from + each, nodes);
  auto size = [&](const Node& x) { return size_of(x, group, c.kv_heads, M, heads); };
  int64_t work[1] = {0}, total[1];
  for (int i = from; i < to; ++i) work[0] += cost_of(size(plan.nodes()[i]));
  threads_before(work, sums, total);
  const int64_t slot = total[0] / kSlots + 1;
  int64_t x_of[2] = {0, 0}, all[2];
  int64_t &units = x_of[0], &rows = x_of[1];  // units and part rows
  for (int i = from; i < to; ++i) {
    const Node& x = plan.nodes()[i];
    const Size z = size(x);
    units += int64_t(z.row_tiles) * chunks_of(z, slot) * z.heads, rows += int64_t(x.tokens) * a.q_heads * chunks_of(z, slot);
  }
  threads_before(x_of, sums + 1, all);
  const bool fits = all[0] <= plan.y.most_units && all[1] <= plan.y.most_rows;
  for (int i = from; fits && i < to; ++i) {
    Node& x = plan.nodes()[i];
    const Size z = size(x);
    x.chunks = chunks_of(z, slot), x.rows = z.rows, x.part = rows;
    x.tiles = (z.key_tiles + x.chunks - 1) / x.chunks;
    lds.first_unit[i] = static_cast<int>(units);
    units += int64_t(z.row_tiles) * x.chunks * z.heads, rows += int64_t(x.tokens) * a.q_heads * x.chunks;
  }
  __syncthreads();
  if (fits) {
    for (int u = tid; u < all[0]; u += kPlan) {
      int i = 0;
      for (int step = 1 << (31 - __clz(nodes)); step; step /= 2)
        if (i + step < nodes && lds.first_unit[i + step] <= u) i += step;
      const Node x = plan.nodes()[i];
      plan.units()[u] = unit_of(c, x, group, size(x).heads, u - lds.first_unit[i]);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {  // what the join has to know
      const int s = tid + i * kPlan;
      if (s >= n) continue;
      PlanSeq& p = mine[i];
#pragma unroll
      for (int v = 0; v <= kLevels; ++v) {
        if (v >= p.levels) continue;
        const Node& x = plan.nodes()[p.of[v].node];
        p.of[v].all = x.tokens * group, p.of[v].M = x.rows, p.of[v].chunks = x.chunks, p.of[v].part = x.part;
      }
      plan.seqs()[s] = p;
    }
  }
  if (tid == 0) *plan.head() = Head{fits ? kMagic : 0, a.T, a.q_heads, fits ? int(all[0]) : 0, nodes, M, {heads, 0}};
}

// Whether the plan is one for this call.
__device__ inline bool planned(const Plan& plan, const KvAttention& a, int M) {
  const Head* h = plan.head();
  return h->magic == kMagic && h->T == a.T && h->q_heads == a.q_heads && h->rows == M;
}

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

// A unit of the plan.
//
// 64 tokens behind one prompt (shapes as above) 34 us a layer, 103 MB read, 64 trees
// of drafts 51: a tile of 128 rows x 64 keys is products, maximum, exponentials,
// products, one behind the other in each wavefront, with two workgroups on a compute
// unit (the matrix cores are 16 to 27 % busy), and a unit takes 5 to 7 us for its
// start and end.  256 tokens of four prompts 203 us, 841 MB, 4.1 TB/s.  Tried and
// slower, with weights of one part: equal shares of the cost, a workgroup each, in a
// loop over their segments (34 -> 52, trees 49 -> 60, 256 tokens 196 -> 235 us:
// registers go to scratch, and every segment starts anew), tiles of 32 keys copied
// three ahead (32.1 -> 32.4, 46.9 -> 49.0, 198 -> 207).
template <int DT, int D, int Shape, int Heads>
__global__ __launch_bounds__(kBlock, D == 256 || (D == 128 && Shape == kFew32) ? 1 : 2) void nodes_kernel(KvCache c, KvAttention a, Plan plan) {
  using Small = FewRows<DT, D, 1, Heads>;
  using Large = typename Body<DT, D, Shape>::Type;
  using Medium = typename Body<DT, D, Shape == kMany128 ? kMany64 : Shape>::Type;
  __shared__ union {
    typename Small::Lds small;
    typename Medium::Lds medium;
    typename Large::Lds large;
  } lds;
  const Unit& at = plan.units()[blockIdx.x];
  if (!planned(plan, a, rows_of(Shape)) || int(blockIdx.x) >= plan.head()->units) return;
  Unit x;
  x.seq = uniform(at.seq), x.key0 = uniform(at.key0), x.keys = uniform(at.keys), x.list = uniform(at.list);
  x.begin = uniform(at.begin), x.n = uniform(at.n), x.len = uniform(at.len), x.all = uniform(at.all);
  x.row0 = uniform(at.row0), x.rows = uniform(at.rows), x.h = uniform(at.h), x.M = uniform(at.M);
  x.tile0 = uniform(at.tile0), x.tile1 = uniform(at.tile1), x.part = uniform(at.part);
  const int group = a.q_heads / c.kv_heads, row0 = x.row0, rows = x.rows;
  const int32_t* table = c.table + int64_t(x.seq) * c.max_pages + (x.key0 >> c.page_shift);
  const int32_t* list = plan.tokens() + max(x.list, 0);
  const bool own = x.list < 0;  // keys of one sequence, its new rows among them
  if (own && x.n > a.max_new) return;
  FewTile t{};
  t.h = x.h;
  if (own) {
    t.q.begin = x.begin, t.q.n = x.n, t.q.len = x.len;
    t.tok0 = row0 / group, t.tok1 = (row0 + rows - 1) / group;
    t.limit = a.parent ? x.keys : x.len + t.tok1 + 1;
  } else {  // all rows see all keys
    a.parent = nullptr;
    t.q.len = t.limit = x.keys;
    t.tok0 = t.tok1 = -1;
  }
  auto query = [&](int h, int r) {
    const int row = row0 + min(r, rows - 1), i = row / group;
    const int token = own ? x.begin + i : list[i];
    return int64_t(token) * a.ldq + int64_t(h * group + row % group) * D;
  };
  auto token = [&](int r) { return own && r < rows ? (row0 + r) / group : -1; };
  const Parts parts = plan.parts();
  auto emit = [&](int h, int r, int column, f32x4 v, float top, float l) {
    if (r >= rows) return;
    const int64_t part = x.part + (h - x.h) * rows + r;
    *reinterpret_cast<f32x4*>(parts.values + part * D + column) = v;
    if (column == 0) parts.stats[part] = float2{top, l};
  };
  auto tiles = [&](int keys) {  // key tiles of this many keys
    t.kt0 = x.tile0 * (kTile / keys);
    t.kt1 = min(x.tile1 * (kTile / keys), (x.keys + keys - 1) / keys);
  };
  auto page_at = [&](int key) { return max(0, min(table[key >> c.page_shift], c.pages - 1)); };
  if (few_rows(Shape, x.M)) {
    tiles(Small::KW);
    Small::run(c, a, lds.small, t, page_at, query, token, emit);
  } else if constexpr (Shape == kFew32) {
    tiles(Large::KW);
    Large::run(c, a, lds.large, t, page_at, query, token, emit);
  } else if constexpr (Shape >= kMany64) {
    auto many = [&](auto body, auto& in) __attribute__((always_inline)) {
      using Rows = decltype(body);
      tiles(Rows::KT);
      Rows::run(c, a, in, t, table, [&](int r) { return query(x.h, r); }, token,
                [&](int r, int column, f32x4 v, float top, float l) { emit(x.h, r, column, v, top, l); });
    };
    if (Shape == kMany128 && x.M == kMedium) many(Medium(), lds.medium);
    else many(Large(), lds.large);
  }
}

// The parts of a token and query head over all its nodes: D / 4 threads to a row,
// or G times as many, each of which take every G-th chunk, where rows are few and
// their chunks many.  Bound by the chain plan, node, statistics, values: 64 tokens
// of 32 heads 8 us for 16 MB, trees of 18 drafts 12 for 31 MB.
template <int DT, int D, int G>
__global__ __launch_bounds__(kBlock) void join_nodes_kernel(KvCache c, KvAttention a, Plan plan, int M) {
  constexpr int kRow = D / 4, kRows = kBlock / (kRow * G);
  __shared__ float2 stats[G > 1 ? kBlock : 1];
  __shared__ f32x4 values[G > 1 ? kBlock : 1];
  const int tid = threadIdx.x, g = tid / kRow % G, column = tid % kRow * 4;
  const int64_t row = min(int64_t(blockIdx.x) * kRows + tid / (kRow * G), int64_t(a.T) * a.q_heads - 1);
  const int t = static_cast<int>(row / a.q_heads), head = static_cast<int>(row % a.q_heads);
  const int group = a.q_heads / c.kv_heads, h = head / group;
  // (what is read from a plan that was not made is not used; the reads do not
  // wait for each other)
  const int s = plan.owner()[t], at = max(0, min(s, c.seqs - 1));
  const PlanSeq p = plan.seqs()[at];
  const bool made = planned(plan, a, M);
  // what the plan was made from
  const bool good = made && s >= 0 && p.levels > 0 && c.status[at] == TMS_OK && p.len == c.length[at] && p.begin == a.start[at] &&
                    p.n <= a.max_new;
  PartSum sum;
  if (good) {
#pragma unroll
    for (int i = 0; i <= kLevels; ++i) {
      if (i >= p.levels) break;
      const auto& of = p.of[i];
      const int r = (of.at + t - p.begin) * group + head % group, rt = r / of.M;
      const int64_t first = part_row(of.part, c.kv_heads, of.all, of.M, of.chunks, rt, 0, h) + r % of.M;
      const int64_t step = part_row(of.part, c.kv_heads, of.all, of.M, of.chunks, rt, 1, h) + r % of.M - first;
      sum.add<D, G == 1 ? 4 : 8>(plan.parts(), (of.chunks - g + G - 1) / G, column, [&](int k) { return first + (g + k * G) * step; });
    }
  }
  if constexpr (G > 1) {
    stats[tid] = float2{sum.top, sum.l}, values[tid] = sum.x;
    __syncthreads();
    if (g) return;
#pragma unroll
    for (int i = 1; i < G; ++i) {
      const float2 y = stats[tid + i * kRow];
      const float top = fmaxf(sum.top, y.x), base = top == -INFINITY ? 0.f : top;
      const float mine = part_weight(sum.top - base), other = part_weight(y.x - base);
      sum.l = sum.l * mine + y.y * other, sum.x = sum.x * mine + values[tid + i * kRow] * other, sum.top = top;
    }
  }
  if (made && s < 0) return;  // a token of nobody: its outputs stay as they are
  store4<DT>(a.out, row * D + column, good ? sum.x * (1.f / sum.l) : f32x4{NAN, NAN, NAN, NAN});
}

template <int DT, int D, int Shape>
hipError_t launch(const KvCache& c, const KvAttention& a, const Plan& plan, hipStream_t s) {
  const int64_t blocks = plan.y.most_units, rows = int64_t(a.T) * a.q_heads;
  constexpr int kRows = kBlock * 4 / D;  // of a workgroup of the join
  constexpr int64_t kFew = 2048;
  if (blocks >= (int64_t(1) << 32) / kBlock || rows >= (int64_t(1) << 32) / kBlock) return hipErrorInvalidValue;
  const int heads = small_heads(c, a.T, a.q_heads);
  if (heads == kMostHeads) nodes_kernel<DT, D, Shape, kMostHeads><<<unsigned(blocks), kBlock, 0, s>>>(c, a, plan);
  else nodes_kernel<DT, D, Shape, 1><<<unsigned(blocks), kBlock, 0, s>>>(c, a, plan);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (rows <= kFew) join_nodes_kernel<DT, D, 4><<<unsigned((4 * rows + kRows - 1) / kRows), kBlock, 0, s>>>(c, a, plan, rows_of(Shape));
  else join_nodes_kernel<DT, D, 1><<<unsigned((rows + kRows - 1) / kRows), kBlock, 0, s>>>(c, a, plan, rows_of(Shape));
  return hipGetLastError();
}

template <int DT, int D>
hipError_t launch(const KvCache& c, const KvAttention& a, const Plan& plan, int shape, hipStream_t s) {
  if (shape == kFew16) return launch<DT, D, kFew16>(c, a, plan, s);
  if constexpr (DT == 1) {
    if (shape == kMany64) return launch<DT, D, kMany64>(c, a, plan, s);
    if (shape == kMany128) return launch<DT, D, kMany128>(c, a, plan, s);
  }
  if constexpr (D == 64 || (DT == 0 && D == 128)) return launch<DT, D, kFew32>(c, a, plan, s);
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
  const Plan plan = plan_of(c, sh, x);
  if (c.seqs > kMeetHere) {
    meet_kernel<<<c.seqs, kWave, 0, s>>>(c, sh.a, plan);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (c.seqs <= kPlan) plan_kernel<1><<<1, kPlan, 0, s>>>(c, sh.a, plan, rows_of(x), small_heads(c, sh.a.T, sh.a.q_heads));
  else plan_kernel<kSeqs / kPlan><<<1, kPlan, 0, s>>>(c, sh.a, plan, rows_of(x), small_heads(c, sh.a.T, sh.a.q_heads));
  return hipGetLastError();
}

hipError_t launch_kv_attention_shared(const KvCache& c, const KvShared& sh, hipStream_t s) {
  // where every sequence has many rows there is nothing to share
  if (int64_t(sh.a.max_new) * (sh.a.q_heads / c.kv_heads) > most_rows_shared(c)) return launch_kv_attention(c, sh.a, s);
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
