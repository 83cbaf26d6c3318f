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

#include "kv_few.h"

namespace tms {
namespace {

constexpr int kLevels = 3;      // nodes of a sequence beside its own
constexpr int kSeqs = 4096;     // sequences of a cache, at most
constexpr int kPlan = 1024;     // threads of plan_kernel
constexpr int kSlots = 512;     // workgroups that a launch should have
constexpr int kMagic = 0x73686172;

// Sequences of more rows of a key head than this read their pages for
// themselves: the products bound them, and many rows share a page's read already.
constexpr int kMostRowsShared = 128;

// Rows of the prefix that are not read again (its rows times the sequences but
// one) have to be at least this for a node.
constexpr int kLeastSaved = 256;

struct Head {
  int32_t magic, T, q_heads, units, nodes, rows, keys, pad;
};

struct PlanSeq {
  int32_t begin, n, len, levels;      // tokens, committed rows; nodes (-1: its outputs are NaN)
  int32_t node[kLevels + 1], at[kLevels + 1];  // nodes, and where its tokens are among a node's
};

struct Node {
  int32_t seq, key0, keys;            // the sequence whose table has the pages; first row, rows
  int32_t tokens, list;               // query tokens; their place in the list, -1: begin ..
  int32_t begin, n, len;              // of one sequence's own: its new tokens, committed rows from key0 on
  int32_t unit, chunks, tiles, pad;   // first unit, chunks of `tiles` key tiles
  int64_t part;                       // first row of its parts
};

// Places in the plan.  M: rows of a tile.
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
  const int64_t tiles = (kLevels + 1) * (int64_t(T) * group / M) + y.most_nodes;
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

// Pages that sequences s and t have in common from page p on, of the first
// `most`, by one wavefront.
__device__ inline int common(const KvCache& c, int s, int t, int p, int most) {
  const int lane = threadIdx.x % kWave;
  const int32_t *x = c.table + int64_t(s) * c.max_pages, *y = c.table + int64_t(t) * c.max_pages;
  constexpr int kLoads = 4;
  for (int j0 = p; j0 < most; j0 += kLoads * kWave) {
    int a[kLoads], b[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int j = min(j0 + i * kWave + lane, most - 1);
      a[i] = x[j], b[i] = y[j];
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint64_t differ = __ballot(a[i] != b[i] || j0 + i * kWave + lane >= most);
      if (differ) return min(j0 + i * kWave + __builtin_ctzll(differ), most) - p;
    }
  }
  return most - p;
}

// One workgroup.  In every round, sequences that have the same next page form a
// group; its first sequence is the leader, and the cut that saves most reads
// (pages in common with the leader, times the sequences that have them but one)
// makes a node.  Its sequences go on behind it in the next round.  Pages are
// compared one by one, so a table that no fork has made is planned rightly too.
__global__ __launch_bounds__(kPlan) void plan_kernel(KvCache c, KvAttention a, Plan plan, int M, int KT) {
  __shared__ int next[kSeqs];    // next page's number; then the leader of the node that it is in
  __shared__ int lead[kSeqs], pos[kSeqs], same[kSeqs], count[kSeqs], whole[kSeqs], cut[kSeqs];
  __shared__ unsigned long long best[kSeqs];
  __shared__ int nodes_s;
  __shared__ int64_t scan[3][kPlan / kWave];
  constexpr int kEach = kSeqs / kPlan;
  const int tid = threadIdx.x, wave = uniform(tid / kWave), lane = tid % kWave, n = c.seqs, group = a.q_heads / c.kv_heads;
  a.max_new = INT_MAX;
  if (tid == 0) nodes_s = 0;
  for (int i = tid; i < a.T; i += kPlan) plan.owner()[i] = -1;
  __syncthreads();
  for (int s = tid; s < n; s += kPlan) {
    const Seq q = sequence(c, a, s, 1, 1);
    const bool on = q.n && !q.bad;
    count[s] = on ? q.n : 0, pos[s] = 0;
    whole[s] = on && int64_t(q.n) * group <= kMostRowsShared ? q.len >> c.page_shift : 0;
    PlanSeq p{};
    p.begin = q.begin, p.n = q.n, p.len = q.len, p.levels = on ? 0 : -1;
    plan.seqs()[s] = p;
  }
  __syncthreads();
  // tokens that two sequences claim (start not ascending) would not fit the lists
  int64_t tokens_of = 0, all_tokens;
  for (int s = tid; s < n; s += kPlan) tokens_of += count[s];
  for (int step = 1; step < kWave; step *= 2) tokens_of += __shfl_xor(tokens_of, step);
  if (lane == 0) scan[0][wave] = tokens_of;
  __syncthreads();
  all_tokens = 0;
  for (int w = 0; w < kPlan / kWave; ++w) all_tokens += scan[0][w];
  if (all_tokens > a.T) {
    if (tid == 0) *plan.head() = Head{};
    return;
  }
  __syncthreads();
  for (int s = wave; s < n; s += kPlan / kWave) {
    const int begin = a.start[s], end = a.start[s + 1];
    if (begin >= 0 && end <= a.T)
      for (int i = begin + lane; i < end; i += kWave) plan.owner()[i] = s;
  }
  for (int round = 0; round < kLevels; ++round) {
    for (int s = tid; s < n; s += kPlan) {
      int x = -1;
      if (pos[s] < whole[s]) x = c.table[int64_t(s) * c.max_pages + pos[s]];
      next[s] = x, best[s] = 0, cut[s] = 0;
    }
    __syncthreads();
    for (int s = tid; s < n; s += kPlan) {
      const int x = next[s], p = pos[s];
      int t = 0;
      if (x >= 0) while (t < s && (next[t] != x || pos[t] != p)) ++t;
      lead[s] = x >= 0 ? t : s;
    }
    __syncthreads();
    for (int s = wave; s < n; s += kPlan / kWave) {
      const int t = lead[s];
      const int d = t == s ? 0 : common(c, s, t, pos[s], min(whole[s], whole[t]));
      if (lane == 0) same[s] = d;
    }
    __syncthreads();
    unsigned long long saved[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int s = tid + i * kPlan;
      saved[i] = 0;
      if (s >= n || lead[s] == s) continue;
      int m = 0;
      for (int t = lead[s] + 1; t < n; ++t) m += lead[t] == lead[s] && same[t] >= same[s];
      saved[i] = static_cast<unsigned long long>(same[s]) * m;
      atomicMax(&best[lead[s]], saved[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int s = tid + i * kPlan;
      if (saved[i] && saved[i] == best[lead[s]] && saved[i] << c.page_shift >= kLeastSaved) atomicMax(&cut[lead[s]], same[s]);
    }
    __syncthreads();
    bool any = false;
    for (int s = tid; s < n; s += kPlan) {
      const int d = cut[lead[s]];
      any |= d > 0;
      next[s] = d > 0 && (lead[s] == s || same[s] >= d) ? lead[s] : INT_MAX;
    }
    if (!__syncthreads_or(any)) break;
    const int first_node = nodes_s;
    __syncthreads();
    for (int s = tid; s < n; s += kPlan) {
      const int mine = next[s];
      if (mine == INT_MAX) continue;
      // the round's list: nodes in the order of their leaders, tokens in the
      // order of their sequences
      int node = first_node, list = 0, at = 0, tokens = 0;
      for (int t = 0; t < n; ++t) {
        const int x = next[t];
        node += x == t && t < mine;
        list += x < mine ? count[t] : 0;
        tokens += x == mine ? count[t] : 0;
        at += x == mine && t < s ? count[t] : 0;
      }
      list += round * a.T;
      PlanSeq& p = plan.seqs()[s];
      for (int i = 0; i < count[s]; ++i) plan.tokens()[list + at + i] = p.begin + i;
      p.node[p.levels] = node, p.at[p.levels] = at;
      ++p.levels;
      if (s == mine) {
        Node x{};
        x.seq = s, x.key0 = pos[s] << c.page_shift, x.keys = cut[s] << c.page_shift;
        x.tokens = tokens, x.list = list;
        plan.nodes()[node] = x;
        atomicAdd(&nodes_s, 1);
      }
    }
    __syncthreads();
    for (int s = tid; s < n; s += kPlan)
      if (next[s] != INT_MAX) pos[s] += cut[next[s]];
    __syncthreads();
  }
  __syncthreads();
  const int shared_nodes = nodes_s;
  __syncthreads();
  // what every sequence has for itself
  for (int s = tid; s < n; s += kPlan) {
    if (!count[s]) continue;
    int node = shared_nodes;
    for (int t = 0; t < s; ++t) node += count[t] > 0;
    PlanSeq& p = plan.seqs()[s];
    Node x{};
    x.seq = s, x.key0 = pos[s] << c.page_shift;
    x.len = p.len - x.key0, x.n = p.n, x.keys = x.len + x.n, x.begin = p.begin;
    x.tokens = p.n, x.list = -1;
    plan.nodes()[node] = x;
    p.node[p.levels] = node, p.at[p.levels] = 0;
    ++p.levels;
    atomicAdd(&nodes_s, 1);
  }
  __syncthreads();
  // chunks of the keys, equal for all, so that there is a workgroup for each slot
  const int nodes = nodes_s, each = (nodes + kPlan - 1) / kPlan, from = tid * each, to = min(from + each, nodes);
  auto row_tiles = [&](const Node& x) { return (int64_t(x.tokens) * group + M - 1) / M; };
  auto key_tiles = [&](const Node& x) { return (x.keys + KT - 1) / KT; };
  auto prefix = [&](int64_t mine, int which, int64_t& total) {
    int64_t incl = mine;
    for (int step = 1; step < kWave; step *= 2) {
      const int64_t x = __shfl_up(incl, step);
      if (lane >= step) incl += x;
    }
    if (lane == kWave - 1) scan[which][wave] = incl;
    __syncthreads();
    int64_t before = incl - mine;
    total = 0;
    for (int w = 0; w < kPlan / kWave; ++w) {
      if (w < wave) before += scan[which][w];
      total += scan[which][w];
    }
    return before;
  };
  int64_t work = 0, total;
  for (int i = from; i < to; ++i) work += row_tiles(plan.nodes()[i]) * key_tiles(plan.nodes()[i]);
  prefix(work, 0, total);
  const int64_t tiles = max(int64_t(4), (total * c.kv_heads + kSlots - 1) / kSlots);
  int64_t units = 0, rows = 0, all_units, all_rows;
  for (int i = from; i < to; ++i) {
    Node& x = plan.nodes()[i];
    x.chunks = static_cast<int>((key_tiles(x) + tiles - 1) / tiles), x.tiles = static_cast<int>(min(tiles, int64_t(key_tiles(x))));
    units += row_tiles(x) * x.chunks, rows += int64_t(x.tokens) * a.q_heads * x.chunks;
  }
  units = prefix(units, 1, all_units), rows = prefix(rows, 2, all_rows);
  for (int i = from; i < to; ++i) {
    Node& x = plan.nodes()[i];
    x.unit = static_cast<int>(units), x.part = rows;
    units += row_tiles(x) * x.chunks, rows += int64_t(x.tokens) * a.q_heads * x.chunks;
  }
  const bool fits = all_units <= plan.y.most_units && all_rows <= plan.y.most_rows;
  __syncthreads();
  if (fits)
    for (int i = wave; i < nodes; i += kPlan / kWave) {
      const Node& x = plan.nodes()[i];
      const int count = static_cast<int>(row_tiles(x)) * x.chunks;
      for (int u = lane; u < count; u += kWave) plan.units()[x.unit + u] = i;
    }
  if (tid == 0) *plan.head() = Head{fits ? kMagic : 0, a.T, a.q_heads, fits ? int(all_units) : 0, nodes, M, KT, 0};
}

// Whether the plan is one for this call.
__device__ inline bool planned(const Plan& plan, const KvAttention& a, int M) {
  const Head* h = plan.head();
  return h->magic == kMagic && h->T == a.T && h->q_heads == a.q_heads && h->rows == M;
}

// First part row of row tile rt, chunk k of a node and key head: a chunk's parts
// are the tile's rows for head 0, then for head 1, ...
__device__ inline int64_t part_row(const KvCache& c, const Node& x, int group, int M, int rt, int k, int h) {
  const int64_t all = int64_t(x.tokens) * group, first = int64_t(rt) * M, rows = min(int64_t(M), all - first);
  return x.part + c.kv_heads * (first * x.chunks + k * rows) + h * rows;
}

// A unit of the plan and a key head.
template <int DT, int D, int MT>
__global__ __launch_bounds__(kBlock) void few_nodes_kernel(KvCache c, KvAttention a, Plan plan) {
  using Rows = FewRows<DT, D, MT>;
  constexpr int M = Rows::M;
  __shared__ typename Rows::Lds lds;
  const int h = blockIdx.x % c.kv_heads, unit = blockIdx.x / c.kv_heads;
  if (!planned(plan, a, M) || unit >= plan.head()->units) return;
  const Node x = plan.nodes()[plan.units()[unit]];
  const int group = a.q_heads / c.kv_heads, all = x.tokens * group;
  const int rt = (unit - x.unit) / x.chunks, k = (unit - x.unit) % x.chunks, row0 = rt * M, rows = min(M, all - row0);
  const int32_t* table = c.table + int64_t(x.seq) * c.max_pages + (x.key0 >> c.page_shift);
  const int32_t* list = x.list < 0 ? nullptr : plan.tokens() + x.list;
  FewTile t{};
  t.h = h, t.kt0 = k * x.tiles, t.kt1 = min(t.kt0 + x.tiles, (x.keys + Rows::KW - 1) / Rows::KW);
  if (list) {  // all rows see all keys
    a.parent = nullptr;
    t.q.len = t.limit = x.keys;
    t.tok0 = t.tok1 = -1;
  } else {
    t.q.begin = x.begin, t.q.n = x.n, t.q.len = x.len;
    t.tok0 = row0 / group, t.tok1 = (row0 + rows - 1) / group;
    t.limit = a.parent ? x.keys : x.len + t.tok1 + 1;
  }
  auto page_at = [&](int key) { return max(0, min(table[key >> c.page_shift], c.pages - 1)); };
  auto query = [&](int r) {
    const int row = row0 + min(r, rows - 1), at = row / group;
    const int token = list ? list[at] : x.begin + at;
    return int64_t(token) * a.ldq + int64_t(h * group + row % group) * D;
  };
  auto token = [&](int r) { return list || r >= rows ? -1 : (row0 + r) / group; };
  const Parts parts = plan.parts();
  const int64_t part = part_row(c, x, group, M, rt, k, h);
  Rows::run(c, a, lds, t, page_at, query, token, [&](int r, int column, f32x4 v, float top, float l) {
    if (r >= rows) return;
    *reinterpret_cast<f32x4*>(parts.values + (part + r) * D + column) = v;
    if (column == 0) parts.stats[part + r] = float2{top, l};
  });
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
        const int r = (p.at[i] + t - p.begin) * group + head % group, rt = r / M;
        const int64_t first = part_row(c, node, group, M, rt, 0, h) + r % M;
        const int64_t step = part_row(c, node, group, M, rt, 1, h) + r % M - first;
        sum.add<D>(plan.parts(), node.chunks, column, [&](int k) { return first + k * step; });
      }
      x = sum.x * (1.f / sum.l);
    }
  }
  store4<DT>(a.out, row * D + column, x);
}

// Rows and keys of a tile.
struct Shape {
  int rows, keys;
};
Shape shape(const KvCache& c, int32_t T, int32_t q_heads) {
  const int64_t rows = int64_t(T) * (q_heads / c.kv_heads);
  return Shape{rows > 16 && (c.dtype == TMS_BF16 || c.head_dim < 256) ? 32 : 16, c.dtype == TMS_F32 ? 16 : 32};
}

template <int DT, int D>
hipError_t launch(const KvCache& c, const KvShared& sh, const Plan& plan, hipStream_t s) {
  const KvAttention& a = sh.a;
  const int M = shape(c, a.T, a.q_heads).rows;
  const int64_t blocks = int64_t(plan.y.most_units) * c.kv_heads, rows = int64_t(a.T) * a.q_heads;
  constexpr int kRows = kBlock * 4 / D;
  if (blocks >= (int64_t(1) << 32) / kBlock || rows >= (int64_t(1) << 32) / kBlock) return hipErrorInvalidValue;
  if (M == 16) few_nodes_kernel<DT, D, 1><<<unsigned(blocks), kBlock, 0, s>>>(c, a, plan);
  else if constexpr (DT == 1 || D < 256) few_nodes_kernel<DT, D, 2><<<unsigned(blocks), kBlock, 0, s>>>(c, a, plan);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  join_nodes_kernel<DT, D><<<unsigned((rows + kRows - 1) / kRows), kBlock, 0, s>>>(c, a, plan, M);
  return hipGetLastError();
}

}  // namespace

int64_t kv_share_bytes(const KvCache& c, int32_t T, int32_t q_heads) {
  return layout(c, T, q_heads, shape(c, T, q_heads).rows).bytes;
}

hipError_t launch_kv_share(const KvCache& c, const KvShared& sh, hipStream_t s) {
  const Shape x = shape(c, sh.a.T, sh.a.q_heads);
  const Plan plan{static_cast<char*>(sh.plan), layout(c, sh.a.T, sh.a.q_heads, x.rows)};
  plan_kernel<<<1, kPlan, 0, s>>>(c, sh.a, plan, x.rows, x.keys);
  return hipGetLastError();
}

hipError_t launch_kv_attention_shared(const KvCache& c, const KvShared& sh, hipStream_t s) {
  // where every sequence has many rows there is nothing to share
  if (int64_t(sh.a.max_new) * (sh.a.q_heads / c.kv_heads) > kMostRowsShared) return launch_kv_attention(c, sh.a, s);
  const Shape x = shape(c, sh.a.T, sh.a.q_heads);
  const Plan plan{static_cast<char*>(sh.plan), layout(c, sh.a.T, sh.a.q_heads, x.rows)};
  if (c.dtype == TMS_F32) {
    if (c.head_dim == 64) return launch<0, 64>(c, sh, plan, s);
    return c.head_dim == 128 ? launch<0, 128>(c, sh, plan, s) : launch<0, 256>(c, sh, plan, s);
  }
  if (c.head_dim == 64) return launch<1, 64>(c, sh, plan, s);
  return c.head_dim == 128 ? launch<1, 128>(c, sh, plan, s) : launch<1, 256>(c, sh, plan, s);
}

}  // namespace tms
