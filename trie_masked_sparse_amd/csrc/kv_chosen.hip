// Attention of new tokens over pages of the cache that were chosen for each of
// them and each key head, for gfx950.
//
// Mathematics.  As kv_attention.hip, over fewer keys: of a token's list the
// rows of every page, then the committed rows behind the last whole page and
// the new rows that the token sees.  They are numbered in this order (row j of
// list entry i is i * page_tokens + j, the rest comes behind), so a tile of
// keys may lie in several pages, and the masks are those of a sequence whose
// committed rows are the listed ones.
#include <algorithm>

#include "kv_few.h"

namespace tms {
namespace {

// Workgroup of a row tile of one token and key head, over `each` entries of
// its list; the last of `splits` workgroups also takes the rows behind.  With
// one split the outputs are final, else parts.
template <int DT, int D>
__global__ __launch_bounds__(kBlock) void chosen_kernel(KvCache c, KvChosen ch, int splits, int each, Parts parts) {
  using Rows = FewRows<DT, D, 1>;
  constexpr int M = Rows::M, KW = Rows::KW;
  __shared__ typename Rows::Lds lds;
  __shared__ int found, wrong, valid;
  extern __shared__ int32_t listed[];  // pages of this workgroup's entries
  KvAttention a = ch.a;
  const int tid = threadIdx.x, group = a.q_heads / c.kv_heads, tiles = (group + M - 1) / M;
  const int h = blockIdx.x % c.kv_heads, rt = blockIdx.x / c.kv_heads % tiles, t = blockIdx.x / c.kv_heads / tiles;
  const int split = blockIdx.y, e0 = split * each, e1 = min(e0 + each, ch.k);
  if (tid == 0) found = -1, wrong = 0, valid = max(e1 - e0, 0);
  __syncthreads();
  for (int s = tid; s < c.seqs; s += kBlock)
    if (a.start[s] <= t && t < a.start[s + 1]) found = s;
  __syncthreads();
  const int s = uniform(found);
  const int row0 = rt * M, rows = min(group - row0, M);
  const int64_t all = int64_t(a.T) * a.q_heads, first_row = int64_t(t) * a.q_heads + h * group + row0;
  if (s < 0) {  // a token of nobody: its outputs stay as they are
    if (splits > 1 && tid < rows) parts.stats[split * all + first_row + tid] = float2{0.f, -1.f};
    return;
  }
  Seq q = uniform(sequence(c, a, s, 1, 1));
  const int whole = q.len >> c.page_shift, i = t - q.begin;
  const int32_t* table = c.table + int64_t(s) * c.max_pages;
  bool bad = q.bad || q.n <= i;
  if (!bad) {
    // entries in ascending order up to the first negative one
    const int32_t* list = ch.chosen + (int64_t(t) * c.kv_heads + h) * ch.k;
    for (int e = e0 + tid; e < e1; e += kBlock) {
      const int32_t v = list[e], before = e ? list[e - 1] : -1;
      if (v < 0) atomicMin(&valid, e - e0);
      else if (v >= whole || (e && (before < 0 || before >= v))) wrong = 1;
      listed[e - e0] = v < 0 || v >= whole ? 0 : max(0, min(table[v], c.pages - 1));
    }
  }
  __syncthreads();
  bad |= wrong != 0;
  FewTile tile;
  const bool rest = split == splits - 1;
  const int from_list = bad ? 0 : valid;
  tile.h = h;
  tile.q = q;
  tile.q.len = from_list << c.page_shift;
  tile.tok0 = tile.tok1 = -1;
  tile.limit = tile.q.len;
  if (rest && !bad) {
    tile.q.len += q.len - (whole << c.page_shift);
    tile.tok0 = tile.tok1 = i;
    tile.limit = tile.q.len + (a.parent ? q.n : i + 1);
  } else {
    a.parent = nullptr;
  }
  if (bad) tile.limit = 0;
  tile.kt0 = 0, tile.kt1 = (tile.limit + KW - 1) / KW;
  const int tok = tile.tok0;
  auto page_at = [&](int key) {
    const int e = key >> c.page_shift;
    if (e < from_list) return listed[e];
    return max(0, min(table[whole + e - from_list], c.pages - 1));
  };
  auto query = [&](int, int r) { return int64_t(t) * a.ldq + int64_t(h * group + row0 + min(r, rows - 1)) * D; };
  auto emit = [&](int, int r, int column, f32x4 x, float top, float l) {
    if (r >= rows) return;
    if (bad) x = f32x4{NAN, NAN, NAN, NAN}, l = 1.f;
    const int64_t row = first_row + r;
    if (splits == 1) {
      store4<DT>(a.out, row * D + column, x * (1.f / l));
    } else {
      const int64_t at = split * all + row;
      *reinterpret_cast<f32x4*>(parts.values + at * D + column) = x;
      if (column == 0) parts.stats[at] = float2{top, l};
    }
  };
  Rows::run(c, a, lds, tile, page_at, query, [&](int r) { return r < rows ? tok : -1; }, emit);
}

// A row's parts joined: D / 4 threads to a row.
template <int DT, int D>
__global__ __launch_bounds__(kBlock) void join_chosen_kernel(KvAttention a, int splits, Parts parts) {
  const int64_t all = int64_t(a.T) * a.q_heads, row = int64_t(blockIdx.x) * (kBlock * 4 / D) + threadIdx.x / (D / 4);
  if (row >= all) return;
  const int column = threadIdx.x % (D / 4) * 4;
  if (parts.stats[row].y < 0.f) return;
  PartSum sum;
  sum.add<D, 8>(parts, splits, column, [&](int i) { return i * all + row; });
  store4<DT>(a.out, row * D + column, sum.x * (1.f / sum.l));
}

Parts parts_at(const KvCache& c, int64_t rows) {
  char* p = static_cast<char*>(c.work) + kWorkCounts;
  return Parts{reinterpret_cast<float*>(p), reinterpret_cast<float2*>(p + rows * c.head_dim * 4)};
}

// Where the tiles of tokens and heads are fewer than the workgroups that the chip
// holds at once, their lists are cut, to no less than kLeast keys a workgroup.
constexpr int kFit = 512, kLeast = 256;

struct Cut {
  int64_t items;
  int splits, each;
};
Cut cut(const KvCache& c, const KvChosen& ch) {
  const int group = ch.a.q_heads / c.kv_heads;
  const int64_t items = int64_t(ch.a.T) * c.kv_heads * ((group + 15) / 16);
  const int64_t most = std::max<int64_t>(1, (int64_t(ch.k) << c.page_shift) / kLeast);
  const int splits = static_cast<int>(std::min(most, std::max<int64_t>(1, kFit / items)));
  const int each = (ch.k + splits - 1) / splits;
  return Cut{items, each ? std::max(1, (ch.k + each - 1) / each) : 1, each};
}

template <int DT, int D>
hipError_t launch(const KvCache& c, const KvChosen& ch, hipStream_t s) {
  const Cut x = cut(c, ch);
  if (x.items >= (int64_t(1) << 32) / kBlock) return hipErrorInvalidValue;
  const int64_t rows = int64_t(ch.a.T) * ch.a.q_heads;
  const Parts parts = parts_at(c, rows * x.splits);
  chosen_kernel<DT, D><<<dim3(unsigned(x.items), x.splits), kBlock, size_t(std::max(x.each, 1)) * 4, s>>>(c, ch, x.splits, x.each, parts);
  if (hipError_t e = hipGetLastError(); e != hipSuccess || x.splits == 1) return e;
  constexpr int kRows = kBlock * 4 / D;
  join_chosen_kernel<DT, D><<<unsigned((rows + kRows - 1) / kRows), kBlock, 0, s>>>(ch.a, x.splits, parts);
  return hipGetLastError();
}

template <int DT>
hipError_t launch(const KvCache& c, const KvChosen& ch, hipStream_t s) {
  if (c.head_dim == 64) return launch<DT, 64>(c, ch, s);
  if (c.head_dim == 128) return launch<DT, 128>(c, ch, s);
  return launch<DT, 256>(c, ch, s);
}

}  // namespace

// At most kFit workgroups of 16 rows have parts.
int64_t kv_chosen_work_bytes(const KvCache& c) { return kWorkCounts + int64_t(kFit) * 16 * (c.head_dim + 2) * 4; }

hipError_t launch_kv_attention_pages(const KvCache& c, const KvChosen& ch, hipStream_t s) {
  return c.dtype == TMS_F32 ? launch<0>(c, ch, s) : launch<1>(c, ch, s);
}

}  // namespace tms
