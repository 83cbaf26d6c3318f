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

constexpr int kHeld = 2048, kWords = 1024;  // pages of a workgroup, words of its sequence's pages (sequences of 32768)

// What a launch is cut into: `splits` workgroups for the pages of a list, in even
// shares of them.  Drafts of a sequence choose mostly the same pages: where there
// are some, a workgroup takes as many tokens of a sequence as fit a row tile, over
// all pages that any of them has chosen (`together`, at most `held` for a
// workgroup: tokens of 3 to 13 drafts of 16 sequences, 24 pages of 32 rows each,
// 62 -> 42 us).
struct Cut {
  int64_t items;
  int splits, together, held, words;  // words of 32 pages in a sequence, at most
};

// Pages of a workgroup's keys, in LDS: of one token the entries of its list, of
// several the pages that any has chosen, each with the tokens that have.
struct Listed {
  int32_t* page;   // [held]
  int32_t* mine;   // [held], of one of several tokens
  uint32_t* bits;  // [words]: a bit for each chosen page, then
  int32_t* before; //   [words]: how many in the words before
  uint16_t* of;    // [held]: tokens, a bit each
};
__host__ __device__ inline int64_t listed_bytes(const Cut& x) {
  return x.together == 1 ? 4 * int64_t(x.held) : 8 * int64_t(x.held) + 8 * int64_t(x.words) + 2 * int64_t(x.held + x.held % 2);
}
__device__ inline Listed listed_at(const Cut& x, int32_t* p) {
  if (x.together == 1) return Listed{p, p, nullptr, nullptr, nullptr};
  int32_t* const bits = p + 2 * x.held;
  return Listed{p, p + x.held, reinterpret_cast<uint32_t*>(bits), bits + x.words, reinterpret_cast<uint16_t*>(bits + 2 * x.words)};
}

// Sum over the threads up to and including this one; sums: of the wavefronts, free
// again behind the next barrier.
__device__ inline int threads_before(int x, int* sums) {
  const int wave = threadIdx.x / kWave;
  x += from_lane<0x111, 0xf>(x);  // 1, 2, 4 and 8 lanes down in rows of 16
  x += from_lane<0x112, 0xf>(x);
  x += from_lane<0x114, 0xf>(x);
  x += from_lane<0x118, 0xf>(x);
  x += from_lane<0x142, 0xa>(x);  // row 0 to row 1, row 2 to row 3
  x += from_lane<0x143, 0xc>(x);  // lane 31 to rows 2 and 3
  if (threadIdx.x % kWave == kWave - 1) sums[wave] = x;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w)
    if (w < wave) x += sums[w];
  return x;
}

// Workgroup of a row tile of one token and key head, or of several tokens of a
// sequence.  The last of the splits also takes the rows behind the last whole
// page.  With one split the outputs are final, else parts, which the last split
// to arrive joins in their order.
//
// Measured (MI355X, bf16): 64 tokens behind 100 to 60000 rows, 64 pages of 64 rows
// each, 32 / 8 heads of 128: 150 us for 742 MB, 4.9 TB/s of the 6.1 that a plain read
// reaches; the longest lists end last.  One token, 32 pages, 16 / 8 heads: 13 us, the
// chain list, page number, keys, join.  3 to 13 drafts of 16 sequences, 24 pages of 32
// rows: 43 us for 116 MB: unions of 24 to 190 pages, so uneven workgroups, and the
// same chain with the union's three passes over the lists before it.
template <int DT, int D, bool Together>
__global__ __launch_bounds__(kBlock, D == 256 ? 1 : 2) void chosen_kernel(KvCache c, KvChosen ch, Cut x, Parts parts) {
  using Rows = FewRows<DT, D, 1>;
  constexpr int M = Rows::M, KW = Rows::KW;
  __shared__ typename Rows::Lds lds;
  __shared__ int found[6], sums[kWaves], count, arrivals;
  __shared__ uint32_t wrong;
  extern __shared__ int32_t dynamic[];
  const Listed listed = listed_at(x, dynamic);
  KvAttention a = ch.a;
  const int tid = threadIdx.x, group = a.q_heads / c.kv_heads, tiles = (group + M - 1) / M;
  const int h = blockIdx.x % c.kv_heads, split = blockIdx.y;
  const int tile_at = blockIdx.x / c.kv_heads;  // of this head
  const int rt = Together ? 0 : tile_at % tiles;
  if (tid == 0) found[0] = -1, wrong = 0, count = 0;
  if constexpr (Together) {
    // tiles of the sequences before each
    for (int i = tid; i < x.words; i += kBlock) listed.bits[i] = 0;
    const int each = (c.seqs + kBlock - 1) / kBlock, s0 = min(tid * each, c.seqs), s1 = min(s0 + each, c.seqs);
    Seq q{};
    int mine = 0;
    for (int s = s0; s < s1; ++s) {
      q = sequence(c, a, s, 1, 1);
      mine += (q.n + x.together - 1) / x.together;
    }
    const int before = threads_before(mine, sums) - mine;
    if (tile_at >= before && tile_at < before + mine) {
      int at = before, s = s0;
      for (; each > 1; ++s) {
        q = sequence(c, a, s, 1, 1);
        const int n = (q.n + x.together - 1) / x.together;
        if (tile_at < at + n) break;
        at += n;
      }
      found[0] = s, found[1] = q.begin, found[2] = q.n, found[3] = q.len, found[4] = q.bad, found[5] = q.begin + (tile_at - at) * x.together;
    }
  } else {
    __syncthreads();
    const int t = tile_at / tiles;
    for (int s = tid; s < c.seqs; s += kBlock) {
      const Seq q = sequence(c, a, s, 1, 1);
      if (q.n && q.begin <= t && t < q.begin + q.n)
        found[0] = s, found[1] = q.begin, found[2] = q.n, found[3] = q.len, found[4] = q.bad, found[5] = t;
    }
  }
  __syncthreads();
  const int s = uniform(found[0]);
  if (s < 0) return;  // a token of nobody (its outputs stay as they are), or no tile
  Seq q{};
  q.begin = uniform(found[1]), q.n = uniform(found[2]), q.len = uniform(found[3]), q.bad = uniform(found[4]);
  const int t = uniform(found[5]), i0 = t - q.begin;  // the first token; which of its sequence's new tokens
  const int row0 = rt * M;
  const int64_t all = int64_t(a.T) * a.q_heads;
  const int tokens = Together ? min(x.together, q.n - i0) : 1;  // of this workgroup
  const int rows = Together ? tokens * group : min(group - row0, M);
  const int whole = q.bad ? 0 : q.len >> c.page_shift, rest = q.len - (whole << c.page_shift);
  const int32_t* table = c.table + int64_t(s) * c.max_pages;
  const bool last = split == x.splits - 1;
  const int32_t* lists = ch.chosen + (int64_t(t) * c.kv_heads + h) * ch.k;  // the next token's kv_heads * k further on
  const int64_t list_step = int64_t(c.kv_heads) * ch.k;
  // entry e of token i: the page, or -1; ascending up to the first negative one
  auto entry = [&](int i, int e) {
    const int32_t* p = lists + i * list_step + e;
    const int32_t v = *p, before = e ? p[-1] : -1;
    if (v < 0) return -1;
    if (v >= whole || (e && (before < 0 || before >= v))) {
      atomicOr(&wrong, 1u << i);
      return -1;
    }
    return v;
  };
  int n_pages = 0;  // of this workgroup
  if (q.bad) {
    if (tid == 0) wrong = ~0u;
  } else if constexpr (!Together) {
    const int e0 = split * x.held, e1 = min(e0 + x.held, ch.k);
    int n = 0;  // entries are a run from the first on
    for (int e = e0 + tid; e < e1; e += kBlock) {
      const int v = entry(0, e);
      // (of a refused entry any page: a good one may follow, and the keys up to it are
      // read, though the outputs are NaN)
      listed.page[e - e0] = v >= 0 ? max(0, min(table[v], c.pages - 1)) : 0;
      if (v >= 0) n = max(n, e - e0 + 1);
    }
    if (n) atomicMax(&count, n);
    __syncthreads();
    n_pages = uniform(count);
  } else {
    const int entries = tokens * ch.k;
    for (int j = tid; j < entries; j += kBlock) {
      const int v = entry(j / ch.k, j % ch.k);
      if (v >= 0) atomicOr(&listed.bits[v >> 5], 1u << (v & 31));
    }
    __syncthreads();
    // pages before each word, and in all
    const int each = (x.words + kBlock - 1) / kBlock, w0 = min(tid * each, x.words), w1 = min(w0 + each, x.words);
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(listed.bits[w]);
    __syncthreads();  // the first use of sums
    int before = threads_before(mine, sums) - mine, chosen = 0;
    for (int w = 0; w < kWaves; ++w) chosen += sums[w];
    const int share = (uniform(chosen) + x.splits - 1) / x.splits;  // at most `held`
    const int u0 = min(split * share, chosen), u1 = min(u0 + share, chosen);
    n_pages = uniform(u1 - u0);
    for (int w = w0; w < w1; ++w) {
      listed.before[w] = before;
      for (uint32_t word = listed.bits[w]; word; word &= word - 1, ++before)
        if (before >= u0 && before < u1) listed.page[before - u0] = max(0, min(table[32 * w + __builtin_ctz(word)], c.pages - 1));
    }
    for (int i = tid; i < (x.held + 1) / 2; i += kBlock) reinterpret_cast<uint32_t*>(listed.of)[i] = 0;
    __syncthreads();
    for (int j = tid; j < entries; j += kBlock) {
      const int i = j / ch.k, v = lists[i * list_step + j % ch.k];
      if (v < 0 || v >= whole || wrong >> i & 1) continue;
      const int u = listed.before[v >> 5] + __popc(listed.bits[v >> 5] & ((1u << (v & 31)) - 1)) - u0;
      if (u >= 0 && u < n_pages) atomicOr(&reinterpret_cast<uint32_t*>(listed.of)[u / 2], 1u << (i + u % 2 * 16));
    }
  }
  __syncthreads();
  const uint32_t bad = wrong;
  FewTile tile{};
  tile.h = h;
  // keys: the rows of n pages, then, in the last split, those behind; of the tokens first .. last
  auto keys = [&](int n, int first, int last_token) {
    tile.q = q;
    tile.q.len = n << c.page_shift;
    tile.tok0 = tile.tok1 = -1;
    tile.limit = tile.q.len;
    if (last && !q.bad) {
      tile.q.len += rest;
      tile.tok0 = first, tile.tok1 = last_token;
      tile.limit = tile.q.len + (a.parent ? q.n : last_token + 1);
    }
    tile.kt0 = 0, tile.kt1 = (tile.limit + KW - 1) / KW;
  };
  if (!last || q.bad) a.parent = nullptr;
  auto row_of = [&](int r) { return int64_t(t) * a.q_heads + (Together ? int64_t(r / group) * a.q_heads + r % group : r) + h * group + row0; };
  auto query = [&](int, int r) {
    r = min(r, rows - 1);
    return (t + (Together ? int64_t(r / group) : 0)) * a.ldq + int64_t(h * group + row0 + (Together ? r % group : r)) * D;
  };
  auto token = [&](int r) { return tile.tok0 < 0 || r >= rows ? -1 : Together ? i0 + r / group : i0; };
  auto emit = [&](int, int r, int column, f32x4 v, float top, float l) {
    if (r >= rows) return;
    if (bad >> (Together ? r / group : 0) & 1) v = f32x4{NAN, NAN, NAN, NAN}, l = 1.f, top = 0.f;
    const int64_t row = row_of(r);
    if (x.splits == 1) {
      store4<DT>(a.out, row * D + column, v * (1.f / l));
    } else {
      const int64_t at = split * all + row;
      part_store<true>(reinterpret_cast<f32x4*>(parts.values + at * D + column), v);
      if (column == 0) part_store<true>(&parts.stats[at].x, top), part_store<true>(&parts.stats[at].y, l);
    }
  };
  auto page_in = [&](const int32_t* list, int n, int key) {
    const int e = key >> c.page_shift;
    if (e < n) return list[e];
    return max(0, min(table[whole + e - n], c.pages - 1));
  };
  if constexpr (!Together) {
    keys(n_pages, i0, i0);
    Rows::run(c, a, lds, tile, [&](int key) { return page_in(listed.page, n_pages, key); }, query, token, emit);
  } else {
    // all tokens at once; where a value is not finite, maybe in a page that only
    // others have chosen, a token after the other
    for (int i = -1; i < tokens; ++i) {
      int n = n_pages;
      const int32_t* list = listed.page;
      if (i >= 0) {
        __syncthreads();
        if (tid < kWave) {
          n = 0;
          for (int u0 = 0; u0 < n_pages; u0 += kWave) {
            const int u = min(u0 + tid, n_pages - 1);
            const bool on = u0 + tid < n_pages && listed.of[u] >> i & 1;
            const uint64_t lanes = __ballot(on);
            if (on) listed.mine[n + __popcll(lanes & ((uint64_t(1) << tid) - 1))] = listed.page[u];
            n += __popcll(lanes);
          }
          if (tid == 0) count = n;
        }
        __syncthreads();
        n = uniform(count), list = listed.mine;
      }
      const int first = i < 0 ? 0 : i, end = i < 0 ? tokens : i + 1;
      keys(n, i0 + first, i0 + end - 1);
      auto mine = [&](int r) { return r >= first * group && r < end * group; };
      const bool done = Rows::run(
          c, a, lds, tile, [&](int key) { return page_in(list, n, key); }, query,
          [&](int r) { return tile.tok0 < 0 || !mine(r) ? -1 : i0 + r / group; },
          [&](int h, int r, int column, f32x4 v, float top, float l) {
            if (mine(r)) emit(h, r, column, v, top, l);
          },
          [&](int key, int r) {
            const int e = key >> c.page_shift;
            return e >= n || i >= 0 || (r < rows && listed.of[e] >> (r / group) & 1);
          },
          i < 0);
      if (i < 0 && done) break;
    }
  }
  if (x.splits == 1) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the parts are written
  __syncthreads();
  if (tid == 0) {
    uint32_t* arrived = static_cast<uint32_t*>(c.work) + blockIdx.x;
    arrivals = atomicAdd(arrived, 1u);
    if (arrivals == x.splits - 1) *arrived = 0;
  }
  __syncthreads();
  if (arrivals != x.splits - 1) return;
  for (int i = tid; i < rows * (D / 4); i += kBlock) {
    const int64_t row = row_of(i / (D / 4));
    const int column = i % (D / 4) * 4;
    PartSum sum;
    sum.add<D, 8, true>(parts, x.splits, column, [&](int k) { return k * all + row; });
    store4<DT>(a.out, row * D + column, sum.x * (1.f / sum.l));
  }
}

Parts parts_at(const KvCache& c, int64_t rows) {
  char* p = static_cast<char*>(c.work) + kWorkCounts;
  return Parts{reinterpret_cast<float*>(p), reinterpret_cast<float2*>(p + rows * c.head_dim * 4)};
}

// Where the tiles of tokens and heads are fewer than the workgroups that the chip
// holds at once, their pages are cut, to no less than kLeast keys a workgroup (one
// token, 32 pages of 64: 13.1 us, with 256 and 512 keys 14.3 and 18.1; kFit 1024: 64
// tokens 150 -> 167 us, 16 sequences of drafts 42 -> 47).
constexpr int kFit = 512, kLeast = 128;
static_assert(kFit * 4 <= kWorkCounts, "a counter for each tile that is cut");

Cut cut(const KvCache& c, const KvChosen& ch) {
  const int64_t group = ch.a.q_heads / c.kv_heads, T = ch.a.T;
  auto splits_of = [&](int64_t tiles, int64_t pages) {
    const int64_t most = std::max<int64_t>(1, (pages << c.page_shift) / kLeast);
    return static_cast<int>(std::min(most, std::max<int64_t>(1, kFit / tiles)));
  };
  if (ch.a.max_new > 1 && group <= 8 && ch.k > 0) {
    const int together = static_cast<int>(16 / group);
    // tiles at most, and about (a sequence's last is half full)
    const int64_t seqs = std::min<int64_t>(c.seqs, T), most = std::min(T, T / together + seqs) * c.kv_heads;
    const int64_t tiles = (T / together + (seqs + 1) / 2) * c.kv_heads;
    const int64_t pages = std::min<int64_t>(c.max_pages, int64_t(together) * ch.k);
    const int splits = splits_of(tiles, std::min<int64_t>(pages, 2 * ch.k));
    const int64_t held = (pages + splits - 1) / splits, words = (int64_t(c.max_pages) + 31) / 32;
    if (held <= kHeld && words <= kWords) return Cut{most, splits, together, int(held), int(words)};
  }
  const int64_t items = T * c.kv_heads * ((group + 15) / 16);
  const int splits = splits_of(items, ch.k), held = (ch.k + splits - 1) / splits;
  return Cut{items, held ? std::max(1, (ch.k + held - 1) / held) : 1, 1, std::max(held, 1), 0};
}

template <int DT, int D>
hipError_t launch(const KvCache& c, const KvChosen& ch, hipStream_t s) {
  const Cut x = cut(c, ch);
  if (x.items >= (int64_t(1) << 32) / kBlock) return hipErrorInvalidValue;
  const int64_t rows = int64_t(ch.a.T) * ch.a.q_heads;
  const Parts parts = parts_at(c, rows * x.splits);
  const dim3 grid(unsigned(x.items), x.splits);
  const size_t bytes = listed_bytes(x);
  if (x.together > 1) chosen_kernel<DT, D, true><<<grid, kBlock, bytes, s>>>(c, ch, x, parts);
  else chosen_kernel<DT, D, false><<<grid, kBlock, bytes, s>>>(c, ch, x, parts);
  return hipGetLastError();
}

template <int DT>
hipError_t launch(const KvCache& c, const KvChosen& ch, hipStream_t s) {
  if (c.head_dim == 64) return launch<DT, 64>(c, ch, s);
  if (c.head_dim == 128) return launch<DT, 128>(c, ch, s);
  return launch<DT, 256>(c, ch, s);
}

}  // namespace

// Parts of every row in each split: where there is more than one, at most those
// of kFit full tiles of 16 rows.
int64_t kv_chosen_work_bytes(const KvCache& c) { return kWorkCounts + int64_t(kFit) * 16 * (c.head_dim + 2) * 4; }

hipError_t launch_kv_attention_pages(const KvCache& c, const KvChosen& ch, hipStream_t s) {
  return c.dtype == TMS_F32 ? launch<0>(c, ch, s) : launch<1>(c, ch, s);
}

}  // namespace tms
