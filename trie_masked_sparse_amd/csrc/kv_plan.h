// What the plan of the shared attention is counted by: its layout in memory, row
// tiles and chunks of nodes, units.  Plain arithmetic, for the host and the
// device alike.
#pragma once
#include <algorithm>

#include "kv_cache.h"

namespace tms {
namespace {

constexpr int kLevels = 3;      // nodes of a sequence beside its own
constexpr int kSlots = 512;     // workgroups that the chip holds at once (work cut for 768 to 2048: 64 answers 34 -> 39 to 44 us)
constexpr int kTile = 64;       // keys that the plan counts in
constexpr int kSmall = 16;      // rows of a small node
constexpr int kMostHeads = 2;   // key heads of a unit of one, at most
constexpr int kMedium = 64;     // of one that takes a row tile half as high, where the others' have 128

// Key tiles of a chunk, at least.
constexpr int kLeastTiles = 4;

// Costs in units of 0.35 us, as measured with two workgroups on a compute unit:
// the start of a unit and its end (queries, page numbers, first keys; joining
// wavefronts, parts), and 64 keys of it.
constexpr int kOpenSmall = 20, kOpenLarge = 18, kTileSmall = 4, kTileLarge = 5;

struct Head {
  int32_t magic, T, q_heads, units, nodes, rows, pad[2];
};

struct PlanSeq {
  int32_t begin, n, len, levels;  // tokens, committed rows; nodes (-1: its outputs are NaN)
  struct {
    int32_t node, at;         // where its tokens are among a node's
    int32_t all, M, chunks;   // of the node: rows, rows of a row tile, chunks, parts
    int32_t pad;
    int64_t part;
  } of[kLevels + 1];
};

// Of a sequence: among those before it the first that has most pages in common
// with it, from the first page on, and how many (0: itself).  Two sequences have
// as many pages in common as the fewest on the way from one to the other along
// these: the trie of the tables' rows.
struct Meet {
  int32_t with, pages;
};

struct Node {
  int32_t seq, key0, keys;   // the sequence whose table has the pages; first row, rows
  int32_t tokens, list;      // query tokens; their place in the list, -1: begin ..
  int32_t begin, n, len;     // of one sequence's own: its new tokens, committed rows from key0 on
  int32_t chunks, tiles, rows, pad;  // chunks of `tiles` key tiles, rows of a row tile
  int64_t part;              // first row of its parts
};

// What a workgroup works on: a row tile and a chunk of the keys of a node, and a
// key head, or several of a small one.  All that it has to know, in one read.
struct Unit {
  int32_t seq, key0, keys, list, begin, n, len, all;  // of its node; all: rows
  int32_t row0, rows, h, tile0, tile1, M;             // M: rows of its node's row tiles
  int64_t part;
};

// Places in the plan.  M: rows of a tile of nodes that are not small.
struct Layout {
  int64_t seqs, meets, nodes, units, tokens, owner, stats, values, bytes;
  int32_t most_nodes;
  int64_t most_units, most_rows;
};

inline int64_t up(int64_t x) { return (x + 255) & ~int64_t(255); }

inline Layout layout(const KvCache& c, int32_t T, int32_t q_heads, int M) {
  Layout y{};
  const int64_t group = q_heads / c.kv_heads, n = std::min<int64_t>(c.seqs, T);
  y.most_nodes = static_cast<int32_t>(2 * n);  // the sequences' own, and places where the trie branches
  // A node's row tiles and heads, and what cuts add: a chunk costs a slot, less
  // one of its tiles, of which it has kLeastTiles or more.  A unit has the rows of
  // a row tile for each of its heads: 32 for the two of a small one, whatever M (and
  // whether there are two, so that more tokens never need less).
  constexpr int kCuts = kSlots * (kLeastTiles + 1) / kLeastTiles;
  const int64_t tiles = (kLevels + 1) * (int64_t(T) * group / std::max(M, kSmall)) + y.most_nodes;
  y.most_units = tiles * c.kv_heads + kCuts;
  y.most_rows = (kLevels + 1) * int64_t(T) * q_heads + kCuts * std::max<int64_t>(M, kMostHeads * kSmall);
  y.seqs = up(sizeof(Head));
  y.meets = up(y.seqs + c.seqs * int64_t(sizeof(PlanSeq)));
  y.nodes = up(y.meets + c.seqs * int64_t(sizeof(Meet)));
  y.units = up(y.nodes + y.most_nodes * int64_t(sizeof(Node)));
  y.tokens = up(y.units + y.most_units * int64_t(sizeof(Unit)));
  y.owner = up(y.tokens + kLevels * int64_t(T) * 4);
  y.stats = up(y.owner + int64_t(T) * 4);
  y.values = up(y.stats + y.most_rows * 8);
  y.bytes = up(y.values + y.most_rows * c.head_dim * 4);
  return y;
}

// How a node is cut.  M: rows of a tile of nodes that are not small; heads: key
// heads of a unit of a small one.
struct Size {
  int rows, row_tiles, key_tiles, heads;  // rows of a tile; heads: units of a row tile and chunk
  bool small;
  int open, tile;  // cost of a unit and of one of its key tiles
};
__host__ __device__ inline Size size_of(const Node& x, int group, int kv_heads, int M, int heads) {
  const int64_t rows = int64_t(x.tokens) * group;
  const bool small = rows <= kSmall;
  const int of = small ? kSmall : rows <= kMedium && M > kMedium ? kMedium : M;
  return Size{of, static_cast<int>((rows + of - 1) / of), (x.keys + kTile - 1) / kTile, small ? kv_heads / heads : kv_heads,
              small, small ? kOpenSmall : kOpenLarge, small ? kTileSmall * heads : kTileLarge};
}
__host__ __device__ inline int64_t cost_of(const Size& z) {
  return (int64_t(z.key_tiles) * z.tile + z.open) * z.row_tiles * z.heads;
}
// Chunks of the keys: of a unit's cost as much as a slot has, or less.
__host__ __device__ inline int chunks_of(const Size& z, int64_t slot) {
  const int64_t most = slot / z.tile > kLeastTiles ? slot / z.tile : kLeastTiles;  // key tiles
  return static_cast<int>((z.key_tiles + most - 1) / most);
}

// What a node that is not small is worked on by.
enum { kFew16 = 0, kFew32, kMany64, kMany128 };
constexpr __host__ __device__ int rows_of(int shape) { return shape == kFew16 ? 16 : shape == kFew32 ? 32 : shape == kMany64 ? 64 : 128; }

inline int shape(const KvCache& c, int32_t T, int32_t q_heads) {
  const int64_t rows = int64_t(T) * (q_heads / c.kv_heads);  // of a node, at most
  if (rows <= 16) return kFew16;
  if (c.dtype == TMS_F32) return c.head_dim < 256 ? kFew32 : kFew16;
  return rows <= 32 && c.head_dim == 64 ? kFew32 : rows <= 64 ? kMany64 : kMany128;
}

// Whether units of row tiles of M rows are worked on as those of small nodes are,
// and by how many key heads at once.
constexpr __host__ __device__ bool few_rows(int shape, int M) { return shape == kFew16 || M == kSmall; }
inline int unit_heads(int shape, int M, int heads) { return few_rows(shape, M) ? heads : 1; }

// Key heads of a unit of a small node: two where there are units enough (64 answers
// 34 -> 31 us; four where they are four times as many 204 -> 214), and where the
// nodes that are not small have taller row tiles (few_rows tells them apart by
// these) or there are none.
inline int small_heads(const KvCache& c, int32_t T, int32_t q_heads) {
  const bool alike = shape(c, T, q_heads) == kFew16 && int64_t(T) * (q_heads / c.kv_heads) > kSmall;
  return !alike && c.kv_heads % 2 == 0 && int64_t(std::min(c.seqs, T)) * c.kv_heads >= kSlots ? kMostHeads : 1;
}

}  // namespace
}  // namespace tms
