// The arithmetic of the shared attention's plan (trie_masked_sparse_amd/csrc/
// kv_plan.h) over batches of every kind, without a GPU: the units and part rows of
// a batch fit the memory that its layout has for them, and a unit is worked on by
// as many key heads as it was cut for.  Prints "ok <batches>".
#include <cstdio>
#include <vector>

#include "kv_plan.h"

using namespace tms;

namespace {

struct Batch {
  KvCache c;
  int T, q_heads;
  std::vector<Node> nodes;
};

// `seqs` sequences of `n` new tokens each, behind runs of pages that `fan[i]` of
// them share (0: none of that level), of keys[i] rows, and `own` rows of their own.
Batch batch(int dtype, int dim, int kv_heads, int group, int seqs, int n, const int (&fan)[kLevels], const int (&keys)[kLevels], int own) {
  Batch b{};
  b.c.dtype = dtype, b.c.head_dim = dim, b.c.kv_heads = kv_heads, b.c.seqs = seqs, b.c.page_shift = 5;
  b.T = seqs * n, b.q_heads = kv_heads * group;
  for (int i = 0; i < kLevels; ++i)
    for (int s = 0; fan[i] && s < seqs; s += fan[i]) {
      Node x{};
      x.tokens = std::min(fan[i], seqs - s) * n, x.keys = keys[i];
      if (x.tokens > n) b.nodes.push_back(x);
    }
  for (int s = 0; s < seqs; ++s) {
    Node x{};
    x.tokens = n, x.keys = own + n, x.list = -1, x.n = n;
    b.nodes.push_back(x);
  }
  return b;
}

bool fits(const Batch& b) {
  const int M = rows_of(shape(b.c, b.T, b.q_heads)), heads = small_heads(b.c, b.T, b.q_heads), group = b.q_heads / b.c.kv_heads;
  for (const Node& x : b.nodes) {
    const Size z = size_of(x, group, b.c.kv_heads, M, heads);
    if (z.heads * unit_heads(shape(b.c, b.T, b.q_heads), z.rows, heads) == b.c.kv_heads) continue;
    std::printf("dtype %d heads %d/%d of %d, %d sequences, %d tokens, a node of %d: %d units of %d key heads\n", b.c.dtype, b.q_heads,
                b.c.kv_heads, b.c.head_dim, b.c.seqs, b.T, x.tokens, z.heads, unit_heads(shape(b.c, b.T, b.q_heads), z.rows, heads));
    return false;
  }
  const Layout y = layout(b.c, b.T, b.q_heads, M);
  int64_t work = 0, units = 0, rows = 0;
  for (const Node& x : b.nodes) work += cost_of(size_of(x, group, b.c.kv_heads, M, heads));
  for (const Node& x : b.nodes) {
    const Size z = size_of(x, group, b.c.kv_heads, M, heads);
    const int chunks = chunks_of(z, work / kSlots + 1);
    units += int64_t(z.row_tiles) * chunks * z.heads, rows += int64_t(x.tokens) * b.q_heads * chunks;
  }
  if (units <= y.most_units && rows <= y.most_rows) return true;
  std::printf("dtype %d heads %d/%d of %d, %d sequences, %d tokens, first node %d keys, own %d: %lld units of %lld, %lld rows of %lld\n",
              b.c.dtype, b.q_heads, b.c.kv_heads, b.c.head_dim, b.c.seqs, b.T, b.nodes[0].keys, b.nodes.back().keys,
              static_cast<long long>(units), static_cast<long long>(y.most_units), static_cast<long long>(rows),
              static_cast<long long>(y.most_rows));
  return false;
}

}  // namespace

int main() {
  long checked = 0, failed = 0;
  const int all_keys[] = {640, 6144, 9024, 20000, 1000000};
  for (int dtype : {int(TMS_F32), int(TMS_BF16)})
    for (int dim : {64, 128, 256})
      for (int kv_heads : {1, 2, 3, 8, 12, 32, 64, 256})
        for (int group : {1, 2, 4, 16})
          for (int seqs : {1, 2, 4, 8, 12, 16, 17, 64, 256, 2050})
            for (int n : {1, 2, 5, 31}) {
              if (n * group > (dim == 256 ? 64 : 128) || seqs * n > 3000) continue;
              for (int own : {0, 20, 1000})
                for (int keys : all_keys)
                  for (int kind = 0; kind < 4; ++kind) {
                    const int one[kLevels] = {seqs, 0, 0}, two[kLevels] = {seqs, 4, 0}, three[kLevels] = {seqs, 16, 2}, none[kLevels] = {0, 0, 0};
                    const int lengths[kLevels] = {keys, keys / 2 + 1, 300};
                    ++checked;
                    failed += !fits(batch(dtype, dim, kv_heads, group, seqs, n, kind == 0 ? one : kind == 1 ? two : kind == 2 ? three : none,
                                          lengths, kind == 3 ? keys : own));
                    if (failed > 10) return 1;
                  }
            }
  if (failed) return 1;
  std::printf("ok %ld\n", checked);
}
