// Plain views of the paged key/value cache shared by its C entry points and
// its kernels.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "tms.h"

namespace tms {

// Device view of a tms_kv (same fields, sizes with their shift).
struct KvCache {
  void* kv;
  int32_t *table, *length, *held, *refs, *status;
  void* work;
  int32_t dtype, layers, pages, kv_heads, page_tokens, page_shift, head_dim, seqs, max_pages;
};

// Layout of KvCache::work.  Its first kWorkCounts bytes are counters, zero
// between calls.  The page operations' scratch and the attention's partial
// results behind them are never live at once (every call leaves nothing
// behind), so they share the same bytes.
//   fork:    int32 table rows [seqs][max_pages], then {length, pages, status, changed} [seqs]
//   reserve: int32 free pages [pages], then {from, to, rows, 0} [seqs]
//   attention: see kv_attention.hip
constexpr int64_t kWorkCounts = TMS_KV_WORK_ZERO;
int64_t kv_page_work_bytes(const KvCache& c);
int64_t kv_attention_work_bytes(const KvCache& c);

struct KvWrite {
  const int32_t* start;
  int32_t T, layer;
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;
  int32_t q_heads;
  void* q_out;
  const void *q_weight, *k_weight;
  float eps;
  const int32_t* pos;
  const float* inv_freq;
  int32_t n_freq, interleaved;
};

struct KvAttention {
  const int32_t* start;
  int32_t T, layer, max_new;
  const void* q;
  int64_t ldq;
  int32_t q_heads;
  const int32_t* parent;
  float scale;
  void* out;
};

// Bounds of the keys of whole pages, [layers][pages][kv_heads][2][head_dim] in the
// cache's type: the lowest and the highest value of each column.
struct KvBounds {
  const int32_t* n_new;  // null: all committed rows
  int32_t max_new;       // of the launch: more rows are looked at all the same
  void* bounds;
};

struct KvSelect {
  KvAttention a;  // start, T, layer, max_new, q, ldq, q_heads, scale
  const void* bounds;
  int32_t k, first, last;
  int32_t* chosen;  // [T][kv_heads][k]
  void* work;
};

constexpr int kMostChosen = 8192;  // pages of a list: their numbers are held in LDS

struct KvChosen {
  KvAttention a;
  const int32_t* chosen;
  int32_t k;
};

struct KvShared {
  KvAttention a;
  void* plan;
};

hipError_t launch_kv_fork(const KvCache& c, const int32_t* src, hipStream_t s);
hipError_t launch_kv_reserve(const KvCache& c, const int32_t* n_new, hipStream_t s);
hipError_t launch_kv_commit(const KvCache& c, const int32_t* n_keep, const int32_t* keep, int32_t keep_stride,
                            hipStream_t s);
hipError_t launch_kv_write(const KvCache& c, const KvWrite& w, hipStream_t s);
hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, hipStream_t s);
hipError_t launch_kv_bounds(const KvCache& c, const KvBounds& b, hipStream_t s);
int64_t kv_select_work_bytes(const KvCache& c, int32_t T);
hipError_t launch_kv_select(const KvCache& c, const KvSelect& a, hipStream_t s);
hipError_t launch_kv_attention_pages(const KvCache& c, const KvChosen& a, hipStream_t s);
int64_t kv_chosen_work_bytes(const KvCache& c);
int64_t kv_share_bytes(const KvCache& c, int32_t T, int32_t q_heads);
hipError_t launch_kv_share(const KvCache& c, const KvShared& a, hipStream_t s);
hipError_t launch_kv_attention_shared(const KvCache& c, const KvShared& a, hipStream_t s);

}  // namespace tms
