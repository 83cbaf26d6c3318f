// Page operations of the paged key/value cache for gfx950: forking by
// reference count, reserving pages (with a copy of a shared last page),
// moving the accepted rows together and giving pages back.
//
// The tables are small integers (a 32-bit word for each page of 10^4..10^6
// bytes), so the bookkeeping is bound by latency: one wavefront for each
// sequence where the sequences are independent, one workgroup where the pages
// are handed out in order.  The rows that move are bound by memory: they are
// copied by a grid over (sequence, keys or values of a head, layer), whose
// contiguous piece is up to page_tokens * head_dim elements.
#include <hip/hip_runtime.h>

#include "kv_cache.h"
#include "tms.h"

namespace tms {
namespace {

constexpr int kWave = 64;

struct ForkRec {
  int32_t length, pages, status, changed;
};
struct CopyRec {
  int32_t from, to, rows, pad;
};

__host__ __device__ inline int64_t round256(int64_t x) { return (x + 255) & ~int64_t(255); }

__device__ inline int pages_of(const KvCache& c, int64_t rows) {
  return static_cast<int>((rows + c.page_tokens - 1) >> c.page_shift);
}

__device__ inline int32_t* fork_rows(const KvCache& c) { return static_cast<int32_t*>(c.work); }
__device__ inline ForkRec* fork_recs(const KvCache& c) {
  return reinterpret_cast<ForkRec*>(static_cast<char*>(c.work) + round256(4ll * c.seqs * c.max_pages));
}
__device__ inline int32_t* free_list(const KvCache& c) { return static_cast<int32_t*>(c.work); }
__device__ inline CopyRec* copy_recs(const KvCache& c) {
  return reinterpret_cast<CopyRec*>(static_cast<char*>(c.work) + round256(4ll * c.pages));
}

__device__ inline bool page_ok(const KvCache& c, int32_t p) { return p >= 0 && p < c.pages; }

// Fork, first half: what every changed sequence becomes, read from the state
// before the call and staged in work (a reordering may replace a sequence
// that others are forked from); the references of the new rows are counted.
__global__ __launch_bounds__(256) void fork_stage_kernel(KvCache c, const int32_t* __restrict__ src) {
  const int s = blockIdx.x * (256 / kWave) + threadIdx.x / kWave, lane = threadIdx.x % kWave;
  if (s >= c.seqs) return;
  const int from = src[s];
  ForkRec r{0, 0, TMS_OK, from != s};
  if (from < -1 || from >= c.seqs) r = ForkRec{0, 0, TMS_ERR_INVALID_ARG, -1};
  if (r.changed == 1 && from >= 0) {
    r.length = c.length[from];
    r.status = c.status[from];
    r.pages = min(pages_of(c, r.length), min(c.held[from], c.max_pages));
    for (int j = lane; j < r.pages; j += kWave) {
      const int32_t p = c.table[int64_t(from) * c.max_pages + j];
      fork_rows(c)[int64_t(s) * c.max_pages + j] = p;
      if (page_ok(c, p)) atomicAdd(&c.refs[p], 1);
    }
  }
  if (lane == 0) fork_recs(c)[s] = r;
}

// Fork, second half: the old rows' references go, the staged rows come in.
__global__ __launch_bounds__(256) void fork_apply_kernel(KvCache c) {
  const int s = blockIdx.x * (256 / kWave) + threadIdx.x / kWave, lane = threadIdx.x % kWave;
  if (s >= c.seqs) return;
  const ForkRec r = fork_recs(c)[s];
  if (r.changed < 0 && lane == 0) c.status[s] = r.status;
  if (r.changed != 1) return;
  int32_t* row = c.table + int64_t(s) * c.max_pages;
  const int old = min(c.held[s], c.max_pages);
  for (int j = lane; j < max(old, r.pages); j += kWave) {
    if (j < old) {
      const int32_t p = row[j];
      if (page_ok(c, p)) atomicSub(&c.refs[p], 1);
    }
    row[j] = j < r.pages ? fork_rows(c)[int64_t(s) * c.max_pages + j] : -1;
  }
  if (lane == 0) {
    c.length[s] = r.length;
    c.held[s] = r.pages;
    c.status[s] = r.status;
  }
}

constexpr int kPlan = 1024;  // threads of the one workgroup that hands out pages

// Sum of v over the threads before this one, and over all of them.  Every
// thread of the workgroup calls it.
__device__ inline int block_before(int v, int* total) {
  __shared__ int wave_total[kPlan / kWave];
  const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
  int incl = v;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == kWave - 1) wave_total[w] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kPlan / kWave; ++i) {
    const int t = wave_total[i];
    if (i < w) before += t;
    all += t;
  }
  __syncthreads();
  *total = all;
  return before + incl - v;
}

// Reserve: demands of all sequences, their prefix sums, the lowest free pages,
// and who gets which.  The order is fixed (sequences ascending, pages
// ascending), so the tables do not depend on timing.
__global__ __launch_bounds__(kPlan) void reserve_plan_kernel(KvCache c, const int32_t* __restrict__ n_new) {
  __shared__ int begin[4096];   // first page of the sequence's share of the free list
  __shared__ int want[4096];    // pages it holds afterwards; -1: left as it is
  const int tid = threadIdx.x;
  CopyRec* recs = copy_recs(c);
  int64_t need = 0;  // all demands (at most pages + 1 counts: more never fits)
  for (int base = 0; base < c.seqs; base += kPlan) {
    const int s = base + tid;
    int more = 0, w = -1;
    CopyRec rec{-1, -1, 0, 0};
    if (s < c.seqs && c.status[s] == TMS_OK && n_new[s] > 0) {
      const int len = c.length[s], held = min(c.held[s], c.max_pages);
      const int64_t rows = int64_t(len) + n_new[s];
      if (rows > int64_t(c.max_pages) << c.page_shift) {
        c.status[s] = TMS_ERR_INVALID_ARG;
      } else {
        w = max(pages_of(c, rows), held);
        more = w - held;
        const int fill = len & (c.page_tokens - 1), last = len >> c.page_shift;
        if (fill && last < held) {
          const int32_t p = c.table[int64_t(s) * c.max_pages + last];
          if (page_ok(c, p) && c.refs[p] > 1) {
            rec = CopyRec{p, -1, fill, 0};
            ++more;
          }
        }
      }
    }
    // a demand above the whole pool never fits; cutting it there keeps the
    // sums below 2^31 (4096 * (pages + 1) could pass it: sum in 64 bits)
    int total;
    more = min(more, c.pages + 1);
    const int hi = more >> 16, lo = more & 0xffff;
    int total_hi;
    const int before_lo = block_before(lo, &total), before_hi = block_before(hi, &total_hi);
    const int64_t at = need + (int64_t(before_hi) << 16) + before_lo;
    if (s < c.seqs) {
      begin[s] = static_cast<int>(min(at, int64_t(c.pages) + 1));
      want[s] = w;
      // the demand itself rides in rec.pad until the pages are known
      rec.pad = more;
      recs[s] = rec;
    }
    need += (int64_t(total_hi) << 16) + total;
  }
  // the lowest free pages, as many as are asked for at most
  const int most = static_cast<int>(min(need, int64_t(c.pages)));
  int32_t* list = free_list(c);
  int found = 0;
  for (int base = 0; base < c.pages && found < most; base += 4 * kPlan) {
    const int p0 = base + 4 * tid;
    int is_free[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      is_free[i] = p0 + i < c.pages && c.refs[p0 + i] == 0;
      n += is_free[i];
    }
    int total;
    int rank = found + block_before(n, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (is_free[i]) {
        if (rank < most) list[rank] = p0 + i;
        ++rank;
      }
    found += total;
  }
  found = min(found, most);
  __syncthreads();
  const int lane = tid % kWave;
  for (int s = tid / kWave; s < c.seqs; s += kPlan / kWave) {
    if (want[s] < 0) continue;
    CopyRec rec = recs[s];
    const int at = begin[s], more = rec.pad;
    rec.pad = 0;
    if (more > 0 && int64_t(at) + more > found) {
      if (lane == 0) {
        c.status[s] = TMS_ERR_OOM;
        recs[s] = CopyRec{-1, -1, 0, 0};
      }
      continue;
    }
    int32_t* row = c.table + int64_t(s) * c.max_pages;
    const int held = min(c.held[s], c.max_pages), split = rec.rows > 0;
    for (int j = held + lane; j < want[s]; j += kWave) {
      const int32_t p = list[at + split + j - held];
      row[j] = p;
      c.refs[p] = 1;
    }
    if (lane == 0) {
      if (split) {
        rec.to = list[at];
        row[c.length[s] >> c.page_shift] = rec.to;
        c.refs[rec.to] = 1;
        atomicSub(&c.refs[rec.from], 1);
      }
      recs[s] = rec;
      c.held[s] = want[s];
    }
  }
}

// The committed rows of every page that reserve replaced by a copy.  One
// workgroup for the keys or values of one head in one layer.
__global__ __launch_bounds__(256) void copy_pages_kernel(KvCache c, int elem_bytes) {
  const int parts = 2 * c.kv_heads;
  const int s = blockIdx.x / parts, part = blockIdx.x % parts, layer = blockIdx.y;
  const CopyRec r = copy_recs(c)[s];
  if (r.rows <= 0) return;
  const int64_t piece = int64_t(c.page_tokens) * c.head_dim * elem_bytes / 16;  // 16-byte words
  const int64_t page0 = (int64_t(layer) * c.pages) * parts;
  const uint4* from = static_cast<const uint4*>(c.kv) + (page0 + int64_t(r.from) * parts + part) * piece;
  uint4* to = static_cast<uint4*>(c.kv) + (page0 + int64_t(r.to) * parts + part) * piece;
  const int n = r.rows * c.head_dim * elem_bytes / 16;
  for (int i = threadIdx.x; i < n; i += 256) to[i] = from[i];
}

// Whether entry i of a sequence's keep list is out of order or past the rows
// it has reserved.
__device__ inline bool keep_bad(const KvCache& c, int s, const int32_t* keep, int i) {
  const int k = keep[i], prev = i ? keep[i - 1] : -1;
  return k <= prev || int64_t(c.length[s]) + k >= int64_t(min(c.held[s], c.max_pages)) << c.page_shift;
}

// Accepted rows moved together, in place.  An ascending list never moves a row
// upwards, so a chunk of rows may be written once every row of the chunk has
// been read: later chunks read only rows at or past their own targets.
constexpr int kMove = 8;  // 16-byte words in flight for each thread

__global__ __launch_bounds__(256) void move_rows_kernel(KvCache c, const int32_t* __restrict__ n_keep,
                                                        const int32_t* __restrict__ keep_all, int keep_stride,
                                                        int elem_bytes) {
  const int parts = 2 * c.kv_heads;
  const int s = blockIdx.x / parts, part = blockIdx.x % parts, layer = blockIdx.y;
  const int n = n_keep[s];
  if (n <= 0 || n > keep_stride || c.status[s] != TMS_OK) return;
  const int32_t* keep = keep_all + int64_t(s) * keep_stride;
  int bad = 0, moves = 0;
  for (int i = threadIdx.x; i < n; i += 256) {
    bad |= keep_bad(c, s, keep, i);
    moves |= keep[i] != i;
  }
  bad = __syncthreads_or(bad);
  moves = __syncthreads_or(moves);
  if (bad || !moves) return;
  const int words = c.head_dim * elem_bytes / 16, shift = __builtin_ctz(words), len = c.length[s];  // words: 8 .. 64
  const int32_t* row = c.table + int64_t(s) * c.max_pages;
  uint4* kv = static_cast<uint4*>(c.kv);
  auto at = [&](int r, int w) -> int64_t {
    const int32_t p = row[r >> c.page_shift];
    if (!page_ok(c, p)) return -1;
    return (((int64_t(layer) * c.pages + p) * parts + part) * c.page_tokens + (r & (c.page_tokens - 1))) * words + w;
  };
  for (int64_t base = 0; base < int64_t(n) << shift; base += 256 * kMove) {
    uint4 v[kMove];
    int64_t to[kMove];
#pragma unroll
    for (int u = 0; u < kMove; ++u) {
      const int64_t i = base + u * 256 + threadIdx.x;
      const int j = static_cast<int>(i >> shift), w = static_cast<int>(i) & (words - 1);
      to[u] = -1;
      if (j < n && keep[j] != j) {
        const int64_t from = at(len + keep[j], w);
        to[u] = at(len + j, w);
        if (from < 0) to[u] = -1;
        if (to[u] >= 0) v[u] = kv[from];
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // every row of the chunk is in registers
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMove; ++u)
      if (to[u] >= 0) kv[to[u]] = v[u];
  }
}

// Lengths after a commit, and the pages past them given back.  One wavefront
// for each sequence.
__global__ __launch_bounds__(256) void commit_kernel(KvCache c, const int32_t* __restrict__ n_keep,
                                                     const int32_t* __restrict__ keep_all, int keep_stride) {
  const int s = blockIdx.x * (256 / kWave) + threadIdx.x / kWave, lane = threadIdx.x % kWave;
  if (s >= c.seqs) return;
  const int n = n_keep[s];
  if (n < 0 || c.status[s] != TMS_OK) return;
  const int len = c.length[s], held = min(c.held[s], c.max_pages);
  bool bad = int64_t(len) + n > int64_t(held) << c.page_shift;
  if (keep_all) {
    bad |= n > keep_stride;
    if (!bad)
      for (int i = lane; i < n; i += kWave) bad |= keep_bad(c, s, keep_all + int64_t(s) * keep_stride, i);
  }
  if (__any(bad)) {
    if (lane == 0) c.status[s] = TMS_ERR_INVALID_ARG;
    return;
  }
  int32_t* row = c.table + int64_t(s) * c.max_pages;
  const int pages = pages_of(c, int64_t(len) + n);
  for (int j = pages + lane; j < held; j += kWave) {
    const int32_t p = row[j];
    if (page_ok(c, p)) atomicSub(&c.refs[p], 1);
    row[j] = -1;
  }
  if (lane == 0) {
    c.length[s] = len + n;
    c.held[s] = pages;
  }
}

int waves_grid(int seqs) { return (seqs + 3) / 4; }
int elem_bytes(const KvCache& c) { return c.dtype == TMS_F32 ? 4 : 2; }

}  // namespace

int64_t kv_page_work_bytes(const KvCache& c) {
  const int64_t fork = round256(4ll * c.seqs * c.max_pages) + int64_t(sizeof(ForkRec)) * c.seqs;
  const int64_t reserve = round256(4ll * c.pages) + int64_t(sizeof(CopyRec)) * c.seqs;
  return round256(fork > reserve ? fork : reserve);
}

hipError_t launch_kv_fork(const KvCache& c, const int32_t* src, hipStream_t s) {
  fork_stage_kernel<<<waves_grid(c.seqs), 256, 0, s>>>(c, src);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  fork_apply_kernel<<<waves_grid(c.seqs), 256, 0, s>>>(c);
  return hipGetLastError();
}

hipError_t launch_kv_reserve(const KvCache& c, const int32_t* n_new, hipStream_t s) {
  reserve_plan_kernel<<<1, kPlan, 0, s>>>(c, n_new);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  copy_pages_kernel<<<dim3(c.seqs * 2 * c.kv_heads, c.layers), 256, 0, s>>>(c, elem_bytes(c));
  return hipGetLastError();
}

hipError_t launch_kv_commit(const KvCache& c, const int32_t* n_keep, const int32_t* keep, int32_t keep_stride,
                            hipStream_t s) {
  if (keep) {
    move_rows_kernel<<<dim3(c.seqs * 2 * c.kv_heads, c.layers), 256, 0, s>>>(c, n_keep, keep, keep_stride,
                                                                             elem_bytes(c));
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  commit_kernel<<<waves_grid(c.seqs), 256, 0, s>>>(c, n_keep, keep, keep_stride);
  return hipGetLastError();
}

}  // namespace tms
