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

#include <algorithm>

#include "kv_cache.h"
#include "tms.h"

namespace tms {
namespace {

constexpr int kWave = 64;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct ForkRec {
  int32_t length, pages, status, changed;
};
struct CopyRec {
  int32_t from, to, rows, pad;  // to: -1 where no page was given, and nothing is copied
};

__host__ __device__ inline int64_t round256(int64_t x) { return (x + 255) & ~int64_t(255); }

__device__ inline int pages_of(const KvCache& c, int64_t rows) {
  return static_cast<int>((rows + c.page_tokens - 1) >> c.page_shift);
}

__device__ inline char* scratch(const KvCache& c) { return static_cast<char*>(c.work) + kWorkCounts; }
__device__ inline int32_t* fork_rows(const KvCache& c) { return reinterpret_cast<int32_t*>(scratch(c)); }
__device__ inline ForkRec* fork_recs(const KvCache& c) {
  return reinterpret_cast<ForkRec*>(scratch(c) + round256(4ll * c.seqs * c.max_pages));
}
__device__ inline int32_t* free_list(const KvCache& c) { return reinterpret_cast<int32_t*>(scratch(c)); }
__device__ inline CopyRec* copy_recs(const KvCache& c) {
  return reinterpret_cast<CopyRec*>(scratch(c) + round256(4ll * c.pages));
}

__device__ inline bool page_ok(const KvCache& c, int32_t p) { return p >= 0 && p < c.pages; }

// Fork, first half, by Lanes lanes: what sequence s becomes, read from the
// state before the call and staged in work (a reordering may replace a sequence
// that others are forked from); the references of the new row are counted.
template <int Lanes>
__device__ inline void fork_stage(const KvCache& c, const int32_t* src, int s, int lane) {
  const int from = src[s];
  ForkRec r{0, 0, TMS_OK, from != s};
  if (from < -1 || from >= c.seqs) r = ForkRec{0, 0, TMS_ERR_INVALID_ARG, -1};
  if (r.changed == 1 && from >= 0) {
    r.length = c.length[from];
    r.status = c.status[from];
    r.pages = min(pages_of(c, r.length), min(c.held[from], c.max_pages));
    for (int j = lane; j < r.pages; j += Lanes) {
      const int32_t p = c.table[int64_t(from) * c.max_pages + j];
      fork_rows(c)[int64_t(s) * c.max_pages + j] = p;
      if (page_ok(c, p)) atomicAdd(&c.refs[p], 1);
    }
  }
  if (lane == 0) fork_recs(c)[s] = r;
}

// Fork, second half: the old row's references go, the staged row comes in.
template <int Lanes>
__device__ inline void fork_apply(const KvCache& c, int s, int lane) {
  const ForkRec r = fork_recs(c)[s];
  if (r.changed < 0 && lane == 0) c.status[s] = r.status;
  if (r.changed != 1) return;
  int32_t* row = c.table + int64_t(s) * c.max_pages;
  const int old = min(c.held[s], c.max_pages);
  for (int j = lane; j < max(old, r.pages); j += Lanes) {
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

// 256 sequences of up to 33 pages: 6.2 and 6.0 us.
__global__ __launch_bounds__(256) void fork_stage_kernel(KvCache c, const int32_t* __restrict__ src) {
  const int s = blockIdx.x * (256 / kWave) + threadIdx.x / kWave;
  if (s < c.seqs) fork_stage<kWave>(c, src, s, threadIdx.x % kWave);
}
__global__ __launch_bounds__(256) void fork_apply_kernel(KvCache c) {
  const int s = blockIdx.x * (256 / kWave) + threadIdx.x / kWave;
  if (s < c.seqs) fork_apply<kWave>(c, s, threadIdx.x % kWave);
}
// Both halves in one workgroup, Lanes lanes for each of at most 1024 / Lanes
// sequences: saves the second launch.  One workgroup makes all the atomics of
// the counts, so with a wavefront for a sequence (up to 16) it is ahead up to
// 1024 pages each, by max_pages, which is what the host knows (16 sequences of 16
// pages 3.8 us against 5.9 of the two kernels, of 1024 pages 18.4 against 17.5,
// of 4096 66 against 58), with 16 lanes only where the tables are short (all
// forked from one: 64 sequences of 4 pages 4.0 against 6.4, 32 of 16 4.8 against
// 6.0, 64 of 16 7.0 against 6.4, 64 of 64 20.7 against 6.8, 64 of 1024 210
// against 21).
template <int Lanes>
__global__ __launch_bounds__(1024) void fork_small_kernel(KvCache c, const int32_t* __restrict__ src) {
  const int s = threadIdx.x / Lanes, lane = threadIdx.x % Lanes;
  if (s < c.seqs) fork_stage<Lanes>(c, src, s, lane);
  __threadfence_block();
  __syncthreads();
  if (s < c.seqs) fork_apply<Lanes>(c, s, lane);
}

constexpr int kPlan = 1024;  // threads of the one workgroup that hands out pages

// The value of a lane before this one (DPP control), 0 where there is none.
template <int Control, int Rows>
__device__ inline int from_lane(int x) {
  return __builtin_amdgcn_update_dpp(0, x, Control, Rows, 0xf, false);
}
// Sum of v over the lanes up to this one.
__device__ inline int wave_sum_to(int v) {
  v += from_lane<0x111, 0xf>(v);  // 1, 2, 4 and 8 lanes down in rows of 16
  v += from_lane<0x112, 0xf>(v);
  v += from_lane<0x114, 0xf>(v);
  v += from_lane<0x118, 0xf>(v);
  v += from_lane<0x142, 0xa>(v);  // row 0 to row 1, row 2 to row 3
  return v + from_lane<0x143, 0xc>(v);  // lane 31 to rows 2 and 3
}

// Sum of v over the threads before this one, and over all of them.  Every
// thread of the workgroup calls it, with another `buffer` than the call before.
__device__ inline int block_before(int v, int* total, int buffer) {
  __shared__ int wave_total[2][kPlan / kWave];
  const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
  const int incl = wave_sum_to(v);
  if (lane == kWave - 1) wave_total[buffer][w] = incl;
  __syncthreads();
  const int sums = wave_sum_to(lane < kPlan / kWave ? wave_total[buffer][lane] : 0);
  const int before = w ? __builtin_amdgcn_readlane(sums, w - 1) : 0;
  *total = __builtin_amdgcn_readlane(sums, kPlan / kWave - 1);
  return before + incl - v;
}

// 16-byte words that a thread has in flight.
constexpr int kFlight = 8;

// The committed rows of a page that reserve replaced by a copy: one piece, the
// keys or values of a head in a layer (contiguous), by `threads` threads.
__device__ inline void copy_piece(const KvCache& c, const CopyRec& r, int piece, int elem_bytes, int tid, int threads) {
  const int parts = 2 * c.kv_heads, words = c.page_tokens * c.head_dim * elem_bytes / 16;
  const int64_t page0 = int64_t(piece / parts) * c.pages;
  const u32x4* __restrict__ from = static_cast<const u32x4*>(c.kv) + ((page0 + r.from) * parts + piece % parts) * words;
  u32x4* __restrict__ to = static_cast<u32x4*>(c.kv) + ((page0 + r.to) * parts + piece % parts) * words;
  const int n = r.rows * c.head_dim * elem_bytes / 16;
  for (int base = tid; base < n; base += threads * (kFlight / 2)) {
    u32x4 v[kFlight / 2];
#pragma unroll
    for (int u = 0; u < kFlight / 2; ++u)
      if (base + u * threads < n) v[u] = from[base + u * threads];
#pragma unroll
    for (int u = 0; u < kFlight / 2; ++u)
      if (base + u * threads < n) to[base + u * threads] = v[u];
  }
}

// Reserve: demands of all sequences, their prefix sums, the lowest free pages,
// and who gets which.  The order is fixed (sequences ascending, pages
// ascending), so the tables do not depend on timing.  pieces: where the copies
// are few, this workgroup makes them too (the pieces of a page; 0: it does not).
// A chain of reads and of sums over the workgroup: 8 sequences with the copies of
// 24 pieces of 4 KB 7.0 us (sums through LDS exchanges: 1.4 more), 256 without
// copies 7.4.  The search for free pages reads the
// counts from the pool's start on, 4096 a turn, until it has enough: where the
// only free ones are at its end, a pool of 10^5 pages takes 28 us more, of 10^6
// 300.
__global__ __launch_bounds__(kPlan) void reserve_plan_kernel(KvCache c, const int32_t* __restrict__ n_new, int elem_bytes,
                                                             int pieces) {
  // of want: the last page is copied; pages are asked for (pages of a sequence
  // stay below 2^28).  begin cannot say the latter: it ends at pages + 1, and
  // all sequences past that point begin and end there.
  constexpr int kSplit = 1 << 30, kMore = 1 << 29;
  __shared__ int begin[4096 + 1];  // first page of the sequence's share of the free list
  __shared__ int want[4096];       // pages it holds afterwards; -1: left as it is
  const int tid = threadIdx.x;
  CopyRec* recs = copy_recs(c);
  int64_t need = 0;
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
            w |= kSplit;
            ++more;
          }
        }
        if (more) w |= kMore;
      }
    }
    // a demand above the whole pool never fits: cut there, up to 1024 of them
    // are summed in two 16-bit halves where they could pass 2^31 together
    more = min(more, c.pages + 1);
    int total_lo, total_hi = 0, before_lo, before_hi = 0;
    if (c.pages < 1 << 20) {
      before_lo = block_before(more, &total_lo, 0);
    } else {
      before_lo = block_before(more & 0xffff, &total_lo, 0), before_hi = block_before(more >> 16, &total_hi, 1);
    }
    __syncthreads();
    const int64_t at = need + (int64_t(before_hi) << 16) + before_lo;
    if (s < c.seqs) {
      begin[s] = static_cast<int>(min(at, int64_t(c.pages) + 1));
      want[s] = w;
      recs[s] = rec;
    }
    need += (int64_t(total_hi) << 16) + total_lo;
  }
  if (tid == 0) begin[c.seqs] = static_cast<int>(min(need, int64_t(c.pages) + 1));
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
    int rank = found + block_before(n, &total, base / (4 * kPlan) & 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (is_free[i]) {
        if (rank < most) list[rank] = p0 + i;
        ++rank;
      }
    found += total;
  }
  found = min(found, most);
  __threadfence_block();
  __syncthreads();
  // every page to its sequence: the last one that begins at or before it (a
  // demand that does not fit ends past the pages found)
  for (int k = tid; k < found; k += kPlan) {
    int s = 0;
    for (int step = 2048; step > 0; step /= 2)
      if (s + step < c.seqs && begin[s + step] <= k) s += step;
    const int i = k - begin[s], split = want[s] >= kSplit;
    if (begin[s + 1] > found) continue;
    const int32_t p = list[k];
    int32_t* row = c.table + int64_t(s) * c.max_pages;
    c.refs[p] = 1;
    if (split && i == 0) {
      const int32_t old = recs[s].from;
      recs[s].to = p;
      row[c.length[s] >> c.page_shift] = p;
      atomicSub(&c.refs[old], 1);
    } else {
      row[min(c.held[s], c.max_pages) + i - split] = p;
    }
  }
  __threadfence_block();
  __syncthreads();
  for (int s = tid; s < c.seqs; s += kPlan) {
    if (want[s] < 0) continue;
    if (want[s] & kMore && begin[s + 1] > found) c.status[s] = TMS_ERR_OOM;
    else c.held[s] = want[s] & (kMore - 1);
  }
  if (pieces) {
    __threadfence_block();
    __syncthreads();
    for (int i = tid / kWave; i < c.seqs * pieces; i += kPlan / kWave) {
      const CopyRec r = recs[i / pieces];
      if (r.to >= 0) copy_piece(c, r, i % pieces, elem_bytes, tid % kWave, kWave);
    }
  }
}

// 256 sequences, 8 layers of 8 heads: 176 MB written in 38 to 42 us, 4.2 to 4.6
// TB/s (the shared pages are read from the cache).
__global__ __launch_bounds__(256) void copy_pages_kernel(KvCache c, int elem_bytes) {
  const int parts = 2 * c.kv_heads;
  const CopyRec r = copy_recs(c)[blockIdx.x / parts];
  if (r.to >= 0) copy_piece(c, r, blockIdx.y * parts + blockIdx.x % parts, elem_bytes, threadIdx.x, 256);
}

// Whether entry i of a sequence's keep list is out of order or past the rows
// it has reserved.
__device__ inline bool keep_bad(const KvCache& c, int s, const int32_t* keep, int i) {
  const int k = keep[i], prev = i ? keep[i - 1] : -1;
  return k <= prev || int64_t(c.length[s]) + k >= int64_t(min(c.held[s], c.max_pages)) << c.page_shift;
}

// Accepted rows of sequence s moved together, in place, in `pieces` of its
// (layer, keys or values of a head) pieces from p0 on, by one workgroup.  An
// ascending list never moves a row upwards, so the rows of a chunk may be
// written once all of them have been read: later chunks read only rows at or
// past their own targets.
constexpr int kRows = 256 * kFlight / 8;  // of a chunk at most: a row has at least 8 words
static_assert(kRows <= 256, "a thread for each row of a chunk");

__device__ inline void move_rows(const KvCache& c, const int32_t* n_keep, const int32_t* keep_all, int keep_stride,
                                 int elem_bytes, int s, int p0, int pieces) {
  __shared__ int32_t from_page[kRows], from_slot[kRows], to_page[kRows], to_slot[kRows];
  __shared__ int count;
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
  const int parts = 2 * c.kv_heads, p1 = min(p0 + pieces, c.layers * parts);
  const int words = c.head_dim * elem_bytes / 16, shift = __builtin_ctz(words), len = c.length[s];  // words: 8 .. 64
  const int32_t* row = c.table + int64_t(s) * c.max_pages;
  u32x4* kv = static_cast<u32x4*>(c.kv);
  auto place = [&](int piece, int page, int slot, int w) {
    return (((int64_t(piece / parts) * c.pages + page) * parts + piece % parts) * c.page_tokens + slot) * words + w;
  };
  const int most = (256 * kFlight) >> shift;  // a chunk of one piece is in flight at once
  for (int j0 = 0; j0 < n; j0 += most) {
    // the chunk's rows that move, packed in their order
    __syncthreads();
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    const int in = min(most, n - j0);
    const bool mine = static_cast<int>(threadIdx.x) < in;
    const int j = j0 + threadIdx.x, k = mine ? keep[j] : 0;
    int32_t fp = -1, tp = -1;
    if (mine && k != j) {
      fp = row[(len + k) >> c.page_shift], tp = row[(len + j) >> c.page_shift];
      if (!page_ok(c, fp) || !page_ok(c, tp)) fp = -1;
    }
    if (fp >= 0) {
      const int at = atomicAdd(&count, 1);  // any order: a chunk is read whole before it is written
      from_page[at] = fp, to_page[at] = tp;
      from_slot[at] = (len + k) & (c.page_tokens - 1), to_slot[at] = (len + j) & (c.page_tokens - 1);
    }
    __syncthreads();
    const int rows = count;
    if (rows == 0) continue;
    const int per = rows << shift, group = max(1, 256 * kFlight / per);  // words of a piece, pieces in flight
    for (int p = p0; p < p1; p += group) {
      const int total = min(group, p1 - p) * per;  // at most 256 * kFlight
      u32x4 v[kFlight];
      int64_t to[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int i = u * 256 + threadIdx.x;
        to[u] = -1;
        if (i < total) {
          const int piece = p + i / per, at = i % per >> shift, w = i & (words - 1);
          v[u] = kv[place(piece, from_page[at], from_slot[at], w)];
          to[u] = place(piece, to_page[at], to_slot[at], w);
        }
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // every row in flight is in registers
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        if (to[u] >= 0) kv[to[u]] = v[u];
    }
  }
}

// Length of sequence s after a commit, and the pages past it given back, by one
// wavefront.
__device__ inline void commit_sequence(const KvCache& c, const int32_t* n_keep, const int32_t* keep_all, int keep_stride,
                                       int s, int lane) {
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

__global__ __launch_bounds__(256) void commit_kernel(KvCache c, const int32_t* __restrict__ n_keep,
                                                     const int32_t* __restrict__ keep_all, int keep_stride) {
  const int s = blockIdx.x * (256 / kWave) + threadIdx.x / kWave;
  if (s < c.seqs) commit_sequence(c, n_keep, keep_all, keep_stride, s, threadIdx.x % kWave);
}

// 256 sequences, 8 layers: 48 MB read and written in 38 us, 2.5 TB/s: reads and
// writes of a chunk wait for each other, rows of 256 bytes lie apart.
__global__ __launch_bounds__(256) void move_rows_kernel(KvCache c, const int32_t* __restrict__ n_keep,
                                                        const int32_t* __restrict__ keep, int keep_stride, int elem_bytes,
                                                        int pieces) {
  move_rows(c, n_keep, keep, keep_stride, elem_bytes, blockIdx.x, blockIdx.y * pieces, pieces);
}
// Where one workgroup moves all pieces of a sequence it does the rest too (8
// sequences, one layer of 2 heads: 5.5 us).
__global__ __launch_bounds__(256) void move_commit_kernel(KvCache c, const int32_t* __restrict__ n_keep,
                                                          const int32_t* __restrict__ keep, int keep_stride,
                                                          int elem_bytes) {
  move_rows(c, n_keep, keep, keep_stride, elem_bytes, blockIdx.x, 0, c.layers * 2 * c.kv_heads);
  __syncthreads();
  if (threadIdx.x < kWave) commit_sequence(c, n_keep, keep, keep_stride, blockIdx.x, threadIdx.x);
}

int waves_grid(int seqs) { return (seqs + 3) / 4; }
int elem_bytes(const KvCache& c) { return c.dtype == TMS_F32 ? 4 : 2; }

}  // namespace

int64_t kv_page_work_bytes(const KvCache& c) {
  const int64_t fork = round256(4ll * c.seqs * c.max_pages) + int64_t(sizeof(ForkRec)) * c.seqs;
  const int64_t reserve = round256(4ll * c.pages) + int64_t(sizeof(CopyRec)) * c.seqs;
  return kWorkCounts + round256(fork > reserve ? fork : reserve);
}

hipError_t launch_kv_fork(const KvCache& c, const int32_t* src, hipStream_t s) {
  if (c.seqs <= 16 && c.max_pages <= 1024) {
    fork_small_kernel<64><<<1, 1024, 0, s>>>(c, src);
    return hipGetLastError();
  }
  if (c.seqs <= 64 && int64_t(c.seqs) * c.max_pages <= 512) {
    fork_small_kernel<16><<<1, 1024, 0, s>>>(c, src);
    return hipGetLastError();
  }
  fork_stage_kernel<<<waves_grid(c.seqs), 256, 0, s>>>(c, src);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  fork_apply_kernel<<<waves_grid(c.seqs), 256, 0, s>>>(c);
  return hipGetLastError();
}

hipError_t launch_kv_reserve(const KvCache& c, const int32_t* n_new, hipStream_t s) {
  // Up to 64 pieces to copy (four for each wavefront of the plan's workgroup) of
  // up to 128 KB in all: beyond, one workgroup copies longer than a launch takes
  // (64 pieces of 2 KB 6.4 to 7.1 us against 6.5 to 7.0, of 4 KB 8.4 against 6.7;
  // 4 of 16 KB 4.2 against 6.6, of 64 KB 7.9 against 6.7; 64 of 1 MB 1100
  // against 40).
  const int64_t pieces = int64_t(c.layers) * 2 * c.kv_heads;
  const int64_t bytes = c.seqs * pieces * c.page_tokens * c.head_dim * elem_bytes(c);
  const bool here = c.seqs * pieces <= 64 && bytes <= 128 * 1024;
  reserve_plan_kernel<<<1, kPlan, 0, s>>>(c, n_new, elem_bytes(c), here ? static_cast<int>(pieces) : 0);
  if (hipError_t e = hipGetLastError(); e != hipSuccess || here) return e;
  copy_pages_kernel<<<dim3(c.seqs * 2 * c.kv_heads, c.layers), 256, 0, s>>>(c, elem_bytes(c));
  return hipGetLastError();
}

hipError_t launch_kv_commit(const KvCache& c, const int32_t* n_keep, const int32_t* keep, int32_t keep_stride,
                            hipStream_t s) {
  if (keep) {
    // About 2048 workgroups in all; one for a sequence where it has few pieces and
    // up to 128 KB to move, which saves a launch (up to 64 sequences, 64 KB each:
    // 4.9 to 5.2 us against 7.1 to 7.8; 128 KB 6.3 against 7.8; 256 KB 13.5 to 17
    // against 7.5; 1 MB 70 against 7).
    const int64_t pieces = int64_t(c.layers) * 2 * c.kv_heads, wgs = std::max<int64_t>(1, 2048 / c.seqs);
    const int64_t bytes = pieces * keep_stride * c.head_dim * elem_bytes(c);
    if ((pieces <= 16 && bytes <= 128 * 1024) || wgs == 1) {
      move_commit_kernel<<<c.seqs, 256, 0, s>>>(c, n_keep, keep, keep_stride, elem_bytes(c));
      return hipGetLastError();
    }
    const int each = static_cast<int>(std::max((pieces + wgs - 1) / wgs, (pieces + 65534) / 65535));
    move_rows_kernel<<<dim3(c.seqs, (pieces + each - 1) / each), 256, 0, s>>>(c, n_keep, keep, keep_stride,
                                                                             elem_bytes(c), each);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  commit_kernel<<<waves_grid(c.seqs), 256, 0, s>>>(c, n_keep, keep, keep_stride);
  return hipGetLastError();
}

}  // namespace tms
