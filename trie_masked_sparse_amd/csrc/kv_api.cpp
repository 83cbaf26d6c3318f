// C ABI of the paged key/value cache (declared in include/tms.h): argument
// checks and launches.  The descriptor's memory is the caller's; nothing is
// allocated here.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "handles.h"
#include "kv_cache.h"

namespace {

#define TMS_KV_HIP(call, what)                               \
  do {                                                       \
    hipError_t e_ = (call);                                  \
    if (e_ != hipSuccess) return tms::api_hip_fail(e_, what); \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

tms_status bad(const char* msg) { return tms::api_fail(TMS_ERR_INVALID_ARG, msg); }

tms_status check_sizes(const tms_kv* c) {
  if (!c) return bad("null cache");
  if (c->dtype != TMS_F32 && c->dtype != TMS_BF16) return bad("dtype must be fp32 or bf16");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return bad("head_dim must be 64, 128 or 256");
  if (c->page_tokens < 8 || c->page_tokens > 1024 || (c->page_tokens & (c->page_tokens - 1)))
    return bad("page_tokens must be a power of two in [8, 1024]");
  if (c->seqs < 1 || c->seqs > 4096) return bad("seqs must be in [1, 4096]");
  if (c->kv_heads < 1 || c->kv_heads > 256) return bad("kv_heads must be in [1, 256]");
  if (c->layers < 1 || c->layers > 65535 || c->pages < 1 || c->max_pages < 1)
    return bad("layers must be in [1, 65535], pages and max_pages positive");
  if (int64_t(c->max_pages) * c->page_tokens >= (int64_t(1) << 31)) return bad("max_pages * page_tokens must be below 2^31");
  return TMS_OK;
}

tms::KvCache view(const tms_kv* c) {
  return tms::KvCache{c->kv,     c->table,    c->length,      c->held,
                      c->refs,   c->status,   c->work,        c->dtype,
                      c->layers, c->pages,    c->kv_heads,    c->page_tokens,
                      __builtin_ctz(unsigned(c->page_tokens)), c->head_dim, c->seqs, c->max_pages};
}

int64_t work_bytes(const tms::KvCache& v) {
  return std::max({tms::kv_page_work_bytes(v), tms::kv_attention_work_bytes(v), tms::kv_chosen_work_bytes(v)});
}

tms_status check_cache(const tms_kv* c) {
  if (const tms_status s = check_sizes(c); s != TMS_OK) return s;
  if (!c->kv || !c->table || !c->length || !c->held || !c->refs || !c->status || !c->work)
    return bad("null pointer in the cache");
  if (!aligned(c->kv, 16) || !aligned(c->work, 256)) return bad("kv not 16-byte or work not 256-byte aligned");
  if (c->work_bytes < work_bytes(view(c))) return bad("work_bytes below tms_kv_work_bytes");
  return TMS_OK;
}

#define TMS_KV_CHECK(c)                                            \
  do {                                                             \
    if (const tms_status s_ = check_cache(c); s_ != TMS_OK) return s_; \
  } while (0)

int elem_size(const tms_kv* c) { return c->dtype == TMS_F32 ? 4 : 2; }

// Packed rows [T][heads][D], ld elements apart.
bool rows_ok(const tms_kv* c, const void* p, int64_t ld, int32_t heads) {
  return p && aligned(p, 16) && ld >= int64_t(heads) * c->head_dim && ld * elem_size(c) % 16 == 0;
}

// What the attention calls have alike.
tms_status check_attention(const tms_kv* c, int32_t layer, const void* q, int64_t ldq, int32_t q_heads,
                           const int32_t* start, int32_t T, int32_t* max_new, const int32_t* parent, const void* out) {
  if (layer < 0 || layer >= c->layers) return bad("layer out of range");
  if (T < 0 || !start) return bad("null start or negative T");
  if (q_heads < 1 || q_heads > 4096 || q_heads % c->kv_heads) return bad("q_heads must be a multiple of kv_heads, at most 4096");
  if (T == 0) return TMS_OK;
  if (*max_new < 1) return bad("max_new must be positive");
  if (*max_new > T) *max_new = T;
  if (parent && *max_new > 1024) return bad("a tree of drafts has at most 1024 tokens (max_new)");
  if (!rows_ok(c, q, ldq, q_heads) || !out || !aligned(out, 16))
    return bad("q or out null or not aligned, or the row stride of q too small or not a multiple of 16 bytes");
  return TMS_OK;
}

tms_status check_share(const tms_kv* c, int32_t T, int32_t q_heads) {
  if (const tms_status s = check_sizes(c); s != TMS_OK) return s;
  if (T < 1 || T > (1 << 24)) return bad("T must be in [1, 2^24]");
  if (q_heads < 1 || q_heads > 4096 || q_heads % c->kv_heads) return bad("q_heads must be a multiple of kv_heads, at most 4096");
  return TMS_OK;
}

tms_status check_plan(const tms_kv* c, int32_t T, int32_t q_heads, const void* plan, int64_t bytes) {
  if (const tms_status s = check_share(c, T, q_heads); s != TMS_OK) return s;
  if (!plan || !aligned(plan, 256)) return bad("plan null or not 256-byte aligned");
  if (bytes < tms::kv_share_bytes(view(c), T, q_heads)) return bad("plan_bytes below tms_kv_share_bytes");
  return TMS_OK;
}

}  // namespace

extern "C" {

tms_status tms_kv_work_bytes(const tms_kv* c, int64_t* bytes) {
  if (const tms_status s = check_sizes(c); s != TMS_OK) return s;
  if (!bytes) return bad("bytes is null");
  *bytes = work_bytes(view(c));
  return TMS_OK;
}

tms_status tms_kv_fork(const tms_kv* c, const int32_t* src, void* stream) {
  TMS_KV_CHECK(c);
  if (!src) return bad("null src");
  TMS_KV_HIP(tms::launch_kv_fork(view(c), src, static_cast<hipStream_t>(stream)), "kv fork launch");
  return TMS_OK;
}

tms_status tms_kv_reserve(const tms_kv* c, const int32_t* n_new, void* stream) {
  TMS_KV_CHECK(c);
  if (!n_new) return bad("null n_new");
  TMS_KV_HIP(tms::launch_kv_reserve(view(c), n_new, static_cast<hipStream_t>(stream)), "kv reserve launch");
  return TMS_OK;
}

tms_status tms_kv_commit(const tms_kv* c, const int32_t* n_keep, const int32_t* keep, int32_t keep_stride,
                         void* stream) {
  TMS_KV_CHECK(c);
  if (!n_keep) return bad("null n_keep");
  if (keep && keep_stride < 1) return bad("keep_stride must be positive");
  TMS_KV_HIP(tms::launch_kv_commit(view(c), n_keep, keep, keep_stride, static_cast<hipStream_t>(stream)),
             "kv commit launch");
  return TMS_OK;
}

tms_status tms_kv_write(const tms_kv* c, int32_t layer, const int32_t* start, int32_t T, const void* q, int64_t ldq,
                        int32_t q_heads, void* q_out, const void* k, int64_t ldk, const void* v, int64_t ldv,
                        const void* q_weight, const void* k_weight, float eps, const int32_t* pos,
                        const float* inv_freq, int32_t n_freq, int32_t interleaved, void* stream) {
  TMS_KV_CHECK(c);
  if (layer < 0 || layer >= c->layers) return bad("layer out of range");
  if (T < 0 || !start) return bad("null start or negative T");
  if (n_freq < 0 || n_freq % 8 || 2 * n_freq > c->head_dim) return bad("n_freq must be a multiple of 8, at most D/2");
  if (n_freq && (!pos || !inv_freq)) return bad("rotation needs pos and inv_freq");
  if (T == 0) return TMS_OK;
  if (q && (q_heads < 1 || q_heads > 4096)) return bad("q_heads must be in [1, 4096]");
  if (q && (!rows_ok(c, q, ldq, q_heads) || !q_out || !aligned(q_out, 16)))
    return bad("q or q_out null or not aligned, or the row stride of q too small or not a multiple of 16 bytes");
  if (!rows_ok(c, k, ldk, c->kv_heads) || !rows_ok(c, v, ldv, c->kv_heads))
    return bad("k or v null or not aligned, or a row stride too small or not a multiple of 16 bytes");
  if ((q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16)))
    return bad("norm weights not 16-byte aligned");
  tms::KvWrite w{start, T, layer, q, k, v, ldq, ldk, ldv, q ? q_heads : 0, q_out, q_weight, k_weight, eps, pos,
                 inv_freq, n_freq, interleaved ? 1 : 0};
  TMS_KV_HIP(tms::launch_kv_write(view(c), w, static_cast<hipStream_t>(stream)), "kv write launch");
  return TMS_OK;
}

tms_status tms_kv_attention(const tms_kv* c, int32_t layer, const void* q, int64_t ldq, int32_t q_heads,
                            const int32_t* start, int32_t T, int32_t max_new, const int32_t* parent, float scale,
                            void* out, void* stream) {
  TMS_KV_CHECK(c);
  if (const tms_status s = check_attention(c, layer, q, ldq, q_heads, start, T, &max_new, parent, out); s != TMS_OK || T == 0)
    return s;
  tms::KvAttention a{start, T, layer, max_new, q, ldq, q_heads, parent, scale, out};
  TMS_KV_HIP(tms::launch_kv_attention(view(c), a, static_cast<hipStream_t>(stream)), "kv attention launch");
  return TMS_OK;
}

tms_status tms_kv_share_bytes(const tms_kv* c, int32_t T, int32_t q_heads, int64_t* bytes) {
  if (const tms_status s = check_share(c, T, q_heads); s != TMS_OK) return s;
  if (!bytes) return bad("bytes is null");
  *bytes = tms::kv_share_bytes(view(c), T, q_heads);
  return TMS_OK;
}

tms_status tms_kv_share(const tms_kv* c, const int32_t* start, int32_t T, int32_t q_heads, void* plan,
                        int64_t plan_bytes, void* stream) {
  TMS_KV_CHECK(c);
  if (!start) return bad("null start");
  if (const tms_status s = check_plan(c, T, q_heads, plan, plan_bytes); s != TMS_OK) return s;
  tms::KvShared a{{start, T, 0, T, nullptr, 0, q_heads, nullptr, 1.f, nullptr}, plan};
  TMS_KV_HIP(tms::launch_kv_share(view(c), a, static_cast<hipStream_t>(stream)), "kv share launch");
  return TMS_OK;
}

tms_status tms_kv_attention_shared(const tms_kv* c, int32_t layer, const void* q, int64_t ldq, int32_t q_heads,
                                   const int32_t* start, int32_t T, int32_t max_new, const int32_t* parent, float scale,
                                   void* out, void* plan, int64_t plan_bytes, void* stream) {
  TMS_KV_CHECK(c);
  if (const tms_status s = check_attention(c, layer, q, ldq, q_heads, start, T, &max_new, parent, out); s != TMS_OK || T == 0)
    return s;
  if (const tms_status s = check_plan(c, T, q_heads, plan, plan_bytes); s != TMS_OK) return s;
  tms::KvShared a{{start, T, layer, max_new, q, ldq, q_heads, parent, scale, out}, plan};
  TMS_KV_HIP(tms::launch_kv_attention_shared(view(c), a, static_cast<hipStream_t>(stream)), "kv shared attention launch");
  return TMS_OK;
}

tms_status tms_kv_bounds(const tms_kv* c, const int32_t* n_new, int32_t max_new, void* bounds, void* stream) {
  TMS_KV_CHECK(c);
  if (!bounds || !aligned(bounds, 16)) return bad("bounds null or not 16-byte aligned");
  if (max_new < 0) return bad("negative max_new");
  tms::KvBounds b{n_new, max_new, bounds};
  TMS_KV_HIP(tms::launch_kv_bounds(view(c), b, static_cast<hipStream_t>(stream)), "kv bounds launch");
  return TMS_OK;
}

tms_status tms_kv_select_bytes(const tms_kv* c, int32_t T, int64_t* bytes) {
  if (const tms_status s = check_sizes(c); s != TMS_OK) return s;
  if (T < 0 || !bytes) return bad("negative T or null bytes");
  *bytes = tms::kv_select_work_bytes(view(c), T);
  return TMS_OK;
}

tms_status tms_kv_select(const tms_kv* c, int32_t layer, const void* q, int64_t ldq, int32_t q_heads,
                         const int32_t* start, int32_t T, int32_t max_new, float scale, const void* bounds, int32_t k,
                         int32_t first, int32_t last, int32_t* chosen, void* work, int64_t work_bytes, void* stream) {
  TMS_KV_CHECK(c);
  if (k < 1 || k > tms::kMostChosen) return bad("k must be in [1, 8192]");
  if (first < 0 || last < 0) return bad("first and last must not be negative");
  // chosen stands for the outputs, which are whole numbers: no alignment
  if (const tms_status s = check_attention(c, layer, q, ldq, q_heads, start, T, &max_new, nullptr, q); s != TMS_OK || T == 0)
    return s;
  if (!chosen || !bounds || !aligned(bounds, 16)) return bad("chosen or bounds null or bounds not 16-byte aligned");
  if (!work || !aligned(work, 256) || work_bytes < tms::kv_select_work_bytes(view(c), T))
    return bad("work null, not 256-byte aligned or below tms_kv_select_bytes");
  tms::KvSelect a{{start, T, layer, max_new, q, ldq, q_heads, nullptr, scale, nullptr}, bounds, k, first, last, chosen, work};
  TMS_KV_HIP(tms::launch_kv_select(view(c), a, static_cast<hipStream_t>(stream)), "kv select launch");
  return TMS_OK;
}

tms_status tms_kv_attention_pages(const tms_kv* c, int32_t layer, const void* q, int64_t ldq, int32_t q_heads,
                                  const int32_t* start, int32_t T, int32_t max_new, const int32_t* parent,
                                  const int32_t* chosen, int32_t k, float scale, void* out, void* stream) {
  TMS_KV_CHECK(c);
  if (k < 0 || k > tms::kMostChosen) return bad("k must be in [0, 8192]");
  if (const tms_status s = check_attention(c, layer, q, ldq, q_heads, start, T, &max_new, parent, out); s != TMS_OK || T == 0)
    return s;
  if (k && !chosen) return bad("null chosen");
  tms::KvChosen a{{start, T, layer, max_new, q, ldq, q_heads, parent, scale, out}, chosen, k};
  TMS_KV_HIP(tms::launch_kv_attention_pages(view(c), a, static_cast<hipStream_t>(stream)), "kv attention over pages launch");
  return TMS_OK;
}

tms_status tms_kv_sync_status(const tms_kv* c, int32_t* host_status, void* stream) {
  TMS_KV_CHECK(c);
  int32_t buf[4096];  // seqs is at most 4096
  TMS_KV_HIP(hipMemcpyAsync(buf, c->status, sizeof(int32_t) * size_t(c->seqs), hipMemcpyDeviceToHost,
                            static_cast<hipStream_t>(stream)), "kv status copy");
  TMS_KV_HIP(hipStreamSynchronize(static_cast<hipStream_t>(stream)), "kv status synchronise");
  tms_status first = TMS_OK;
  for (int32_t s = 0; s < c->seqs; ++s) {
    if (host_status) host_status[s] = buf[s];
    if (first == TMS_OK && buf[s] != TMS_OK) {
      first = static_cast<tms_status>(buf[s]);
      tms::api_fail(first, "sequence " + std::to_string(s) + ": " + tms_status_str(first));
    }
  }
  return first;
}

}  // extern "C"
