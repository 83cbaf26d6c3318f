// Attention of new tokens (one, a tree of drafts, a whole prompt) over the
// paged key/value cache, for gfx950.
#include <hip/hip_runtime.h>

#include "kv_cache.h"
#include "tms.h"

namespace tms {
namespace {

constexpr int kWave = 64;

template <int DT>
__device__ inline float load1(const void* p, int64_t i) {
  if constexpr (DT == 0) return static_cast<const float*>(p)[i];
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}
template <int DT>
__device__ inline void store1(void* p, int64_t i, float x) {
  if constexpr (DT == 0) static_cast<float*>(p)[i] = x;
  else static_cast<__bf16*>(p)[i] = static_cast<__bf16>(x);
}

// One wavefront for a token and a query head: a lane takes a key of 64, then
// the weights are broadcast and a lane takes D/64 values of the output.
template <int DT, int D>
__global__ __launch_bounds__(64) void attention_kernel(KvCache c, KvAttention a) {
  constexpr int E = D / kWave;
  __shared__ float q[D];
  __shared__ uint32_t seen[32];
  const int lane = threadIdx.x, t = blockIdx.x, h = blockIdx.y, kh = h / (a.q_heads / c.kv_heads);
  int s = 0;
  for (int base = 0; base < c.seqs; base += kWave) {
    const int i = base + lane + 1;
    s += __popcll(__ballot(i <= c.seqs && a.start[min(i, c.seqs)] <= t));
  }
  const int64_t out = (int64_t(t) * a.q_heads + h) * D;
  int begin = 0, n = -1, len = 0;
  if (s < c.seqs && c.status[s] == TMS_OK) {
    begin = a.start[s], len = c.length[s], n = a.start[s + 1] - begin;
    if (begin < 0 || t < begin || a.start[s + 1] > a.T || n > a.max_new ||
        int64_t(len) + n > int64_t(min(c.held[s], c.max_pages)) << c.page_shift)
      n = -1;
  }
  if (n < 0) {
    for (int e = 0; e < E; ++e) store1<DT>(a.out, out + lane + e * kWave, NAN);
    return;
  }
  const int i = t - begin;
  for (int e = lane; e < D; e += kWave) q[e] = load1<DT>(a.q, int64_t(t) * a.ldq + h * D + e) * a.scale;
  if (a.parent) {
    if (lane < 32) seen[lane] = 0;
    __syncthreads();
    if (lane == 0)
      for (int j = i; j >= 0;) {
        seen[j >> 5] |= 1u << (j & 31);
        const int p = a.parent[begin + j];
        j = p < j ? p : -1;
      }
  }
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[E] = {};
  const int keys = len + (a.parent ? n : i + 1);
  for (int base = 0; base < keys; base += kWave) {
    const int r = base + lane;
    float x = -INFINITY;
    int64_t row = 0;
    if (r < keys) {
      const int32_t p = c.table[int64_t(s) * c.max_pages + (r >> c.page_shift)];
      row = (((int64_t(a.layer) * c.pages + p) * 2 * c.kv_heads + kh) * c.page_tokens + (r & (c.page_tokens - 1))) * D;
      const int j = r - len;
      if (j < 0 || !a.parent || (seen[j >> 5] >> (j & 31) & 1)) {
        x = 0.f;
        for (int e = 0; e < D; ++e) x = fmaf(q[e], load1<DT>(c.kv, row + e), x);
      }
    }
    float top = x;
    for (int d = 1; d < kWave; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    const float m2 = fmaxf(m, top);
    const float p = x == -INFINITY ? 0.f : expf(x - m2), turn = m == -INFINITY ? 0.f : expf(m - m2);
    float sum = p;
    for (int d = 1; d < kWave; d *= 2) sum += __shfl_xor(sum, d);
    l = l * turn + sum;
    for (int e = 0; e < E; ++e) o[e] *= turn;
    m = m2;
    for (int j = 0; j < min(kWave, keys - base); ++j) {
      const float w = __shfl(p, j);
      const int64_t v = __shfl(row, j) + int64_t(c.kv_heads) * c.page_tokens * D;
      if (w != 0.f)
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, load1<DT>(c.kv, v + lane + e * kWave), o[e]);
    }
  }
  for (int e = 0; e < E; ++e) store1<DT>(a.out, out + lane + e * kWave, o[e] / l);
}

template <int DT>
hipError_t launch(const KvCache& c, const KvAttention& a, hipStream_t s) {
  const dim3 grid(a.T, a.q_heads);
  if (c.head_dim == 64) attention_kernel<DT, 64><<<grid, kWave, 0, s>>>(c, a);
  else if (c.head_dim == 128) attention_kernel<DT, 128><<<grid, kWave, 0, s>>>(c, a);
  else attention_kernel<DT, 256><<<grid, kWave, 0, s>>>(c, a);
  return hipGetLastError();
}

}  // namespace

int64_t kv_attention_work_bytes(const KvCache&) { return 256; }

hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, hipStream_t s) {
  return c.dtype == TMS_F32 ? launch<0>(c, a, s) : launch<1>(c, a, s);
}

}  // namespace tms
