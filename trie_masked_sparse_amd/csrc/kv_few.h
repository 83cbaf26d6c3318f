// One tile of up to 16 MT query rows of one key head over a run of keys: what a
// workgroup of the attention over chosen pages does, and of the shared attention
// in fp32 or, in bf16, where the rows are few (up to 16; 32 with heads of 64).
#pragma once
#include <type_traits>

#include "kv_tiles.h"

namespace tms {
namespace {

// What the rows of a tile see.  Keys are numbered as the caller likes (a
// sequence's rows from some page on, the rows of a list of pages): q.len of
// them are seen by all rows, then come new rows, which a row sees as its token
// does (sees() in kv_tiles.h).  Rows that see all keys and no new ones have
// token -1, and tok0 = tok1 = -1, a.parent null, limit = q.len.
struct FewTile {
  Seq q;           // begin, n and len, in this numbering
  int h;           // key head
  int tok0, tok1;  // tokens of the tile, among the sequence's new ones
  int kt0, kt1;    // key tiles to work on
  int limit;       // keys that any row sees: none is read from there on
};

// Four wavefronts for Heads key heads from t.h on: each holds all rows of one head
// and takes every Step-th key tile, K straight
// into registers, V through its own part of LDS, the next tile's loads in
// flight during the softmax and the second product; no barrier among them until
// their parts are joined.  Softmax statistics and outputs are fp32; bf16
// weights go into the second product as two bf16 parts (16 bits).
template <int DT, int D, int MT, int Heads = 1>
struct FewRows {
  using T = Tile<DT, D>;
  static constexpr int Step = kWaves / Heads;  // wavefronts of a head
  static constexpr int M = 16 * MT, KW = T::Keys, DB = D / 16, L = T::Loads;
  static constexpr int kVWords = KW * T::Chunks;  // 16-byte words of a V tile
  static constexpr int kLds = kWaves * kVWords > kWaves * M * D / 4 ? kWaves * kVWords : kWaves * M * D / 4;
  struct Lds {
    u32x4 tiles[kLds];
    float stat[kWaves][2][M];
    uint32_t seen[M * kTreeWords];
    int32_t par[kTree];
    uint32_t nonfinite[Heads][kMixedWords];
  };

  // page_at(key): its page, clamped to the pool.  query(r): element of q of row r, in bounds for every r < M;
  // token(r): its token, -1 where there is none.  emit(h, r, column, x, top, l): 4
  // values of a row, not yet divided by the sum l of its weights relative to 2^top.
  // visible(key, r): whether row r sees key .. key + 3 (a multiple of 4), where that
  // is not all that a.parent and the token say; rows then differ in keys that may
  // hold anything, so where an output is not finite nothing is emitted: returns
  // whether it was.
  struct Everything {};
  template <class PageAt, class Query, class Token, class Emit, class Visible = Everything>
  static __device__ inline bool run(const KvCache& c, const KvAttention& a, Lds& lds, const FewTile& t, PageAt page_at,
                                    Query query, Token token, Emit emit, Visible visible = Visible(), bool finite_only = false) {
    constexpr bool kChosen = !std::is_same<Visible, Everything>::value;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int col = lane % 16, g = lane / 16, part = wave % Step, head = wave / Step, h = t.h + head;
    // a scale of 0 clears q instead: a masked score stays -inf
    const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
    const uint32_t flip = a.scale < 0.f ? (DT == 0 ? 0x80000000u : 0x80008000u) : 0u, on = a.scale == 0.f ? 0u : ~0u;
    const Seq& q = t.q;
    const int limit = t.limit, end = min(t.kt1, (limit + KW - 1) / KW);
    const int64_t head_stride = int64_t(c.page_tokens) * T::Chunks;  // 16-byte words
    const u32x4* kv = static_cast<const u32x4*>(c.kv) + (int64_t(a.layer) * c.pages * 2 * c.kv_heads + h) * head_stride;
    const int64_t v_off = c.kv_heads * head_stride, page_stride = 2 * v_off;
    // keys past the last one to be used are read from that one: in bounds, and masked
    auto page_of = [&](int kt, int i) { return page_at(min(kt * KW + i * 16 + col, limit - 1)); };
    u32x4* vt = lds.tiles + wave * kVWords;
    const Mixed mixed = mixed_rows(a, q, t.tok0, t.tok1, lds.nonfinite[head]);
    for (int again = 0;; ++again) {  // a second pass where a value is not finite
      int kt = t.kt0 + part;
      int32_t pg[T::Sub];
      if (kt < end)
#pragma unroll
        for (int i = 0; i < T::Sub; ++i) pg[i] = page_of(kt, i);
      // the queries: B operand, row = lane % 16; asked for before the first keys,
      // used after them
      u32x4 qr[MT][L];
      int tok[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + query(h, m * 16 + col) * (DT == 0 ? 4 : 2));
        tok[m] = token(m * 16 + col);
#pragma unroll
        for (int i = 0; i < L; ++i) qr[m][i] = p[i * 4 + g];
      }
      u32x4 kr[T::Sub][L], vr[T::Sub][L];
      auto load = [&](int kt) {
#pragma unroll
        for (int i = 0; i < T::Sub; ++i) {
          const int r = min(kt * KW + i * 16 + col, limit - 1);
          const u32x4* p = kv + pg[i] * page_stride + int64_t(r & (c.page_tokens - 1)) * T::Chunks + g;
#pragma unroll
          for (int j = 0; j < L; ++j) kr[i][j] = p[j * 4];
#pragma unroll
          for (int j = 0; j < L; ++j) vr[i][j] = p[v_off + j * 4];
        }
      };
      if (kt < end) {
        load(kt);
#pragma unroll
        for (int i = 0; i < T::Sub; ++i) pg[i] = page_of(min(kt + Step, end - 1), i);
      }
      if (a.parent && end * KW > q.len) walk_tree<kBlock>(a, q, t.tok0, t.tok1, lds.par, lds.seen, kTreeWords);
      bool odd = false;
      if (again)
        for (int i = 0; i < Heads; ++i) {
          const Mixed m = mixed_rows(a, q, t.tok0, t.tok1, lds.nonfinite[i]);
          odd |= find_nonfinite<kBlock, DT, D>(c, page_at, kv + v_off + (i - head) * head_stride, page_stride, m);
        }
      f32x4 o[MT][DB];
      float mx[MT], sum[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mx[m] = -INFINITY, sum[m] = 0.f;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < L; ++i) qr[m][i] = (qr[m][i] ^ flip) & on;
      }
      for (; kt < end; kt += Step) {
        // V to LDS, S^T from the registers
#pragma unroll
        for (int i = 0; i < T::Sub; ++i)
#pragma unroll
          for (int j = 0; j < L; ++j) vt[T::at(i * 16 + col, j * 4 + g)] = vr[i][j];
        f32x4 sc[MT][T::Sub];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < T::Sub; ++i) {
            f32x4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < L; ++j) {
              if constexpr (DT == 1) {
                x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kr[i][j]),
                                                            __builtin_bit_cast(bf16x8, qr[m][j]), x, 0, 0, 0);
              } else {
                const f32x4 k4 = __builtin_bit_cast(f32x4, kr[i][j]), q4 = __builtin_bit_cast(f32x4, qr[m][j]);
#pragma unroll
                for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_16x16x4f32(k4[e], q4[e], x, 0, 0, 0);
              }
            }
            sc[m][i] = x;
          }
        if (kt + Step < end) {
          load(kt + Step);
#pragma unroll
          for (int i = 0; i < T::Sub; ++i) pg[i] = page_of(min(kt + 2 * Step, end - 1), i);
        }
        if ((kt + 1) * KW > q.len) {  // new rows among the keys, or none behind them: who sees them
          const int first = kt * KW, at = first & 31;  // key and bit of the tile's first key
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t word = sees(a, q, tok[m], t.tok0, first & ~31, lds.seen, kTreeWords) >> (at + 4 * g);
#pragma unroll
            for (int i = 0; i < T::Sub; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[m][i][e] = word >> (16 * i + e) & 1 ? sc[m][i][e] : -INFINITY;
          }
        }
        if constexpr (kChosen) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < T::Sub; ++i) {
              const bool on = visible(kt * KW + 16 * i + 4 * g, m * 16 + col);
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[m][i][e] = on ? sc[m][i][e] : -INFINITY;
            }
        }
        u32x4 pw[MT], pl[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float top = sc[m][0][0];
#pragma unroll
          for (int i = 0; i < T::Sub; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[m][i][e]);
          top = row_max(top) * scale;
          if (top > mx[m]) {
            const float turn = exp2_fast(mx[m] - top);  // 0 for the first tile
            mx[m] = top;
            sum[m] *= turn;
#pragma unroll
            for (int d = 0; d < DB; ++d) o[m][d] *= turn;
          }
          const float at = mx[m] == -INFINITY ? 0.f : mx[m];
#pragma unroll
          for (int i = 0; i < T::Sub; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sc[m][i][e] = exp2_fast(fmaf(sc[m][i][e], scale, -at));
              sum[m] += sc[m][i][e];
            }
          if constexpr (DT == 1)
            split_bf16({sc[m][0][0], sc[m][0][1], sc[m][0][2], sc[m][0][3], sc[m][1][0], sc[m][1][1], sc[m][1][2], sc[m][1][3]},
                       &pw[m], &pl[m]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (odd) {
          for (uint32_t word = mixed.word(kt * KW & ~31) >> (kt * KW & 31) & T::Mask; word; word &= word - 1) {
            const int r = __builtin_ctz(word);
            for (int i = lane; i < T::Chunks; i += kWave) vt[r * T::Chunks + i] = keep_finite<DT>(vt[r * T::Chunks + i], true);
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          if constexpr (DT == 1) {
            // 4 keys of column 16 d + lane % 16, from both halves
            const int r = 4 * g + col / 4, half = col % 4 / 2;
            const char* p0 = reinterpret_cast<const char*>(vt + T::at(r, 2 * d + half)) + col % 2 * 8;
            const char* p1 = reinterpret_cast<const char*>(vt + T::at(16 + r, 2 * d + half)) + col % 2 * 8;
            const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p0));
            const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p1));
            const bf16x8 va = __builtin_bit_cast(bf16x8, s16x8(__builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7)));
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              o[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, __builtin_bit_cast(bf16x8, pl[m]), o[m][d], 0, 0, 0);
              o[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, __builtin_bit_cast(bf16x8, pw[m]), o[m][d], 0, 0, 0);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v = reinterpret_cast<const float*>(vt + T::at(4 * g + e, 4 * d + col / 4))[col % 4];
#pragma unroll
              for (int m = 0; m < MT; ++m)
                o[m][d] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, sc[m][0][e], o[m][d], 0, 0, 0);
            }
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }

      float z = 0.f;
      if ((kChosen && finite_only) || (!again && end * KW > mixed.first))
#pragma unroll
        for (int m = 0; m < MT; ++m) z = zero_or_nan(o[m], z);
      // every wavefront is done with its tiles
      if (__syncthreads_or(z != z)) {
        if (kChosen && finite_only) return false;
        continue;
      }
      // a head's wavefronts' parts joined; each ends with as many of the
      // columns
      f32x4* buf = reinterpret_cast<f32x4*>(lds.tiles);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        sum[m] = row_sum(sum[m]);
        if (g == 0) lds.stat[wave][0][m * 16 + col] = mx[m], lds.stat[wave][1][m * 16 + col] = sum[m];
#pragma unroll
        for (int d = 0; d < DB; ++d) buf[((wave * MT + m) * DB + d) * kWave + lane] = o[m][d];
      }
      if (odd)  // every wavefront for the tiles that it had
        for (kt = t.kt0 + part; kt < end; kt += Step)
          for (uint32_t word = mixed.word(kt * KW & ~31) >> (kt * KW & 31) & T::Mask; word; word &= word - 1) {
            const int row = kt * KW + __builtin_ctz(word);
            if (row >= limit) break;
            const u32x4* p = value_row(c, page_at, kv + v_off, page_stride, T::Chunks, row);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              if (sees(a, q, tok[m], t.tok0, row & ~31, lds.seen, kTreeWords) >> (row & 31) & 1)
#pragma unroll 1
                for (int d = 0; d < DB; ++d)
                  buf[((wave * MT + m) * DB + d) * kWave + lane] += odd_values<DT>(p, 16 * d + 4 * g);
          }
      __syncthreads();
      constexpr int Q = DB / Step;
      const int first = head * Step;  // wavefront of the head
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r = m * 16 + col;
        float top = -INFINITY, weight[Step], l = 0.f;
#pragma unroll
        for (int w = 0; w < Step; ++w) top = fmaxf(top, lds.stat[first + w][0][r]);
        const float at = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < Step; ++w) {
          weight[w] = part_weight(lds.stat[first + w][0][r] - at);
          l += weight[w] * lds.stat[first + w][1][r];
        }
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          const int d = part * Q + i;
          f32x4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < Step; ++w) x += buf[(((first + w) * MT + m) * DB + d) * kWave + lane] * weight[w];
          emit(h, r, 16 * d + 4 * g, x, top, l);
        }
      }
      return true;
    }
  }
};

// Parts of query rows: the values [rows][D], not yet divided, and of each row
// the maximum's exponent and the sum of the weights relative to it.
struct Parts {
  float* values;
  float2* stats;
};

// One row's 4 values from column `column` on over `count` parts: part i is row
// at(i) of the parts.  A running maximum; kParts of them are in flight.  Shared:
// other workgroups of the launch have written them (part_store in kv_tiles.h).
struct PartSum {
  float top = -INFINITY, l = 0.f;
  f32x4 x{0.f, 0.f, 0.f, 0.f};

  template <int D, int kParts, bool Shared = false, class At>
  __device__ void add(const Parts& p, int count, int column, At at) {
    for (int i = 0; i < count; i += kParts) {
      float2 s[kParts];
      f32x4 y[kParts];
#pragma unroll
      for (int u = 0; u < kParts; ++u) {
        s[u] = float2{-INFINITY, 0.f}, y[u] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (i + u < count) {
          const int64_t row = at(i + u);
          if constexpr (Shared) s[u] = float2{part_load<true>(&p.stats[row].x), part_load<true>(&p.stats[row].y)};
          else s[u] = p.stats[row];
          y[u] = part_load<Shared>(reinterpret_cast<const f32x4*>(p.values + row * D + column));
        }
      }
      float next = top;
#pragma unroll
      for (int u = 0; u < kParts; ++u) next = fmaxf(next, s[u].x);
      const float base = next == -INFINITY ? 0.f : next, old = part_weight(top - base);
      top = next;
      l *= old, x *= old;
#pragma unroll
      for (int u = 0; u < kParts; ++u) {
        const float now = part_weight(s[u].x - base);
        l += s[u].y * now;
        x += y[u] * now;
      }
    }
  }
};

}  // namespace
}  // namespace tms
