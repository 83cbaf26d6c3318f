// One tile of up to 32 RW query rows of one key head over a run of keys, in
// bf16: what a workgroup of the shared attention does where many rows see the
// same keys.
#pragma once
#include "kv_few.h"

namespace tms {
namespace {

// RW x KS wavefronts: each holds 32 rows and takes 1 / KS of the keys of every
// tile of 64; K and V tiles are copied from the cache straight into LDS, one tile
// ahead of the products.  The weights go into the second product as two bf16 parts
// (16 bits), so that what a token gets does not depend on how many others share its
// pages: of 128 rows, one part was quicker (64 answers behind one prompt 103.4 ->
// 105.2 us for plan and two layers, trees of 5 to 31 drafts 138 -> 150, 256 answers
// 238 -> 245), and off by up to 2^-8 of each weight.  Their sum is taken from the
// fp32 weights (by products with ones, of both parts: 106.2, 153, 248).  A tile of 64
// keys took a wavefront 1.8 us, weights of one part, where two workgroups of 128 rows
// share a compute unit: the chain from scores to weights, not the copies (tiles of 32
// keys three ahead took no less).  Heads of 256, 64 answers over 9000 rows: 128 rows
// of a workgroup 44 us, 64 rows 58.
template <int D, int RW, int KS>
struct ManyRows {
  static constexpr int W = RW * KS, M = 32 * RW, CH = D / 8, KK = D / 16, DB = D / 32, Threads = W * kWave;
  static constexpr int KT = 64, TileWords = KT * CH;       // keys of a tile, its 16-byte words
  static constexpr int NB = KT / 32 / KS;                  // 32-key blocks of a tile for each wavefront
  static constexpr int Bufs = 2;
  static constexpr int RPI = kWave / CH, P = KT / RPI / W;  // rows of a copying instruction, instructions of a wavefront
  static constexpr int Ahead = 3;                           // products that the reads of LDS run ahead
  // a sequence's new tokens: its rows fit a tile of 128
  static constexpr int MostNew = 128, Words = MostNew / 32 + 1;
  struct Lds {
    u32x4 tiles[2 * Bufs * TileWords];  // K tiles, then V tiles; the outputs of the second half of the keys at the end
    float stat[KS == 2 ? 2 * M : 1];
    uint32_t seen[M * Words];
    int32_t par[MostNew];
    uint32_t nonfinite[kMixedWords];
  };

  // table: the pages of the keys, the same for all lanes, as all of t; a tree has
  // at most MostNew drafts.  query, token and emit as in FewRows.
  template <class Query, class Token, class Emit>
  static __device__ inline void run(const KvCache& c, const KvAttention& a, Lds& lds, const FewTile& t, const int32_t* table,
                                    Query query, Token token, Emit emit) {
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int rw = wave % RW, ks = wave / RW, col = lane % 32, hi2 = lane / 32;
    const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u, on = a.scale == 0.f ? 0u : ~0u;
    const int tiles_at = static_cast<int>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)lds.tiles));
    // places in LDS: K is read 16 bytes of 16 rows at a time, V 64 bytes of 4, each
    // from 64 different banks (but K of 64-value heads, where pairs of rows meet)
    constexpr int Mask = (CH < 16 ? CH : 16) - 1, VShift = D == 64 ? 1 : 2;
    auto k_at = [](int r, int ch) { return r * CH + (ch ^ (r & Mask)); };
    auto v_at = [](int r, int ch) { return r * CH + (ch ^ (r << VShift & Mask)); };
    const Seq& q = t.q;
    const int limit = t.limit, kt0 = t.kt0, end = max(kt0, min(t.kt1, (limit + KT - 1) / KT));
    const int r = rw * 32 + col, tok = token(r);
    const int64_t head_stride = int64_t(c.page_tokens) * CH;  // 16-byte words
    const u32x4* kv = static_cast<const u32x4*>(c.kv) + (int64_t(a.layer) * c.pages * 2 * c.kv_heads + t.h) * head_stride;
    const int64_t v_off = c.kv_heads * head_stride, page_stride = 2 * v_off;
    const Mixed mixed = mixed_rows(a, q, t.tok0, t.tok1, lds.nonfinite);
    // keys that all rows of the workgroup see
    const int clear = a.parent ? q.len : q.len + t.tok0 + 1;
    for (int again = 0;; ++again) {  // a second pass where a value is not finite
      u32x4 qr[KK];  // asked for here, used after the first copies are
      {
        const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + query(r) * 2);
#pragma unroll
        for (int i = 0; i < KK; ++i) qr[i] = p[2 * i + hi2];
      }
      const f32x16 zero = {};
      f32x16 o[DB], sc[NB];
      float mx = -INFINITY, sum = 0.f;  // sum: of this lane's weights
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
      // Copies from the cache straight into LDS, 1 KB an instruction: rows r0 ..
      // r0 + RPI - 1 of a tile, in one page (a page has at least 8 rows).  LDS
      // fills in the lanes' order, so the lanes take the words in the order that
      // k_at and v_at have them.  Rows past the last one to be used are filled
      // with that one: in bounds, and masked or never used.
      const int final_row = uniform(max(min(limit, end * KT) - 1, 0));
      const int my_row = lane / CH, k_ch = lane % CH ^ ((wave * RPI + my_row) & Mask),
                v_ch = lane % CH ^ ((wave * RPI + my_row) << VShift & Mask);
      // Step x copies K of tile x + 2 and V of tile x + 1; a tile's page numbers
      // are asked for one step before its K, its addresses are kept for its V.
      const const_i32 pages = (const_i32)(table);
      const uint32_t page_words = 2 * c.kv_heads * c.page_tokens * CH;
      int next_page[P], row_at[P];
      int64_t from[P];  // addresses
      auto look = [&](int kt, int i) __attribute__((always_inline)) {
        next_page[i] = pages[uint32_t(min(kt * KT + (i * W + wave) * RPI, final_row)) >> c.page_shift];
      };
      auto find = [&](int kt, int i) __attribute__((always_inline)) {
        const int r0 = kt * KT + (i * W + wave) * RPI, first = min(r0, final_row & ~(RPI - 1));
        const uint32_t page = uniform(max(0, min(next_page[i], c.pages - 1)));
        from[i] = uniform(reinterpret_cast<int64_t>(kv) +
                          (int64_t(uint64_t(page) * page_words) + uint32_t(first & (c.page_tokens - 1)) * CH) * 16);
        row_at[i] = (min(r0 + my_row, final_row) - first) * (CH * 16);
      };
      auto copy = [&](int64_t off, int ch, int step, int to, int i) __attribute__((always_inline)) {
        copy_to_lds(from[i] + off, row_at[i] + (ch ^ (i * W * RPI * step & Mask)) * 16,
                    tiles_at + to * (TileWords * 16) + (i * W + wave) * (kWave * 16));
      };
      // buffers of the V tile and of the K tile of the next step
      int to_v = 0, to_k = 1;
      auto ask = [&](int x, int piece) __attribute__((always_inline)) {
        const int i = piece % P;
        if (piece < P) {
          copy(v_off * 16, v_ch, 1 << VShift, Bufs + to_v, i);
        } else {
          find(x + 2, i);
          copy(0, k_ch, 1, to_k, i);
          look(x + 3, i);
        }
        if (piece == 2 * P - 1) to_v ^= 1, to_k ^= 1;
      };
      // words of LDS that the products read.  V^T: lane (d = lane % 32 of the
      // block, keys 4 hi2 .. +3 of two groups of 8) as the weights have them
      const int vrow = 4 * hi2 + lane % 16 / 4, vch = 2 * (lane % 32 / 16) + lane % 4 / 2, vb = lane % 2 * 8;
      int k_at_lds[KK], v_at_lds[DB];
#pragma unroll
      for (int j = 0; j < KK; ++j) k_at_lds[j] = tiles_at + k_at(ks * NB * 32 + col, 2 * j + hi2) * 16;
#pragma unroll
      for (int d = 0; d < DB; ++d)
        v_at_lds[d] = tiles_at + (Bufs * TileWords + v_at(ks * NB * 32 + vrow, 4 * d + vch)) * 16 + vb;
      auto k_words = [&](int at) __attribute__((always_inline)) { return __builtin_bit_cast(bf16x8, *(lds_u32x4)(at)); };
      auto v_words = [&](int at) __attribute__((always_inline)) {
        const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at));
        const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at + 8 * CH * 16));
        return __builtin_bit_cast(bf16x8, s16x8(__builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7)));
      };
      int odd = 0;
      if (kt0 < end) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          look(kt0, i);
          find(kt0, i);
          copy(0, k_ch, 1, 0, i);
          look(kt0 + 1, i);
        }
#pragma unroll
        for (int i = 0; i < 2 * P; ++i) ask(kt0 - 1, i);
        // the tree is walked while the first copies are on their way
        if (a.parent && end * KT > q.len) walk_tree<Threads>(a, q, t.tok0, t.tok1, lds.par, lds.seen, Words);
        if (again) odd = uniform(find_nonfinite<Threads, 1, D>(c, table, kv + v_off, page_stride, mixed));
#pragma unroll
        for (int i = 0; i < KK; ++i) qr[i] = (qr[i] ^ flip) & on;
        wait_copies<2 * P>();
        lds_barrier();
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < KK; ++j)
            sc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k_words(k_at_lds[j] + i * 32 * CH * 16), __builtin_bit_cast(bf16x8, qr[j]), j ? sc[i] : zero, 0, 0, 0);
        lds_barrier();
      }
      // a tile: softmax, output, the scores of the next tile (past the last one:
      // not used)
      int v_buf = 0, k_buf = 1;
      for (int kt = kt0; kt < end; ++kt) {
        if ((kt + 1) * KT > clear) {
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const int first = kt * KT + 32 * (ks * NB + i);
            uint32_t word = first < q.len ? ~0u : 0u;
            if (!a.parent || (first + 32 > q.len && first < limit)) word = sees(a, q, tok, t.tok0, first, lds.seen, Words);
            word >>= 4 * hi2;
#pragma unroll
            for (int e = 0; e < 16; ++e) sc[i][e] = word >> (8 * (e / 4) + e % 4) & 1 ? sc[i][e] : -INFINITY;
          }
        }
        float top = sc[0][0];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[i][e]);
        {
          auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
          top = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])) * scale;
        }
        // the maximum is moved only when a row has outgrown it by 2^8: weights
        // stay below 256, and most tiles need no rescaling
        if (__any(top > mx + 8.f)) {
          const float next = fmaxf(mx, top), turn = next == -INFINITY ? 1.f : exp2_fast(mx - next);
          mx = next;
          sum *= turn;
#pragma unroll
          for (int d = 0; d < DB; ++d) o[d] *= turn;
        }
        const float at = mx == -INFINITY ? 0.f : mx;
        // the weights, and between them the copies of a step: all at once they
        // would wait for each other's way to LDS
        u32x4 pw[2 * NB], pl[2 * NB];
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) {
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            w[e] = exp2_fast(fmaf(sc[j / 2][j % 2 * 8 + e], scale, -at));
            sum += w[e];
          }
          split_bf16(w, &pw[j], &pl[j]);
#pragma unroll
          for (int i = j * P / NB; i < (j + 1) * P / NB; ++i) ask(kt, i);
          __builtin_amdgcn_sched_barrier(0);
        }
        // K of tile kt + 1 and V of tile kt are there, of all wavefronts behind the barrier
        wait_copies<2 * P>();
        lds_barrier();
        // O^T += V^T P^T, then the scores of the next tile.  The operands come
        // from LDS some products before their use; the order is fixed here because
        // the compiler's own puts every read next to its product
        constexpr int PV = DB * 2 * NB, QK = NB * KK;
        if (odd) {  // the wavefronts write the same
          for (int i = 0; i < NB; ++i) {
            const int block = ks * NB + i;
            for (uint32_t word = mixed.word(kt * KT + 32 * block); word; word &= word - 1) {
              u32x4* p = lds.tiles + (Bufs + v_buf) * TileWords + (32 * block + __builtin_ctz(word)) * CH;
              if (lane < CH) p[lane] = keep_finite<1>(p[lane], true);
            }
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        int k_now[KK], v_now[DB];
#pragma unroll
        for (int j = 0; j < KK; ++j) k_now[j] = k_at_lds[j] + k_buf * (TileWords * 16);
#pragma unroll
        for (int d = 0; d < DB; ++d) v_now[d] = v_at_lds[d] + v_buf * (TileWords * 16);
        v_buf ^= 1, k_buf ^= 1;
        auto fetch = [&](int i) __attribute__((always_inline)) {
          if (i < PV) return v_words(v_now[i % DB] + i / DB * (16 * CH * 16));
          return k_words(k_now[(i - PV) / NB] + (i - PV) % NB * (32 * CH * 16));
        };
        bf16x8 f[Ahead];
#pragma unroll
        for (int i = 0; i < Ahead; ++i) f[i] = fetch(i);
#pragma unroll
        for (int i = 0; i < PV + QK; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          if (i < PV) {
            const int j = i / DB, d = i % DB;
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % Ahead], __builtin_bit_cast(bf16x8, pl[j]), o[d], 0, 0, 0);
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % Ahead], __builtin_bit_cast(bf16x8, pw[j]), o[d], 0, 0, 0);
          } else {
            const int j = (i - PV) / NB, k = (i - PV) % NB;
            sc[k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % Ahead], __builtin_bit_cast(bf16x8, qr[j]), j ? sc[k] : zero, 0, 0, 0);
          }
          if (i + Ahead < PV + QK) f[i % Ahead] = fetch(i + Ahead);
        }
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
      }
      if (kt0 < end) {  // the copies asked for past the end, before LDS is used for anything else
        wait_copies<0>();
        lds_barrier();
      }
      if (!again && kt0 < end && end * KT > mixed.first) {
        const float z = zero_or_nan(o);
        if (__syncthreads_or(z != z)) continue;
      }
      {
        auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum), __float_as_uint(sum), false, false);
        sum = __uint_as_float(x[0]) + __uint_as_float(x[1]);
      }
      if constexpr (KS == 2) {  // the two halves of the keys joined
        static_assert(KS == 1 || RW * DB * 4 * kWave <= 2 * Bufs * TileWords, "the outputs of one half fit the tiles");
        f32x4* buf = reinterpret_cast<f32x4*>(lds.tiles);
        if (ks == 1) {
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              buf[((rw * DB + d) * 4 + j) * kWave + lane] =
                  f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
          if (hi2 == 0) lds.stat[rw * 64 + col] = mx, lds.stat[rw * 64 + 32 + col] = sum;
        }
        lds_barrier();
        if (ks == 1) return;
        const float m1 = lds.stat[rw * 64 + col], top = fmaxf(mx, m1), at = top == -INFINITY ? 0.f : top;
        const float mine = part_weight(mx - at), other = part_weight(m1 - at);
        mx = top;
        sum = sum * mine + lds.stat[rw * 64 + 32 + col] * other;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 y = buf[((rw * DB + d) * 4 + j) * kWave + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][4 * j + e] = o[d][4 * j + e] * mine + y[e] * other;
          }
      }
      if (odd) {  // values that are not finite, to the rows that see them
        for (int at = kt0 * KT; at < end * KT; at += 32)
          for (uint32_t word = mixed.word(at); word; word &= word - 1) {
            const int row = at + __builtin_ctz(word);
            if (row >= limit) break;
            if (!(sees(a, q, tok, t.tok0, at, lds.seen, Words) >> (row & 31) & 1)) continue;
            const u32x4* p = value_row(c, table, kv + v_off, page_stride, CH, row);
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const f32x4 x = odd_values<1>(p, 32 * d + 8 * j + 4 * hi2);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[d][4 * j + e] += x[e];
              }
          }
      }
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          emit(r, 32 * d + 8 * j + 4 * hi2, f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]}, mx, sum);
      return;
    }
  }
};

}  // namespace
}  // namespace tms
