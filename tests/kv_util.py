"""Plain 64-bit forms of the paged-cache operators for the tests, on the CPU
and without the library, and the bounds that the kernels are held to.

Bounds (u = 2^-24 and h = 2^-8, the relative errors of rounding to fp32 and bf16):
  attention  a score is a dot product of D fp32 products, scaled: its error is
      at most e = gamma(D + 4) * scale * sum|q_i k_i|.  A weight is exp of it
      relative to a maximum with the same error, so it is off by a factor
      within exp(2 e), the exponential itself and the rescaling of a running
      maximum by a few 2^-22; the sums over n keys add gamma(n + 64).  All
      that, rel, is in the numerator and in the denominator; rounding the
      weights to bf16 (h) in the numerator only.  With A = sum_j w_j |v_j| (the
      weights normalised) the output is within (2 * rel + h) * A of the exact
      one, and rounding it adds h |out|;
      Up to 64 query rows of a key head the weights are cut to bf16 (at most 2 h
      of them is left) and what is left is rounded to bf16: within 2 h^2
      (attention_fine);
  write      the sum of squares gamma(D + 8), its root and the products a few u,
      the angle (a turn in fp64 rounded to fp32) 2 pi u, sine and cosine 4 u:
      32 u + gamma(D + 8) relative to |a| + |b|, and h |out| for bf16.
"""
import math

import numpy as np

U32, UBF16 = 2.0 ** -24, 2.0 ** -8


def gamma(n):
    return n * U32 / (1 - n * U32)


def ancestors(parent):
    """sees[i][j]: draft j is draft i or an ancestor of it."""
    n = len(parent)
    sees = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            sees[i, j] = True
            j = parent[j] if -1 <= parent[j] < j else -1
    return sees


def attention(q, k, v, length, scale, parent, bf16):
    """(out, bound) of one sequence: q [n][Hq][D], k, v [length+n][Hkv][D] in
    fp64; parent [n] or None."""
    n, hq, D = q.shape
    group = hq // k.shape[1]
    sees = np.ones((n, length + n), bool)
    sees[:, length:] = np.tril(np.ones((n, n), bool)) if parent is None else ancestors(parent)
    out, bound = np.zeros_like(q), np.zeros_like(q)
    if np.isfinite(k).all() and np.isfinite(v).all():  # the same, a head at once
        rel = 2.0 ** -20 + gamma(sees.sum(1) + 64)[:, None]
        for h in range(hq):
            kk, vv = k[:, h // group], v[:, h // group]
            x = np.where(sees, scale * (q[:, h] @ kk.T), -np.inf)
            e = gamma(D + 4) * abs(scale) * np.where(sees, np.abs(q[:, h]) @ np.abs(kk).T, 0).max(1, keepdims=True)
            w = np.exp(x - x.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[:, h] = w @ vv
            bound[:, h] = (2 * (np.expm1(2 * e) + rel) + (UBF16 if bf16 else 0)) * (w @ np.abs(vv)) + \
                (UBF16 if bf16 else U32) * np.abs(out[:, h])
        return out, bound
    with np.errstate(invalid="ignore"):
        for h in range(hq):
            kk, vv = k[:, h // group], v[:, h // group]
            for i in range(n):
                on = sees[i]
                x = scale * (kk[on] @ q[i, h])
                e = gamma(D + 4) * abs(scale) * (np.abs(kk[on]) @ np.abs(q[i, h])).max()
                w = np.exp(x - x.max())
                w /= w.sum()
                out[i, h] = w @ vv[on]
                rel = math.expm1(2 * e) + 2.0 ** -20 + gamma(int(on.sum()) + 64)
                bound[i, h] = (2 * rel + (UBF16 if bf16 else 0)) * (w @ np.abs(vv[on])) + \
                    (UBF16 if bf16 else U32) * np.abs(out[i, h])
    return out, bound


def attention_fine(q, k, v, length, scale, parent):
    """attention in bf16 of up to 64 query rows of a key head."""
    out, bound = attention(q, k, v, length, scale, parent, False)
    mass, _ = attention(q, k, np.abs(v), length, scale, parent, False)
    return out, bound + 2 * UBF16 ** 2 * mass + (UBF16 - U32) * np.abs(out)


def marked_values(rows, kv_heads, dim, block=16):
    """V whose rows of `block` are 1 in a column of their own, 0 elsewhere (the
    columns in turn): an output's column is the weight of its blocks alone, so
    a block that is left out, or counted twice, shows as a share of the column
    that far outgrows the bound, which is relative to the column too."""
    v = np.zeros((rows, kv_heads, dim))
    v[np.arange(rows), :, np.arange(rows) // block % dim] = 1.0
    return v


def head(x, weight, eps, pos, inv_freq, interleaved, bf16):
    """(out, bound) of x [T][heads][D] in fp64."""
    D = x.shape[-1]
    y, size = x.copy(), np.abs(x)
    if weight is not None:
        y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * weight
        size = np.abs(y)
    if inv_freq is not None and len(inv_freq):
        half = len(inv_freq)
        z, s2 = y.copy(), size.copy()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            t = (pos.astype(np.float64) * np.float64(inv_freq[i]))[:, None]
            z[..., a] = y[..., a] * np.cos(t) - y[..., b] * np.sin(t)
            z[..., b] = y[..., b] * np.cos(t) + y[..., a] * np.sin(t)
            s2[..., a] = s2[..., b] = size[..., a] + size[..., b]
        y, size = z, s2
    plain = weight is None and (inv_freq is None or not len(inv_freq))
    bound = (0 if plain else (32 * U32 + gamma(D + 8)) * size) + (0 if plain or not bf16 else UBF16) * np.abs(y)
    return y, bound


class Pages:
    """The page operations on Python lists: what every row holds and which
    pages a sequence has, with the library's rules of order."""

    OK, INVALID, OOM = 0, 1, 9

    def __init__(self, seqs, pages, page, max_pages):
        self.page, self.max_pages, self.pages = page, max_pages, pages
        self.table = [[] for _ in range(seqs)]
        self.rows = [[] for _ in range(seqs)]      # committed rows
        self.status = [0] * seqs

    def refs(self):
        r = [0] * self.pages
        for t in self.table:
            for p in t:
                r[p] += 1
        return r

    def fork(self, src):
        table, rows, status = [list(t) for t in self.table], [list(r) for r in self.rows], list(self.status)
        for s, x in enumerate(src):
            if x == s:
                continue
            if x < -1 or x >= len(src):
                self.status[s] = self.INVALID
            elif x == -1:
                self.table[s], self.rows[s], self.status[s] = [], [], 0
            else:
                self.table[s] = table[x][:-(-len(rows[x]) // self.page)]
                self.rows[s], self.status[s] = list(rows[x]), status[x]

    def reserve(self, n_new):
        refs = self.refs()
        free = [p for p in range(self.pages) if refs[p] == 0]
        taken = 0
        for s, n in enumerate(n_new):
            if n <= 0 or self.status[s]:
                continue
            want = -(-(len(self.rows[s]) + n) // self.page)
            if want > self.max_pages:
                self.status[s] = self.INVALID
                continue
            last, t = len(self.rows[s]) // self.page, self.table[s]
            split = len(self.rows[s]) % self.page > 0 and last < len(t) and refs[t[last]] > 1
            more = max(want - len(t), 0) + split
            if more and taken + more > len(free):
                self.status[s] = self.OOM
            elif more:
                mine = free[taken:taken + more]
                if split:
                    t[last] = mine.pop(0)
                t.extend(mine)
            taken += more

    def commit(self, n_keep, keep, drafts):
        """drafts[s]: the rows written past the committed ones."""
        for s, n in enumerate(n_keep):
            if n < 0 or self.status[s]:
                continue
            k = list(range(n)) if keep is None else [int(x) for x in keep[s][:n]]
            room = len(self.table[s]) * self.page - len(self.rows[s])
            if (keep is not None and n > len(keep[s])) or any(b <= a for a, b in zip([-1] + k, k)) or (k and k[-1] >= room) or n > room:
                self.status[s] = self.INVALID
                continue
            self.rows[s] += [drafts[s][i] for i in k]
            self.table[s] = self.table[s][:-(-len(self.rows[s]) // self.page)]


def choice(q, bounds, k, scale, first, last):
    """The pages that one token reads: q [Hq][D], bounds [pages][Hkv][2][D] in
    fp64 -> [Hkv][k], ascending, -1 past the pages."""
    pages, hkv = bounds.shape[:2]
    out = np.full((hkv, k), -1, np.int32)
    group = q.shape[0] // hkv
    for h in range(hkv):
        x = np.sign(scale) * q[h * group:(h + 1) * group] if scale else np.zeros((group, q.shape[1]))
        with np.errstate(invalid="ignore"):
            over, under = np.maximum(x, 0).sum(0), np.minimum(x, 0).sum(0)
            score = (over * bounds[:, h, 1] + under * bounds[:, h, 0]).sum(-1)
        always = [j for j in range(pages) if j < first or j >= pages - last]
        score[always] = np.inf
        # NaN above all, then by score, of equal ones the lower page
        order = sorted(range(pages), key=lambda j: (not np.isnan(score[j]), -score[j] if not np.isnan(score[j]) else 0, j))
        best = sorted(order[:k])
        out[h, :len(best)] = best
    return out
