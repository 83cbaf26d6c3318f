"""Long contexts of the paged cache on the GPU against plain 64-bit forms
(kv_util.py, which also derives the bounds): attention of batches that share
pages, bounds of pages, the choice of pages by them, and attention over chosen
pages."""
import numpy as np
import pytest
import torch

import trie_masked_sparse_amd as tms
from kv_util import attention, attention_fine, choice, marked_values
from test_gpu_kv import BF, F, dev32, filled, offsets, tree

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 64), (16, 8, 128), (8, 1, 128), (3, 3, 64), (10, 2, 256)]
ids = dict(ids=lambda h: "x".join(map(str, h)) if isinstance(h, tuple) else None)


# ------------------------------------------------------------------ shared pages

class Branches:
    """A cache whose sequences are paths of named runs of whole pages (a run of
    one name is the same pages for all that have it behind the same runs), and
    rows of their own: seqs = [(((name, pages), ...), own rows, new rows)]."""

    def __init__(self, rng, dtype, kv_heads, dim, page, seqs, layers=1, spare=3, marked=False):
        self.lens = [sum(p for _, p in path) * page + own for path, own, _ in seqs]
        self.new = [new for _, _, new in seqs]
        need = [-(-(a + b) // page) for a, b in zip(self.lens, self.new)]
        total, width = sum(need) + spare, max(max(need), 1)
        pool = list(rng.permutation(total))
        kv = torch.full((layers, total, 2, kv_heads, page, dim), float("nan"), dtype=dtype)
        table, refs, known = np.full((len(seqs), width), -1, np.int32), np.zeros(total, np.int32), {}
        self.ks, self.vs = [[] for _ in range(layers)], [[] for _ in range(layers)]
        for s, (path, own, new) in enumerate(seqs):
            at, where, rows = 0, (), self.lens[s] + new
            for name, count in path:
                where += ((name, count),)
                for i in range(count):
                    if (where, i) not in known:
                        known[where, i] = int(pool.pop())
                        kv[:, known[where, i]] = self.values(rng, (layers, 2, kv_heads, page, dim), dtype)
                    table[s, at] = known[where, i]
                    at += 1
            for j in range(at, need[s]):
                table[s, j] = pool.pop()
                have = min(page, rows - j * page)
                kv[:, table[s, j], :, :, :have] = self.values(rng, (layers, 2, kv_heads, have, dim), dtype)
            if marked and not (table[s, :at] < 0).any():  # values of a page by its place: the same for all that share it
                v = torch.from_numpy(marked_values(width * page, kv_heads, dim)).to(dtype)
                for j in range(need[s]):
                    have = min(page, rows - j * page)
                    kv[:, table[s, j], 1, :, :have] = v[j * page:j * page + have].transpose(0, 1)
            for p in table[s, :need[s]]:
                refs[p] += 1
        for layer in range(layers):
            for s in range(len(seqs)):
                both = kv[layer, table[s, :need[s]].tolist()].double().numpy()  # [pages][2][heads][page][dim]
                both = both.transpose(1, 0, 3, 2, 4).reshape(2, -1, kv_heads, dim)[:, :self.lens[s] + self.new[s]]
                self.ks[layer].append(both[0])
                self.vs[layer].append(both[1])
        self.page, self.table, self.need = page, table, need
        self.cache = tms.PagedCache(kv.cuda(), dev32(table), dev32(self.lens), dev32(need), dev32(refs), dev32([0] * len(seqs)))

    @staticmethod
    def values(rng, shape, dtype):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def queries(rng, b, heads, dim, dtype):
    return torch.from_numpy(rng.standard_normal((sum(b.new), heads, dim)).astype(np.float32)).to(dtype).cuda()


def run_shared(b, q, parents=None, scale=None, layer=0, plan=None, max_new=None, stream=None, out=None):
    if out is None:
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    start = dev32(offsets(b.new))
    par = None if parents is None else dev32([p for t in parents for p in t])
    if plan is None:
        plan = tms.SharedPlan(b.cache, q.shape[0], q.shape[1])
        tms.kv_share(b.cache, plan, start, stream=stream)
    tms.kv_attention_shared(b.cache, layer, q, start, out, plan, scale, parent=par, max_new=max_new or max(b.new), stream=stream)
    return out


def check_shared(b, q, out, scale, parents, where="", layer=0, of=None):
    bf16 = q.dtype == BF
    q, out, at = q.double().cpu().numpy(), out.double().cpu().numpy(), offsets(b.new)
    for s, (a, n) in enumerate(zip(b.lens, b.new)):
        if n and (of is None or s in of):
            want, bound = attention(q[at[s]:at[s + 1]], b.ks[layer][s], b.vs[layer][s], a, scale,
                                    None if parents is None else parents[s], bf16)
            err = np.abs(out[at[s]:at[s + 1]] - want)
            assert (err <= bound).all(), (where, s, a, n, float(np.nanmax(err / bound)), int((~(err <= bound)).sum()))


A, B_, C_ = ("a", 40), ("b", 33), ("c", 1)
SHARED = [
    # (page, sequences)
    (16, [((A,), 3, 1)] * 2),
    (64, [((A,), i, 1) for i in range(9)]),
    (8, [((("p", 200),), i % 5, i % 3) for i in range(40)]),
    # two prompts with one beginning, a sequence of the beginning alone, one of nothing, some without new tokens
    (16, [((A, B_), 5, 1), ((A, ("d", 50)), 0, 2), ((A, B_), 17, 4), ((A,), 1, 3), ((), 0, 1), ((A, ("d", 50)), 100, 0),
          ((), 700, 5), ((A, ("d", 50)), 15, 1), ((("e", 80),), 2, 2), ((("e", 80),), 0, 7)]),
    # a chain of beginnings, longer than the runs that are shared
    (32, [((("x", 9),) * d, 0, 2) for d in (1, 2, 3, 4, 5, 6, 6)]),
    # runs that are too short to be shared, pages larger than a tile
    (128, [((C_,), 0, 1), ((C_,), 5, 1), ((("y", 7),), 9, 30), ((("y", 7),), 0, 31), ((("y", 7),), 128, 16)]),
    # sequences of many rows beside some of few
    (16, [((A,), 0, 200), ((A,), 7, 1), ((A,), 9, 3), ((A,), 11, 150)]),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS, **ids)
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_shared_matches_the_64_bit_form(dtype, heads, kind):
    hq, hkv, D = heads
    for n, (page, seqs) in enumerate(SHARED):
        print(f"shared {dtype} {heads} {kind} batch {n} page {page}", flush=True)
        rng = np.random.default_rng(17 * n + D + hq)
        b = Branches(rng, dtype, hkv, D, page, seqs, layers=2)
        q = queries(rng, b, hq, D, dtype)
        parents = [tree(rng, x) for x in b.new] if kind == "tree" else None
        out = run_shared(b, q, parents, layer=1)
        check_shared(b, q, out, D ** -0.5, parents, (n, kind), layer=1)
        assert torch.equal(out, run_shared(b, q, parents, layer=1))  # no order depends on timing


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_shared_large_batches(dtype):
    rng = np.random.default_rng(3)
    few = dict(page=16, dim=64, heads=(4, 2))
    for seqs in ([((("p", 300),), int(x), 1) for x in rng.integers(0, 40, 256)],
                 [((("p", 20), (f"q{i % 7}", 30), (f"r{i % 14}", 11)), int(x), int(y))
                  for i, (x, y) in enumerate(zip(rng.integers(0, 90, 300), rng.integers(0, 4, 300)))],
                 [(((f"p{i % 500}", 20),), 0, 1) for i in range(1500)],
                 [((("p", 4000),), 3, 2)] * 3):
        print(f"shared {dtype} {len(seqs)} sequences", flush=True)
        b = Branches(rng, dtype, few["heads"][1], few["dim"], few["page"], seqs)
        q = queries(rng, b, few["heads"][0], few["dim"], dtype)
        out = run_shared(b, q)
        check_shared(b, q, out, few["dim"] ** -0.5, None)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 4, 128), (8, 1, 256)], **ids)
def test_shared_counts_every_key_once(dtype, heads):
    hq, hkv, D = heads
    for n, (page, seqs) in enumerate([(16, [((("p", 900),), i, 1) for i in range(5)]),
                                      (64, [((("p", 90), (f"q{i % 2}", 40)), 30 * i, 1) for i in range(20)]),
                                      (8, [((("p", 500),), 900 * i, 3) for i in range(4)])]):
        print(f"marked {dtype} {heads} batch {n}", flush=True)
        rng = np.random.default_rng(n)
        b = Branches(rng, dtype, hkv, D, page, seqs, marked=True)
        q = 0.7 * queries(rng, b, hq, D, dtype)
        check_shared(b, q, run_shared(b, q), D ** -0.5, None, n)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_shared_tables_that_no_fork_makes(dtype):
    """Pages in common behind different ones, a page twice in a sequence, tables
    that agree, differ and agree again."""
    rng = np.random.default_rng(8)
    page, dim = 16, 64
    b = Branches(rng, dtype, 2, dim, page, [((("p", 60),), 4, 1), ((("q", 60),), 4, 2), ((("r", 60),), 4, 1), ((("s", 60),), 4, 1)])
    table = b.table.copy()
    table[1, 20:60] = table[0, 20:60]
    table[2, :10], table[2, 11:40] = table[0, :10], table[0, 11:40]
    table[3, 30] = table[3, 2]
    table[3, :2] = table[2, :2]
    kv = b.cache.kv[0].cpu()
    for s in range(4):
        both = kv[table[s, :b.need[s]].tolist()].double().numpy().transpose(1, 0, 3, 2, 4).reshape(2, -1, 2, dim)
        b.ks[0][s], b.vs[0][s] = both[0, :b.lens[s] + b.new[s]], both[1, :b.lens[s] + b.new[s]]
    b.cache.table.copy_(dev32(table))
    q = queries(rng, b, 4, dim, dtype)
    check_shared(b, q, run_shared(b, q), dim ** -0.5, None)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_shared_scales_strides_and_another_stream(dtype):
    rng = np.random.default_rng(4)
    b = Branches(rng, dtype, 2, 128, 32, [((("p", 30),), i, 1 + i % 3) for i in range(6)])
    T = sum(b.new)
    wide = torch.from_numpy(rng.standard_normal((T, 8 + 4, 128)).astype(np.float32)).to(dtype).cuda()
    q = wide[:, 2:10]
    for scale in (4.0, -2.0, 0.0):
        check_shared(b, q, run_shared(b, q, scale=scale), scale, None, scale)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    start = dev32(offsets(b.new))
    plan = tms.SharedPlan(b.cache, T, 8)
    torch.cuda.synchronize()
    tms.kv_share(b.cache, plan, start, stream=s)
    tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=3, stream=s)
    s.synchronize()
    check_shared(b, q, out, 128 ** -0.5, None, "stream")


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["causal", "tree"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (4, 2, 128), (8, 2, 256)], **ids)
def test_shared_rows_not_seen_may_hold_anything(dtype, kind, heads):
    """Infinities and NaN of drafts and later tokens reach only who sees them; an
    infinite value of a token itself stays infinite."""
    hq, hkv, D = heads
    rng = np.random.default_rng(21)
    b = Branches(rng, dtype, hkv, D, 16, [((("p", 40),), 5, 6), ((("p", 40),), 0, 3), ((("p", 40),), 30, 1)])
    for s, i, which, value in ((0, 3, 1, float("inf")), (0, 5, 0, float("nan")), (1, 2, 1, float("nan"))):
        row = b.lens[s] + i
        b.cache.kv[0, int(b.table[s, row // 16]), which, :, row % 16, 1] = value
        (b.ks if which == 0 else b.vs)[0][s][row, :, 1] = value
    parents = [[-1, 0, 0, 1, 1, 2], [-1, 0, 0], [-1]] if kind == "tree" else None
    q = queries(rng, b, hq, D, dtype)
    out = run_shared(b, q, parents).double().cpu().numpy()
    at = offsets(b.new)
    for s in range(3):
        with np.errstate(invalid="ignore"):
            want, bound = attention(q[at[s]:at[s + 1]].double().cpu().numpy(), b.ks[0][s], b.vs[0][s], b.lens[s], D ** -0.5,
                                    None if parents is None else parents[s], dtype == BF)
        got = out[at[s]:at[s + 1]]
        for i in range(b.new[s]):
            fine = np.isfinite(want[i])
            assert (np.isnan(got[i]) == np.isnan(want[i])).all() and (got[i][np.isinf(want[i])] == np.inf).all(), (s, i)
            assert (np.abs(got[i] - want[i])[fine] <= bound[i][fine]).all(), (s, i)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_shared_an_infinite_value_of_the_last_shared_row(dtype):
    """Rows that fill up a tile behind it weigh nothing."""
    rng = np.random.default_rng(6)
    for page in (8, 16, 64):
        b = Branches(rng, dtype, 2, 64, page, [((("p", 41),), i, 1) for i in range(4)])
        b.cache.kv[0, int(b.table[0, 40]), 1, :, page - 1, 7] = float("inf")
        q = queries(rng, b, 4, 64, dtype)
        q[:, :, :] *= 0.1
        out = run_shared(b, q)
        assert torch.isinf(out[..., 7]).all(), page
        rest = torch.cat((out[..., :7], out[..., 8:]), -1)
        assert torch.isfinite(rest).all()


def test_shared_sequences_in_error_stale_plans_and_tokens_of_nobody():
    rng = np.random.default_rng(2)
    b = Branches(rng, BF, 2, 64, 16, [((("p", 40),), i, 1) for i in range(4)])
    q = queries(rng, b, 4, 64, BF)
    start = dev32(offsets(b.new))
    b.cache.status_codes[1] = tms.ERR_OOM
    out = run_shared(b, q)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2, 3]]).all()
    check_shared(b, q, out, 0.125, None, of=(0, 2, 3))
    b.cache.status_codes[1] = 0
    # a plan that is older than the lengths
    plan = tms.SharedPlan(b.cache, 4, 4)
    out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="made for 0"):
        tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=1)
    plan._planned = 4  # (the library's own check)
    tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=1)  # never made
    assert torch.isnan(out).all()
    tms.kv_share(b.cache, plan, start)
    b.cache.length[2] -= 1
    tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=1)
    assert torch.isnan(out[2]).all() and torch.isfinite(out[[0, 1, 3]]).all()
    b.cache.length[2] += 1
    # of other tokens
    tms.kv_share(b.cache, plan, dev32([0, 1, 2, 3, 3]), tokens=3)
    with pytest.raises(ValueError, match="made for 3"):
        tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=1)
    plan._planned = 4
    tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=1)
    assert torch.isnan(out).all()
    out.fill_(7.0)
    few = dev32([0, 1, 1, 2, 2])
    tms.kv_share(b.cache, plan, few, tokens=4)
    tms.kv_attention_shared(b.cache, 0, q, few, out, plan, max_new=1)
    assert (out[2:] == 7.0).all() and torch.isfinite(out[:2]).all()
    # too many tokens of a sequence for max_new
    b2 = Branches(rng, BF, 2, 64, 16, [((("p", 40),), i, 1 + i) for i in range(3)])
    q2 = queries(rng, b2, 4, 64, BF)
    out = run_shared(b2, q2, max_new=2)
    assert torch.isnan(out[3:]).all()
    check_shared(b2, q2, out, 0.125, None, of=(0, 1))


@pytest.mark.parametrize("n", [2, 3, 4, 15, 17, 40, 63, 64, 65, 100, 200, 1030])
@pytest.mark.parametrize("prompts", [1, 2])
def test_shared_pages_are_read_once(n, prompts):
    """Pages of sequences other than the first of a prompt are replaced behind the
    plan by one that holds NaN: whoever shares the first one's does not notice."""
    rng = np.random.default_rng(n)
    b = Branches(rng, BF, 1, 64, 16, [(((f"p{i % prompts}", 60),), i % 5, 1) for i in range(n)])
    q = queries(rng, b, 2, 64, BF)
    start = dev32(offsets(b.new))
    plan = tms.SharedPlan(b.cache, n, 2)
    tms.kv_share(b.cache, plan, start)
    nobody = [p for p in range(b.cache.pages) if int(b.cache.refs[p]) == 0][0]
    assert torch.isnan(b.cache.kv[0, nobody].float()).all()
    b.cache.table[prompts:, :60] = nobody
    out = run_shared(b, q, plan=plan)
    alone = [s for s in range(n) if n // prompts < 2 or (n == 3 and prompts == 2 and s == 1)]
    check_shared(b, q, out, 0.125, None, n, of=[s for s in range(n) if s < prompts or s not in alone])


@pytest.mark.parametrize("branch", [3, 40])
def test_shared_beginnings_of_prompts_are_read_once_where_it_pays(branch):
    """Prompts of one beginning: a run of its own if it is long, else part of each
    prompt's."""
    rng = np.random.default_rng(branch)
    b = Branches(rng, BF, 1, 64, 16, [((("a", branch), (f"p{i % 4}", 50)), 3, 1) for i in range(64)])
    q = queries(rng, b, 2, 64, BF)
    plan = tms.SharedPlan(b.cache, 64, 2)
    tms.kv_share(b.cache, plan, dev32(offsets(b.new)))
    nobody = [p for p in range(b.cache.pages) if int(b.cache.refs[p]) == 0][0]
    keep = b.cache.table.clone()
    b.cache.table[4:, :branch + 50] = nobody
    check_shared(b, q, run_shared(b, q, plan=plan), 0.125, None, branch)
    b.cache.table.copy_(keep)
    b.cache.table[1:, :branch] = nobody
    out = run_shared(b, q, plan=plan)
    if branch == 40:
        check_shared(b, q, out, 0.125, None, branch)
    else:
        assert torch.isfinite(out[0::4]).all() and torch.isnan(out[1::4]).all()


def test_shared_starts_out_of_order_are_refused_without_harm():
    rng = np.random.default_rng(2)
    b = Branches(rng, BF, 2, 64, 16, [((("p", 40),), 0, 4)] * 4)
    q = queries(rng, b, 4, 64, BF)
    bad = dev32([0, 10, 4, 14, 16])  # tokens of two sequences
    b.cache.held.fill_(44)
    out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    plan = tms.SharedPlan(b.cache, 16, 4)
    tms.kv_share(b.cache, plan, bad)
    tms.kv_attention_shared(b.cache, 0, q, bad, out, plan, max_new=16)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ bounds

@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 64, 1024])
def test_bounds_are_the_lowest_and_highest_keys(dtype, dim, page):
    rng = np.random.default_rng(dim + page)
    lens = [0, 1, page - 1, page, page + 1, 3 * page + 5, 7 * page]
    cache, ks, _ = filled(rng, dtype, 5, dim, page, lens, [0] * len(lens), layers=2, layer=1)
    cache.kv[0].copy_(cache.kv[1])
    table = cache.table.cpu().numpy()
    for n_new in (None, [0, 1, 3, 1, 1, page + 5, 2 * page], [9, -4, 0, page, 0, 5, 6 * page + 1]):
        print(f"bounds {dtype} {dim} {page} {n_new}", flush=True)
        index = tms.PageIndex(cache, torch.full((2, cache.pages, 5, 2, dim), 7.0, dtype=dtype, device="cuda"))
        want = torch.full_like(index.bounds, 7.0).cpu()
        for s, a in enumerate(lens):
            n = a if n_new is None else min(max(n_new[s], 0), a)
            for j in range((a - n) // page, a // page):
                keys = torch.from_numpy(ks[s][j * page:(j + 1) * page])
                want[:, table[s, j], :, 0], want[:, table[s, j], :, 1] = keys.amin(0).to(dtype), keys.amax(0).to(dtype)
        for most in (None, 1):
            index.bounds.fill_(7.0)
            tms.kv_bounds(cache, index, None if n_new is None else dev32(n_new), max_new=most)
            assert torch.equal(index.bounds.cpu(), want), (n_new, most)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_bounds_of_keys_that_are_not_finite(dtype):
    rng = np.random.default_rng(1)
    cache, _, _ = filled(rng, dtype, 2, 64, 16, [32], [0])
    a, b = (int(x) for x in cache.table[0, :2])
    cache.kv[0, a, 0, 0, 3, 5] = float("nan")
    cache.kv[0, a, 0, 1, 15, 6] = float("inf")
    cache.kv[0, b, 0, 0, 0, 7] = -float("inf")
    cache.kv[0, b, 0, 1, :, 8] = -float("inf")
    index = tms.PageIndex(cache)
    tms.kv_bounds(cache, index)
    got = index.bounds[0]
    keys = cache.kv[0, [a, b], 0]
    assert torch.equal(torch.nan_to_num(got[[a, b]], nan=77.0),
                       torch.nan_to_num(torch.stack((keys.amin(2), keys.amax(2)), 2), nan=77.0))
    assert torch.isnan(got[a, 0, :, 5]).all() and got[a, 1, 1, 6] == float("inf") and got[b, 1, 1, 8] == -float("inf")


def test_bounds_of_sequences_in_error_are_left():
    rng = np.random.default_rng(1)
    cache, _, _ = filled(rng, BF, 2, 64, 16, [32, 32], [0, 0])
    cache.status_codes[0] = tms.ERR_OOM
    index = tms.PageIndex(cache)
    tms.kv_bounds(cache, index)
    table = cache.table.cpu()
    assert (index.bounds[0, table[0, :2].tolist()] == 0).all() and (index.bounds[0, table[1, :2].tolist()] != 0).any()


# ------------------------------------------------------------------ choice

def run_select(cache, index, q, new, k, scale=None, first=1, last=1, max_new=None):
    chosen = torch.full((q.shape[0], cache.kv_heads, k), 77, dtype=torch.int32, device="cuda")
    tms.kv_select(cache, 0, q, dev32(offsets(new)), index, chosen, scale, first=first, last=last, max_new=max_new or max(max(new), 1))
    return chosen.cpu().numpy()


def check_select(cache, index, q, lens, new, k, chosen, scale=1.0, first=1, last=1):
    table, at = cache.table.cpu().numpy(), offsets(new)
    bounds, q = index.bounds[0].double().cpu().numpy(), q.double().cpu().numpy()
    for s, (a, n) in enumerate(zip(lens, new)):
        whole = a // cache.page_tokens
        for t in range(at[s], at[s + 1]):
            want = choice(q[t], bounds[table[s, :whole]], k, scale, first, last)
            assert (chosen[t] == want).all(), (s, t, a, k)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS, **ids)
def test_select_matches_the_64_bit_form(dtype, heads):
    hq, hkv, D = heads
    for n, (page, lens, new, k, first, last) in enumerate([
            (16, [700], [1], 8, 1, 1), (8, [9000, 3, 64, 65, 0], [1, 1, 2, 0, 1], 8, 0, 0),
            (16, [333, 1000, 17, 2500], [5, 1, 3, 13], 20, 2, 3), (64, [1500, 640], [1, 1], 1, 0, 0),
            (8, [40000], [2], 300, 1, 2), (32, [900, 800], [1, 2], 5, 4, 4), (16, [700, 100], [3, 2], 8192, 1, 1)]):
        print(f"select {dtype} {heads} {n}", flush=True)
        rng = np.random.default_rng(n + D)
        cache, _, _ = filled(rng, dtype, hkv, D, page, lens, new)
        index = tms.PageIndex(cache, tokens=sum(new))
        tms.kv_bounds(cache, index)
        q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
        for scale in (None, -0.5):
            chosen = run_select(cache, index, q, new, k, scale, first, last)
            check_select(cache, index, q, lens, new, k, chosen, scale or 1.0, first, last)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_select_equal_scores_and_values_that_are_not_finite(dtype):
    rng = np.random.default_rng(5)
    lens, new, k = [16 * 300 + 3, 16 * 40], [1, 2], 10
    cache, _, _ = filled(rng, dtype, 2, 64, 16, lens, new)
    index = tms.PageIndex(cache, tokens=3)
    tms.kv_bounds(cache, index)
    table = cache.table.cpu()
    p = table[0, :300].long().cuda()
    index.bounds[0, p] = index.bounds[0, p[torch.arange(300) % 7]].clone()  # seven kinds of pages
    q = torch.from_numpy(rng.standard_normal((3, 4, 64)).astype(np.float32)).to(dtype).cuda()
    check_select(cache, index, q, lens, new, k, run_select(cache, index, q, new, k))
    # a scale of 0: all equal
    assert (run_select(cache, index, q, new, k, 0.0, 0, 0)[0] == np.arange(k)).all()
    assert (run_select(cache, index, q, new, k, 0.0, 0, 3)[0] == np.r_[np.arange(7), 297:300]).all()
    index.bounds[0, p[123], 0, 1, 5] = float("nan")
    index.bounds[0, p[200], :, 1] = float("inf")
    index.bounds[0, p[210], :, 0] = float("-inf")
    index.bounds[0, p[220], :, 1] = float("-inf")
    chosen = run_select(cache, index, q, new, k)
    check_select(cache, index, q, lens, new, k, chosen)
    assert 123 in chosen[0, 0] and 123 not in chosen[0, 1] and 200 in chosen[0, 0] and 210 in chosen[0, 0]
    q[0, 1, 3] = float("nan")  # a query: every page the same
    chosen = run_select(cache, index, q, new, k, first=0, last=0)
    assert (chosen[0, 0] == np.arange(k)).all()
    cache.status_codes[1] = tms.ERR_OOM
    assert (run_select(cache, index, q, new, k)[1:] == -1).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("pages,cut", [(40, False), (5000, False), (5000, True)], ids=["short", "past_lds", "cut"])
def test_select_borders_among_nan_infinite_and_always_chosen_pages(dtype, pages, cut):
    """Every place that the border can have: among NaN, among infinite scores and
    the first and last pages (by place), among finite ones; more first and last
    pages than are taken; equal scores at the border."""
    rng = np.random.default_rng(pages)
    # (a list is taken by one workgroup where there are many)
    T = 1 if cut else 300 if pages > 1000 else 1
    cache, _, _ = filled(rng, dtype, 1, 64, 8, [8 * pages + 2], [T])
    index = tms.PageIndex(cache, tokens=T)
    tms.kv_bounds(cache, index)
    p = cache.table[0, :pages].long()
    base = index.bounds[0, p].clone()
    q = torch.from_numpy(np.abs(rng.standard_normal((1, 2, 64))).astype(np.float32)).to(dtype).cuda().expand(T, 2, 64).contiguous()
    for nans, infs, same, low in ((0, 0, 0, 0), (3, 0, 0, 0), (20, 0, 0, 0), (0, 20, 0, 0), (4, 9, 0, 3), (0, 0, pages, 0), (2, 1, pages // 2, 1)):
        b = base.clone()
        where = torch.from_numpy(rng.permutation(pages)).cuda()
        b[where[:same]] = base[0]
        b[where[same // 2:same // 2 + nans], 0, 1, 3] = float("nan")
        b[where[-infs - 1:-1] if infs else where[:0], 0, 1, 5] = float("inf")
        b[where[5:5 + low], 0, 1, 7] = float("-inf")
        index.bounds[0, p] = b
        for k, first, last in ((1, 0, 0), (10, 0, 0), (10, 2, 3), (10, 7, 9), (pages - 1, 1, 1), (16, 0, 16)):
            if k > 8192:
                continue
            chosen = run_select(cache, index, q, [T], k, None, first, last)
            want = choice(q[0].double().cpu().numpy(), index.bounds[0, p].double().cpu().numpy(), k, 1.0, first, last)
            assert (chosen == want[None]).all(), (nans, infs, same, low, k, first, last)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_select_gives_the_same_on_memory_that_holds_anything(dtype):
    rng = np.random.default_rng(8)
    lens, new = [9000, 40, 3000], [2, 1, 3]
    cache, _, _ = filled(rng, dtype, 2, 128, 16, lens, new)
    index = tms.PageIndex(cache, tokens=6)
    tms.kv_bounds(cache, index)
    q = torch.from_numpy(rng.standard_normal((6, 8, 128)).astype(np.float32)).to(dtype).cuda()
    first = run_select(cache, index, q, new, 12)
    check_select(cache, index, q, lens, new, 12, first)
    index.memory.fill_(0xff)
    cache.work[tms.KV_WORK_ZERO:].fill_(0xff)
    assert (run_select(cache, index, q, new, 12) == first).all()
    assert (cache.work[:tms.KV_WORK_ZERO] == 0).all()


def test_select_leaves_tokens_of_nobody():
    rng = np.random.default_rng(5)
    cache, _, _ = filled(rng, BF, 2, 64, 16, [100, 200], [1, 1])
    index = tms.PageIndex(cache, tokens=4)
    tms.kv_bounds(cache, index)
    q = torch.zeros((4, 4, 64), dtype=BF, device="cuda")
    chosen = torch.full((4, 2, 3), 77, dtype=torch.int32, device="cuda")
    tms.kv_select(cache, 0, q, dev32([0, 1, 2]), index, chosen, max_new=1)
    assert (chosen[2:] == 77).all() and (chosen[:2] >= 0).all()


# ------------------------------------------------------------------ attention over chosen pages

def lists(rng, lens, new, kv_heads, page, k):
    out = np.full((sum(new), kv_heads, k), -1, np.int32)
    at = offsets(new)
    for s, a in enumerate(lens):
        whole = a // page
        for t in range(at[s], at[s + 1]):
            for h in range(kv_heads):
                m = min(int(rng.integers(0, k + 1)) if rng.random() < 0.3 else k, whole)
                out[t, h, :m] = np.sort(rng.permutation(whole)[:m])
    return out


def run_pages(cache, q, new, chosen, parents=None, scale=None, max_new=None, stream=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    par = None if parents is None else dev32([p for t in parents for p in t])
    tms.kv_attention_pages(cache, 0, q, dev32(offsets(new)), dev32(chosen), out, scale, parent=par,
                           max_new=max_new or max(max(new), 1), stream=stream)
    return out


def check_pages(cache, q, out, ks, vs, lens, new, chosen, scale, parents, where=""):
    bf16, page = q.dtype == BF, cache.page_tokens
    q, out, at = q.double().cpu().numpy(), out.double().cpu().numpy(), offsets(new)
    group = q.shape[1] // cache.kv_heads
    for s, (a, n) in enumerate(zip(lens, new)):
        for i in range(n):
            t, mine = at[s] + i, [i] if parents is None else []
            j = i
            while parents is not None and j >= 0:
                mine.append(j)
                p = parents[s][j]
                j = p if -1 <= p < j else -1
            mine = list(range(i + 1)) if parents is None else sorted(mine)
            for h in range(cache.kv_heads):
                rows = [r for p in chosen[t, h] if p >= 0 for r in range(p * page, (p + 1) * page)]
                rows += list(range(a // page * page, a)) + [a + m for m in mine]
                x = q[t:t + 1, h * group:(h + 1) * group]
                k, v = ks[s][rows, h:h + 1], vs[s][rows, h:h + 1]
                want, bound = (attention_fine(x, k, v, len(rows) - 1, scale, None) if bf16 else
                               attention(x, k, v, len(rows) - 1, scale, None, False))
                err = np.abs(out[t:t + 1, h * group:(h + 1) * group] - want)
                assert (err <= bound).all(), (where, s, i, h, a, n, float(np.nanmax(err / bound)))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS + [(40, 2, 64)], **ids)
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_pages_match_the_64_bit_form(dtype, heads, kind):
    hq, hkv, D = heads
    for n, (page, lens, new, k) in enumerate([
            (16, [0], [1], 0), (16, [700], [1], 5), (64, [6000], [1], 30), (8, [100, 0, 9, 333], [3, 1, 9, 20], 7),
            (32, [4000] * 5, [1] * 5, 9), (16, [250, 15], [30, 1], 12), (128, [1000, 1], [1, 2], 3), (8, [9], [70], 1)]):
        print(f"pages {dtype} {heads} {kind} {n}", flush=True)
        rng = np.random.default_rng(31 * n + D + hq)
        cache, ks, vs = filled(rng, dtype, hkv, D, page, lens, new)
        q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
        parents = [tree(rng, x) for x in new] if kind == "tree" else None
        chosen = lists(rng, lens, new, hkv, page, k)
        out = run_pages(cache, q, new, chosen, parents)
        check_pages(cache, q, out, ks, vs, lens, new, chosen, D ** -0.5, parents, n)
        assert torch.equal(out, run_pages(cache, q, new, chosen, parents))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_pages_long_lists_and_many_tokens(dtype):
    rng = np.random.default_rng(9)
    for page, lens, new, k in ((8, [40000], [1], 4000), (16, [int(x) for x in rng.integers(0, 900, 70)], [1] * 70, 11),
                               (16, [500, 600], [150, 90], 6)):
        print(f"pages long {dtype} {page} {k}", flush=True)
        cache, ks, vs = filled(rng, dtype, 2, 64, page, lens, new)
        q = torch.from_numpy(rng.standard_normal((sum(new), 4, 64)).astype(np.float32)).to(dtype).cuda()
        chosen = lists(rng, lens, new, 2, page, k)
        check_pages(cache, q, run_pages(cache, q, new, chosen), ks, vs, lens, new, chosen, 0.125, None)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_pages_of_all_are_the_whole_attention(dtype):
    rng = np.random.default_rng(10)
    lens, new = [700, 16, 5], [4, 1, 2]
    cache, ks, vs = filled(rng, dtype, 2, 128, 16, lens, new)
    q = torch.from_numpy(rng.standard_normal((7, 8, 128)).astype(np.float32)).to(dtype).cuda()
    index = tms.PageIndex(cache, tokens=7)
    tms.kv_bounds(cache, index)
    chosen = run_select(cache, index, q, new, 64)
    for scale in (0.3, -1.0, 0.0):
        out = run_pages(cache, q, new, chosen, scale=scale).double().cpu().numpy()
        at = offsets(new)
        for s in range(3):
            want, bound = attention(q[at[s]:at[s + 1]].double().cpu().numpy(), ks[s], vs[s], lens[s], scale, None, dtype == BF)
            assert (np.abs(out[at[s]:at[s + 1]] - want) <= bound).all(), (s, scale)


def test_pages_lists_that_are_wrong_give_nan():
    rng = np.random.default_rng(12)
    lens, new = [330, 330], [2, 1]
    cache, ks, vs = filled(rng, BF, 2, 64, 16, lens, new)
    q = torch.from_numpy(rng.standard_normal((3, 4, 64)).astype(np.float32)).to(BF).cuda()
    good = np.tile(np.array([1, 5, 19, -1], np.int32), (3, 2, 1))
    for wrong in ([1, 1, 2, 3], [5, 4, 6, 7], [1, 2, 20, -1], [0, -1, 3, -1], [2000000000, 3, 4, 5], [0, 1, 2, 21]):
        chosen = good.copy()
        chosen[0, 1] = wrong
        out = run_pages(cache, q, new, chosen)
        assert torch.isnan(out[0, 2:]).all(), wrong
        assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1:]).all(), wrong
    chosen = good.copy()
    chosen[0, 0] = [-1, -1, -1, -1]
    chosen[0, 1] = [3, -7, -1, -2000000000]
    check_pages(cache, q, run_pages(cache, q, new, chosen), ks, vs, lens, new, chosen, 0.125, None)
    cache.status_codes[1] = tms.ERR_OOM
    out = run_pages(cache, q, new, good)
    assert torch.isnan(out[2]).all() and torch.isfinite(out[:2]).all()
    cache.status_codes[1] = 0
    out = run_pages(cache, q, new, good, max_new=1)
    assert torch.isnan(out[:2]).all() and torch.isfinite(out[2]).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(2, 2, 64), (16, 4, 128), (8, 1, 256), (20, 2, 64)], **ids)
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_pages_of_drafts_in_every_kind_of_batch(dtype, heads, kind):
    """Tokens of a sequence that share a workgroup: ones that do not fill a row
    tile, sequences without tokens, lists with nothing in common, one list for
    all, more pages than are held at once, sequences of many pages."""
    hq, hkv, D = heads
    for n, (page, lens, new, k, same) in enumerate([
            (8, [700, 0, 90, 2000], [17, 3, 0, 40], 20, False), (16, [3000] * 3, [2, 16, 33], 30, True), (64, [5000, 64], [8, 7], 70, False),
            (8, [20000], [20], 900, False), (8, [40] * 60, [int(x) for x in np.arange(60) % 4], 3, False)]):
        if D == 256 and k > 100 or k > 100 and heads != (2, 2, 64) and dtype == F:
            continue
        print(f"pages of drafts {dtype} {heads} {kind} {n}", flush=True)
        rng = np.random.default_rng(3 * n + D)
        cache, ks, vs = filled(rng, dtype, hkv, D, page, lens, new)
        q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
        parents = [tree(rng, x) for x in new] if kind == "tree" else None
        chosen = lists(rng, lens, new, hkv, page, k)
        if same:
            at = offsets(new)
            for s in range(len(new)):
                chosen[at[s]:at[s + 1]] = chosen[at[s]]
        out = run_pages(cache, q, new, chosen, parents)
        check_pages(cache, q, out, ks, vs, lens, new, chosen, D ** -0.5, parents, n)
        cache.work[tms.KV_WORK_ZERO:].fill_(0xff)
        assert torch.equal(out, run_pages(cache, q, new, chosen, parents))
        assert (cache.work[:tms.KV_WORK_ZERO] == 0).all()


def test_pages_of_sequences_too_long_for_their_pages_to_be_counted_together():
    """More than 32768 pages a sequence: tokens take workgroups of their own."""
    rng = np.random.default_rng(1)
    cache = tms.PagedCache.empty(1, 50, 2, 8, 64, 2, 40000, dtype=BF)
    cache.kv.copy_(torch.randn(cache.kv.shape, device="cuda"))
    table = cache.table
    lens, new = [8 * 39990, 100], [3, 5]
    table[0, :39995] = torch.from_numpy(rng.integers(0, 40, 39995).astype(np.int32)).cuda()
    table[1, :14] = torch.arange(36, 50, dtype=torch.int32, device="cuda")
    cache.length.copy_(dev32(lens))
    cache.held.copy_(dev32([39995, 14]))
    chosen = lists(rng, lens, new, 2, 8, 9)
    q = torch.from_numpy(rng.standard_normal((8, 4, 64)).astype(np.float32)).to(BF).cuda()
    out = run_pages(cache, q, new, chosen)
    kv = cache.kv[0].double().cpu().numpy()
    at = offsets(new)
    for s in range(2):
        rows = np.arange(lens[s] + new[s])
        pages = table[s].cpu().numpy()[rows // 8]
        ks, vs = kv[pages, 0, :, rows % 8], kv[pages, 1, :, rows % 8]
        check_pages(cache, q[at[s]:at[s + 1]], out[at[s]:at[s + 1]], [ks], [vs], [lens[s]], [new[s]], chosen[at[s]:at[s + 1]], 0.125, None, s)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_pages_values_that_are_not_finite_in_pages_that_other_drafts_chose(dtype):
    """In every split of the work."""
    rng = np.random.default_rng(14)
    lens, new, page, k = [8000], [7], 16, 40
    cache, ks, vs = filled(rng, dtype, 2, 64, page, lens, new)
    chosen = lists(rng, lens, new, 2, page, k)
    q = 0.1 * torch.from_numpy(rng.standard_normal((7, 4, 64)).astype(np.float32)).to(dtype).cuda()
    for t in range(7):
        for h in range(2):
            others = set(chosen[[u for u in range(7) if u != t], h].ravel().tolist())
            alone = [p for p in chosen[t, h] if p >= 0 and p not in others]
            if t % 2 and alone:
                p = alone[t % len(alone)]
                cache.kv[0, int(cache.table[0, p]), 1, h, 5, 9] = float("nan")
                vs[0][p * page + 5, h, 9] = np.nan
    out = run_pages(cache, q, new, chosen).double().cpu().numpy()
    for t in range(7):
        for h in range(2):
            rows = [r for p in chosen[t, h] if p >= 0 for r in range(p * page, (p + 1) * page)] + list(range(8000, 8001 + t))
            hit = np.isnan(vs[0][rows, h, 9]).any()
            got = out[t, 2 * h:2 * h + 2]
            assert np.isnan(got[:, 9]).all() == hit, (t, h)
            assert np.isfinite(np.delete(got, 9, 1)).all(), (t, h)


@pytest.mark.parametrize("k", [0, 3, 400])
def test_pages_leave_tokens_of_nobody(k):
    rng = np.random.default_rng(12)
    cache, _, _ = filled(rng, BF, 2, 64, 16, [8000, 20], [1, 1])
    q = torch.from_numpy(rng.standard_normal((5, 4, 64)).astype(np.float32)).to(BF).cuda()
    out = torch.full((5, 4, 64), 7.0, dtype=BF, device="cuda")
    chosen = dev32(lists(rng, [8000, 20, 0], [1, 1, 3], 2, 16, k))
    tms.kv_attention_pages(cache, 0, q, dev32([0, 1, 2]), chosen, out, max_new=1)
    assert (out[2:] == 7.0).all() and torch.isfinite(out[:2]).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_pages_rows_not_seen_may_hold_anything(dtype, kind):
    rng = np.random.default_rng(13)
    lens, new, page = [330], [6], 16
    cache, ks, vs = filled(rng, dtype, 2, 64, page, lens, new)
    for i, which, value in ((3, 1, float("inf")), (5, 0, float("nan")), (4, 1, float("nan"))):
        row = lens[0] + i
        cache.kv[0, int(cache.table[0, row // page]), which, :, row % page, 1] = value
        (ks if which == 0 else vs)[0][row, :, 1] = value
    unseen = int(cache.table[0, 7])
    cache.kv[0, unseen] = float("nan")  # a page that no token has chosen
    parents = [[-1, 0, 0, 1, 1, 2]] if kind == "tree" else None
    chosen = np.tile(np.array([0, 2, 6, 8, 19], np.int32), (6, 2, 1))
    q = torch.from_numpy(rng.standard_normal((6, 4, 64)).astype(np.float32)).to(dtype).cuda()
    out = run_pages(cache, q, new, chosen, parents).cpu()
    seen = {"causal": [set(range(i + 1)) for i in range(6)], "tree": [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 1, 4}, {0, 2, 5}]}[kind]
    for i in range(6):
        rest = torch.cat((out[i, :, :1], out[i, :, 2:]), -1)
        if 5 in seen[i]:
            assert torch.isnan(out[i]).all(), i
        else:
            assert torch.isfinite(rest).all(), i
            assert torch.isnan(out[i, :, 1]).all() if 4 in seen[i] else (out[i, :, 1] == float("inf")).all() if 3 in seen[i] \
                else torch.isfinite(out[i, :, 1]).all(), i


# ------------------------------------------------------------------ together

def test_a_step_over_long_contexts_replays_in_a_graph():
    """What a serving step does: fork, reserve, write, plan, shared attention in
    one layer and chosen pages in another, commit, bounds; recorded once and
    replayed, each replay against the same calls made eagerly."""
    def build():
        rng = np.random.default_rng(77)
        cache = tms.PagedCache.empty(2, 400, 2, 16, 64, 9, 60, dtype=BF)
        index, plan = tms.PageIndex(cache, tokens=40), tms.SharedPlan(cache, 40, 4)
        n = dev32([700] + [0] * 8)
        tms.kv_reserve(cache, n)
        for layer in range(2):
            x = torch.from_numpy(rng.standard_normal((700, 4, 64)).astype(np.float32)).to(BF).cuda()
            tms.kv_write(cache, layer, x[:, :2], x[:, 2:], dev32([0] + [700] * 9))
        tms.kv_commit(cache, n)
        tms.kv_bounds(cache, index)
        tms.kv_fork(cache, dev32([0] * 9))
        return cache, index, plan

    new = [0] + [3, 1, 5, 2, 4, 1, 1, 6]
    T = sum(new)
    rng = np.random.default_rng(78)
    steps = [torch.from_numpy(rng.standard_normal((2, T, 8, 64)).astype(np.float32)).to(BF).cuda() for _ in range(4)]
    x = steps[0].clone()
    n_new, start, n_keep = dev32(new), dev32(offsets(new)), dev32([0, 3, 1, 2, 1, 4, 1, 0, 5])
    chosen = torch.zeros((T, 2, 6), dtype=torch.int32, device="cuda")
    out = torch.zeros((2, T, 4, 64), dtype=BF, device="cuda")

    def step(cache, index, plan):
        tms.kv_reserve(cache, n_new, check=False)
        tms.kv_share(cache, plan, start, tokens=T)
        for layer in range(2):
            q, k, v = x[layer].split([4, 2, 2], 1)
            tms.kv_write(cache, layer, k, v, start)
            if layer == 0:
                tms.kv_attention_shared(cache, layer, q, start, out[layer], plan, max_new=6)
            else:
                tms.kv_select(cache, layer, q, start, index, chosen, max_new=6)
                tms.kv_attention_pages(cache, layer, q, start, chosen, out[layer], max_new=6)
        tms.kv_commit(cache, n_keep, check=False)
        tms.kv_bounds(cache, index, n_keep, max_new=6)

    eager, results = build(), []
    for i, s in enumerate(steps):
        x.copy_(s)
        step(*eager)
        results.append((out.clone(), chosen.clone()))
    torch.cuda.synchronize()
    assert (eager[0].status() == tms.OK).all()
    recorded = build()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step(*recorded)
    for i, s in enumerate(steps):
        x.copy_(s)
        torch.zeros(1000, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, results[i][0]) and torch.equal(chosen, results[i][1]), i
    assert torch.equal(recorded[0].length, eager[0].length) and torch.equal(recorded[1].bounds, eager[1].bounds)
    # every whole page has its bounds
    cache, index = recorded[0], recorded[1]
    for s in range(9):
        for p in cache.table[s, :int(cache.length[s]) // 16].long():
            keys = cache.kv[:, p, 0]
            assert torch.equal(index.bounds[:, p], torch.stack((keys.amin(2), keys.amax(2)), 2))


def test_binding_refusals_of_the_long_context_calls():
    rng = np.random.default_rng(1)
    cache, _, _ = filled(rng, BF, 2, 64, 16, [100, 200], [1, 1])
    start = dev32([0, 1, 2])
    q = torch.zeros((2, 4, 64), dtype=BF, device="cuda")
    out = torch.zeros_like(q)
    plan, index = tms.SharedPlan(cache, 2, 4), tms.PageIndex(cache, tokens=2)
    with pytest.raises(tms.TmsError):
        tms.SharedPlan(cache, 0, 4)
    with pytest.raises(tms.TmsError):
        tms.SharedPlan(cache, 2, 3)
    with pytest.raises(ValueError, match="heads"):
        tms.kv_attention_shared(cache, 0, q[:, :2], start, out, plan)
    with pytest.raises(tms.TmsError, match="plan_bytes"):
        tms.kv_share(cache, plan, start, tokens=20000)
    tms.kv_share(cache, plan, start)
    with pytest.raises(tms.TmsError, match="layer"):
        tms.kv_attention_shared(cache, 1, q, start, out, plan)
    with pytest.raises(TypeError):
        tms.kv_share(cache, plan, start.long())
    with pytest.raises(ValueError, match="bounds"):
        tms.PageIndex(cache, torch.zeros((1, 3), device="cuda"))
    with pytest.raises(TypeError):
        tms.PageIndex(cache, index.bounds.float())
    other, _, _ = filled(rng, BF, 2, 64, 16, [1000, 200], [1, 1])
    with pytest.raises(ValueError, match="other sizes"):
        tms.kv_bounds(other, index)
    with pytest.raises(ValueError, match="other sizes"):
        tms.kv_share(other, plan, start)
    chosen = torch.zeros((2, 2, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="other sizes"):
        tms.kv_select(other, 0, q, start, index, chosen)
    with pytest.raises(ValueError, match="chosen"):
        tms.kv_select(cache, 0, q, start, index, chosen[:1])
    with pytest.raises(ValueError, match="chosen"):
        tms.kv_attention_pages(cache, 0, q, start, chosen[:, :1], out)
    with pytest.raises(TypeError):
        tms.kv_attention_pages(cache, 0, q, start, chosen.long(), out)
    with pytest.raises(tms.TmsError, match="first"):
        tms.kv_select(cache, 0, q, start, index, chosen, first=-1)
    with pytest.raises(tms.TmsError, match="work"):
        tms.kv_select(cache, 0, torch.zeros((40000, 4, 64), dtype=BF, device="cuda"), start, index,
                      torch.zeros((40000, 2, 4), dtype=torch.int32, device="cuda"))
    with pytest.raises(tms.TmsError, match="k must"):
        tms.kv_select(cache, 0, q, start, index, torch.zeros((2, 2, 0), dtype=torch.int32, device="cuda"))


def test_shared_plans_older_than_the_tables_or_of_another_cache_are_refused():
    """A fork may leave every length as it was, so the library cannot see it."""
    rng = np.random.default_rng(30)
    b = Branches(rng, BF, 2, 64, 16, [((("p", 40),), 3, 1), ((("p", 40),), 3, 1), ((("q", 40),), 3, 1)])
    q = queries(rng, b, 4, 64, BF)
    start, out = dev32(offsets(b.new)), torch.zeros_like(q)
    plan = tms.SharedPlan(b.cache, 3, 4)
    zero = dev32([0, 0, 0])
    for change in (lambda: tms.kv_fork(b.cache, dev32([0, 1, 2])), lambda: tms.kv_reserve(b.cache, zero),
                   lambda: tms.kv_commit(b.cache, dev32([-1, -1, -1]))):
        tms.kv_share(b.cache, plan, start)
        tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=1)
        change()
        with pytest.raises(ValueError, match="before the cache's last"):
            tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=1)
    other = Branches(rng, BF, 2, 64, 16, [((("p", 40),), 3, 1), ((("p", 40),), 3, 1), ((("q", 40),), 3, 1)])
    tms.kv_share(other.cache, plan, start)
    with pytest.raises(ValueError, match="another cache"):
        tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=1)
    check_shared(other, q, run_shared(other, q, plan=plan), 0.125, None)


def test_pools_past_32_bits_a_later_layer_another_stream_and_strided_queries():
    """A pool of more than 2^32 elements a layer, pages at its end, bounds past 2^32
    bytes; queries inside a wider row."""
    rng = np.random.default_rng(31)
    hq, hkv, D, page, pages = 16, 8, 128, 8, 272000  # 4.5 G elements a layer of keys and values, four layers
    kv = torch.empty((4, pages, 2, hkv, page, D), dtype=BF, device="cuda")
    index_of = torch.empty((4, pages, hkv, 2, D), dtype=BF, device="cuda")
    assert kv[0].numel() > 2 ** 32 and index_of.numel() * 2 > 2 ** 32
    lens, new, common = [500, 497], [1, 2], 60
    table = np.full((2, 63), -1, np.int32)
    table[0] = [pages - 1 - i if i % 2 else i for i in range(63)]
    table[1] = table[0]
    table[1, common:] = [pages - 100, 100, pages - 101]
    refs = np.zeros(pages, np.int32)
    for p in table.reshape(-1):
        refs[p] += 1
    used = torch.from_numpy(np.unique(table)).long().cuda()
    kv[3, used] = torch.from_numpy(rng.standard_normal((len(used), 2, hkv, page, D)).astype(np.float32)).to(BF).cuda()
    cache = tms.PagedCache(kv, dev32(table), dev32(lens), dev32([63, 63]), dev32(refs), dev32([0, 0]))
    ks, vs = [], []
    for s in range(2):
        both = kv[3, torch.from_numpy(table[s]).long().cuda()].double().cpu().numpy().transpose(1, 0, 3, 2, 4).reshape(2, -1, hkv, D)
        ks.append(both[0, :lens[s] + new[s]])
        vs.append(both[1, :lens[s] + new[s]])
    wide = torch.from_numpy(rng.standard_normal((3, hq + 9, D)).astype(np.float32)).to(BF).cuda()
    q, start = wide[:, 5:5 + hq], dev32([0, 1, 3])
    index, plan = tms.PageIndex(cache, index_of, tokens=3), tms.SharedPlan(cache, 3, hq)
    chosen = torch.full((3, hkv, 6), 77, dtype=torch.int32, device="cuda")
    shared, paged = torch.zeros((2, 3, hq, D), dtype=BF, device="cuda").unbind(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tms.kv_bounds(cache, index, stream=side)
    tms.kv_share(cache, plan, start, stream=side)
    tms.kv_attention_shared(cache, 3, q, start, shared, plan, max_new=2, stream=side)
    tms.kv_select(cache, 3, q, start, index, chosen, max_new=2, stream=side)
    tms.kv_attention_pages(cache, 3, q, start, chosen, paged, max_new=2, stream=side)
    side.synchronize()
    x, lists_of, at = q.double().cpu().numpy(), chosen.cpu().numpy(), offsets(new)
    for s in range(2):
        whole = lens[s] // page
        bounds = np.stack([ks[s][:whole * page].reshape(whole, page, hkv, D).min(1),
                           ks[s][:whole * page].reshape(whole, page, hkv, D).max(1)], 2)  # [pages][heads][2][D]
        assert (index.bounds[3, torch.from_numpy(table[s, :whole]).long().cuda()].double().cpu().numpy() == bounds).all()
        for t in range(at[s], at[s + 1]):
            assert (lists_of[t] == choice(x[t], bounds, 6, 1.0, 1, 1)).all(), (s, t)
        want, bound = attention(x[at[s]:at[s + 1]], ks[s], vs[s], lens[s], D ** -0.5, None, True)
        assert (np.abs(shared[at[s]:at[s + 1]].double().cpu().numpy() - want) <= bound).all(), s
    check_pages(cache, q, paged, ks, vs, lens, new, lists_of, D ** -0.5, None)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(4096, 1, 64), (256, 256, 64)], **ids)
def test_the_most_heads(dtype, heads):
    hq, hkv, D = heads
    print(f"{dtype} {heads}", flush=True)
    rng = np.random.default_rng(hq)
    lens, new = [300, 77], [1, 1]
    cache, ks, vs = filled(rng, dtype, hkv, D, 16, lens, new)
    q = torch.from_numpy(rng.standard_normal((2, hq, D)).astype(np.float32)).to(dtype).cuda()
    index, start = tms.PageIndex(cache, tokens=2), dev32([0, 1, 2])
    tms.kv_bounds(cache, index)
    chosen = run_select(cache, index, q, new, 6)
    check_select(cache, index, q, lens, new, 6, chosen)
    check_pages(cache, q, run_pages(cache, q, new, chosen), ks, vs, lens, new, chosen, 0.125, None)
    plan, out = tms.SharedPlan(cache, 2, hq), torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    tms.kv_share(cache, plan, start)
    tms.kv_attention_shared(cache, 0, q, start, out, plan, max_new=1)
    x, out = q.double().cpu().numpy(), out.double().cpu().numpy()
    for s in range(2):
        want, bound = attention(x[s:s + 1], ks[s], vs[s], lens[s], 0.125, None, dtype == BF)
        assert (np.abs(out[s:s + 1] - want) <= bound).all(), s


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_the_most_sequences(dtype):
    """4096, of two prompts, most of them without a new token."""
    rng = np.random.default_rng(33)
    new = [0] * 4096
    for s in rng.permutation(4096)[:60]:
        new[s] = int(rng.integers(1, 4))
    new[0] = new[4095] = 1
    b = Branches(rng, dtype, 1, 64, 8, [(((f"p{s % 2}", 40),), s % 11, new[s]) for s in range(4096)])
    q = queries(rng, b, 2, 64, dtype)
    check_shared(b, q, run_shared(b, q), 0.125, None)
    index = tms.PageIndex(b.cache, tokens=sum(new))
    tms.kv_bounds(b.cache, index)
    chosen = run_select(b.cache, index, q, new, 7)
    check_select(b.cache, index, q, b.lens, new, 7, chosen)
    check_pages(b.cache, q, run_pages(b.cache, q, new, chosen), b.ks[0], b.vs[0], b.lens, new, chosen, 0.125, None)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_pages_longest_lists_of_the_widest_heads(dtype):
    """Lists and unions that take the most LDS, beside tiles that do: 8192 pages of a
    workgroup, and 2048 of several tokens."""
    rng = np.random.default_rng(34)
    print(f"{dtype} 8192 pages a list", flush=True)
    new, lens, page = [512], [8 * 8192 + 3], 8
    cache, ks, vs = filled(rng, dtype, 1, 256, page, lens, new)
    q = torch.from_numpy(rng.standard_normal((512, 16, 256)).astype(np.float32)).to(dtype).cuda()
    chosen = np.tile(np.arange(8192, dtype=np.int32), (512, 1, 1))
    out = run_pages(cache, q, new, chosen)
    for t in (0, 1, 300, 511):
        x = q[t:t + 1].double().cpu().numpy()
        k, v = ks[0][:lens[0] + t + 1], vs[0][:lens[0] + t + 1]
        want, bound = (attention_fine(x, k, v, len(k) - 1, 1 / 16, None) if dtype == BF else
                       attention(x, k, v, len(k) - 1, 1 / 16, None, False))
        assert (np.abs(out[t:t + 1].double().cpu().numpy() - want) <= bound).all(), t
    print(f"{dtype} 2048 pages of several tokens", flush=True)
    new, lens = [300, 300], [8 * 2010 + 1, 900]
    cache, ks, vs = filled(rng, dtype, 8, 256, page, lens, new)
    q = torch.from_numpy(rng.standard_normal((600, 8, 256)).astype(np.float32)).to(dtype).cuda()
    chosen = lists(rng, lens, new, 8, page, 150)
    check_pages(cache, q, run_pages(cache, q, new, chosen), ks, vs, lens, new, chosen, 1 / 16, None)


# ------------------------------------------------------------------ one prompt

class OnePrompt:
    """Sequences behind one prompt of whole pages, each with rows of its own and one
    new token, without a 64-bit copy of the prompt for each: `want` puts the rows
    of a sequence together where they are compared."""

    def __init__(self, rng, dtype, kv_heads, dim, page, prompt, own, layers=1):
        self.rows, self.page, seqs = prompt * page, page, len(own)
        self.lens = [self.rows + x for x in own]
        mine = [-(-(x + 1) // page) for x in own]
        total = prompt + sum(mine) + 1
        kv = torch.from_numpy(rng.standard_normal((layers, total, 2, kv_heads, page, dim)).astype(np.float32)).to(dtype)
        order = rng.permutation(total)
        table, refs, at = np.full((seqs, prompt + max(mine)), -1, np.int32), np.zeros(total, np.int32), prompt
        for s in range(seqs):
            table[s, :prompt] = order[:prompt]
            table[s, prompt:prompt + mine[s]] = order[at:at + mine[s]]
            at += mine[s]
            np.add.at(refs, table[s, :prompt + mine[s]], 1)
        self.kv, self.table = kv, table
        self.cache = tms.PagedCache(kv.cuda(), dev32(table), dev32(self.lens), dev32([prompt + m for m in mine]), dev32(refs),
                                    dev32([0] * seqs))
        self.new = [1] * seqs

    def check(self, q, out, of, layer=0, scale=None, fine=False):
        bf16, scale = q.dtype == BF, q.shape[2] ** -0.5 if scale is None else scale
        for s in of:
            n = self.lens[s] + 1
            both = self.kv[layer, self.table[s, :-(-n // self.page)].tolist()].double().numpy().transpose(1, 0, 3, 2, 4)
            both = both.reshape(2, -1, both.shape[3], both.shape[4])[:, :n]
            x = q[s:s + 1].double().cpu().numpy()
            want, bound = attention_fine(x, both[0], both[1], n - 1, scale, None) if bf16 and fine else \
                attention(x, both[0], both[1], n - 1, scale, None, bf16)
            err = np.abs(out[s:s + 1].double().cpu().numpy() - want)
            assert (err <= bound).all(), (s, n, float(np.nanmax(err / bound)), int((~(err <= bound)).sum()))


@pytest.mark.parametrize("dtype,heads,seqs,prompt", [
    (BF, (32, 32, 64), 16, 282), (F, (32, 32, 64), 16, 282), (BF, (32, 32, 128), 16, 288), (F, (32, 32, 256), 16, 192),
    (BF, (128, 64, 64), 8, 282), (BF, (40, 40, 64), 16, 700)], ids=lambda x: str(x).replace("torch.", ""))
def test_shared_plans_of_many_key_heads_and_few_rows_fit(dtype, heads, seqs, prompt):
    """Units of two key heads whose row tiles have 16 rows: the parts of a long prompt's
    chunks take twice the rows of one head's."""
    hq, hkv, D = heads
    print(f"{dtype} {heads} {seqs} sequences behind {prompt} pages", flush=True)
    rng = np.random.default_rng(prompt)
    b = OnePrompt(rng, dtype, hkv, D, 32, prompt, [20 + s % 3 for s in range(seqs)])
    q = queries(rng, b, hq, D, dtype)
    out = run_shared(b, q)
    assert torch.isfinite(out).all()
    b.check(q, out, (0, seqs // 2, seqs - 1))


@pytest.mark.parametrize("heads,seqs,prompt,own", [((8, 2, 256), 256, 40, 3), ((32, 8, 256), 64, 30, 40), ((2, 2, 256), 300, 25, 0)])
def test_shared_wide_heads_in_fp32_of_many_sequences(heads, seqs, prompt, own):
    """Row tiles of 16 for nodes of any size: the shared run is worked on a key head a
    unit, however many units there are."""
    hq, hkv, D = heads
    print(f"{heads} {seqs} sequences", flush=True)
    rng = np.random.default_rng(seqs)
    b = OnePrompt(rng, F, hkv, D, 16, prompt, [own + s % 2 for s in range(seqs)], layers=2)
    q = queries(rng, b, hq, D, F)
    out = run_shared(b, q, layer=1)
    assert torch.equal(out, run_shared(b, q, layer=1))
    b.check(q, out, range(0, seqs, 5), layer=1)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads,new", [((4, 2, 64), [1, 1, 1]), ((40, 2, 128), [2, 1, 3]), ((8, 1, 256), [1, 0, 1])], ids=["one", "wide", "256"])
@pytest.mark.parametrize("k", [4, 37, 200])
def test_pages_wrong_lists_of_tokens_that_are_alone_in_a_workgroup(dtype, heads, new, k):
    """Entries that are out of order, equal, out of range or behind a negative one, in
    every part of a list: NaN for their token and head, and nothing changes for the
    others."""
    hq, hkv, D = heads
    print(f"{dtype} {heads} {k}", flush=True)
    rng = np.random.default_rng(k)
    lens, page = [16 * 300 + 5, 700, 16 * 260], 16
    cache, ks, vs = filled(rng, dtype, hkv, D, page, lens, new)
    q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
    good = lists(rng, lens, new, hkv, page, k)
    t, h = sum(new) - 1, hkv - 1  # of the last sequence, which has 260 whole pages
    good[t, h] = np.arange(k)
    right = run_pages(cache, q, new, good)
    check_pages(cache, q, right, ks, vs, lens, new, good, D ** -0.5, None)
    mine = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    mine[t, h * hq // hkv:(h + 1) * hq // hkv] = True
    for at in sorted({1, 2, k // 3, k // 2, k - 2, k - 1} - {0}):
        for entry in (at - 1, max(at - 2, 0), 259 if at < k - 1 else 260, 300, 2 ** 31 - 1, -1, -2 ** 31):
            wrong = good.copy()
            wrong[t, h, at] = entry
            if entry < 0 and at == k - 1:  # the list ends there
                continue
            out = run_pages(cache, q, new, wrong)
            assert torch.isnan(out[mine]).all(), (at, entry)
            assert torch.equal(out[~mine], right[~mine]), (at, entry)
    for first in (260, -1, 2 ** 31 - 1):  # the first entry
        wrong = good.copy()
        wrong[t, h, 0] = first
        out = run_pages(cache, q, new, wrong)
        assert torch.isnan(out[mine]).all() and torch.equal(out[~mine], right[~mine]), first
    assert (cache.work[:tms.KV_WORK_ZERO] == 0).all()


@pytest.mark.parametrize("heads", [(8, 2, 64), (16, 4, 128), (8, 2, 256)], **ids)
@pytest.mark.parametrize("seqs,kind", [(64, "token"), (24, "tree")])
def test_shared_weights_keep_16_bits_however_many_rows_share_a_run(heads, seqs, kind):
    """Runs of more than 64 query rows of a key head, whose weights are those of single
    tokens: what a token gets does not depend on how many others share its prompt.
    A peaked softmax: weights of 8 bits are off by 1.1 to 3.7 of the bound."""
    hq, hkv, D = heads
    rng = np.random.default_rng(seqs + D)
    b = Branches(rng, BF, hkv, D, 16, [((("p", 20),), s % 7, 1 if kind == "token" else 5 + s % 3) for s in range(seqs)])
    q = 2 * queries(rng, b, hq, D, BF)
    parents = [tree(rng, n) for n in b.new] if kind == "tree" else None
    out, at = run_shared(b, q, parents).double().cpu().numpy(), offsets(b.new)
    x = q.double().cpu().numpy()
    for s in range(seqs):
        want, bound = attention_fine(x[at[s]:at[s + 1]], b.ks[0][s], b.vs[0][s], b.lens[s], D ** -0.5, None if parents is None else parents[s])
        err = np.abs(out[at[s]:at[s + 1]] - want)
        assert (err <= bound).all(), (s, float((err / bound).max()), int((err > bound).sum()))


def test_an_index_of_another_cache_is_refused():
    """Of the same sizes too: its bounds would be of other keys."""
    rng = np.random.default_rng(40)
    cache, _, _ = filled(rng, BF, 2, 64, 16, [100, 200], [1, 1])
    other, _, _ = filled(rng, BF, 2, 64, 16, [100, 200], [1, 1])
    index, start = tms.PageIndex(cache, tokens=2), dev32([0, 1, 2])
    tms.kv_bounds(cache, index)
    before = index.bounds.clone()
    q = torch.zeros((2, 4, 64), dtype=BF, device="cuda")
    chosen = torch.full((2, 2, 4), 77, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="another cache"):
        tms.kv_select(other, 0, q, start, index, chosen, max_new=1)
    with pytest.raises(ValueError, match="another cache"):
        tms.kv_bounds(other, index)
    assert (chosen == 77).all() and torch.equal(index.bounds, before)
    # the same tensors in a cache made anew are the same keys
    again = tms.PagedCache(cache.kv, cache.table, cache.length, cache.held, cache.refs, cache.status_codes)
    tms.kv_select(again, 0, q, start, index, chosen, max_new=1)
    assert (chosen >= 0).all()
    # bounds that were kept may be given to an index for the cache that they are of
    del other
    tms.kv_select(cache, 0, q, start, tms.PageIndex(cache, before, tokens=2), chosen, max_new=1)
    assert (chosen >= 0).all()


def test_shared_plans_of_tokens_that_two_sequences_claim_give_nan():
    """And leave the plan's memory good for the next plan."""
    rng = np.random.default_rng(41)
    b = Branches(rng, BF, 2, 64, 16, [((("p", 40),), 0, 4)] * 4)
    q = queries(rng, b, 4, 64, BF)
    held = b.cache.held.clone()
    b.cache.held.fill_(44)
    plan = tms.SharedPlan(b.cache, 16, 4)
    for bad in ([0, 10, 4, 14, 16], [0, 16, 0, 16, 16], [0, 9, 8, 16, 16]):
        out, start = torch.full(q.shape, 7.0, dtype=BF, device="cuda"), dev32(bad)
        tms.kv_share(b.cache, plan, start)
        tms.kv_attention_shared(b.cache, 0, q, start, out, plan, max_new=16)
        assert torch.isnan(out).all(), bad
    b.cache.held.copy_(held)
    start = dev32(offsets(b.new))
    tms.kv_share(b.cache, plan, start)
    check_shared(b, q, run_shared(b, q, plan=plan), 0.125, None)
