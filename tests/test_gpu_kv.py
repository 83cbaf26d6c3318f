"""The paged key/value cache on the GPU against plain 64-bit forms
(kv_util.py, which also derives the bounds): attention of single tokens, trees
of drafts and prompts, cache writes, page operations, and their refusals."""
import numpy as np
import pytest
import torch

import trie_masked_sparse_amd as tms
from kv_util import Pages, attention, head
from kv_util import attention_fine, marked_values

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def dev32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def tree(rng, n, back=5):
    return [-1 if i == 0 or rng.random() < 0.1 else int(rng.integers(max(0, i - back), i)) for i in range(n)]


def filled(rng, dtype, kv_heads, dim, page, lens, new, layers=1, layer=0, spare=2, fill=float("nan")):
    """A cache whose sequences hold lens committed and new further rows of
    normal values, in pages of random order; every other value is `fill`.
    Returns (cache, [k of every sequence], [v ...]) in fp64."""
    need = [-(-(a + b) // page) for a, b in zip(lens, new)]
    total, width = sum(need) + spare, max(max(need), 1)
    order = list(rng.permutation(total))
    kv = torch.full((layers, total, 2, kv_heads, page, dim), fill, dtype=dtype)
    table, refs = np.full((len(lens), width), -1, np.int32), np.zeros(total, np.int32)
    ks, vs = [], []
    for s, (a, b) in enumerate(zip(lens, new)):
        both = torch.from_numpy(rng.standard_normal((2, kv_heads, a + b, dim)).astype(np.float32)).to(dtype)
        for j in range(need[s]):
            p = int(order.pop())
            table[s, j], refs[p] = p, 1
            rows = both[:, :, j * page:(j + 1) * page]
            kv[layer, p, :, :, :rows.shape[2]] = rows
        ks.append(both[0].transpose(0, 1).double().numpy())
        vs.append(both[1].transpose(0, 1).double().numpy())
    cache = tms.PagedCache(kv.cuda(), dev32(table), dev32(lens), dev32(need), dev32(refs), dev32([0] * len(lens)))
    return cache, ks, vs


def run_attention(cache, q, new, parents=None, max_new=None, scale=None, layer=0, stream=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    par = None if parents is None else dev32([p for t in parents for p in t])
    tms.kv_attention(cache, layer, q, dev32(offsets(new)), out, scale, parent=par,
                     max_new=max_new or max(max(new), 1), stream=stream)
    return out


def check_attention(q, out, ks, vs, lens, new, scale, parents, bf16, where=""):
    q, out = q.double().cpu().numpy(), out.double().cpu().numpy()
    at = offsets(new)
    for s, (a, b) in enumerate(zip(lens, new)):
        if b:
            want, bound = attention(q[at[s]:at[s + 1]], ks[s], vs[s], a, scale, None if parents is None else parents[s],
                                    bf16)
            err = np.abs(out[at[s]:at[s + 1]] - want)
            assert (err <= bound).all(), (where, s, a, b, float(np.nanmax(err / bound)), int((~(err <= bound)).sum()))


SHAPES = [
    # lens, new
    ([0], [1]), ([1], [1]), ([63], [1]), ([64], [1]), ([517], [1]),
    ([0, 1, 0, 130], [0, 1, 3, 2]), ([33, 0, 700, 15, 16, 17], [5, 31, 1, 0, 13, 64]),
    ([2000, 3], [63, 100]), ([0, 90], [257, 129]),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 8, 128), (8, 1, 128), (3, 3, 64), (10, 2, 256)],
                         ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_attention_matches_the_64_bit_form(dtype, heads, kind):
    hq, hkv, D = heads
    for n, (lens, new) in enumerate(SHAPES):
        page = [16, 64, 8, 128][n % 4]
        print(f"attention {dtype} {heads} {kind} lens {lens} new {new} page {page}", flush=True)
        rng = np.random.default_rng(100 * n + D + hq)
        # rows past the end of a sequence and pages of nobody hold NaN
        cache, ks, vs = filled(rng, dtype, hkv, D, page, lens, new, layers=2, layer=1)
        q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
        parents = [tree(rng, b) for b in new] if kind == "tree" else None
        out = run_attention(cache, q, new, parents, layer=1)
        check_attention(q, out, ks, vs, lens, new, D ** -0.5, parents, dtype == BF, (n, kind))
        assert (cache.status() == tms.OK).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_attention_many_sequences_and_long_contexts(dtype):
    """Work split over the context: many ragged sequences, and one long one."""
    rng = np.random.default_rng(5)
    for lens, new in (([int(x) for x in rng.integers(0, 900, 70)], [int(x) for x in rng.integers(0, 4, 70)]),
                      ([20011], [1]), ([9001, 0, 12], [37, 2, 20])):
        print(f"attention long {dtype} {len(lens)} sequences, longest {max(lens)}", flush=True)
        cache, ks, vs = filled(rng, dtype, 2, 128, 32, lens, new)
        q = torch.from_numpy(rng.standard_normal((sum(new), 8, 128)).astype(np.float32)).to(dtype).cuda()
        for parents in (None, [tree(rng, b) for b in new]):
            out = run_attention(cache, q, new, parents)
            check_attention(q, out, ks, vs, lens, new, 128 ** -0.5, parents, dtype == BF)
            again = run_attention(cache, q, new, parents)
            assert torch.equal(out, again)  # no order depends on timing


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_attention_scores_far_apart(dtype):
    """Scores of several thousand, positive and negative, infinities in the
    keys of rows nobody sees, negative and zero scale."""
    rng = np.random.default_rng(11)
    lens, new = [100, 5], [6, 9]
    for scale in (8.0, -3.0, 0.0):
        cache, ks, vs = filled(rng, dtype, 2, 64, 16, lens, new, fill=float("inf"))
        q = torch.from_numpy(20 * rng.standard_normal((sum(new), 4, 64)).astype(np.float32)).to(dtype).cuda()
        parents = [tree(rng, b) for b in new]
        for p in (None, parents):
            out = run_attention(cache, q, new, p, scale=scale)
            assert torch.isfinite(out.float()).all()
            check_attention(q, out, ks, vs, lens, new, scale, p, dtype == BF, scale)


BATCHES = [
    # heads of queries, of keys, head_dim, committed rows, new rows, trees; what is taken by it
    (8, 2, 64, [100, 0, 7], [700, 333, 1], False),        # causal row tiles in pairs, an odd count of them
    (4, 1, 128, [1000, 0], [257, 600], False),
    (4, 2, 256, [64, 9], [400, 130], False),
    (2, 2, 256, [0], [40], False),
    (8, 8, 64, [3] * 20, [210] * 20, False),              # whole segments: fp32
    (128, 16, 64, [10], [1100], False),                   # whole segments of 256 rows
    (32, 8, 64, [0, 5] * 32, [70, 64] * 32, False),       # short prompts
    (8, 4, 256, [0, 5] * 32, [70, 64] * 32, False),
    (5, 5, 128, [50, 0], [20, 32], False),                # 17 .. 32 rows
    (6, 2, 128, [50, 900], [20, 1], False),               # 33 .. 64 rows, of three heads
    (6, 2, 64, [50, 0], [30, 42], False),                 # 65 .. 128 rows
    (5, 5, 128, [50, 0], [20, 32], True),
    (6, 2, 128, [50, 900], [20, 1], True),
    (6, 2, 64, [31, 0], [30, 42], True),
    (2, 2, 64, [33, 500], [600, 513], True),              # more drafts than one row of the table
    (2, 2, 128, [95], [1024], True),
    (2, 2, 128, [95], [512], True),
    (4, 2, 64, [31, 0], [1024, 700], True),
    (4, 2, 256, [31, 200], [80, 300], True),
    (2, 1, 64, [9, 0, 40] * 200, [1, 2, 0] * 200, False),  # several sequences to a thread of the plan
    (2, 1, 64, [9, 0, 40] * 400, [20, 3, 0] * 400, True),
    (4, 2, 64, [20000], [18], True),                      # many parts of few segments
    (8, 1, 128, [15000, 300], [30, 2], True),
    (4, 2, 64, [30000, 17], [2, 1], True),
    (8, 2, 256, [9000], [1], False),
    (2, 1, 256, [9000, 0], [60, 3], False),
    (16, 8, 64, [20000] + [0] * 40, [100] * 41, False),   # one context much longer than the others
    (8, 4, 128, [0, 9000, 3], [900, 30, 700], False),
    (4, 4, 64, [0] * 7 + [12000], [300] * 8, False),
    (16, 8, 128, [0, 700, 3000, 40] * 12, [10, 20, 9, 32] * 12, True),  # parts joined by the last workgroup
    (8, 8, 64, [0, 700, 3000, 40] * 12, [10, 20, 9, 32] * 12, False),
    (8, 4, 256, [0, 700, 3000, 40] * 20, [10, 20, 9, 32] * 20, True),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(BATCHES)))
def test_attention_of_every_kind_of_batch(dtype, case):
    hq, hkv, D, lens, new, trees = BATCHES[case]
    print(f"attention {dtype} {BATCHES[case][:3]} {len(new)} sequences, new <= {max(new)}, trees {trees}", flush=True)
    rng = np.random.default_rng(300 + case)
    cache, ks, vs = filled(rng, dtype, hkv, D, 32, lens, new)
    q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
    parents = [tree(rng, b) for b in new] if trees else None
    for _ in range(2):  # the counters in the work memory are zero again after a call
        out = run_attention(cache, q, new, parents)
        check_attention(q, out, ks, vs, lens, new, D ** -0.5, parents, dtype == BF, case)
        assert not cache.work[:2048].any()


LONG = [
    (8, 2, 64, [20000, 3], [1, 1], False),
    (16, 1, 128, [20000], [1], False),
    (8, 4, 128, [30000], [8], True),                      # 17 .. 64 rows, many parts
    (4, 1, 256, [30000, 100], [16, 2], False),
    (8, 1, 64, [30000], [16], True),                      # 65 .. 128
    (8, 1, 128, [20000, 0, 500], [63, 5, 1], True),       # over 128
    (4, 2, 256, [20000], [80], True),
    (2, 2, 128, [20000], [600], True),
    (16, 8, 128, [4096] * 40, [1] * 40, False),
    (16, 8, 128, [2048, 2000, 63, 0] * 12, [9, 20, 31, 5] * 12, True),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(LONG) + len(BATCHES)))
def test_attention_counts_every_key_once(dtype, case):
    """Values that tell the blocks of 16 keys apart: no tile, share or part is
    left out or counted twice, however small its part of the whole."""
    hq, hkv, D, lens, new, trees = (LONG + BATCHES)[case]
    print(f"attention marked {dtype} {hq, hkv, D} {len(new)} sequences, longest {max(lens)}, trees {trees}", flush=True)
    rng = np.random.default_rng(800 + case)
    cache, ks, vs = filled(rng, dtype, hkv, D, 32, lens, new)
    for s, (a, b) in enumerate(zip(lens, new)):
        if a + b == 0:
            continue
        vs[s] = marked_values(a + b, hkv, D)
        values = torch.zeros((-(-(a + b) // 32) * 32, hkv, D))
        values[:a + b] = torch.from_numpy(vs[s]).float()
        pages = cache.table[s, :len(values) // 32].long()
        cache.kv[0, pages, 1] = values.unflatten(0, (-1, 32)).transpose(1, 2).to(dtype).cuda()
    q = torch.from_numpy(0.7 * rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
    parents = [tree(rng, b) for b in new] if trees else None
    check_attention(q, run_attention(cache, q, new, parents), ks, vs, lens, new, D ** -0.5, parents, dtype == BF, case)


@pytest.mark.parametrize("heads", [(4, 4, 64), (16, 8, 128), (8, 1, 128), (10, 2, 256), (8, 2, 64)],
                         ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_attention_weights_of_up_to_64_rows_keep_16_bits(heads, kind):
    """Outputs near 0 beside values of 1: no more than the rounding of the output
    and 2^-15 of each weight."""
    hq, hkv, D = heads
    most = 64 // (hq // hkv)
    for n, (lens, new) in enumerate((([60], [1]), ([700, 0, 90], [1, 1, 1]), ([5, 333], [most // 4, most // 8]), ([4000], [most]),
                                     ([100, 60, 1000], [most // 2, 1, most]), ([9000], [most // 4]))):
        print(f"attention 16 bits {heads} {kind} lens {lens} new {new}", flush=True)
        rng = np.random.default_rng(900 + n)
        cache, ks, vs = filled(rng, BF, hkv, D, 16, lens, new)
        q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(BF).cuda()
        parents = [tree(rng, b) for b in new] if kind == "tree" else None
        out, qd, at = run_attention(cache, q, new, parents).double().cpu().numpy(), q.double().cpu().numpy(), offsets(new)
        for s, (a, b) in enumerate(zip(lens, new)):
            want, bound = attention_fine(qd[at[s]:at[s + 1]], ks[s], vs[s], a, D ** -0.5, parents and parents[s])
            err = np.abs(out[at[s]:at[s + 1]] - want)
            assert (err <= bound).all(), (n, s, float((err / bound).max()))


def test_the_work_memory_behind_its_counters_may_hold_anything():
    """Only the counters have to be zero, and are zero again after every call."""
    cache = tms.PagedCache.empty(1, 4, 2, 16, 256, 1, 4)
    assert not cache.work[:tms.KV_WORK_ZERO].any()
    for case in (0, 5, 7, 12, 21, 22, 24, 26, 29, 31):
        hq, hkv, D, lens, new, trees = BATCHES[case]
        for dtype in (BF, F):
            print(f"work memory {dtype} {BATCHES[case][:3]} {len(new)} sequences", flush=True)
            rng = np.random.default_rng(700 + case)
            cache, ks, vs = filled(rng, dtype, hkv, D, 32, lens, new)
            q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
            parents = [tree(rng, b) for b in new] if trees else None
            want = run_attention(cache, q, new, parents)
            for byte in (0xff, 0x7f):
                cache.work[tms.KV_WORK_ZERO:] = byte
                assert torch.equal(run_attention(cache, q, new, parents), want)
                assert not cache.work[:tms.KV_WORK_ZERO].any()
            cache.work[tms.KV_WORK_ZERO:] = 0xff
            src, n_keep = list(range(len(new))), [min(b, 1) for b in new]
            src[0] = len(new) - 1
            tms.kv_fork(cache, dev32(src), check=False)
            cache.work[tms.KV_WORK_ZERO:] = 0xff
            tms.kv_reserve(cache, dev32([1] * len(new)), check=False)
            tms.kv_commit(cache, dev32(n_keep), check=False)
            assert all(x in (tms.OK, tms.ERR_OOM) for x in cache.status().tolist())
            held = torch.bincount(cache.table[cache.table >= 0].long(), minlength=cache.pages)
            assert torch.equal(held.int(), cache.refs) and not cache.work[:tms.KV_WORK_ZERO].any()


def set_row(cache, s, row, which, column, value):
    page = cache.kv.shape[4]
    cache.kv[0, int(cache.table[s, row // page]), which, :, row % page, column] = value


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (4, 2, 128), (8, 2, 256)], ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_attention_rows_not_seen_may_hold_anything(dtype, heads, kind):
    """Infinities and NaN in a draft's or a later token's key and value reach the
    rows that see it, in its columns, and no others."""
    hq, hkv, D = heads
    for n, (lens, new) in enumerate((([50], [7]), ([3000], [8]), ([33, 40], [25, 3]), ([1000, 64], [70, 33]), ([31], [150]),
                                     ([700, 20], [300, 5]), ([0, 700, 2500, 40] * 30, [10, 20, 9, 32] * 30))):
        print(f"attention not finite {dtype} {heads} {kind} lens {lens} new {new}", flush=True)
        rng = np.random.default_rng(400 + n)
        cache, ks, vs = filled(rng, dtype, hkv, D, 16, lens, new)
        parents = [tree(rng, b) for b in new] if kind == "tree" else None
        for s, (a, b) in enumerate(zip(lens, new)):
            for row, which, column, value in ((a + b // 2, 1, 3, np.inf), (a + b // 2 + 1, 1, 21, -np.inf),
                                              (a + b - 1, 1, 5, np.nan), (a + b - 2, 0, 7, np.nan)):
                set_row(cache, s, row, which, column, value)
                (vs if which else ks)[s][row, :, column] = value
        q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
        out = run_attention(cache, q, new, parents).double().cpu().numpy()
        qd, at = q.double().cpu().numpy(), offsets(new)
        for s, (a, b) in enumerate(zip(lens, new)):
            want, bound = attention(qd[at[s]:at[s + 1]], ks[s], vs[s], a, D ** -0.5, parents and parents[s], dtype == BF)
            got, fine = out[at[s]:at[s + 1]], np.isfinite(want)
            assert fine.any() and not fine.all()
            assert (np.abs(got[fine] - want[fine]) <= bound[fine]).all(), (n, s)
            assert np.array_equal(got[~fine], want[~fine], equal_nan=True), (n, s)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (4, 2, 128), (8, 2, 256), (32, 1, 128)], ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_attention_a_last_token_whose_value_is_not_finite(dtype, heads, kind):
    """The last row of a sequence fills its key tile up: infinities of its own
    value stay infinities in its columns, also where it is the only new token
    or alone in its row tile."""
    hq, hkv, D = heads
    group = hq // hkv
    for n, (lens, new) in enumerate((([0], [1]), ([40], [1]), ([63], [1]), ([5, 700, 31, 2000], [1, 1, 1, 1]), ([9000], [1]),
                                     ([33, 3], [256 // group + 1, 1]), ([100], [2]), ([17], [64 // group + 1]))):
        for most in (None, 200):  # also by the kernels for more rows
            print(f"attention last value not finite {dtype} {heads} {kind} lens {lens} new {new} max_new {most}", flush=True)
            rng = np.random.default_rng(500 + n)
            cache, ks, vs = filled(rng, dtype, hkv, D, 16, lens, new)
            # every draft follows the context itself: nobody else sees the last one
            parents = [[-1] * b for b in new] if kind == "tree" else None
            for s, (a, b) in enumerate(zip(lens, new)):
                for column, value in ((3, np.inf), (21, -np.inf), (5, np.nan), (D - 1, np.inf)):
                    set_row(cache, s, a + b - 1, 1, column, value)
                    vs[s][a + b - 1, :, column] = value
            q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype).cuda()
            out = run_attention(cache, q, new, parents, max_new=most and max(most, max(new))).double().cpu().numpy()
            qd, at = q.double().cpu().numpy(), offsets(new)
            for s, (a, b) in enumerate(zip(lens, new)):
                want, bound = attention(qd[at[s]:at[s + 1]], ks[s], vs[s], a, D ** -0.5, parents and parents[s], dtype == BF)
                got, fine = out[at[s]:at[s + 1]], np.isfinite(want)
                assert np.isposinf(want).any() and np.isneginf(want).any() and np.isnan(want).any()
                assert (np.abs(got[fine] - want[fine]) <= bound[fine]).all(), (n, s)
                assert np.array_equal(got[~fine], want[~fine], equal_nan=True), (n, s)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (4, 2, 128), (8, 2, 256), (8, 1, 64)], ids=lambda h: "x".join(map(str, h)))
def test_attention_an_infinite_value_behind_a_part_of_little_weight(dtype, heads):
    """A draft's infinite value whose weight, and that of every key worked on
    with it, is below what fp32 holds: the sum is infinite all the same."""
    hq, hkv, D = heads
    for n, (lens, new) in enumerate((([40], [1]), ([500], [3]), ([9000], [2]), ([3000, 70], [20, 9]), ([2000], [70]))):
        print(f"attention infinite value of little weight {dtype} {heads} lens {lens} new {new}", flush=True)
        rng = np.random.default_rng(600 + n)
        cache, ks, vs = filled(rng, dtype, hkv, D, 16, lens, new)
        q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype)
        q[:, :, 0] = 64.0
        for s, (a, b) in enumerate(zip(lens, new)):
            for row in range(a + b):  # scores of the first row lead those of all later ones by hundreds
                set_row(cache, s, row, 0, 0, 0.0 if row == 0 else -64.0)
                ks[s][row, :, 0] = 0.0 if row == 0 else -64.0
            set_row(cache, s, a + b - 1, 1, 7, np.inf)
            vs[s][a + b - 1, :, 7] = np.inf
        out = run_attention(cache, q.cuda(), new).double().cpu().numpy()
        at = offsets(new)
        for s, (a, b) in enumerate(zip(lens, new)):
            last = out[at[s + 1] - 1]
            assert np.isposinf(last[:, 7]).all(), (n, s, last[:, 7])
            others = np.delete(out[at[s]:at[s + 1]], 7, 2)
            want = np.repeat(np.delete(vs[s][0], 7, 1), hq // hkv, 0)[None]  # the first row has all the weight
            assert (np.abs(others - want) <= (2.0 ** -8 if dtype == BF else 2.0 ** -18) * np.abs(want) + 2.0 ** -100).all(), (n, s)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (4, 2, 128), (8, 2, 256), (8, 1, 64)], ids=lambda h: "x".join(map(str, h)))
def test_attention_infinite_values_of_committed_rows(dtype, heads):
    """All tokens see them: infinite in their columns, NaN where both signs are."""
    hq, hkv, D = heads
    for n, (lens, new) in enumerate((([40], [1]), ([70, 3, 20], [1, 1, 1]), ([3000, 70], [6, 9]), ([9000], [2]), ([500], [30]),
                                     ([333, 2000], [90, 3]), ([700], [400]))):
        for rows_alike in (False, True):
            print(f"attention infinite committed {dtype} {heads} lens {lens} new {new}", flush=True)
            rng = np.random.default_rng(1000 + n)
            cache, ks, vs = filled(rng, dtype, hkv, D, 16, lens, new)
            q = torch.from_numpy(rng.standard_normal((sum(new), hq, D)).astype(np.float32)).to(dtype)
            if rows_alike:  # weights that are powers of two: nothing is left of them in fewer bits
                q.zero_()
            for s, a in enumerate(lens):
                for row, column, value in ((0, 3, np.inf), (a - 1, 21, -np.inf), (a // 2, 5, np.inf), (a // 3, 5, -np.inf),
                                           (a // 2, D - 1, np.inf), (a - 1, D - 1, np.inf), (1, 9, np.nan)):
                    set_row(cache, s, row, 1, column, value)
                    vs[s][row, :, column] = value
            out = run_attention(cache, q.cuda(), new).double().cpu().numpy()
            qd, at = q.double().numpy(), offsets(new)
            for s, (a, b) in enumerate(zip(lens, new)):
                want, bound = attention(qd[at[s]:at[s + 1]], ks[s], vs[s], a, D ** -0.5, None, dtype == BF)
                got, fine = out[at[s]:at[s + 1]], np.isfinite(want)
                assert np.isposinf(want[:, :, [3, D - 1]]).all() and np.isneginf(want[:, :, 21]).all()
                assert (np.abs(got[fine] - want[fine]) <= bound[fine]).all(), (n, s)
                assert np.array_equal(got[~fine], want[~fine], equal_nan=True), (n, s)


def test_attention_parents_that_are_not_earlier_tokens_count_as_none():
    rng = np.random.default_rng(12)
    lens, new = [20], [6]
    cache, ks, vs = filled(rng, BF, 2, 64, 16, lens, new)
    q = torch.from_numpy(rng.standard_normal((6, 4, 64)).astype(np.float32)).to(BF).cuda()
    odd = [[-5, 0, 2, 9, 3, 2 ** 31 - 1]]
    out = run_attention(cache, q, new, odd)
    check_attention(q, out, ks, vs, lens, new, 64 ** -0.5, [[-1, 0, -1, -1, 3, -1]], True)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_attention_strided_queries_and_another_stream(dtype):
    rng = np.random.default_rng(13)
    lens, new = [40, 300], [3, 1]
    cache, ks, vs = filled(rng, dtype, 2, 128, 64, lens, new)
    wide = torch.from_numpy(rng.standard_normal((4, 11, 128)).astype(np.float32)).to(dtype).cuda()
    q = wide[:, 2:10]
    assert not q.is_contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty((4, 8, 128), dtype=dtype, device="cuda")
    start = dev32(offsets(new))
    side.wait_stream(torch.cuda.current_stream())
    tms.kv_attention(cache, 0, q, start, out, max_new=3, stream=side)
    side.synchronize()
    check_attention(q, out, ks, vs, lens, new, 128 ** -0.5, None, dtype == BF)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_attention_sequences_in_error_give_nan(dtype):
    rng = np.random.default_rng(14)
    lens, new = [10, 20, 30, 40], [2, 3, 2, 2]
    cache, ks, vs = filled(rng, dtype, 2, 64, 16, lens, new)
    cache.status_codes[0] = tms.ERR_OOM
    cache.held[2] = 1  # 16 rows held, 32 needed
    q = torch.from_numpy(rng.standard_normal((sum(new), 4, 64)).astype(np.float32)).to(dtype).cuda()
    out = run_attention(cache, q, new, max_new=2)  # sequence 1 has more than max_new tokens
    assert torch.isnan(out[:7].float()).all()
    check_attention(q[7:], out[7:], ks[3:], vs[3:], lens[3:], new[3:], 64 ** -0.5, None, dtype == BF)


def test_one_token_of_a_projection_whose_width_is_odd():
    """With one token there is no next row: the distance to it says nothing."""
    rng = np.random.default_rng(18)
    cache, ks, vs = filled(rng, BF, 2, 64, 16, [20], [1])
    wide = torch.from_numpy(rng.standard_normal((1, 8 * 64 + 3)).astype(np.float32)).to(BF).cuda()
    q, k, v = (wide.as_strided((1, b - a, 64), (wide.shape[1], 64, 1), a * 64) for a, b in ((0, 4), (4, 6), (6, 8)))
    assert q.stride(0) % 8
    out, q_out = torch.zeros((1, 4, 64), dtype=BF, device="cuda"), torch.zeros((1, 4, 64), dtype=BF, device="cuda")
    tms.kv_write(cache, 0, k, v, dev32([0, 1]), q=q, q_out=q_out)
    assert (cache.status() == tms.OK).all() and torch.equal(q_out, q)
    tms.kv_attention(cache, 0, q, dev32([0, 1]), out, max_new=1)
    ks[0][20], vs[0][20] = k[0].double().cpu().numpy(), v[0].double().cpu().numpy()
    check_attention(q, out, ks, vs, [20], [1], 64 ** -0.5, None, True)


def test_attention_max_new_of_a_batch_of_trees():
    """The limit of 1024 drafts is a tree's, not the batch's: without max_new,
    on another stream too, and with a max_new above all tokens there are."""
    rng = np.random.default_rng(17)
    lens, new = [int(x) for x in rng.integers(0, 200, 64)], [31] * 63 + [3]
    cache, ks, vs = filled(rng, BF, 2, 64, 16, lens, new)
    q = torch.from_numpy(rng.standard_normal((sum(new), 4, 64)).astype(np.float32)).to(BF).cuda()
    parents = [tree(rng, b) for b in new]
    start, parent, side = dev32(offsets(new)), dev32([p for t in parents for p in t]), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for max_new, stream in ((None, None), (None, side), (31, None)):
        out = torch.zeros_like(q)
        side.wait_stream(torch.cuda.current_stream())
        tms.kv_attention(cache, 0, q, start, out, parent=parent, max_new=max_new, stream=stream)
        side.synchronize()
        check_attention(q, out, ks, vs, lens, new, 64 ** -0.5, parents, True)
    few, n = dev32([0, 31, 62] + [62] * 62), 62
    out = torch.zeros_like(q[:n])
    tms.kv_attention(cache, 0, q[:n], few, out, parent=parent[:n], max_new=5000)
    check_attention(q[:n], out, ks[:2], vs[:2], lens[:2], new[:2], 64 ** -0.5, parents[:2], True)
    with pytest.raises(tms.TmsError) as ei:  # a tree of all tokens is too large
        tms.kv_attention(cache, 0, q, dev32([0] + [sum(new)] * 64), torch.zeros_like(q), parent=parent)
    assert "1024" in str(ei.value)


def test_caches_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements, pages at its end."""
    rng = np.random.default_rng(15)
    hkv, D, page, pages = 8, 128, 64, 17000  # 262144 bytes a page: 4.4 GB a layer of bf16, two layers
    kv = torch.empty((2, pages, 2, hkv, page, D), dtype=BF, device="cuda")
    assert kv.numel() > 2 ** 31 and kv.numel() * 2 > 2 ** 33
    lens, new = [100], [5]
    table, refs = np.array([[pages - 1, 0]], np.int32), np.zeros(pages, np.int32)
    refs[[pages - 1, 0]] = 1
    cache = tms.PagedCache(kv, dev32(table), dev32([0]), dev32([2]), dev32(refs), dev32([0]))
    k = torch.from_numpy(rng.standard_normal((2, 105, hkv, D)).astype(np.float32)).to(BF).cuda()
    tms.kv_write(cache, 1, k[0], k[1], dev32([0, 105]))
    assert torch.equal(kv[1, pages - 1, 0].transpose(0, 1), k[0, :64]) and torch.equal(kv[1, 0, 1, :, :41].transpose(0, 1), k[1, 64:])
    cache.length.fill_(100)
    q = torch.from_numpy(rng.standard_normal((5, 16, D)).astype(np.float32)).to(BF).cuda()
    out = run_attention(cache, q, new, layer=1)
    ks, vs = ([k[i].double().cpu().numpy()] for i in (0, 1))
    check_attention(q, out, ks, vs, lens, new, D ** -0.5, None, True)
    # a fork and its copy, from and to pages past 2^31 elements
    cache2 = tms.PagedCache(kv, torch.cat([cache.table, torch.full_like(cache.table, -1)]), dev32([40, 0]), dev32([1, 0]),
                            cache.refs, dev32([0, 0]))
    cache2.refs.fill_(1)
    cache2.refs[pages - 2] = 0
    tms.kv_fork(cache2, dev32([0, 0]))
    tms.kv_reserve(cache2, dev32([0, 3]))
    assert cache2.table[1, 0].item() == pages - 2
    assert torch.equal(kv[1, pages - 2, :, :, :40], kv[1, pages - 1, :, :, :40])
    tms.kv_write(cache2, 1, k[0, 60:63], k[1, 60:63], dev32([0, 0, 3]))
    tms.kv_commit(cache2, dev32([0, 2]), dev32([[0, 0], [0, 2]]))
    assert torch.equal(kv[1, pages - 2, 0, :, 40:42].transpose(0, 1), k[0, [60, 62]])


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 30, 300])
def test_attention_row_numbers_at_the_end_of_32_bits_give_nan(dtype, new):
    """A table that holds one page 2^25 - 1 times: rows that cannot be counted on
    from are refused, and a short sequence beside them is not."""
    print(f"attention {dtype} {new} tokens behind 2^31 - 64 rows", flush=True)
    rng = np.random.default_rng(16)
    small, ks, vs = filled(rng, dtype, 2, 64, 64, [70], [new])
    most = 2 ** 25 - 1
    table = torch.zeros((2, most), dtype=torch.int32, device="cuda")
    table[1, :small.table.shape[1]] = small.table[0]
    cache = tms.PagedCache(small.kv, table, dev32([64 * most - new, 70]), dev32([most, int(small.held[0])]), small.refs,
                           dev32([0, 0]))
    q = torch.from_numpy(rng.standard_normal((2 * new, 4, 64)).astype(np.float32)).to(dtype).cuda()
    out = run_attention(cache, q, [new, new])
    assert torch.isnan(out[:new].float()).all()
    check_attention(q[new:], out[new:], ks, vs, [70], [new], 64 ** -0.5, None, dtype == BF)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim,n_freq,interleaved", [(64, 32, False), (64, 32, True), (128, 64, False), (128, 16, False),
                                                    (128, 16, True), (256, 128, False), (64, 0, False), (256, 8, True)])
def test_write_matches_the_64_bit_form(dtype, dim, n_freq, interleaved):
    rng = np.random.default_rng(dim + n_freq)
    hq, hkv, page = 5, 3, 16
    for lens, new in (([0], [1]), ([5, 0, 31, 16], [0, 17, 33, 1]), (list(range(70)), [i % 3 for i in range(70)])):
        print(f"write {dtype} D={dim} n_freq={n_freq} {interleaved} {len(lens)} sequences", flush=True)
        for norm in (True, False):
            cache, _, _ = filled(rng, dtype, hkv, dim, page, lens, new, layers=3, layer=1, fill=3.0)
            before, T = cache.kv.clone(), sum(new)
            fused = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, dim)).astype(np.float32)).to(dtype).cuda()
            q, k, v = fused.split([hq, hkv, hkv], 1)
            w = [torch.from_numpy((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)).to(dtype).cuda() for _ in range(2)]
            pos = rng.integers(0, 200000, T)
            inv = (10000.0 ** -(np.arange(n_freq) / max(n_freq, 1))).astype(np.float32)
            q_out = torch.empty((T, hq, dim), dtype=dtype, device="cuda")
            tms.kv_write(cache, 1, k, v, dev32(offsets(new)), q=q, q_out=q_out, q_weight=w[0] if norm else None,
                         k_weight=w[1] if norm else None, eps=1e-5, pos=dev32(pos),
                         inv_freq=torch.from_numpy(inv).cuda() if n_freq else None, interleaved=interleaved)
            assert (cache.status() == tms.OK).all()
            got = {"q": q_out}
            seq = np.repeat(np.arange(len(lens)), new)
            row = np.concatenate([a + np.arange(b) for a, b in zip(lens, new)]).astype(np.int64)
            page_of = cache.table.cpu().numpy()[seq, row // page]
            at = (torch.from_numpy(page_of).long().cuda(), torch.from_numpy(row % page).cuda())
            got["k"], got["v"] = cache.kv[1][at[0], 0, :, at[1]], cache.kv[1][at[0], 1, :, at[1]]
            for name, x, weight in (("q", q, w[0]), ("k", k, w[1])):
                want, bound = head(x.double().cpu().numpy(), weight.double().cpu().numpy() if norm else None, 1e-5, pos,
                                   inv, interleaved, dtype == BF)
                err = np.abs(got[name].double().cpu().numpy() - want)
                assert (err <= bound).all(), (name, float((err / np.maximum(bound, 1e-30)).max()))
            assert torch.equal(got["v"], v)
            # nothing else moved
            before[1][at[0], 0, :, at[1]], before[1][at[0], 1, :, at[1]] = got["k"], got["v"]
            assert torch.equal(before, cache.kv)


def test_write_refuses_rows_that_are_not_reserved():
    cache = tms.PagedCache.empty(1, 4, 1, 16, 64, 2, 2, dtype=F)
    k = torch.ones((5, 1, 64), device="cuda")
    tms.kv_reserve(cache, dev32([3, 0]))
    tms.kv_write(cache, 0, k, k, dev32([0, 3, 5]))
    assert cache.status().tolist() == [tms.OK, tms.ERR_INVALID_ARG]
    with pytest.raises(tms.TmsError) as ei:
        tms.kv_reserve(cache, dev32([1, 1]))
    assert ei.value.code == tms.ERR_INVALID_ARG
    tms.kv_fork(cache, dev32([0, -1]))  # new content clears the error
    assert (cache.status() == tms.OK).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_write_refuses_all_rows_of_a_sequence_that_does_not_fit(dtype):
    """Not the ones that happen to come before its status is set: no row of it
    is written, every row of the others is, and queries come out of all."""
    hkv, hq, D, page = 2, 3, 128, 16
    for lens, new, held in (([5, 0, 9], [20, 1000, 30], [2, 62, 3]), ([0] * 70, [2] * 70, [i % 3 for i in range(70)]),
                            ([3, 30], [30, 3], [2, 3])):
        print(f"write that does not fit {dtype} {len(lens)} sequences", flush=True)
        rng = np.random.default_rng(len(lens))
        cache, _, _ = filled(rng, dtype, hkv, D, page, lens, new, layers=2, layer=1, fill=3.0)
        cache.held.copy_(dev32(held))
        before, T, at = cache.kv.clone(), sum(new), offsets(new)
        fused = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, D)).astype(np.float32)).to(dtype).cuda()
        q, k, v = fused.split([hq, hkv, hkv], 1)
        q_out = torch.empty((T, hq, D), dtype=dtype, device="cuda")
        tms.kv_write(cache, 1, k, v, dev32(at), q=q, q_out=q_out)
        fits = [a + b <= page * h for a, b, h in zip(lens, new, held)]
        assert not all(fits) and any(fits)
        assert cache.status().tolist() == [tms.OK if x else tms.ERR_INVALID_ARG for x in fits]
        table = cache.table.cpu().numpy()
        for s, (a, b) in enumerate(zip(lens, new)):
            if fits[s]:
                row = np.arange(a, a + b)
                where = torch.from_numpy(table[s, row // page]).long().cuda(), torch.from_numpy(row % page).cuda()
                before[1][where[0], 0, :, where[1]] = k[at[s]:at[s + 1]]
                before[1][where[0], 1, :, where[1]] = v[at[s]:at[s + 1]]
        assert torch.equal(before, cache.kv) and torch.equal(q_out, q)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_write_refuses_a_page_that_others_hold(dtype):
    """After a fork and without a reserve the next rows would land in a page of
    the other sequences too; with it, or from a page's edge on, they do not."""
    rng = np.random.default_rng(31)
    for rows in (40, 48, 5, 70):
        cache = tms.PagedCache.empty(2, 40, 2, 16, 64, 4, 8, dtype=dtype)
        cache.kv.fill_(2.0)
        k = torch.from_numpy(rng.standard_normal((2, 100, 2, 64)).astype(np.float32)).to(dtype).cuda()
        tms.kv_reserve(cache, dev32([rows + 20, 9, 0, 0]))
        tms.kv_write(cache, 0, k[0, :rows + 9], k[1, :rows + 9], dev32([0, rows, rows + 9, rows + 9, rows + 9]))
        tms.kv_commit(cache, dev32([rows, 9, 0, 0]))
        tms.kv_fork(cache, dev32([0, 1, 0, 0]))
        before = cache.kv.clone()
        start = dev32([0, 0, 3, 33, 34])  # the sequence of 9 rows is its own, the others share
        tms.kv_write(cache, 0, k[0, :34], k[1, :34], start)
        # the copies' rows past the edge have no page yet either
        assert cache.status().tolist() == [tms.OK, tms.OK, tms.ERR_INVALID_ARG, tms.ERR_INVALID_ARG], rows
        page = int(cache.table[1, 0])
        before[0, page, 0, :, 9:12], before[0, page, 1, :, 9:12] = k[0, :3].transpose(0, 1), k[1, :3].transpose(0, 1)
        assert torch.equal(before, cache.kv)
        tms.kv_fork(cache, dev32([0, 1, 0, -1]))
        tms.kv_write(cache, 0, k[0, :3], k[1, :3], dev32([0, 1, 1, 3, 3]))
        want = tms.ERR_INVALID_ARG  # the source shares as well, and what lies past the edge is not reserved here
        assert cache.status().tolist() == [want, tms.OK, want, tms.OK], rows
        assert torch.equal(before, cache.kv)
        # given anew and reserved: pages of their own
        cache.status_codes.zero_()
        tms.kv_reserve(cache, dev32([30, 1, 30, 0]))
        tms.kv_write(cache, 0, k[0, :61], k[1, :61], dev32([0, 30, 31, 61, 61]))
        assert (cache.status() == tms.OK).all()
        for s, at, length, n in ((0, 0, rows, 30), (1, 30, 9, 1), (2, 31, rows, 30)):
            r = torch.arange(length, length + n, device="cuda")
            page = cache.table[s].long()[r // 16]
            assert torch.equal(cache.kv[0][page, 0, :, r % 16], k[0, at:at + n]), (rows, s)
            r = torch.arange(length, device="cuda")  # the committed ones
            page = cache.table[s].long()[r // 16]
            first = {0: 0, 1: rows, 2: 0}[s]
            assert torch.equal(cache.kv[0][page, 0, :, r % 16], k[0, first:first + length]), (rows, s)


def _live_rows(cache, s):
    page = cache.page_tokens
    n = int(cache.length[s])
    t = cache.table[s].tolist()
    return [float(cache.kv[0, t[r // page], 0, 0, r % page, 0]) for r in range(n)]


@pytest.mark.parametrize("seqs,pages,page,max_pages,seed", [(1, 3, 8, 3, 0), (5, 12, 8, 4, 1), (7, 64, 16, 5, 2),
                                                            (70, 300, 8, 6, 3), (300, 5000, 8, 9, 4)])
def test_page_operations_follow_the_model(seqs, pages, page, max_pages, seed):
    """Random forks, reorderings, reservations (some past the pool), writes and
    commits: tables, counts, statuses and the rows of every sequence after each."""
    rng = np.random.default_rng(seed)
    cache = tms.PagedCache.empty(1, pages, 1, page, 64, seqs, max_pages, dtype=F)
    cache.kv.fill_(-1.0)
    model, mark = Pages(seqs, pages, page, max_pages), 0
    for step in range(12 if seqs > 100 else 40):
        print(f"pages {seqs}/{pages} step {step}", flush=True)
        src = np.arange(seqs)
        kind = rng.integers(4)
        if kind == 0:
            src = rng.integers(0, seqs, seqs)
        elif kind == 1:
            some = rng.random(seqs) < 0.3
            src = np.where(some, rng.integers(-1, seqs, seqs), src)
        if step % 7 == 5:
            src[rng.integers(seqs)] = seqs + 3
        tms.kv_fork(cache, dev32(src), check=False)
        model.fork(src.tolist())
        n_new = np.where(rng.random(seqs) < 0.7, rng.integers(0, 2 * page, seqs), -1)
        tms.kv_reserve(cache, dev32(n_new), check=False)
        model.reserve(n_new.tolist())
        ok = [n if n > 0 and not model.status[s] else 0 for s, n in enumerate(n_new.tolist())]
        drafts = []
        for n in ok:
            drafts.append([float(mark + i + 1) for i in range(n)])
            mark += n
        rows = torch.tensor([x for d in drafts for x in d], device="cuda")
        k = rows[:, None, None].expand(-1, 1, 64).contiguous()
        tms.kv_write(cache, 0, k, -k, dev32(offsets(ok)))
        keep = np.zeros((seqs, 2 * page), np.int32)
        n_keep = np.zeros(seqs, np.int32)
        for s, n in enumerate(ok):
            idx = np.sort(rng.permutation(n)[: rng.integers(0, n + 1)])
            n_keep[s] = len(idx)
            keep[s, :len(idx)] = idx
        if step % 5 == 3:
            s = int(rng.integers(seqs))
            if n_keep[s] >= 2:
                keep[s, :2] = keep[s, 1::-1]  # not ascending
        if step % 6 == 2:
            n_keep = np.where(rng.random(seqs) < 0.5, np.minimum(n_keep, 1), n_keep).astype(np.int32)
            tms.kv_commit(cache, dev32(n_keep), check=False)
            model.commit(n_keep.tolist(), None, drafts)
        else:
            tms.kv_commit(cache, dev32(n_keep), dev32(keep), check=False)
            model.commit(n_keep.tolist(), keep, drafts)
        table = np.full((seqs, max_pages), -1)
        for s, t in enumerate(model.table):
            table[s, :len(t)] = t
        assert cache.status().tolist() == model.status, step
        assert np.array_equal(cache.table.cpu().numpy(), table), step
        assert cache.refs.tolist() == model.refs(), step
        assert cache.held.tolist() == [len(t) for t in model.table], step
        assert cache.length.tolist() == [len(r) for r in model.rows], step
        kv = cache.kv.cpu()
        for s in range(seqs):
            r = np.arange(len(model.rows[s]))
            at = table[s][r // page], r % page
            want = np.array(model.rows[s])
            assert np.array_equal(kv[0][at[0], 0, 0, at[1]].numpy(), np.repeat(want[:, None], 64, 1)), (step, s)
            assert np.array_equal(kv[0][at[0], 1, 0, at[1]].numpy(), np.repeat(-want[:, None], 64, 1)), (step, s)
        if any(model.status) and step % 3 == 0:  # errors stay until new content comes
            clear = [-1 if x else s for s, x in enumerate(model.status)]
            tms.kv_fork(cache, dev32(clear), check=False)
            model.fork(clear)


@pytest.mark.parametrize("seqs,pages,page,max_pages,seed", [(16, 200, 8, 1025, 5), (33, 400, 8, 15, 6), (33, 400, 8, 16, 7),
                                                            (64, 700, 8, 8, 8), (64, 2000, 8, 60, 9)])
def test_page_operations_where_the_fork_changes_its_form(seqs, pages, page, max_pages, seed):
    test_page_operations_follow_the_model(seqs, pages, page, max_pages, seed)


def check_reserve(cache, model, n_new):
    """Reserves on the device and on the model; tables, counts, statuses and
    every page: a page that was given as a copy has its rows, the others are
    bit for bit what they were."""
    before, tables = cache.kv.clone(), [list(t) for t in model.table]
    tms.kv_reserve(cache, dev32(n_new), check=False)
    model.reserve(n_new)
    table = np.full((cache.seqs, cache.max_pages), -1)
    for s, t in enumerate(model.table):
        table[s, :len(t)] = t
    assert cache.status().tolist() == model.status
    assert np.array_equal(cache.table.cpu().numpy(), table)
    assert np.array_equal(cache.refs.cpu().numpy(), model.refs())
    assert cache.held.tolist() == [len(t) for t in model.table]
    assert cache.length.tolist() == [len(r) for r in model.rows]
    for s, (old, now) in enumerate(zip(tables, model.table)):
        last, fill = len(model.rows[s]) // cache.page_tokens, len(model.rows[s]) % cache.page_tokens
        if last < len(old) and old[last] != now[last]:
            before[:, now[last], :, :, :fill] = before[:, old[last], :, :, :fill]
    assert torch.equal(before, cache.kv)


@pytest.mark.parametrize("layers,kv_heads", [(1, 1), (3, 4)], ids=["in_the_plan", "by_a_launch"])
def test_reserve_past_the_pool_refuses_everyone_after(layers, kv_heads):
    """Demands that pass the whole pool: every later demand gets OOM too, with or
    without a copy of its last page, and holds what it held; who asks for
    nothing stays."""
    for seqs, n_new in ((4, [60, 60, 3, 3]), (6, [200, 0, 3, 20, 1, 2]), (6, [9, 200, 0, 3, 3, -1]), (5, [3, 3, 400, 400, 3])):
        print(f"reserve past the pool {layers} layers n_new {n_new}", flush=True)
        cache = tms.PagedCache.empty(layers, 10, kv_heads, 8, 64, seqs, 60, dtype=F)
        cache.kv.copy_(torch.arange(cache.kv.numel(), device="cuda").view(cache.kv.shape) % 1000003)
        model = Pages(seqs, 10, 8, 60)
        check_reserve(cache, model, [5] + [0] * (seqs - 1))
        tms.kv_commit(cache, dev32([5] + [0] * (seqs - 1)))
        model.commit([5] + [0] * (seqs - 1), None, [[1] * 5] + [[]] * (seqs - 1))
        tms.kv_fork(cache, dev32([0] * seqs))
        model.fork([0] * seqs)
        check_reserve(cache, model, n_new)
        assert model.status.count(Pages.OOM) >= 2
        clear = [-1 if x else s for s, x in enumerate(model.status)]
        tms.kv_fork(cache, dev32(clear))
        model.fork(clear)
        check_reserve(cache, model, [4] * seqs)


@pytest.mark.parametrize("seqs,pages,max_pages,most", [(8, 12, 40, 100), (70, 90, 200, 400), (1500, 4000, 40, 60),
                                                       (2500, 900, 40, 60), (4096, 9000, 30, 40)])
def test_reserve_follows_the_model_in_pools_too_small(seqs, pages, max_pages, most):
    """Also more sequences than the plan takes in one turn."""
    rng = np.random.default_rng(seqs)
    cache = tms.PagedCache.empty(2, pages, 1, 8, 64, seqs, max_pages)
    cache.kv.copy_(torch.arange(cache.kv.numel(), device="cuda").view(cache.kv.shape) % 251)
    model = Pages(seqs, pages, 8, max_pages)
    for step in range(6):
        print(f"reserve {seqs} sequences, {pages} pages, step {step}", flush=True)
        check_reserve(cache, model, [int(x) for x in rng.integers(-2, most if step % 2 else 12, seqs)])
        grown = [min(int(rng.integers(0, 20)), len(t) * 8 - len(r)) for t, r in zip(model.table, model.rows)]
        tms.kv_commit(cache, dev32(grown), check=False)
        model.commit(grown, None, [[1] * n for n in grown])
        src = np.where(rng.random(seqs) < 0.4, rng.integers(-1, seqs, seqs), np.arange(seqs))
        src = [-1 if model.status[s] and x == s else int(x) for s, x in enumerate(src)]
        tms.kv_fork(cache, dev32(src), check=False)
        model.fork(src)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_copies_and_moves_by_the_plan_and_by_launches(dtype, page):
    """Last pages of a few rows up to all but one, few pieces of every size, then
    rows moved together, by short lists and long ones."""
    rng = np.random.default_rng(page)
    for layers, kv_heads, D, seqs in ((1, 1, 64, 4), (1, 1, 256, 3), (2, 2, 128, 4), (1, 8, 64, 2), (3, 4, 64, 3)):
        for rows in (1, page - 1, page + page // 2):
            print(f"copies {dtype} page {page} {layers} layers {kv_heads}x{D} {seqs} sequences {rows} rows", flush=True)
            new = 2 * page + 5
            cache = tms.PagedCache.empty(layers, 5 * seqs + 3, kv_heads, page, D, seqs, 5, dtype=dtype)
            k = torch.from_numpy(rng.standard_normal((2, rows + seqs * new, kv_heads, D)).astype(np.float32)).to(dtype).cuda()
            tms.kv_reserve(cache, dev32([rows] + [0] * (seqs - 1)))
            for layer in range(layers):
                tms.kv_write(cache, layer, k[layer % 2, :rows], k[1 - layer % 2, :rows], dev32([0] + [rows] * seqs))
            tms.kv_commit(cache, dev32([rows] + [0] * (seqs - 1)))
            tms.kv_fork(cache, dev32([0] * seqs))
            tms.kv_reserve(cache, dev32([new] * seqs))
            for layer in range(layers):
                tms.kv_write(cache, layer, k[layer % 2, rows:], k[1 - layer % 2, rows:], dev32(np.arange(seqs + 1) * new))
            for kept in (3, new - 2):
                keep = np.stack([np.sort(rng.permutation(new - (4 if kept > 3 else 0))[:kept - (4 if kept > 3 else 0)])
                                 for _ in range(seqs)])
                saved = [t.clone() for t in (cache.kv, cache.table, cache.length, cache.held, cache.refs)]
                tms.kv_commit(cache, dev32([keep.shape[1]] * seqs), dev32(keep))
                r = torch.arange(rows + keep.shape[1], device="cuda")
                for s in range(seqs):
                    at = torch.from_numpy(np.r_[0:rows, rows + s * new + keep[s]]).cuda()
                    where = cache.table[s].long()[r // page]
                    for layer in range(layers):
                        assert torch.equal(cache.kv[layer][where, 0, :, r % page], k[layer % 2][at]), (rows, kept, s, layer)
                        assert torch.equal(cache.kv[layer][where, 1, :, r % page], k[1 - layer % 2][at]), (rows, kept, s, layer)
                for t, x in zip((cache.kv, cache.table, cache.length, cache.held, cache.refs), saved):
                    t.copy_(x)


def test_reserve_from_a_pool_of_a_million_pages():
    """2^20 pages and more: demands above 2^16 pages, summed in two halves."""
    pages, max_pages = (1 << 20) + 77, 700000
    cache = tms.PagedCache.empty(1, pages, 1, 8, 64, 5, max_pages)
    for n_new, status in (([8 * 70000 - 3, 5, 8 * 650000, 8 * 400000, 9], [0, 0, 0, 9, 9]),
                          ([8 * 65536, 8 * 65535, 0, 5, 5], [0, 0, 0, 0, 0])):
        print(f"reserve {n_new} of {pages} pages", flush=True)
        tms.kv_reserve(cache, dev32(n_new), check=False)
        assert cache.status().tolist() == status
        held = cache.held.tolist()
        assert held == [-(-n // 8) if n > 0 and not x else 0 for n, x in zip(n_new, status)]
        at = 0
        for s, h in enumerate(held):  # ascending pages, sequence after sequence
            assert torch.equal(cache.table[s, :h], torch.arange(at, at + h, dtype=torch.int32, device="cuda"))
            assert (cache.table[s, h:] == -1).all()
            at += h
        assert (cache.refs[:at] == 1).all() and not cache.refs[at:].any()
        tms.kv_fork(cache, dev32([-1] * 5))
        assert not cache.refs.any() and (cache.table == -1).all() and not cache.held.any()


def test_commit_moves_long_keep_lists_in_place():
    """Several hundred rows that overlap their targets, in every layer and head."""
    rng = np.random.default_rng(21)
    for dtype, dim in ((BF, 128), (F, 256)):
        n = 700
        cache = tms.PagedCache.empty(2, 60, 2, 16, dim, 2, 50, dtype=dtype)
        tms.kv_reserve(cache, dev32([n, 5]))
        k = torch.from_numpy(rng.standard_normal((2, n + 5, 2, dim)).astype(np.float32)).to(dtype).cuda()
        for layer in (0, 1):
            tms.kv_write(cache, layer, k[layer], k[1 - layer], dev32([0, n, n + 5]))
        idx = np.sort(rng.permutation(n)[:650])
        idx[0] = 0
        keep = np.zeros((2, 660), np.int32)
        keep[0, :650] = idx
        tms.kv_commit(cache, dev32([650, 0]), dev32(keep))
        t = cache.table[0].tolist()
        r = np.arange(650)
        at = torch.tensor([t[i // 16] for i in r]).cuda(), torch.tensor(r % 16).cuda()
        for layer in (0, 1):
            assert torch.equal(cache.kv[layer][at[0], 0, :, at[1]], k[layer][idx])
            assert torch.equal(cache.kv[layer][at[0], 1, :, at[1]], k[1 - layer][idx])
        assert cache.length.tolist() == [650, 0] and cache.held.tolist() == [41, 0]


@pytest.mark.parametrize("seqs", [1, 130])
def test_commit_moves_chunks_of_the_narrowest_rows(seqs):
    """Rows of 128 bytes: 256 to a chunk, with lists of one row more and less,
    by one workgroup for all pieces of a sequence or by several."""
    rng = np.random.default_rng(23)
    for n, kept, layers in ((257, 256, 1), (260, 257, 1), (600, 513, 9), (256, 255, 9)):
        print(f"commit {seqs} sequences keep {kept} of {n} rows, {layers} layers", flush=True)
        cache = tms.PagedCache.empty(layers, seqs * 40, 1, 16, 64, seqs, 40)
        tms.kv_reserve(cache, dev32([n] * seqs))
        k = torch.from_numpy(rng.standard_normal((2, seqs * n, 1, 64)).astype(np.float32)).to(BF).cuda()
        for layer in range(layers):
            tms.kv_write(cache, layer, k[layer % 2], k[1 - layer % 2], dev32(np.arange(seqs + 1) * n))
        keep = np.stack([np.sort(rng.permutation(n)[:kept]) for _ in range(seqs)])
        tms.kv_commit(cache, dev32([kept] * seqs), dev32(keep))
        assert cache.length.tolist() == [kept] * seqs
        r = torch.arange(kept, device="cuda")
        for s in range(seqs):
            page, at = cache.table[s].long()[r // 16], torch.from_numpy(keep[s] + s * n).cuda()
            for layer in range(layers):
                assert torch.equal(cache.kv[layer][page, 0, :, r % 16], k[layer % 2][at]), (s, layer)
                assert torch.equal(cache.kv[layer][page, 1, :, r % 16], k[1 - layer % 2][at]), (s, layer)


def test_a_whole_step_replays_in_a_graph():
    """Fork, reserve, write, attend and commit recorded once: every replay
    gives the eager results (the branches start from the same root each time)."""
    rng = np.random.default_rng(22)
    seqs, page, hq, hkv, D = 6, 16, 4, 2, 64
    lens = [45] + [0] * 5
    new = [0, 3, 1, 7, 0, 5]
    cache, _, _ = filled(rng, BF, hkv, D, page, lens, [0] * seqs, spare=30, fill=0.0)
    cache = tms.PagedCache(cache.kv, torch.cat([cache.table, torch.full((seqs, 3), -1, dtype=torch.int32, device="cuda")], 1).contiguous(),
                           cache.length, cache.held, cache.refs, cache.status_codes)
    T = sum(new)
    fused = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, D)).astype(np.float32)).to(BF).cuda()
    q, k, v = fused.split([hq, hkv, hkv], 1)
    start, src, n_new = dev32(offsets(new)), dev32([0] * seqs), dev32(new)
    parent = dev32([p for n in new for p in tree(rng, n)])
    n_keep, keep = dev32([0, 2, 1, 3, 0, 0]), dev32([[0, 0, 0], [0, 2, 0], [0, 0, 0], [1, 4, 6], [0, 0, 0], [0, 0, 0]])
    pos, inv = dev32(rng.integers(0, 99, T)), torch.tensor([1.0 / (i + 1) for i in range(32)], device="cuda")
    q_out, out = torch.empty((T, hq, D), dtype=BF, device="cuda"), torch.empty((T, hq, D), dtype=BF, device="cuda")

    def step():
        tms.kv_fork(cache, src, check=False)
        tms.kv_reserve(cache, n_new, check=False)
        tms.kv_write(cache, 0, k, v, start, q=q, q_out=q_out, pos=pos, inv_freq=inv)
        tms.kv_attention(cache, 0, q_out, start, out, parent=parent, max_new=7)
        tms.kv_commit(cache, n_keep, keep, check=False)

    def results():
        torch.cuda.synchronize()
        assert (cache.status() == tms.OK).all()
        return [t.clone() for t in (out, q_out, cache.kv, cache.table, cache.length, cache.held, cache.refs)]

    step()
    want = results()
    assert torch.isfinite(want[0].float()).all()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        out.fill_(9.0)
        q_out.fill_(9.0)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
        step()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    with torch.cuda.stream(side):
        g2 = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g2, stream=side):
            with pytest.raises(tms.TmsError) as ei:
                tms.kv_fork(cache, src)
            assert "recorded" in str(ei.value)


def test_a_cache_dropped_while_another_stream_works_on_it():
    """Its memory is handed on only when that stream is done, whichever stream
    was current when the cache was made of them."""
    side = torch.cuda.Stream()
    for made_on in (torch.cuda.current_stream(), side):
        kv = torch.zeros((1, 4096, 2, 2, 16, 64), device="cuda")
        ints = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((1, 300000), 1, 1, 4096, 1)]
        torch.cuda.synchronize()
        with torch.cuda.stream(made_on):
            cache = tms.PagedCache(kv, *ints)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # some tenths of a second
            tms.kv_reserve(cache, torch.full((1,), 64, dtype=torch.int32, device="cuda"), check=False)
        owned = [cache.kv, cache.table, cache.length, cache.held, cache.refs, cache.status_codes, cache.work]
        shapes, places = [(t.shape, t.dtype) for t in owned], [t.data_ptr() for t in owned]
        stream, done = torch.cuda.current_stream() if made_on == side else made_on, torch.cuda.Event()
        done.record(side)
        del cache, kv, ints, owned
        with torch.cuda.stream(stream):
            fresh = [torch.empty(a, dtype=b, device="cuda") for a, b in shapes]
        early = [t.data_ptr() in places for t in fresh]
        assert not done.query()
        torch.cuda.synchronize()
        assert not any(early), early
        del fresh


def test_binding_refusals():
    cache = tms.PagedCache.empty(2, 8, 2, 16, 64, 3, 4)
    start, q = dev32([0, 1, 1, 2]), torch.zeros((2, 4, 64), dtype=BF, device="cuda")
    k, out = q[:, :2].contiguous(), torch.empty_like(q)
    for call, what in (
            (lambda: tms.kv_attention(cache, 2, q, start, out), "layer"),
            (lambda: tms.kv_attention(cache, -1, q, start, out), "layer"),
            (lambda: tms.kv_attention(cache, 0, q[:, :3].contiguous(), start, out), "kv_heads"),
            (lambda: tms.kv_attention(cache, 0, q, start, out, max_new=0), "max_new"),
            (lambda: tms.kv_write(cache, 5, k, k, start), "layer"),
            (lambda: tms.kv_write(cache, 0, k, k, start, pos=dev32([0, 1]), inv_freq=torch.ones(40, device="cuda")), "n_freq"),
            (lambda: tms.kv_write(cache, 0, k, k, start, pos=dev32([0, 1]), inv_freq=torch.ones(4, device="cuda")), "n_freq")):
        with pytest.raises(tms.TmsError) as ei:
            call()
        assert ei.value.code == tms.ERR_INVALID_ARG and what in str(ei.value)
    big = torch.zeros((1100, 4, 64), dtype=BF, device="cuda")
    with pytest.raises(tms.TmsError) as ei:
        tms.kv_attention(cache, 0, big, dev32([0, 1100, 1100, 1100]), torch.empty_like(big), parent=dev32([0] * 1100))
    assert "1024" in str(ei.value)
    for call in (
            lambda: tms.kv_attention(cache, 0, q, start[:3].contiguous(), out),
            lambda: tms.kv_attention(cache, 0, q, start, out[:1]),
            lambda: tms.kv_attention(cache, 0, q.float(), start, out),
            lambda: tms.kv_attention(cache, 0, q.transpose(0, 1), start, out),
            lambda: tms.kv_attention(cache, 0, q, start, out, parent=dev32([0])),
            lambda: tms.kv_write(cache, 0, k, k[:1], start),
            lambda: tms.kv_write(cache, 0, q, q, start),
            lambda: tms.kv_write(cache, 0, k, k, start, q=q),
            lambda: tms.kv_write(cache, 0, k, k, start, inv_freq=torch.ones(8, device="cuda")),
            lambda: tms.kv_write(cache, 0, k, k, start, q_weight=None, k_weight=torch.ones(64, device="cuda")),
            lambda: tms.kv_fork(cache, dev32([0, 1])),
            lambda: tms.kv_fork(cache, torch.zeros(3, dtype=torch.int32)),
            lambda: tms.kv_commit(cache, dev32([0, 0, 0]), dev32([[0], [0]])),
            lambda: tms.PagedCache(cache.kv.half(), cache.table, cache.length, cache.held, cache.refs, cache.status_codes),
            lambda: tms.PagedCache(cache.kv, cache.table, cache.length, cache.held, cache.refs[:4], cache.status_codes)):
        with pytest.raises((TypeError, ValueError)):
            call()
    # no tokens at all: nothing to do
    none = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    tms.kv_attention(cache, 0, none, dev32([0, 0, 0, 0]), none, max_new=1)
    tms.kv_write(cache, 0, none[:, :2], none[:, :2], dev32([0, 0, 0, 0]))
    assert (cache.status() == tms.OK).all()


def test_the_example_decodes_the_same_with_and_without_drafts():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "tree_decode.py")
    spec = importlib.util.spec_from_file_location("tree_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    c = ex.CONFIGS["tiny"]
    rng = np.random.default_rng(8)
    trie = tms.Trie(ex.catalog("tiny"), c.vocab, c.sep, c.stop)
    model = ex.Model(torch.from_numpy(ex.embedding("tiny").copy()).cuda(), seed=1)
    prompt, questions = rng.integers(0, c.sep, 50).tolist(), [rng.integers(0, c.sep, n).tolist() for n in (1, 7, 3)]
    plain, many = ex.decode(trie, model, prompt, questions, c.k, 0)
    answers, passes = ex.decode(trie, model, prompt, questions, c.k, 40)
    assert answers == plain and passes < many
    entries = {tuple(e) for e in ex.catalog("tiny")}
    for a in answers:  # k different entries, separated, and stop
        parts, part = [], []
        for t in a[:-1]:
            if t == c.sep:
                parts.append(tuple(part))
                part = []
            else:
                part.append(t)
        parts.append(tuple(part))
        assert a[-1] == c.stop and len(parts) == c.k and len(set(parts)) == c.k and set(parts) <= entries
    trie.close()
