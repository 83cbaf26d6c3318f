"""Argument checks of the calls over long contexts of the paged cache that are
made before any GPU call (no GPU needed), and the host forms of their tests."""
import ctypes as C

import numpy as np
import pytest

import trie_masked_sparse_amd as tms
from kv_util import choice
from test_kv_host import descriptor, refused

P = 1 << 20


def long_call(name, **over):
    """One of the calls with good arguments, some of them replaced."""
    L, r = tms.lib(), C.byref(descriptor())
    attention = dict(layer=0, q=P, ldq=256, q_heads=4, start=P, T=1, max_new=1)
    args = {
        "share_bytes": dict(T=1, q_heads=4, bytes=C.byref(C.c_int64())),
        "share": dict(start=P, T=1, q_heads=4, plan=P, plan_bytes=1 << 40, stream=None),
        "attention_shared": dict(attention, parent=None, scale=1.0, out=P, plan=P, plan_bytes=1 << 40, stream=None),
        "bounds": dict(n_new=P, max_new=1, bounds=P, stream=None),
        "select_bytes": dict(T=1, bytes=C.byref(C.c_int64())),
        "select": dict(attention, scale=1.0, bounds=P, k=4, first=1, last=1, chosen=P, work=P, work_bytes=1 << 40, stream=None),
        "attention_pages": dict(attention, parent=None, chosen=P, k=4, scale=1.0, out=P, stream=None),
    }[name]
    assert set(over) <= set(args)
    return getattr(L, "tms_kv_" + name)(r, *{**args, **over}.values())


ATTENTION = [(dict(layer=2), "layer"), (dict(layer=-1), "layer"), (dict(start=None), "start"), (dict(T=-1), "T"),
             (dict(q_heads=3), "q_heads"), (dict(q_heads=0), "q_heads"), (dict(max_new=0), "max_new"), (dict(q=None), "null"),
             (dict(q=P + 8), "aligned"), (dict(ldq=255), "stride"), (dict(ldq=260), "stride")]


@pytest.mark.parametrize("name,over,what",
                         [("attention_shared", *x) for x in ATTENTION] + [("select", *x) for x in ATTENTION] +
                         [("attention_pages", *x) for x in ATTENTION] + [
    ("share_bytes", dict(T=0), "T must"), ("share_bytes", dict(T=(1 << 24) + 1), "T must"), ("share_bytes", dict(q_heads=3), "q_heads"),
    ("share_bytes", dict(q_heads=4098), "q_heads"), ("share_bytes", dict(bytes=None), "null"),
    ("share", dict(start=None), "start"), ("share", dict(T=0), "T must"), ("share", dict(q_heads=1), "q_heads"),
    ("share", dict(plan=None), "plan"), ("share", dict(plan=P + 128), "plan"), ("share", dict(plan_bytes=1000), "plan_bytes"),
    ("attention_shared", dict(out=None), "null"), ("attention_shared", dict(plan=None), "plan"),
    ("attention_shared", dict(plan_bytes=1000), "plan_bytes"), ("attention_shared", dict(T=2000, max_new=1025, parent=P), "1024"),
    ("bounds", dict(bounds=None), "bounds"), ("bounds", dict(bounds=P + 8), "bounds"), ("bounds", dict(max_new=-1), "max_new"),
    ("select_bytes", dict(T=-1), "T"), ("select_bytes", dict(bytes=None), "null"),
    ("select", dict(k=0), "k must"), ("select", dict(k=8193), "k must"), ("select", dict(first=-1), "first"),
    ("select", dict(last=-1), "last"), ("select", dict(chosen=None), "chosen"), ("select", dict(bounds=None), "bounds"),
    ("select", dict(bounds=P + 8), "bounds"), ("select", dict(work=None), "work"), ("select", dict(work=P + 16), "work"),
    ("select", dict(work_bytes=8), "work"),
    ("attention_pages", dict(k=-1), "k must"), ("attention_pages", dict(k=8193), "k must"),
    ("attention_pages", dict(chosen=None), "chosen"), ("attention_pages", dict(out=P + 4), "aligned"),
    ("attention_pages", dict(T=2000, max_new=1025, parent=P), "1024"),
])
def test_arguments_are_checked(name, over, what):
    refused(long_call(name, **over), what)


def test_no_tokens_is_nothing_to_do():
    for name in ("attention_shared", "select", "attention_pages"):
        assert long_call(name, T=0) == tms.OK
    assert long_call("select_bytes", T=0) == tms.OK


@pytest.mark.parametrize("over", [dict(head_dim=96), dict(page_tokens=4), dict(seqs=0), dict(dtype=7), dict(pages=0)])
def test_sizes_of_the_cache_are_checked(over):
    n, L, d = C.c_int64(), tms.lib(), descriptor(**over)
    assert L.tms_kv_share_bytes(C.byref(d), 1, 4, C.byref(n)) == tms.ERR_INVALID_ARG
    assert L.tms_kv_select_bytes(C.byref(d), 1, C.byref(n)) == tms.ERR_INVALID_ARG
    assert L.tms_kv_bounds(C.byref(d), None, 1, P, None) == tms.ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [tms.BF16, tms.F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_plan_for_more_tokens_is_one_for_fewer(dtype, dim):
    L, n = tms.lib(), C.c_int64()
    for seqs, heads, kv_heads in ((1, 4, 2), (64, 32, 8), (4096, 8, 1), (3, 6, 6)):
        d = descriptor(dtype=dtype, head_dim=dim, seqs=seqs, kv_heads=kv_heads)
        sizes = []
        for T in [*range(1, 300), 1000, 5000, 100000]:
            assert L.tms_kv_share_bytes(C.byref(d), T, heads, C.byref(n)) == tms.OK
            assert n.value % 256 == 0
            sizes.append(n.value)
        assert sizes == sorted(sizes)


def test_the_plain_form_of_the_choice():
    bounds = np.zeros((5, 1, 2, 2))
    bounds[:, 0, 1, 0] = [1, 5, 3, 3, 0]      # highest of column 0
    bounds[:, 0, 0, 1] = [-1, 0, -4, -4, -9]  # lowest of column 1
    q = np.array([[1.0, 0.0], [1.0, -0.5]])
    # 2 hi_0 - 0.5 lo_1: 2.5, 10, 8, 8, 4.5
    assert choice(q, bounds, 2, 1.0, 0, 0).tolist() == [[1, 2]]
    assert choice(q, bounds, 3, 1.0, 1, 1).tolist() == [[0, 1, 4]]
    assert choice(q, bounds, 7, 1.0, 0, 0).tolist() == [[0, 1, 2, 3, 4, -1, -1]]
    assert choice(q, bounds, 2, 0.0, 0, 1).tolist() == [[0, 4]]
    bounds[3, 0, 1, 0] = np.nan
    assert choice(q, bounds, 2, 1.0, 0, 0).tolist() == [[1, 3]]
    # no key within the bounds has a larger product than the score
    rng = np.random.default_rng(0)
    keys, x = rng.standard_normal((30, 8)), rng.standard_normal((1, 8))
    b = np.stack((keys.min(0), keys.max(0)))
    score = (np.maximum(x, 0).sum(0) * b[1] + np.minimum(x, 0).sum(0) * b[0]).sum()
    assert (keys @ x[0]).max() <= score
