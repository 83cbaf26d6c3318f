"""Argument checks of the paged-cache entry points that are made before any
GPU call (no GPU needed), and the host forms of the tests themselves."""
import ctypes as C

import numpy as np
import pytest

import trie_masked_sparse_amd as tms
from kv_util import Pages, ancestors, attention, head
from kv_util import marked_values


def descriptor(**over):
    d = dict(kv=1 << 20, table=4096, length=4096, held=4096, refs=4096, status=4096, work=1 << 20, work_bytes=1 << 40,
             dtype=tms.BF16, layers=2, pages=10, kv_heads=2, page_tokens=16, head_dim=64, seqs=3, max_pages=4)
    d.update(over)
    return tms.KvDescriptor(**d)


def refused(rc, what):
    assert rc == tms.ERR_INVALID_ARG
    assert what in tms.lib().tms_last_error().decode(), tms.lib().tms_last_error()


@pytest.mark.parametrize("over,what", [
    (dict(dtype=2), "dtype"), (dict(head_dim=96), "head_dim"), (dict(head_dim=0), "head_dim"),
    (dict(page_tokens=12), "page_tokens"), (dict(page_tokens=4), "page_tokens"), (dict(page_tokens=2048), "page_tokens"),
    (dict(seqs=0), "seqs"), (dict(seqs=4097), "seqs"), (dict(kv_heads=0), "kv_heads"), (dict(layers=0), "layers"),
    (dict(pages=0), "pages"), (dict(max_pages=0), "max_pages"), (dict(max_pages=1 << 28), "2^31"),
])
def test_sizes_are_checked(over, what):
    n = C.c_int64()
    refused(tms.lib().tms_kv_work_bytes(C.byref(descriptor(**over)), C.byref(n)), what)


@pytest.mark.parametrize("over,what", [
    (dict(kv=None), "null"), (dict(table=None), "null"), (dict(status=None), "null"), (dict(work=None), "null"),
    (dict(kv=(1 << 20) + 8), "aligned"), (dict(work=(1 << 20) + 16), "aligned"), (dict(work_bytes=16), "work_bytes"),
])
def test_pointers_are_checked(over, what):
    L, d = tms.lib(), descriptor(**over)
    refused(L.tms_kv_fork(C.byref(d), 4096, None), what)
    refused(L.tms_kv_reserve(C.byref(d), 4096, None), what)
    refused(L.tms_kv_commit(C.byref(d), 4096, None, 0, None), what)


def test_null_arguments_and_strides():
    L, d = tms.lib(), descriptor()
    r = C.byref(d)
    n = C.c_int64()
    assert L.tms_kv_work_bytes(r, C.byref(n)) == tms.OK and n.value > 0 and n.value % 256 == 0
    refused(L.tms_kv_work_bytes(r, None), "null")
    refused(L.tms_kv_fork(None, 4096, None), "null")
    refused(L.tms_kv_fork(r, None, None), "null")
    refused(L.tms_kv_reserve(r, None, None), "null")
    refused(L.tms_kv_commit(r, None, None, 0, None), "null")
    refused(L.tms_kv_commit(r, 4096, 4096, 0, None), "keep_stride")
    P = 1 << 20
    # layer, q, ldq, q_heads, start, T, max_new, parent, scale, out
    refused(L.tms_kv_attention(r, 2, P, 256, 4, P, 1, 1, None, 1.0, P, None), "layer")
    refused(L.tms_kv_attention(r, 0, P, 256, 3, P, 1, 1, None, 1.0, P, None), "q_heads")
    refused(L.tms_kv_attention(r, 0, P, 255, 4, P, 1, 1, None, 1.0, P, None), "stride")
    refused(L.tms_kv_attention(r, 0, P, 260, 4, P, 1, 1, None, 1.0, P, None), "stride")
    refused(L.tms_kv_attention(r, 0, P + 8, 256, 4, P, 1, 1, None, 1.0, P, None), "aligned")
    refused(L.tms_kv_attention(r, 0, P, 256, 4, P, 1, 1, None, 1.0, None, None), "null")
    refused(L.tms_kv_attention(r, 0, P, 256, 4, P, 1, 0, None, 1.0, P, None), "max_new")
    refused(L.tms_kv_attention(r, 0, P, 256, 4, P, 2000, 1025, P, 1.0, P, None), "1024")
    refused(L.tms_kv_attention(r, 0, P, 256, 4, P, -1, 1, None, 1.0, P, None), "T")
    # layer, start, T, q, ldq, q_heads, q_out, k, ldk, v, ldv, q_weight, k_weight, eps, pos, inv_freq, n_freq, interleaved
    def write(**o):
        a = dict(layer=0, start=P, T=1, q=P, ldq=256, q_heads=4, q_out=P, k=P, ldk=128, v=P, ldv=128, q_weight=None,
                 k_weight=None, eps=1e-6, pos=P, inv_freq=P, n_freq=32, interleaved=0)
        a.update(o)
        return L.tms_kv_write(r, *a.values(), None)
    for over, what in ((dict(layer=-1), "layer"), (dict(start=None), "start"), (dict(T=-1), "T"), (dict(n_freq=12), "n_freq"),
                       (dict(n_freq=40), "n_freq"), (dict(pos=None), "pos"), (dict(q_out=None), "q_out"),
                       (dict(q_heads=0), "q_heads"), (dict(ldq=128), "stride"), (dict(k=None), "null"), (dict(ldv=100), "stride"),
                       (dict(ldk=132), "stride"), (dict(k_weight=P + 4), "weights")):
        refused(write(**over), what)
    assert write(T=0) == tms.OK
    assert L.tms_kv_attention(r, 0, P, 256, 4, P, 0, 1, None, 1.0, P, None) == tms.OK


def test_the_package_imports_with_a_torch_without_gpus():
    """Tries are compiled on the host: importing needs nothing of a GPU build."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(tms.__file__))
    subprocess.run([sys.executable, "-c", "import torch; del torch._C._cuda_getCurrentRawStream; "
                    "import trie_masked_sparse_amd as tms; assert tms.OK == 0"], cwd=root, check=True)


def test_the_zeroed_part_of_the_work_memory_is_the_headers():
    import os
    import re
    header = open(os.path.join(os.path.dirname(tms.__file__), os.pardir, "include", "tms.h")).read()
    assert tms.KV_WORK_ZERO == int(re.search(r"#define TMS_KV_WORK_ZERO (\d+)", header).group(1))


@pytest.mark.parametrize("length,new,dim,bf16", [(20000, 18, 64, True), (30000, 2, 64, True), (15000, 30, 128, False),
                                                 (9000, 60, 256, True), (700, 3, 64, False)])
def test_marked_values_show_any_block_left_out_or_counted_twice(length, new, dim, bf16):
    """Mistakes planted in the plain form: keys of 16 or more dropped or twice."""
    rng = np.random.default_rng(length)
    q, k = 0.7 * rng.standard_normal((new, 1, dim)), rng.standard_normal((length + new, 1, dim))
    v = marked_values(length + new, 1, dim)
    want, bound = attention(q, k, v, length, dim ** -0.5, None, bf16)
    for size in (16, 32, 64, 128):
        for t in rng.integers(0, length // size, 5) * size:
            keep = np.r_[0:t, t + size:length + new]
            out, _ = attention(q, k[keep], v[keep], length - size, dim ** -0.5, None, bf16)
            assert (np.abs(out - want) > 2 * bound).any(axis=(1, 2)).all(), (size, t)
            twice = np.r_[0:t + size, t:length + new]
            out, _ = attention(q, k[twice], v[twice], length + size, dim ** -0.5, None, bf16)
            assert (np.abs(out - want) > 2 * bound).any(axis=(1, 2)).all(), (size, t)


def test_the_plain_forms():
    """The oracles against cases worked out by hand."""
    assert ancestors([-1, 0, 0, 2, 7]).tolist() == [
        [True, False, False, False, False], [True, True, False, False, False], [True, False, True, False, False],
        [True, False, True, True, False], [False, False, False, False, True]]
    q = np.zeros((2, 1, 64))
    k = np.zeros((3, 1, 64))
    v = np.arange(3.0)[:, None, None] * np.ones((3, 1, 64))
    out, bound = attention(q, k, v, 1, 1.0, None, False)  # equal weights: means of what a token sees
    assert np.allclose(out[0], 0.5) and np.allclose(out[1], 1.0) and (bound < 1e-4).all()
    out, _ = attention(q, k, v, 1, 1.0, [-1, -1], False)
    assert np.allclose(out[0], 0.5) and np.allclose(out[1], 1.0)
    x = np.zeros((1, 1, 64))
    x[..., 0], x[..., 32] = 3.0, 4.0
    y, _ = head(x, None, 0.0, np.array([1]), np.full(32, np.pi / 2, np.float32), False, False)
    assert np.allclose(y[0, 0, [0, 32]], [-4.0, 3.0], atol=1e-6)
    y, _ = head(x, np.full(64, 2.0), 0.0, np.array([0]), None, False, False)
    assert np.allclose(y[0, 0, 0], 2 * 3.0 / np.sqrt(25 / 64))
    m = Pages(3, 4, 8, 3)
    m.reserve([5, 0, 0])
    m.commit([5, 0, 0], None, [list("abcde"), [], []])
    m.fork([0, 0, -1])
    m.reserve([1, 4, 0])
    assert m.table == [[1], [2, 3], []] and m.refs() == [0, 1, 1, 1]
    m.commit([0, 2, 0], [[0, 0], [1, 3], [0, 0]], [["x"], list("wxyz"), []])
    assert m.rows[1] == list("abcdexz") and m.table[1] == [2]
    m.reserve([20, 20, 0])
    assert m.status == [Pages.INVALID, Pages.INVALID, 0]
