"""The plan of the shared attention without a GPU: its arithmetic
(trie_masked_sparse_amd/csrc/kv_plan.h) is compiled for the host and taken over
batches of every kind by tests/sanitize/kv_plan_driver.cpp."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

import trie_masked_sparse_amd as tms
from test_kv_host import descriptor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_units_and_parts_fit_the_plan(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "driver")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{ROOT}/include",
                    f"-I{ROOT}/trie_masked_sparse_amd/csrc", f"{ROOT}/tests/sanitize/kv_plan_driver.cpp", "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("ok ") and int(r.stdout.split()[1]) > 100000


@pytest.mark.parametrize("dtype", [tms.BF16, tms.F32])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("seqs,q_heads,kv_heads", [(16, 32, 32), (16, 64, 64), (4096, 32, 8), (300, 8, 2), (4096, 512, 256)])
def test_a_plan_for_more_tokens_is_one_for_fewer_of_many_key_heads(dtype, dim, seqs, q_heads, kv_heads):
    """Around the numbers of tokens from which small nodes have units of two heads,
    and taller row tiles."""
    L, n = tms.lib(), C.c_int64()
    d = descriptor(dtype=dtype, head_dim=dim, seqs=seqs, kv_heads=kv_heads)
    sizes = []
    for T in range(1, 600):
        assert L.tms_kv_share_bytes(C.byref(d), T, q_heads, C.byref(n)) == tms.OK
        sizes.append(n.value)
    assert sizes == sorted(sizes)
