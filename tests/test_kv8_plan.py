"""The KV cache attention's workspace: what kv8_attention_workspace gives holds what any call of these sizes or
smaller ones plans (CPU)."""

import ctypes
import os
import re
import subprocess

import pytest

import nvfp4_weight_dense_amd as nv
from nvfp4_weight_dense_amd import build
from test_kv8_checks import P, _attention, _batch, _cache, _lib

HERE = os.path.dirname(os.path.abspath(__file__))


def test_plans_fit_their_bound(tmp_path):
    exe = str(tmp_path / "sweep")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", f"-I{build.CSRC}", "-o", exe,
                    os.path.join(HERE, "kv8_plan_sweep.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    got = re.search(r"^checked=(\d+) over=(\d+)$", r.stdout, re.M)
    assert got and int(got[1]) > 200000 and int(got[2]) == 0, r.stdout + r.stderr


def _bytes(weights=None, heads=8, q_heads=32, dim=128, pages=8, **kw):
    n = _lib().kv8_attention_workspace(q_heads, ctypes.byref(_cache(weights=weights, heads=heads, dim=dim, pages=pages,
                                                                    page=128)),
                                       ctypes.byref(_batch(cols=1 << 16, **kw)))
    assert n > 0, nv.nvfp4_last_error()
    return n


@pytest.mark.parametrize("weights", [None, P])
@pytest.mark.parametrize("rows", [1, 4, 32, 200])
def test_smaller_calls_need_no_more(rows, weights):
    """Lengths up to where a sequence's pieces are taken in two and three rounds."""
    lens = [1, 3968, 3969, 131072, 422923, 507904, 507905, 600000, 1015808, 1015809, 1 << 21]
    sizes = [_bytes(weights, seqs=8, rows=8 * rows, max_rows=rows, max_len=n) for n in lens]
    assert sizes == sorted(sizes)
    for n, size in zip(lens, sizes):
        assert _bytes(weights, seqs=8, rows=8, max_rows=1, max_len=n) <= size


def test_a_workspace_short_of_the_call_is_refused():
    """A window's own plan counts: here its pieces take 58 MB beside the counters."""
    cache = _cache(weights=None, heads=8, dim=128, page=128)
    batch = _batch(seqs=8, rows=8, max_rows=1, cols=4096, max_len=524288)
    for size in (0, 35 << 20, 58 << 20):
        assert _attention(cache=cache, batch=batch, q_heads=32, window=454351, lse=None, workspace=P,
                          size=size) == nv.NVFP4_EINVAL
        assert "workspace" in nv.nvfp4_last_error()
