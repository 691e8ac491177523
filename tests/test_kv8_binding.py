"""What the KV cache's binding asks of its arguments beyond their shapes (CPU)."""

import ctypes

import pytest
import torch

import nvfp4_weight_dense_amd as nv
from test_kv8_checks import P, _batch, _cache, _lib, _py


@pytest.mark.parametrize("current,tensors", [(0, 1), (1, 0), (3, 2)])
def test_another_current_device_is_refused(monkeypatch, current, tensors):
    """The library's scratch and its launches are the current device's."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    with pytest.raises(ValueError, match=f"cuda:{tensors}.*cuda:{current}"):
        nv._kv8_on(tensors)
    nv._kv8_on(current)


def _noalloc(cache=None, batch=None, new_table=P, new_cols=1 << 12, keep=32, recent=8, sink=2, new_lens=P, kept=P,
             workspace=None, size=0):
    r = ctypes.byref
    return _lib().kv8_evict_noalloc(r(cache or _cache()), r(batch or _batch(rows=0, max_rows=0)), new_table, new_cols,
                                    keep, recent, sink, new_lens, kept, workspace, size, None)


def test_eviction_workspace_sizes_and_refusals():
    L, r = _lib(), ctypes.byref
    lens = [0, 1, 32768, 32769, 36000, 130001, 1 << 20]
    for seqs in (1, 3):
        got = [L.kv8_evict_workspace(r(_cache()), r(_batch(seqs=seqs, cols=1 << 16, rows=0, max_rows=0, max_len=n)))
               for n in lens]
        assert got[:3] == [0, 0, 0] and got == sorted(got) and all(x > 4 * seqs * n for x, n in zip(got[3:], lens[3:]))
    assert L.kv8_evict_workspace(r(_cache(dim=96)), r(_batch())) == nv.NVFP4_ESHAPE
    long = _batch(rows=0, max_rows=0, cols=1 << 12, max_len=40000)
    need = L.kv8_evict_workspace(r(_cache()), r(long))
    for workspace, size in ((None, need), (P, need - 1), (P, -1), (P + 16, need)):
        assert _noalloc(batch=long, workspace=workspace, size=size) == nv.NVFP4_EINVAL
        assert f"{need} bytes" in nv.nvfp4_last_error()
    for kw in (dict(cache=_cache(weights=None)), dict(keep=0), dict(recent=31), dict(new_table=None), dict(kept=P + 1)):
        assert _noalloc(**kw) == nv.NVFP4_EINVAL and "kv8_evict_noalloc" in nv.nvfp4_last_error()
    assert _noalloc(new_cols=1) == nv.NVFP4_ESHAPE
    assert _noalloc(batch=_batch(seqs=0, table=None, lens=None, rows=0)) == nv.NVFP4_OK
    with pytest.raises(ValueError, match="workspace"):
        nv.kv8_evict(**_py(), new_table=torch.zeros(2, 2, dtype=torch.int32), keep=8, workspace=torch.zeros(4))


@pytest.mark.parametrize("kw,text", [(dict(keep=2 ** 32 + 5), "keep"), (dict(recent=2 ** 32), "recent"),
                                     (dict(sink=2 ** 32 + 1), "sink"), (dict(recent=-2 ** 32), "recent")])
def test_numbers_past_32_bits_are_refused(kw, text):
    """(ctypes would take them modulo 2^32)"""
    with pytest.raises(ValueError, match=text):
        nv.kv8_evict(**_py(), new_table=torch.zeros(2, 4, dtype=torch.int32), **{"keep": 8, **kw})


def test_lengths_past_the_table_are_held_to_it():
    a = _py()
    sizes = [nv.kv8_workspace(4, a["cache"], a["table"], a["lens"], 2, max_len=n).numel() for n in (None, 64, 2 ** 40)]
    assert sizes[0] == sizes[1] == sizes[2]
    starts = torch.tensor([0, 1, 2], dtype=torch.int32)
    sizes = [nv.kv8_workspace(4, a["cache"], a["table"], a["lens"], 2, starts, max_rows=n).numel() for n in (None, 2 ** 40)]
    assert sizes[0] == sizes[1]
