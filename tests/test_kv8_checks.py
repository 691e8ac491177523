"""Refusals of the KV cache's entry points, through the C ABI and the binding (CPU: no call here launches)."""

import ctypes
import os

import pytest
import torch

import nvfp4_weight_dense_amd as nv

P = 0x100000  # a 16-byte aligned address that is never read


def _lib():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_weight_dense_amd import build
        build.build()
    return nv.load_library()


def _cache(**kw):
    a = dict(k_codes=P, v_codes=P, k_scales=P, v_scales=P, weights=P, pages=8, heads=2, dim=64, page=16)
    a.update(kw)
    return nv._CKv8Cache(**a)


def _batch(**kw):
    a = dict(table=P, lens=P, starts=None, seqs=2, cols=4, rows=2, max_rows=1, max_len=64)
    a.update(kw)
    return nv._CKv8Batch(**a)


def _rows(ptr=P, row_stride=128, head_stride=64):
    return nv._CKv8Rows(ptr, row_stride, head_stride)


def _append(cache=None, batch=None, k=None, v=None):
    L = _lib()
    r = ctypes.byref
    return L.kv8_append(r(k or _rows()), r(v or _rows()), r(cache or _cache()), r(batch or _batch()), None)


def _attention(cache=None, batch=None, q=None, q_heads=4, scale=1.0, window=0, out=P, lse=P, accumulate=0,
               workspace=None, size=0):
    L = _lib()
    r = ctypes.byref
    return L.kv8_attention(r(q or _rows()), q_heads, scale, window, r(cache or _cache()), r(batch or _batch()), out,
                           lse, accumulate, workspace, size, None)


def _evict(cache=None, batch=None, new_table=P, new_cols=4, keep=32, recent=8, sink=2, new_lens=P, kept=P):
    L = _lib()
    r = ctypes.byref
    return L.kv8_evict(r(cache or _cache()), r(batch or _batch(rows=0, max_rows=0)), new_table, new_cols, keep,
                       recent, sink, new_lens, kept, None)


BAD_CACHES = [
    (dict(k_codes=None), nv.NVFP4_EINVAL, "null codes"), (dict(v_scales=None), nv.NVFP4_EINVAL, "null codes"),
    (dict(v_codes=P + 8), nv.NVFP4_EINVAL, "16-byte"), (dict(weights=P + 2), nv.NVFP4_EINVAL, "4-byte"),
    (dict(pages=0), nv.NVFP4_ESHAPE, "pages=0"), (dict(heads=0), nv.NVFP4_ESHAPE, "heads=0"),
    (dict(dim=96), nv.NVFP4_ESHAPE, "dim=96"), (dict(page=24), nv.NVFP4_ESHAPE, "page=24"),
    (dict(page=256), nv.NVFP4_ESHAPE, "page=256"),
]
BAD_BATCHES = [
    (dict(table=None), nv.NVFP4_EINVAL, "null table"), (dict(lens=None), nv.NVFP4_EINVAL, "null table or lens"),
    (dict(lens=P + 2), nv.NVFP4_EINVAL, "4-byte"), (dict(seqs=-1), nv.NVFP4_EINVAL, "seqs=-1"),
    (dict(seqs=65536, rows=65536), nv.NVFP4_ESHAPE, "65535"), (dict(cols=0), nv.NVFP4_ESHAPE, "cols=0"),
    (dict(cols=1 << 25), nv.NVFP4_ESHAPE, "2^28"), (dict(max_len=-1), nv.NVFP4_EINVAL, "max_len=-1"),
]
BAD_ROWS = [
    (dict(ptr=None), nv.NVFP4_EINVAL, "null pointer"), (dict(ptr=P + 2), nv.NVFP4_EINVAL, "16-byte"),
    (dict(row_stride=130), nv.NVFP4_ESHAPE, "multiples of 8"), (dict(head_stride=-64), nv.NVFP4_ESHAPE, "not negative"),
]


@pytest.mark.parametrize("kw,code,text", BAD_CACHES)
@pytest.mark.parametrize("call", [_append, _attention, _evict])
def test_caches(call, kw, code, text):
    assert call(cache=_cache(**kw)) == code
    assert text in nv.nvfp4_last_error()


@pytest.mark.parametrize("kw,code,text", BAD_BATCHES)
@pytest.mark.parametrize("call", [_append, _attention, _evict])
def test_batches(call, kw, code, text):
    assert call(batch=_batch(**kw)) == code
    assert text in nv.nvfp4_last_error()


@pytest.mark.parametrize("kw,code,text", BAD_ROWS)
def test_rows(kw, code, text):
    for rc in (_append(k=_rows(**kw)), _append(v=_rows(**kw)), _attention(q=_rows(**kw))):
        assert rc == code
        assert text in nv.nvfp4_last_error()
    assert _append(batch=_batch(rows=3)) == nv.NVFP4_ESHAPE       # 3 rows over 2 sequences
    assert "without starts" in nv.nvfp4_last_error()
    assert _append(batch=_batch(rows=(1 << 24) + 2)) == nv.NVFP4_ESHAPE


def test_attention_arguments():
    assert _attention(q_heads=3) == nv.NVFP4_ESHAPE and "q_heads=3" in nv.nvfp4_last_error()
    assert _attention(q_heads=0) == nv.NVFP4_ESHAPE
    assert _attention(scale=float("nan")) == nv.NVFP4_EINVAL and "scale" in nv.nvfp4_last_error()
    assert _attention(scale=float("inf")) == nv.NVFP4_EINVAL
    assert _attention(window=-1) == nv.NVFP4_EINVAL and "window" in nv.nvfp4_last_error()
    assert _attention(out=None) == nv.NVFP4_EINVAL and _attention(out=P + 2) == nv.NVFP4_EINVAL
    assert _attention(lse=P + 2) == nv.NVFP4_EINVAL
    assert _attention(lse=None, accumulate=1) == nv.NVFP4_EINVAL and "accumulate" in nv.nvfp4_last_error()
    assert _attention(cache=_cache(weights=None), accumulate=1) == nv.NVFP4_EINVAL
    assert _attention(workspace=P, size=-1) == nv.NVFP4_EINVAL and "workspace" in nv.nvfp4_last_error()
    assert _attention(workspace=P + 16, size=1 << 40) == nv.NVFP4_EINVAL


def test_evict_arguments():
    assert _evict(cache=_cache(weights=None)) == nv.NVFP4_EINVAL and "no weights" in nv.nvfp4_last_error()
    assert _evict(keep=0) == nv.NVFP4_EINVAL and _evict(recent=-1) == nv.NVFP4_EINVAL
    assert _evict(recent=30, sink=3) == nv.NVFP4_EINVAL and "sink=3" in nv.nvfp4_last_error()
    assert _evict(recent=2 ** 31 - 1, sink=2 ** 31 - 1) == nv.NVFP4_EINVAL
    assert _evict(keep=65) == nv.NVFP4_ESHAPE and "keep=65" in nv.nvfp4_last_error()
    assert _evict(new_table=None) == nv.NVFP4_EINVAL and _evict(kept=None) == nv.NVFP4_EINVAL
    assert _evict(new_lens=P + 1) == nv.NVFP4_EINVAL


def test_empty_calls_do_nothing():
    none = _batch(seqs=0, table=None, lens=None, rows=0)
    assert _append(batch=none) == nv.NVFP4_OK and _attention(batch=none) == nv.NVFP4_OK
    assert _evict(batch=none) == nv.NVFP4_OK
    assert _append(batch=_batch(rows=0)) == nv.NVFP4_OK and _attention(batch=_batch(max_rows=0)) == nv.NVFP4_OK


def test_workspace_sizes():
    L = _lib()
    assert L.kv8_attention_workspace(4, ctypes.byref(_cache()), ctypes.byref(_batch())) >= 0
    assert L.kv8_attention_workspace(3, ctypes.byref(_cache()), ctypes.byref(_batch())) == nv.NVFP4_ESHAPE
    assert L.kv8_attention_workspace(4, None, ctypes.byref(_batch())) == nv.NVFP4_EINVAL


def _py():
    c = nv.kv8_cache(8, 2, 64, 16, weights=True, device="cpu")
    return dict(cache=c, table=torch.zeros(2, 4, dtype=torch.int32), lens=torch.ones(2, dtype=torch.int32))


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_refusals():
    a = _py()
    call = lambda k=None, v=None, **kw: nv.kv8_append(_bf(2, 2, 64) if k is None else k,  # noqa: E731
                                                      _bf(2, 2, 64) if v is None else v, **{**a, **kw})
    for kw, text in [(dict(k=torch.zeros(2, 2, 64)), "bfloat16"), (dict(k=_bf(2, 3, 64)), "2 heads"),
                     (dict(k=_bf(2, 2, 128)), "size 64"), (dict(v=_bf(4, 2, 64)), "4 rows"),
                     (dict(k=_bf(2, 64, 2).transpose(1, 2)), "strides"),
                     (dict(k=_bf(2, 2, 68)[..., :64]), "multiples of 8"),
                     (dict(table=torch.zeros(2, 4)), "table"), (dict(lens=torch.ones(3, dtype=torch.int32)), "lens"),
                     (dict(starts=torch.zeros(2, dtype=torch.int32)), "starts"),
                     (dict(), "GPU")]:
        with pytest.raises(ValueError, match=text):
            call(**kw)
    q = _bf(2, 4, 64)
    for kw, text in [(dict(out=torch.zeros(2, 4, 64)), "out"), (dict(lse=torch.zeros(2, 3)), "lse"),
                     (dict(workspace=torch.zeros(4)), "workspace"), (dict(), "GPU")]:
        with pytest.raises(ValueError, match=text):
            nv.kv8_attention(q, **{**a, **kw})
    new = torch.zeros(2, 2, dtype=torch.int32)
    for kw, text in [(dict(new_table=new[:1]), "new_table"), (dict(keep=0), "keep"), (dict(), "GPU")]:
        with pytest.raises(ValueError, match=text):
            nv.kv8_evict(**{**a, "new_table": new, "keep": 8, **kw})
    for field, bad in [("k_codes", torch.zeros(8, 2, 16, 64)), ("v_codes", torch.zeros(8, 2, 16, 128, dtype=torch.uint8)),
                       ("k_scales", torch.zeros(8, 3, dtype=torch.uint8)), ("weights", torch.zeros(8, 15))]:
        c = _py()["cache"]
        setattr(c, field, bad)
        with pytest.raises(ValueError, match=field):
            call(cache=c)


@pytest.mark.parametrize("kw", [dict(seqs=0, rows=0), dict(rows=0, max_rows=0), dict(max_len=0), dict(cols=1, max_len=1),
                                dict(rows=1 << 24, max_rows=1 << 23, cols=1 << 24, max_len=1 << 28)])
def test_workspace_sizes_at_the_ends(kw):
    L = _lib()
    small = L.kv8_attention_workspace(4, ctypes.byref(_cache()), ctypes.byref(_batch(seqs=0, rows=0)))
    got = L.kv8_attention_workspace(4, ctypes.byref(_cache()), ctypes.byref(_batch(**kw)))
    assert got >= small >= 0
