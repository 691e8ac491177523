"""Refusals of the int8 products and the norms, through the C ABI and the binding (CPU: no call here launches)."""

import ctypes
import math
import os

import pytest
import torch

import int8_ref as ref
import nvfp4_weight_dense_amd as nv

P = 0x100000  # a 16-byte aligned address that is never read


def _lib():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_weight_dense_amd import build
        build.build()
    return nv.load_library()


def _w(n=64, k=64, codes=P, scales=P):
    return nv._CInt8Weight(codes, scales, n, k)


def _gemm(m=2, w=None, x=P, xs=None, y=2 * P, workspace=None, size=0):
    return _lib().int8_gemm_w8a8(x, xs, m, None if w is None else ctypes.byref(w), y, workspace, size, None)


def _ffn(m=2, hidden=64, inter=96, wg=None, wu=None, wd=None, x=P, xs=None, out=P, workspace=None, size=0):
    r = ctypes.byref
    return _lib().dense_ffn_forward_int8(x, xs, m, hidden, inter, r(wg or _w(inter, hidden)), r(wu or _w(inter, hidden)),
                                         r(wd or _w(hidden, inter)), out, workspace, size, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(w=None), nv.NVFP4_EINVAL, "null weight"), (dict(w=_w(codes=None)), nv.NVFP4_EINVAL, "null codes"),
    (dict(w=_w(scales=None)), nv.NVFP4_EINVAL, "null codes or scales"), (dict(w=_w(n=0)), nv.NVFP4_ESHAPE, "positive"),
    (dict(w=_w(k=48)), nv.NVFP4_ESHAPE, "multiple of 32"), (dict(w=_w(k=131104)), nv.NVFP4_ESHAPE, "exceed"),
    (dict(w=_w(n=(1 << 21) + 1)), nv.NVFP4_ESHAPE, "exceed"), (dict(w=_w(codes=P + 8)), nv.NVFP4_EINVAL, "16-byte"),
    (dict(w=_w(scales=P + 2)), nv.NVFP4_EINVAL, "4-byte"), (dict(w=_w(), m=-1), nv.NVFP4_EINVAL, "negative"),
    (dict(w=_w(), m=4194241), nv.NVFP4_ESHAPE, "exceeds"), (dict(w=_w(), x=None), nv.NVFP4_EINVAL, "x: null"),
    (dict(w=_w(), x=P + 2), nv.NVFP4_EINVAL, "x: must be"), (dict(w=_w(), y=None), nv.NVFP4_EINVAL, "y: null"),
    (dict(w=_w(), xs=P + 1), nv.NVFP4_EINVAL, "row_scale"),
    (dict(w=_w(), workspace=P + 16, size=1 << 30), nv.NVFP4_EINVAL, "256-byte"),
    (dict(w=_w(), workspace=P, size=1), nv.NVFP4_EINVAL, "bytes"),
    (dict(w=_w(), workspace=P, size=-1), nv.NVFP4_EINVAL, "bytes"),
    (dict(w=_w(), y=P), nv.NVFP4_EINVAL, "y is x"),
    (dict(w=_w(), m=0), nv.NVFP4_OK, ""), (dict(w=_w(), m=0, x=None, y=None), nv.NVFP4_OK, ""),
])
def test_product_refusals(kw, code, text):
    assert _gemm(**kw) == code and text in nv.nvfp4_last_error()


@pytest.mark.parametrize("kw,code,text", [
    (dict(wd=_w(96, 64)), nv.NVFP4_ESHAPE, "wd must be"), (dict(wu=_w(96, 32)), nv.NVFP4_ESHAPE, "wg/wu must be"),
    (dict(wg=_w(64, 64)), nv.NVFP4_ESHAPE, "wg/wu must be"), (dict(hidden=0, wg=_w()), nv.NVFP4_ESHAPE, "positive"),
    (dict(wg=_w(96, 64, scales=None)), nv.NVFP4_EINVAL, "wg: null"), (dict(out=P + 4), nv.NVFP4_EINVAL, "out"),
    (dict(xs=P + 2), nv.NVFP4_EINVAL, "row_scale"), (dict(m=-3), nv.NVFP4_EINVAL, "negative"),
    (dict(workspace=P, size=256), nv.NVFP4_EINVAL, "dense_ffn_forward_int8: the workspace"), (dict(m=0), nv.NVFP4_OK, ""),
])
def test_ffn_refusals(kw, code, text):
    assert _ffn(**kw) == code and text in nv.nvfp4_last_error()


def test_workspace_sizes():
    """They grow with the rows, hold what the call asks for, and refuse what the call refuses."""
    L, r = _lib(), ctypes.byref
    rows = [0, 1, 2, 16, 17, 33, 64, 65, 128, 129, 256, 257, 511, 512, 513, 1024, 2048, 4096, 8191, 65536, 4194240]
    for n, k in ((1, 32), (7001, 4128), (17408, 5120), (5120, 17408), (256, 131072)):
        got = [L.int8_gemm_workspace(m, r(_w(n, k))) for m in rows]
        assert got == sorted(got) and all(x >= m * (k + 4) for x, m in zip(got, rows))
    for h, i in ((32, 32), (4096, 12288), (5120, 17408)):
        got = [L.dense_ffn_int8_workspace(m, h, i) for m in rows]
        assert got == sorted(got)
    assert L.int8_gemm_workspace(-1, r(_w())) == nv.NVFP4_EINVAL
    assert L.int8_gemm_workspace(1, r(_w(k=16))) == nv.NVFP4_ESHAPE
    assert L.dense_ffn_int8_workspace(1, 48, 64) == nv.NVFP4_ESHAPE
    assert L.dense_ffn_int8_workspace(1, 64, 131104) == nv.NVFP4_ESHAPE
    w = nv.Int8Weight(torch.zeros(64, 64, dtype=torch.int8), torch.zeros(64))
    assert nv.int8_workspace(5, w).numel() == L.int8_gemm_workspace(5, r(_w())) and not nv.int8_workspace(5, w).any()
    with pytest.raises(ValueError, match="2 weights"):
        nv.int8_workspace(5, w, w)
    with pytest.raises(ValueError, match="32 bits"):
        nv.int8_workspace(2 ** 32 + 1, w)


def _quant(m=2, k=64, x=P, codes=P, rs=P):
    return _lib().int8_quantize_rows(x, m, k, codes, rs, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(k=12), nv.NVFP4_ESHAPE, "multiple of 8"), (dict(k=0), nv.NVFP4_ESHAPE, "positive"),
    (dict(k=131080), nv.NVFP4_ESHAPE, "131072"), (dict(codes=None), nv.NVFP4_EINVAL, "null"),
    (dict(rs=None), nv.NVFP4_EINVAL, "null"), (dict(codes=P + 8), nv.NVFP4_EINVAL, "16-byte"),
    (dict(rs=P + 2), nv.NVFP4_EINVAL, "4-byte"), (dict(x=P + 2), nv.NVFP4_EINVAL, "16-byte"), (dict(m=0), nv.NVFP4_OK, ""),
])
def test_quantizer_refusals(kw, code, text):
    assert _quant(**kw) == code and text in nv.nvfp4_last_error()


def _norm(m=2, k=64, x=P, weight=P, offset=0.0, eps=1e-6, out=P, codes=None, rs=None):
    return _lib().rms_norm(x, m, k, weight, offset, eps, out, codes, rs, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(k=20), nv.NVFP4_ESHAPE, "multiple of 8"), (dict(k=131080), nv.NVFP4_ESHAPE, "131072"),
    (dict(weight=P + 2), nv.NVFP4_EINVAL, "weights"), (dict(offset=math.inf), nv.NVFP4_EINVAL, "offset"),
    (dict(eps=0.0), nv.NVFP4_EINVAL, "eps"), (dict(eps=-1.0), nv.NVFP4_EINVAL, "eps"), (dict(eps=2.0), nv.NVFP4_EINVAL, "eps"),
    (dict(eps=math.nan), nv.NVFP4_EINVAL, "eps"), (dict(out=None), nv.NVFP4_EINVAL, "expected out"),
    (dict(codes=P, rs=P), nv.NVFP4_EINVAL, "expected out"), (dict(out=None, codes=P), nv.NVFP4_EINVAL, "expected out"),
    (dict(out=None, rs=P), nv.NVFP4_EINVAL, "expected out"), (dict(out=P + 2), nv.NVFP4_EINVAL, "16-byte"),
    (dict(out=None, codes=P + 4, rs=P), nv.NVFP4_EINVAL, "16-byte"), (dict(x=None), nv.NVFP4_EINVAL, "null"),
    (dict(m=0), nv.NVFP4_OK, ""),
])
def test_norm_refusals(kw, code, text):
    assert _norm(**kw) == code and text in nv.nvfp4_last_error()


def _residual(m=6, k=64, residual=P, y=P, post=1, pw=P, gate=None, gates=0, scale=1.0, next=1, nw=P, offset=0.0, eps=1e-6,
              h=P, out=2 * P, codes=None, rs=None):
    return _lib().rms_norm_residual(residual, y, m, k, post, pw, gate, gates, scale, next, nw, offset, eps, h, out, codes,
                                    rs, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(residual=None), nv.NVFP4_EINVAL, "residual"), (dict(y=P + 2), nv.NVFP4_EINVAL, "y:"), (dict(h=None), nv.NVFP4_EINVAL, "h:"),
    (dict(k=4), nv.NVFP4_ESHAPE, "multiple of 8"), (dict(pw=P + 1), nv.NVFP4_EINVAL, "weights"),
    (dict(nw=P + 1), nv.NVFP4_EINVAL, "weights"), (dict(scale=math.nan), nv.NVFP4_EINVAL, "scale"),
    (dict(gate=P), nv.NVFP4_EINVAL, "gates=0"), (dict(gates=2), nv.NVFP4_EINVAL, "gates=2"),
    (dict(gate=P, gates=-2), nv.NVFP4_EINVAL, "gates=-2"), (dict(gate=P, gates=4), nv.NVFP4_ESHAPE, "divide"),
    (dict(gate=P + 8, gates=2), nv.NVFP4_EINVAL, "gate must"), (dict(out=None), nv.NVFP4_EINVAL, "expected out"),
    (dict(next=0), nv.NVFP4_EINVAL, "without a next norm"), (dict(next=0, out=None, codes=P), nv.NVFP4_EINVAL, "without"),
    (dict(out=P), nv.NVFP4_EINVAL, "one array"),
    (dict(eps=0.0), nv.NVFP4_EINVAL, "eps"), (dict(m=0), nv.NVFP4_OK, ""), (dict(m=0, gate=P, gates=4), nv.NVFP4_OK, ""),
])
def test_residual_refusals(kw, code, text):
    assert _residual(**kw) == code and text in nv.nvfp4_last_error()


@pytest.mark.parametrize("call,kw", [
    (_quant, dict()), (_norm, dict(out=None, codes=P, rs=2 * P)), (_residual, dict(out=None, codes=P, rs=2 * P, y=3 * P, h=4 * P)),
    (_residual, dict(out=None, codes=P, rs=2 * P, residual=3 * P, h=4 * P)),
    (_residual, dict(out=None, codes=P, rs=2 * P, residual=3 * P, y=4 * P)),
])
def test_codes_are_no_input(call, kw):
    """A row's codes lie where other rows' values would still be read."""
    assert call(**kw) == nv.NVFP4_EINVAL and "codes is" in nv.nvfp4_last_error()


BF = torch.bfloat16


def test_binding_refusals():
    """Shapes and types first, then the device (these tensors are on the CPU)."""
    _lib()
    x = torch.zeros(2, 64, dtype=BF)
    W = lambda n=8, k=64: nv.Int8Weight(torch.zeros(n, k, dtype=torch.int8), torch.zeros(n))  # noqa: E731

    def bad(text, fn, *a, **kw):
        with pytest.raises(ValueError, match=text):
            fn(*a, **kw)

    bad("codes", nv.int8_gemm_w8a8, x, nv.Int8Weight(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8)))
    bad("scales", nv.int8_gemm_w8a8, x, nv.Int8Weight(torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8, dtype=BF)))
    bad("scales", nv.int8_gemm_w8a8, x, nv.Int8Weight(torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8, 1)))
    bad("columns", nv.int8_gemm_w8a8, x, W(8, 32))
    bad("2-D", nv.int8_gemm_w8a8, x.float(), W())
    bad("2-D", nv.int8_gemm_w8a8, x.t(), W(8, 2))
    bad("y:", nv.int8_gemm_w8a8, x, W(), torch.zeros(2, 9, dtype=BF))
    bad("workspace", nv.int8_gemm_w8a8, x, W(), workspace=torch.zeros(256))
    rows = lambda m=2, k=64, n=2: nv.Int8Rows(torch.zeros(m, k, dtype=torch.int8), torch.zeros(n))  # noqa: E731
    bad("row_scale", nv.int8_gemm_w8a8, rows(n=3), W())
    bad("columns", nv.int8_gemm_w8a8, rows(k=32), W())
    bad("x codes", nv.int8_gemm_w8a8, nv.Int8Rows(x, torch.zeros(2)), W())
    bad("GPU", nv.int8_gemm_w8a8, rows(), W())
    bad("wd", nv.dense_ffn_forward_int8, x, W(96), W(96), W(96))
    bad("wu", nv.dense_ffn_forward_int8, x, W(96), W(64), W(64, 96))
    bad("out:", nv.dense_ffn_forward_int8, x, W(96), W(96), W(64, 96), torch.zeros(2, 96, dtype=BF))
    bad("GPU", nv.dense_ffn_forward_int8, x, W(96), W(96), W(64, 96))
    bad("2-D", nv.int8_quantize_rows, x[0])
    bad("GPU", nv.int8_quantize_rows, x)
    bad("weight", nv.rms_norm, x, torch.zeros(32, dtype=BF))
    bad("weight", nv.rms_norm, x, torch.zeros(64))
    bad("out", nv.rms_norm, x, int8=True, out=x)
    bad("out:", nv.rms_norm, x, out=torch.zeros(2, 32, dtype=BF))
    bad("GPU", nv.rms_norm, x)
    bad("y:", nv.rms_norm_residual, x, torch.zeros(3, 64, dtype=BF))
    bad("post", nv.rms_norm_residual, x, x, post=torch.zeros(32, dtype=BF))
    bad("norm", nv.rms_norm_residual, x, x, norm=torch.zeros(2, 64, dtype=BF))
    bad("gate", nv.rms_norm_residual, x, x, gate=torch.zeros(64))
    bad("gate", nv.rms_norm_residual, x, x, gate=torch.zeros(2, 32, dtype=BF))
    bad("divide", nv.rms_norm_residual, x, x, gate=torch.zeros(3, 64, dtype=BF))
    bad("divide", nv.rms_norm_residual, x, x, gate=torch.zeros(0, 64, dtype=BF))
    bad("int8", nv.rms_norm_residual, x, x, int8=True)
    bad("out", nv.rms_norm_residual, x, x, out=x)
    bad("h:", nv.rms_norm_residual, x, x, h=torch.zeros(2, 64))
    bad("GPU", nv.rms_norm_residual, x, x, norm=True)


@pytest.mark.parametrize("current,tensors", [(0, 1), (2, 0)])
def test_another_current_device_is_refused(monkeypatch, current, tensors):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    monkeypatch.setattr(nv, "_gpu", lambda *t: None)

    class On:
        device = f"cuda:{tensors}"

        def get_device(self):
            return tensors
    with pytest.raises(ValueError, match=f"cuda:{tensors}.*cuda:{current}"):
        nv._on_current(On())


def test_reference_quantizer_by_hand():
    """amax 127 -> s = 1; ties go to the even code; a row of zeros; rows with an infinity or a NaN."""
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 0.0], [0.0] * 8, [1.0, math.inf] + [2.0] * 6,
                      [1.0, math.nan] + [2.0] * 6, [254.0, 1.0, 3.0, -254.0, 5.0, 253.0, -1.0, 2.0]]).bfloat16()
    codes, s = ref.quantize(x)
    assert codes.tolist()[0] == [127, 0, 2, 2, 0, -2, -126, 0] and codes.tolist()[1] == [0] * 8
    assert codes[2:4].abs().sum() == 0 and s.isnan().tolist() == [False, False, True, True, False]
    assert s[[0, 1, 4]].tolist() == [1.0, 1.0, 2.0]
    assert codes.tolist()[4] == [127, 0, 2, -127, 2, 126, 0, 1]


def test_reference_norm_by_hand():
    x = torch.tensor([[3.0, 4.0, 0.0, 0.0, 0.0, 0.0, 0.0, 5.0]]).bfloat16()  # mean of squares 50/8 = 6.25
    w = torch.full((8,), 0.5).bfloat16()
    got = ref.norm(x, w, 1.0, 1e-18)
    assert torch.allclose(got, x.double() / 2.5 * 1.5, rtol=1e-12)
    h, _ = ref.residual(x, x, True, torch.full((1, 8), 2.0).bfloat16(), 0.25, 0.0, 1e-18)
    assert torch.allclose(h, x.double() * 1.2, rtol=1e-12)
