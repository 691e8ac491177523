"""Outputs that share memory with what other rows still read are refused, through the C ABI (CPU: no call here launches)."""

import ctypes
import os

import pytest

import nvfp4_weight_dense_amd as nv

M, K = 6, 64
ROWS = 2 * M * K  # bytes of bf16 rows
P = [0x100000 * (i + 1) for i in range(12)]  # aligned addresses far apart that are never read


def _lib():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_weight_dense_amd import build
        build.build()
    return nv.load_library()


def _quant(x=P[0], codes=P[1], rs=P[2]):
    return _lib().int8_quantize_rows(x, M, K, codes, rs, None)


def _norm(x=P[0], weight=P[1], out=None, codes=None, rs=None):
    return _lib().rms_norm(x, M, K, weight, 0.0, 1e-6, out, codes, rs, None)


def _residual(residual=P[0], y=P[1], post=1, pw=P[2], gate=P[3], gates=2, next=1, nw=P[4], h=P[5], out=None, codes=None, rs=None):
    return _lib().rms_norm_residual(residual, y, M, K, post, pw, gate, gates, 1.0, next, nw, 0.0, 1e-6, h, out, codes, rs, None)


def _gemm(x=P[0], xs=None, w=P[1], ws=P[2], y=P[3], workspace=P[4]):
    return _lib().int8_gemm_w8a8(x, xs, M, ctypes.byref(nv._CInt8Weight(w, ws, 96, K)), y, workspace, 1 << 30, None)


def _ffn(x=P[0], wd=P[1], ds=P[2], out=P[3], workspace=P[4]):
    w = nv._CInt8Weight(P[5], P[6], 96, K)
    d = nv._CInt8Weight(wd, ds, K, 96)
    r = ctypes.byref
    return _lib().dense_ffn_forward_int8(x, None, M, K, 96, r(w), r(w), r(d), out, workspace, 1 << 30, None)


INT8 = dict(codes=P[8], rs=P[9])


@pytest.mark.parametrize("call,kw,text", [
    (_quant, dict(codes=P[0]), "codes is"), (_quant, dict(codes=P[0] + 16), "codes"), (_quant, dict(codes=P[0] + ROWS - 16), "codes"),
    (_quant, dict(codes=P[0] - M * K + 16), "codes"), (_quant, dict(rs=P[0] + 4), "row_scale"), (_quant, dict(rs=P[1] + 64), "row_scale"),
    (_quant, dict(rs=P[1] - 4 * M + 4), "row_scale"),
    (_norm, dict(out=P[0] + 2 * K), "out"), (_norm, dict(out=P[0] - 2 * K), "out"), (_norm, dict(out=P[1]), "out"),
    (_norm, dict(out=P[1] - ROWS + 16), "out"), (_norm, dict(codes=P[1], rs=P[9]), "codes"), (_norm, dict(codes=P[0] + 16, rs=P[9]), "codes"),
    (_norm, dict(codes=P[8], rs=P[1]), "row_scale"), (_norm, dict(codes=P[8], rs=P[0] + ROWS - 4), "row_scale"),
    (_norm, dict(codes=P[8], rs=P[8]), "row_scale"),
    (_residual, dict(h=P[3], out=P[6]), "h"), (_residual, dict(h=P[2], out=P[6]), "h"), (_residual, dict(h=P[4], out=P[6]), "h"),
    (_residual, dict(h=P[0] + 2 * K, out=P[6]), "h"), (_residual, dict(h=P[1] - 2 * K, out=P[6]), "h"),
    (_residual, dict(h=P[3] - ROWS + 16, out=P[6]), "h"),
    (_residual, dict(out=P[3]), "out"), (_residual, dict(out=P[3] + 2 * K), "out"), (_residual, dict(out=P[2]), "out"),
    (_residual, dict(out=P[4]), "out"), (_residual, dict(out=P[5] + 2 * K), "out"), (_residual, dict(out=P[1] + 16), "out"),
    (_residual, {**INT8, "codes": P[3]}, "codes"), (_residual, {**INT8, "codes": P[2]}, "codes"), (_residual, {**INT8, "codes": P[4]}, "codes"),
    (_residual, {**INT8, "codes": P[0] + 16}, "codes"), (_residual, {**INT8, "codes": P[5] + 16}, "codes"),
    (_residual, {**INT8, "rs": P[3]}, "row_scale"), (_residual, {**INT8, "rs": P[4]}, "row_scale"), (_residual, {**INT8, "rs": P[1] + 8}, "row_scale"),
    (_residual, {**INT8, "rs": P[5]}, "row_scale"), (_residual, {**INT8, "rs": P[8]}, "row_scale"),
    (_gemm, dict(y=P[0] + 16), "y"), (_gemm, dict(y=P[0] - 16), "y"), (_gemm, dict(y=P[1]), "y"), (_gemm, dict(y=P[2]), "y"),
    (_gemm, dict(xs=P[7], y=P[7]), "y"), (_gemm, dict(xs=P[7], y=P[0] + M * K - 16), "y"),
    (_ffn, dict(out=P[1]), "out"), (_ffn, dict(out=P[1] + 96 * K - 16), "out"), (_ffn, dict(out=P[2]), "out"),
])
def test_refused(call, kw, text):
    assert call(**kw) == nv.NVFP4_EINVAL
    assert text in nv.nvfp4_last_error() and "expected" not in nv.nvfp4_last_error()


@pytest.mark.parametrize("call,kw", [
    (_quant, dict()), (_quant, dict(codes=P[0] + ROWS)), (_quant, dict(codes=P[0] - M * K)), (_norm, dict(out=P[0])), (_norm, dict(out=P[5])),
    (_norm, INT8), (_norm, dict(out=P[1] + 2 * K)), (_norm, dict(out=P[6], weight=None)), (_residual, dict(out=P[6])),
    (_residual, INT8), (_residual, dict(h=P[0], out=P[1])), (_residual, dict(h=P[1], out=P[0])), (_residual, dict(h=P[0], **INT8)),
    (_residual, dict(out=P[3] + 4 * K)), (_residual, dict(out=P[2], post=0)), (_residual, dict(h=P[4], next=0)), (_gemm, dict()),
    (_gemm, dict(y=P[0] + ROWS)), (_ffn, dict()), (_ffn, dict(out=P[0])),
])
def test_not_refused(call, kw, monkeypatch):
    """What may share memory, or lies next to it: it gets as far as the device (there is none here, or it is not asked)."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("these addresses are not memory")
    assert call(**kw) in (nv.NVFP4_EHIP, nv.NVFP4_ENOMEM), nv.nvfp4_last_error()
