"""The int8 operators and the norms on arrays whose offsets pass 32 bits, on the GPU: rows on either side of each 2^31st
and 2^32nd byte and element have the bits that they have in a small batch."""

import pytest
import torch

import nvfp4_weight_dense_amd as nv

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _places(m, row_bytes):
    """Rows around the places in an array of rows of so many bytes, where 31 or 32 bits of an offset end."""
    at = {0, m - 1}
    for b in (2 ** 31, 2 ** 32):
        at |= {b // row_bytes - 1, b // row_bytes, b // row_bytes + 1}
    return sorted(r for r in at if 0 <= r < m)


def test_rows_far_apart():
    k = 65536
    m = 2 ** 32 // k + 3  # elements past 2^32
    print("far rows", m, k, flush=True)
    places = sorted({r for b in (1, 2) for r in _places(m, b * k)})
    g = torch.Generator(device="cuda").manual_seed(1)
    some, other = (torch.randn(len(places), k, generator=g, device="cuda").to(BF) for _ in range(2))
    w = torch.randn(k, generator=g, device="cuda").to(BF)
    x = torch.zeros(m, k, dtype=BF, device="cuda")
    x[places] = some
    q, few = nv.int8_quantize_rows(x), nv.int8_quantize_rows(some)
    assert torch.equal(q.codes[places], few.codes) and torch.equal(q.row_scale[places], few.row_scale)
    weight = nv.Int8Weight(torch.randint(-127, 128, (40, k), generator=g, device="cuda").to(torch.int8), torch.ones(40, device="cuda"))
    assert torch.equal(nv.int8_gemm_w8a8(q, weight)[places], nv.int8_gemm_w8a8(few, weight))
    del q
    assert torch.equal(nv.rms_norm(x, w)[places], nv.rms_norm(some, w))
    y = torch.zeros(m, k, dtype=BF, device="cuda")
    y[places] = other
    h, n = nv.rms_norm_residual(x, y, post=True, scale=0.5, norm=w, int8=True)
    h2, n2 = nv.rms_norm_residual(some, other, post=True, scale=0.5, norm=w, int8=True)
    assert torch.equal(h[places], h2) and torch.equal(n.codes[places], n2.codes) and torch.equal(n.row_scale[places], n2.row_scale)


def test_results_far_apart():
    m, n, k = 131077, 32771, 64  # results past 2^32
    print("far results", m, n, k, flush=True)
    places = sorted({r for b in (1, 2) for r in _places(m, b * n)})
    g = torch.Generator(device="cuda").manual_seed(2)
    x = nv.Int8Rows(torch.randint(-127, 128, (m, k), generator=g, device="cuda").to(torch.int8), torch.rand(m, generator=g, device="cuda"))
    w = nv.Int8Weight(torch.randint(-127, 128, (n, k), generator=g, device="cuda").to(torch.int8), torch.rand(n, generator=g, device="cuda"))
    y = nv.int8_gemm_w8a8(x, w)
    assert torch.equal(y[places], nv.int8_gemm_w8a8(nv.Int8Rows(x.codes[places], x.row_scale[places]), w))
