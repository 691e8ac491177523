"""The int8 products through every kernel that their plans choose, and every way through it, on the GPU
(tests/int8_shapes.py)."""

import math

import pytest
import torch

import int8_ref as ref
import int8_shapes as shapes
import nvfp4_weight_dense_amd as nv

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda").to(torch.int8)


@pytest.mark.parametrize("m,n,k", shapes.ONE)
def test_one_matrix(m, n, k):
    """Against the sum in 64 bits (exact: whole numbers below 2^53); what lies behind the last row is left as it was."""
    print("product", m, n, k, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x = nv.Int8Rows(_codes(g, m, k), torch.rand(m, generator=g, device="cuda") + 0.5)
    w = nv.Int8Weight(_codes(g, n, k), torch.rand(n, generator=g, device="cuda") + 0.5)
    y = torch.full((m * n + 64,), 7.0, dtype=BF, device="cuda")
    got = nv.int8_gemm_w8a8(x, w, y[:m * n].view(m, n))
    for r in range(0, m, 512):
        want = x.codes[r:r + 512].double() @ w.codes.double().t()
        want *= x.row_scale[r:r + 512].double()[:, None] * w.scales.double()
        over = ((got[r:r + 512].double() - want).abs() / ref.product_bound(want)).nan_to_num(nan=math.inf)
        assert float(over.max()) <= 1.0, (m, n, k, r)
    assert bool((y[m * n:] == 7.0).all())


@pytest.mark.parametrize("m,inter,hidden", shapes.TWO)
def test_two_matrices(m, inter, hidden):
    """An FFN has the bits of its steps one by one, each a kernel of one matrix.  The down projection's weight is a
    unit matrix (repeated where hidden is the longer), so that every value of act is seen in the result, as the code
    that it was given."""
    print("gate and up", m, inter, hidden, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + inter + hidden)
    x = nv.Int8Rows(_codes(g, m, hidden), torch.rand(m, generator=g, device="cuda") + 0.5)
    scale = lambda n: (torch.rand(n, generator=g, device="cuda") + 0.5) * (hidden ** -0.5 / 5000)  # noqa: E731
    wg, wu = (nv.Int8Weight(_codes(g, inter, hidden), scale(inter)) for _ in range(2))
    d = torch.zeros(hidden, inter, dtype=torch.int8, device="cuda")
    at = torch.arange(max(hidden, inter), device="cuda")
    d[at % hidden, at % inter] = (1 + at % 100).to(torch.int8)
    wd = nv.Int8Weight(d, torch.rand(hidden, generator=g, device="cuda") + 0.5)
    out = torch.full((m + 2, hidden), 7.0, dtype=BF, device="cuda")
    got = nv.dense_ffn_forward_int8(x, wg, wu, wd, out[:m])
    act = nv.silu_mul(nv.int8_gemm_w8a8(x, wg), nv.int8_gemm_w8a8(x, wu))
    assert torch.equal(got, nv.int8_gemm_w8a8(act, wd))
    assert bool((out[m:] == 7.0).all()) and bool(got.any())


# where the kernel for few rows takes bf16 rows no more (longest rows of 3 and 4, of 1 and 2), and where its LDS ends
@pytest.mark.parametrize("k", [16352, 16384, 16416, 18464, 32768, 32800])
@pytest.mark.parametrize("m", [1, 2, 3, 4])
def test_few_long_rows(m, k):
    """The bits of the same rows among more, as bf16 and as int8."""
    print("few rows", m, k, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + k)
    x = torch.randn(7, k, generator=g, device="cuda").to(BF)
    w = nv.Int8Weight(_codes(g, 300, k), torch.rand(300, generator=g, device="cuda") + 0.5)
    want = nv.int8_gemm_w8a8(x, w)[:m]
    assert torch.equal(nv.int8_gemm_w8a8(x[:m], w), want)
    assert torch.equal(nv.int8_gemm_w8a8(nv.int8_quantize_rows(x[:m]), w), want)
