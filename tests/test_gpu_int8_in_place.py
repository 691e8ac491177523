"""Outputs in place of inputs, where the header allows it, on the GPU."""

import pytest
import torch

import nvfp4_weight_dense_amd as nv

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _weight(g, n, k):
    return nv.Int8Weight(torch.randint(-127, 128, (n, k), generator=g, device="cuda").to(torch.int8),
                         (torch.rand(n, generator=g, device="cuda") + 0.5) * (k ** -0.5 / 74))


@pytest.mark.parametrize("m", [1, 4, 40, 100, 700])
def test_ffn_over_its_input(m):
    print("ffn in place", m, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m)
    W = [_weight(g, 1056, 512), _weight(g, 1056, 512), _weight(g, 512, 1056)]
    x = torch.randn(m, 512, generator=g, device="cuda").to(BF)
    want = nv.dense_ffn_forward_int8(x, *W)
    assert torch.equal(nv.dense_ffn_forward_int8(x, *W, x), want) and torch.equal(x, want)


# widths of one piece a thread, of several that are held and of several that are read again, and past 65536
@pytest.mark.parametrize("k", [264, 5120, 40000, 70000])
def test_end_of_a_block_over_its_inputs(k):
    """h and out over residual and y, either way round; h over either with int8 rows."""
    print("residual in place", k, flush=True)
    g = torch.Generator(device="cuda").manual_seed(k)
    r, y = (torch.randn(37, k, generator=g, device="cuda").to(BF) for _ in range(2))
    w, gate = (torch.randn(k, generator=g, device="cuda").to(BF) for _ in range(2))
    call = lambda a, b, **kw: nv.rms_norm_residual(a, b, post=w, gate=gate, scale=0.5, norm=w, **kw)  # noqa: E731
    h, n = call(r, y)
    for into in ("ry", "yr"):
        a, b = r.clone(), y.clone()
        h2, n2 = call(a, b, **dict(zip(("h", "out"), (a, b) if into == "ry" else (b, a))))
        assert torch.equal(h2, h) and torch.equal(n2, n), into
    q = call(r, y, int8=True)[1]
    for over in (0, 1):
        ab = r.clone(), y.clone()
        h2, q2 = call(*ab, h=ab[over], int8=True)
        assert torch.equal(h2, h) and torch.equal(q2.codes, q.codes) and torch.equal(q2.row_scale, q.row_scale), over
