"""silu(gate) * up against 64 bits for every gate there is, on the GPU: fp32 up to its rounding to bf16."""

import pytest
import torch

import nvfp4_weight_dense_amd as nv

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# Before it is rounded to bf16 the product is off by at most eight steps of 2^-24: exp(-t) by 2 (one ulp of the
# hardware's), 1 (its correction's rounding) and 1.7 (the correction's second order, (t * 4.9e-6)^2 / 2 at t = -92),
# the sum, the quotient and the product with up by 1 each.
REL = 8 * 2.0 ** -24
# below t = -92 silu is a subnormal fp32 number, a step of those (2^-149) off with the errors above, times up < 2
ABS = 2.0 ** -148


def _edges(v):
    """v (64 bits) rounded to bf16, half to even."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 8).clamp(min=-133))
    return torch.round(v / step) * step


@pytest.mark.parametrize("seed", range(4))
def test_every_gate(seed):
    print("silu", seed, flush=True)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    g = bits[torch.isfinite(bits.float())]
    u = (1 + torch.rand(g.numel(), generator=torch.Generator().manual_seed(seed))).to(BF).clamp(max=1.9921875)
    u = torch.where(torch.arange(g.numel()) % 2 > 0, -u, u)
    got = nv.silu_mul(g.cuda()[None], u.cuda()[None])[0].cpu().double()
    want = g.double() * torch.sigmoid(g.double()) * u.double()
    off = want.abs() * REL + ABS
    lo, hi = _edges(want - off), _edges(want + off)
    past = torch.tensor(torch.finfo(BF).max, dtype=torch.float64)
    fine = want.abs() < past
    bad = fine & ~((lo <= got) & (got <= hi))
    assert not bad.any(), (int(bad.sum()), g[bad][:5].tolist(), u[bad][:5].tolist(), got[bad][:5].tolist(), want[bad][:5].tolist())
    assert torch.isinf(got[~fine & (want.abs() > past * (1 + 2.0 ** -8))]).all()


def test_gates_that_are_not_finite():
    print("silu inf", flush=True)
    g = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0], dtype=BF)
    got = nv.silu_mul(g.cuda()[None], torch.ones(1, 5, dtype=BF, device="cuda"))[0].cpu()
    assert got[0] == float("inf") and got[1:3].isnan().all() and (got[3:] == 0).all()
