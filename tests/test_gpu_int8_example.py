"""The decoder layer example in 8-bit integers: norms, projections, cache, attention and FFN together, on the GPU."""

import importlib.util
import os

import pytest
import torch

import int8_ref as ref
import nvfp4_weight_dense_amd as nv

pytestmark = pytest.mark.gpu
_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decode_layer.py")


def _example():
    spec = importlib.util.spec_from_file_location("decode_layer", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _run(ex, steps, budget, lens=(90, 5, 200, 1)):
    layer = ex.Layer(hidden=256, inter=512, q_heads=4, kv_heads=2, dim=64, int8=True)
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randn(n, 256, generator=g).bfloat16().cuda() for n in lens]
    return (layer,) + ex.generate(layer, prompts, steps, budget, page=16, sink=4, recent=16)


@pytest.mark.parametrize("steps,budget", [(1, 400), (60, 96)])
def test_layer_in_int8(steps, budget):
    """It runs to the lengths that the eviction rule gives, twice with the same bits."""
    ex = _example()
    a, b = _run(ex, steps, budget), _run(ex, steps, budget)
    want = []
    for m in (90, 5, 200, 1):
        for _ in range(steps):
            m = (budget // 2 if m >= budget else m) + 1
        want.append(m)
    assert a[5] == want and a[6].tolist() == want
    assert a[1].shape == (4, 256) and bool(torch.isfinite(a[1].float()).all())
    assert torch.equal(a[1], b[1]) and torch.equal(a[2].weights, b[2].weights)


def test_layer_is_its_steps():
    """One call of the layer, step by step, each held to its definition from what the one before gave."""
    ex = _example()
    layer = ex.Layer(hidden=256, inter=512, q_heads=4, kv_heads=2, dim=64, int8=True)
    x = torch.randn(37, 256, generator=torch.Generator().manual_seed(5)).bfloat16()
    cache = nv.kv8_cache(4, 2, 64, 16, weights=True)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([37], dtype=torch.int32, device="cuda")
    got = layer(x.cuda(), cache, table, lens)
    a = layer.last[1]
    o = nv.int8_gemm_w8a8(a.view(37, -1), layer.wo).cpu()
    codes, s = ref.quantize(a.view(37, -1).cpu())
    want = ref.product(codes, s, layer.wo.codes.cpu(), layer.wo.scales.cpu())
    assert bool(((o.double() - want).abs() <= ref.product_bound(want)).all())
    h, n = nv.rms_norm_residual(x.cuda(), o.cuda(), norm=True, int8=True)
    want, bound = ref.residual(x, o, None, None, 1.0, 0.0, 1e-6)
    assert bool(((h.cpu().double() - want).abs() <= bound).all())
    y = nv.dense_ffn_forward_int8(n, layer.wg, layer.wu, layer.wd).cpu()
    want, bound = ref.residual(h.cpu(), y, None, None, 1.0, 0.0, 1e-6)
    assert bool(((got.cpu().double() - want).abs() <= bound).all())
