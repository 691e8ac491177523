"""The decoder layer example: projections, cache, attention, FFN and eviction together, on the GPU."""

import importlib.util
import math
import os

import pytest
import torch

import kv8_ref as ref

pytestmark = pytest.mark.gpu
_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decode_layer.py")


def _example():
    spec = importlib.util.spec_from_file_location("decode_layer", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _run(ex, steps, budget, lens=(90, 5, 200, 1)):
    layer = ex.Layer(hidden=256, inter=512, q_heads=4, kv_heads=2, dim=64)
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randn(n, 256, generator=g).bfloat16().cuda() for n in lens]
    return (layer,) + ex.generate(layer, prompts, steps, budget, page=16, sink=4, recent=16)


@pytest.mark.parametrize("steps,budget", [(1, 400), (30, 96), (150, 96)])
def test_layer(steps, budget):
    """Pages and lengths are what the eviction rule gives, and the last step's attention is that of the cache."""
    ex = _example()
    layer, x, cache, pages, table, lens, n = _run(ex, steps, budget)
    want = []
    for m in (90, 5, 200, 1):
        for _ in range(steps):
            m = (budget // 2 if m >= budget else m) + 1
        want.append(m)
    assert lens == want and n.tolist() == want
    own = [p for o in pages.own for p in o]
    assert sorted(own + pages.free) == list(range(cache.k_codes.shape[0]))
    assert [len(o) for o in pages.own] == [-(-m // 16) for m in want]
    assert x.shape == (4, 256) and bool(torch.isfinite(x.float()).all())
    q, a = layer.last
    out, _, bound, _, _ = ref.Pool(cache).attention(q.cpu(), table.cpu(), want, [1] * 4, 64 ** -0.5)
    over = ((a.cpu().double() - out).abs() / bound.clamp(min=1e-300)).max()
    assert float(over) <= 1.0
    # each step hands out a weight of q_heads; evicted tokens take theirs with them
    w = ref.Pool(cache)
    for b, m in enumerate(want):
        page, slot = w.where(table.cpu(), b, torch.arange(m))
        got = float(w.weights[page, slot].double().sum())
        assert got >= 4 * (1 - 1e-5)
        if budget == 400:
            handed = 4 * ((90, 5, 200, 1)[b] + steps)
            assert abs(got - handed) <= 1e-4 * handed
    assert math.isfinite(float(x.float().square().mean()))


def test_the_same_again():
    ex = _example()
    a, b = _run(ex, 40, 96), _run(ex, 40, 96)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2].weights, b[2].weights)
