"""The int8 row quantizer and the norms before and after a block against their 64-bit definitions, on the GPU."""

import math

import pytest
import torch

import int8_ref as ref
import nvfp4_weight_dense_amd as nv

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _say(*a):
    print(*a, flush=True)


def _rows(m, k, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.exp(spread * torch.randn(m, 1, generator=g))
    return torch.where(torch.rand(m, k, generator=g) < 0.01, 20 * x, x).to(BF)


def _vec(k, seed, *lead):
    return torch.randn(*lead, k, generator=torch.Generator().manual_seed(seed)).to(BF)


def _check(got, want, bound, what=""):
    over = ((got.cpu().double() - want).abs() / bound).nan_to_num(nan=math.inf)
    assert not over.numel() or float(over.max()) <= 1.0, (what, float(over.max()))


def _same_rows(got, want):
    """int8 rows with the same bits (a NaN scale is one)."""
    return torch.equal(got[0].cpu(), want[0].cpu()) and torch.equal(got[1].cpu().view(torch.int32).where(
        ~got[1].cpu().isnan(), torch.tensor(0, dtype=torch.int32)), want[1].cpu().view(torch.int32).where(
            ~want[1].cpu().isnan(), torch.tensor(0, dtype=torch.int32))) and torch.equal(got[1].cpu().isnan(), want[1].cpu().isnan())


# widths at which the threads or the pieces that a thread holds change, and ones between
WIDTHS = [8, 16, 40, 256, 504, 512, 520, 1000, 2048, 4096, 4104, 5120, 8192, 8200, 12288, 16384, 17408, 32768, 32776, 65536,
          65544, 131072]
COUNTS = [(1, 4096), (2, 256), (37, 5120), (700, 264), (3000, 1024), (4099, 4096), (70000, 8)]


@pytest.mark.parametrize("m,k", [(3, k) for k in WIDTHS] + COUNTS)
def test_quantizer(m, k):
    _say("quantize", m, k)
    x = _rows(m, k, k)
    got = nv.int8_quantize_rows(x.cuda())
    assert _same_rows(got, ref.quantize(x))


def test_quantizer_special_rows():
    """Zeros of both signs, infinities, NaN, subnormal and largest values, a single value that is not zero."""
    _say("quantize special")
    k = 264
    x = _rows(12, k, 1, 0.0)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 5] = math.inf
    x[3, 263] = -math.inf
    x[4, 0] = math.nan
    x[5] = torch.randint(0, 128, (k,), generator=torch.Generator().manual_seed(1)).to(torch.int16).view(BF)  # subnormal
    x[6] = torch.tensor(1, dtype=torch.int16).view(BF)
    x[7] = x[7].float().mul(2.0 ** 120).clamp(-3e38, 3e38).to(BF)
    x[8] = 0.0
    x[8, 100] = -3.0
    x[9] = x[9].float().mul(2.0 ** -100).to(BF)
    x[10, 3] = 3.3895e38
    got, want = nv.int8_quantize_rows(x.cuda()), ref.quantize(x)
    assert _same_rows(got, want)
    assert want[1].isnan().tolist() == [False, False, True, True, True] + 7 * [False]


def test_every_bf16_value_at_every_size():
    """Each finite bf16 value under rows' scales of many sizes: all quotients that can come up are encoded as defined."""
    _say("quantize all")
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(BF)
    rows = []
    for e in (-125, -91, -90, -50, -10, -1, 0, 3, 30, 99, 107, 120):
        for top in (1.0, 1.2421875, 1.9921875):
            amax = torch.tensor(top * 2.0 ** e).to(BF)
            some = bits[bits.float() <= amax.float()][-3000:]
            sign = torch.where(torch.arange(3000) % 2 > 0, -1.0, 1.0).to(BF)
            rows.append(torch.nn.functional.pad(some, (0, 3000 - some.numel())) * sign)
    x = torch.stack(rows)
    assert _same_rows(nv.int8_quantize_rows(x.cuda()), ref.quantize(x))


@pytest.mark.parametrize("m,k", [(3, k) for k in WIDTHS] + COUNTS[:-1])
def test_norm(m, k):
    """With and without a weight and its offset; in place; to int8 with the bits of the two calls."""
    _say("norm", m, k)
    x, w = _rows(m, k, k), _vec(k, 3)
    for weight, offset, eps in ((None, 0.0, 1e-6), (w, 0.0, 1e-5), (w, 1.0, 1e-18)):
        gw = None if weight is None else weight.cuda()
        buf = torch.full((m + 2, k), 7.0, dtype=BF, device="cuda")
        buf[:m] = x.cuda()
        got = nv.rms_norm(buf[:m], gw, eps=eps, weight_offset=offset, out=buf[:m])
        want = ref.norm(x, weight, offset, eps)
        _check(got, want, ref.norm_bound(want, k))
        assert bool((buf[m:] == 7.0).all())
        assert torch.equal(nv.rms_norm(x.cuda(), gw, eps=eps, weight_offset=offset), got)
        rows = nv.rms_norm(x.cuda(), gw, eps=eps, weight_offset=offset, int8=True)
        assert _same_rows(rows, ref.quantize(got.cpu()))


def test_norm_range():
    """Rows whose squares leave fp32's range above or below it, zeros, and rows with an infinity or a NaN."""
    _say("norm range")
    k = 1032
    x = _rows(9, k, 4, 0.0).double()
    for r, e in enumerate((120, 66, 50, 0, -40, -70, -120)):
        x[r] = (x[r] * 2.0 ** e).clamp(-3e38, 3e38)
    x = x.to(BF)
    x[7] = 0.0
    x[8] = 3.3895e38
    for eps in (1e-18, 1e-6, 1.0):
        want = ref.norm(x, None, 0.0, eps)
        got = nv.rms_norm(x.cuda(), eps=eps)
        _check(got, want, ref.norm_bound(want, k) + 2.0 ** -126)
        assert _same_rows(nv.rms_norm(x.cuda(), eps=eps, int8=True), ref.quantize(got.cpu()))
    y = _rows(3, k, 5)
    y[0, 3], y[1, 1031] = math.inf, math.nan
    got = nv.rms_norm(y.cuda()).cpu()
    assert got[0].isnan().sum() == 1 and got[0, 3].isnan() and (got[0][:3] == 0).all() and got[1].isnan().all()
    assert torch.isfinite(got[2]).all()
    rows = nv.rms_norm(y.cuda(), int8=True)
    assert rows.row_scale.isnan().tolist() == [True, True, False] and not rows.codes[:2].any()


@pytest.mark.parametrize("m,k", [(6, k) for k in WIDTHS] + [(1, 4096), (700, 264), (4099, 1024)])
def test_residual(m, k):
    """Every combination of norm, gate and next norm once or more; h in place of residual or of y; int8."""
    _say("residual", m, k)
    r, y = _rows(m, k, 2 * k), _rows(m, k, 2 * k + 1)
    pw, nw = _vec(k, 5), _vec(k, 6)
    some = max(d for d in range(1, min(m, 64) + 1) if m % d == 0)
    for i, (post, gates, norm, offset, scale) in enumerate((
            (None, 0, None, 0.0, 1.0), (True, 0, True, 0.0, 0.5), (pw, 1, None, 1.0, -0.3), (None, m, nw, 1.0, 1.0),
            (pw, some, nw, 0.0, 0.22), (True, 1, nw, 0.0, 0.0))):
        gate = _vec(k, 7 + i, gates) if gates else None
        cuda = lambda t: t.cuda() if isinstance(t, torch.Tensor) else t  # noqa: E731
        args = dict(post=cuda(post), gate=cuda(gate), scale=scale, norm=cuda(norm), weight_offset=offset)
        want, bound = ref.residual(r, y, post, gate, scale, offset, 1e-6)
        rb = torch.full((m + 2, k), 7.0, dtype=BF, device="cuda")
        rb[:m] = r.cuda()
        h, n = nv.rms_norm_residual(rb[:m], y.cuda(), h=rb[:m], **args)
        _check(h, want, bound, i)
        assert bool((rb[m:] == 7.0).all())
        yb = y.cuda()
        h2, n2 = nv.rms_norm_residual(r.cuda(), yb, h=yb, **args)
        assert torch.equal(h2, h) and h2.data_ptr() == yb.data_ptr()
        if norm is None:
            assert n is None and n2 is None
            continue
        assert torch.equal(n, n2)
        # the next norm has the bits of the call of its own
        assert torch.equal(n, nv.rms_norm(h, None if norm is True else norm.cuda(), weight_offset=offset))
        h3, q = nv.rms_norm_residual(r.cuda(), y.cuda(), int8=True, **args)
        assert torch.equal(h3, h) and _same_rows(q, nv.int8_quantize_rows(n))


def test_gate_of_one_dimension_and_other_stream():
    _say("gate, stream")
    r, y, g = _rows(64, 512, 1).cuda(), _rows(64, 512, 2).cuda(), _vec(512, 3).cuda()
    want = nv.rms_norm_residual(r, y, gate=g[None], norm=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.rms_norm_residual(r, y, gate=g, norm=True, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_residual_with_nan_or_infinity():
    _say("residual nan")
    r, y = _rows(4, 264, 1), _rows(4, 264, 2)
    r[0, 5], y[1, 6], y[2, 7] = math.nan, math.nan, math.inf
    h, n = nv.rms_norm_residual(r.cuda(), y.cuda(), norm=True)
    assert h.isnan().sum(1).tolist() == [1, 1, 0, 0] and h.isinf().sum(1).tolist() == [0, 0, 1, 0]
    assert n.isnan().sum(1).tolist() == [264, 264, 1, 0]
    h, q = nv.rms_norm_residual(r.cuda(), y.cuda(), post=True, norm=True, int8=True)
    assert q.row_scale.isnan().tolist() == [True, True, True, False] and not q.codes[:3].any()


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    assert nv.int8_quantize_rows(x).codes.shape == (0, 64)
    assert nv.rms_norm(x).shape == (0, 64) and nv.rms_norm(x, int8=True).codes.shape == (0, 64)
    h, n = nv.rms_norm_residual(x, x, norm=True, gate=torch.ones(64, dtype=BF, device="cuda"))
    assert h.shape == n.shape == (0, 64)


@pytest.mark.parametrize("k", [8, 4096, 5128, 17408, 40000])
def test_a_row_does_not_depend_on_its_batch(k):
    _say("rows alone", k)
    m, few = 1100 if k < 17408 else 300, (1, 7, 257)
    r, y, w = _rows(m, k, 11).cuda(), _rows(m, k, 12).cuda(), _vec(k, 13).cuda()
    norm, quant = nv.rms_norm(y, w), nv.int8_quantize_rows(y)
    h, n = nv.rms_norm_residual(r, y, post=w, scale=0.5, norm=True)
    for i in few:
        assert torch.equal(nv.rms_norm(y[:i], w), norm[:i])
        assert _same_rows(nv.int8_quantize_rows(y[:i]), (quant.codes[:i], quant.row_scale[:i]))
        h2, n2 = nv.rms_norm_residual(r[:i], y[:i], post=w, scale=0.5, norm=True)
        assert torch.equal(h2, h[:i]) and torch.equal(n2, n[:i])
