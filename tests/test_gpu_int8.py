"""Products and the FFN in 8-bit integers against their 64-bit definitions (tests/int8_ref.py), on the GPU."""

import math
import random

import pytest
import torch

import int8_ref as ref
import nvfp4_weight_dense_amd as nv

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _say(*a):
    print(*a, flush=True)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _x(m, k, seed=0):
    g = _gen(seed)
    x = torch.randn(m, k, generator=g)
    return torch.where(torch.rand(m, k, generator=g) < 0.01, 20 * x, x).to(BF)


def _w(n, k, seed=1):
    g = _gen(seed)
    codes = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8)
    return codes, (0.5 + torch.rand(n, generator=g)) * (k ** -0.5 / 74)


def _gw(w):
    return nv.Int8Weight(w[0].cuda(), w[1].cuda())


def _check(got, want, bound, what=""):
    got = got.cpu().double()
    assert got.shape == want.shape
    over = ((got - want).abs() / bound).nan_to_num(nan=math.inf)
    assert not over.numel() or float(over.max()) <= 1.0, (what, float(over.max()))


# sizes at which a tile, a step of K, a split or a variant begins or ends, and ones between
SHAPES = [(1, 1, 32), (1, 17, 64), (2, 48, 96), (3, 128, 256), (5, 65, 160), (8, 513, 1024), (15, 64, 4128), (16, 256, 768),
          (17, 129, 416), (31, 100, 2048), (32, 1000, 544), (33, 768, 256), (47, 255, 8192), (63, 320, 4096), (64, 96, 17408),
          (65, 257, 1056), (96, 192, 160), (127, 700, 512), (128, 384, 3008), (129, 31, 4096), (200, 512, 2080),
          (255, 300, 96), (256, 256, 1024), (257, 513, 288), (300, 1030, 704), (384, 4096, 256), (512, 640, 1536),
          (513, 2049, 160), (777, 333, 1184), (1024, 1024, 64), (1500, 130, 2592), (2049, 300, 352), (4100, 64, 128),
          (1, 70000, 128), (40, 33000, 64), (6, 40, 131072), (300, 40, 65536)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k):
    """bf16 rows and int8 rows; rows behind the last are left as they were."""
    _say("product", m, n, k)
    x, w = _x(m, k, m + n), _w(n, k, k + n)
    codes, s = ref.quantize(x)
    want = ref.product(codes, s, *w)
    gw = _gw(w)
    y = torch.full((m + 3, n), 7.0, dtype=BF, device="cuda")
    got = nv.int8_gemm_w8a8(x.cuda(), gw, y[:m])
    assert got.data_ptr() == y.data_ptr()
    _check(got, want, ref.product_bound(want))
    assert bool((y[m:] == 7.0).all())
    rows = nv.Int8Rows(codes.cuda(), s.cuda())
    assert torch.equal(nv.int8_gemm_w8a8(rows, gw), got)


def _large(m, n, k, seed):
    """A product against the sum in 64 bits, taken on the GPU (exact: whole numbers below 2^53)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = nv.Int8Rows(torch.randint(-127, 128, (m, k), generator=g, device="cuda").to(torch.int8),
                    torch.rand(m, generator=g, device="cuda") + 0.5)
    w = nv.Int8Weight(torch.randint(-128, 128, (n, k), generator=g, device="cuda").to(torch.int8),
                      torch.rand(n, generator=g, device="cuda") + 0.5)
    y = torch.full((m * n + 64,), 7.0, dtype=BF, device="cuda")
    got = nv.int8_gemm_w8a8(x, w, y[:m * n].view(m, n))
    for r in range(0, m, 1024):
        want = x.codes[r:r + 1024].double() @ w.codes.double().t()
        want *= x.row_scale[r:r + 1024].double()[:, None] * w.scales.double()
        over = ((got[r:r + 1024].double() - want).abs() / ref.product_bound(want)).nan_to_num(nan=math.inf)
        assert float(over.max()) <= 1.0, (m, n, k, r)
    assert bool((y[m * n:] == 7.0).all())


# whole rounds of tiles with columns left over, tiles cut along K, more groups than workgroups
@pytest.mark.parametrize("m,n,k", [(2048, 17408, 512), (2048, 5120, 17408), (513, 17408, 1024), (512, 5120, 17408),
                                   (1025, 8200, 4096), (4099, 4104, 1056), (300, 40000, 160), (128, 5120, 17408), (66, 70001, 96),
                                   (96, 33000, 2048), (64, 17408, 5120), (33, 17416, 4096), (17, 50000, 512), (9, 5120, 17408),
                                   (4, 130000, 256), (2, 300000, 64), (1, 17408, 5120), (1024, 64, 131072), (40, 64, 131072)])
def test_product_large(m, n, k):
    _say("product", m, n, k)
    _large(m, n, k, m + n + k)


@pytest.mark.parametrize("seed", range(40))
def test_product_of_any_size(seed):
    r = random.Random(seed)
    log = lambda lo, hi: int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    m, n, k = log(1, 3000), log(1, 20000), 32 * log(1, 600)
    _say("product", m, n, k)
    _large(m, n, k, seed)


@pytest.mark.parametrize("n,k", [(129, 4128), (5120, 96), (48, 17408)])
def test_rows_do_not_depend_on_the_others(n, k):
    """A row's bits are the same alone, among few and among many."""
    _say("rows", n, k)
    x, w = _x(700, k).cuda(), _gw(_w(n, k))
    whole = nv.int8_gemm_w8a8(x, w)
    for m in (1, 4, 16, 17, 40, 64, 65, 130, 256, 257, 400):
        assert torch.equal(nv.int8_gemm_w8a8(x[:m], w), whole[:m]), m


def test_extremes_of_the_sum():
    """The largest sums there are: 127 * 128 * 131072, and its negative."""
    _say("extremes")
    k = 131072
    x = torch.full((2, k), 3.0, dtype=BF)
    x[1] = -5.0
    w = torch.full((40, k), -128, dtype=torch.int8)
    w[1], w[2], w[3, ::2] = 127, 0, 127
    ws = torch.linspace(0.5, 2, 40)
    codes, s = ref.quantize(x)
    want = ref.product(codes, s, w, ws)
    _check(nv.int8_gemm_w8a8(x.cuda(), _gw((w, ws))), want, ref.product_bound(want))
    big = x[:1].expand(300, k).contiguous()
    got = nv.int8_gemm_w8a8(big.cuda(), _gw((w, ws)))
    _check(got, want[:1].expand(300, 40), ref.product_bound(want[:1]))


def test_scales_far_apart():
    """The product of the scales, or the sum with one of them, leaves fp32's range; the result does not.  Results past
    bf16's range are infinite, those below it 0; a NaN or an infinity in a row makes the row NaN."""
    _say("scales")
    g = _gen(3)
    size = 2.0 ** torch.tensor([-130.0, -100, -60, 0, 60, 100, 119, 0, 0, -132])
    x = (torch.randn(10, 256, generator=g).clamp(-2, 2) * size[:, None]).to(BF)
    x[7, 9], x[8, 200] = math.inf, math.nan
    w = torch.randint(-127, 128, (24, 256), generator=g, dtype=torch.int8)
    ws = 2.0 ** torch.linspace(-140, 110, 24)
    codes, s = ref.quantize(x)
    want = ref.product(codes, s, w, ws)
    for rows in (x, x.repeat(8, 1), x.repeat(60, 1)):
        m = rows.shape[0]
        got = nv.int8_gemm_w8a8(rows.cuda(), _gw((w, ws))).cpu().double()
        wide = want.repeat(m // 10, 1)
        fine = torch.isfinite(wide) & (wide.abs() < 3.38e38)
        assert torch.isnan(got[torch.isnan(wide)]).all() and torch.isinf(got[wide.abs() > 3.4e38]).all()
        _check(got[fine], wide[fine], ref.product_bound(wide[fine]))


def test_special_weights_scales():
    """A channel whose scale is 0, infinite or NaN touches no other channel."""
    _say("weight scales")
    for m in (1, 40, 300):
        x, (w, ws) = _x(m, 128), _w(70, 128)
        ws[3], ws[20], ws[69] = 0.0, math.inf, math.nan
        got = nv.int8_gemm_w8a8(x.cuda(), _gw((w, ws))).cpu()
        assert (got[:, 3] == 0).all() and torch.isnan(got[:, 69]).all() and not torch.isfinite(got[:, 20]).any()
        rest = [c for c in range(70) if c not in (3, 20, 69)]
        codes, s = ref.quantize(x)
        want = ref.product(codes, s, w[rest], ws[rest])
        _check(got[:, rest], want, ref.product_bound(want))


FFN = [(1, 32, 32), (1, 256, 768), (2, 4096, 160), (4, 96, 8192), (7, 512, 1056), (16, 640, 416), (33, 160, 1536), (64, 1024, 2816),
       (100, 352, 608), (130, 256, 768), (256, 768, 96), (257, 128, 4128), (600, 1024, 544), (1300, 416, 1184)]


@pytest.mark.parametrize("m,hidden,inter", FFN)
def test_ffn_is_its_steps(m, hidden, inter):
    """The FFN gives the bits of its steps one by one, whose own tests hold them to their definitions."""
    _say("ffn", m, hidden, inter)
    x = _x(m, hidden, m).cuda()
    wg, wu, wd = _gw(_w(inter, hidden, 1)), _gw(_w(inter, hidden, 2)), _gw(_w(hidden, inter, 3))
    out = torch.full((m + 2, hidden), 7.0, dtype=BF, device="cuda")
    got = nv.dense_ffn_forward_int8(x, wg, wu, wd, out[:m])
    act = nv.silu_mul(nv.int8_gemm_w8a8(x, wg), nv.int8_gemm_w8a8(x, wu))
    assert torch.equal(got, nv.int8_gemm_w8a8(act, wd))
    assert bool((out[m:] == 7.0).all())
    rows = nv.int8_quantize_rows(x)
    assert torch.equal(nv.dense_ffn_forward_int8(rows, wg, wu, wd), got)


@pytest.mark.parametrize("m,hidden,inter", [(1, 256, 768), (9, 512, 1056), (70, 256, 768), (300, 128, 416)])
def test_ffn_against_64_bits(m, hidden, inter):
    """A value of gate, up or act that the GPU rounds the other way moves it by one bf16 step (2^-7 of itself), and a
    code of act by at most one: per output at most the sum over those elements of |w| * 1.01 codes.  The elements that
    lie within 2^-20 of themselves of a rounding edge are few; the bound below lets a tenth of the row move, as a
    random walk would, and adds the last rounding."""
    _say("ffn 64", m, hidden, inter)
    x = _x(m, hidden, 5)
    wg, wu, wd = _w(inter, hidden, 1), _w(inter, hidden, 2), _w(hidden, inter, 3)
    codes, s = ref.quantize(x)
    gate, up = (ref.product(codes, s, *w).to(BF).double() for w in (wg, wu))
    act = (gate * torch.sigmoid(gate) * up).to(BF)
    ac, a_s = ref.quantize(act)
    want = ref.product(ac, a_s, *wd)
    moved = (0.1 * (wd[0].double() ** 2).sum(1)).sqrt() * wd[1].double() * a_s.double()[:, None]
    got = nv.dense_ffn_forward_int8(x.cuda(), _gw(wg), _gw(wu), _gw(wd))
    _check(got, want, ref.product_bound(want) + moved)


def test_rows_with_nan_stay_apart():
    """A row with a NaN gives NaN, the rows beside it what they give without it."""
    _say("nan rows")
    hidden, inter = 256, 768
    W = [_gw(_w(inter, hidden, 1)), _gw(_w(inter, hidden, 2)), _gw(_w(hidden, inter, 3))]
    for m in (3, 20, 70, 300):
        x = _x(m, hidden, 2).cuda()
        want = nv.dense_ffn_forward_int8(x, *W)
        x[1, 7], x[2, 0] = math.nan, -math.inf
        got = nv.dense_ffn_forward_int8(x, *W)
        assert torch.isnan(got[1:3]).all()
        keep = [r for r in range(m) if r not in (1, 2)]
        assert torch.equal(got[keep], want[keep])


def test_no_rows():
    _say("no rows")
    w, wd = _gw(_w(96, 64)), _gw(_w(64, 96))
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    assert nv.int8_gemm_w8a8(x, w).shape == (0, 96)
    assert nv.dense_ffn_forward_int8(x, w, w, wd).shape == (0, 64)
    rows = nv.int8_quantize_rows(x)
    assert rows.codes.shape == (0, 64) and nv.int8_gemm_w8a8(rows, w).shape == (0, 96)


CALLS = [(1, 4096, 1024), (3, 64, 17408), (20, 1000, 2048), (64, 5120, 1024), (100, 257, 8192), (256, 640, 4096),
         (300, 5120, 2048), (700, 300, 4096)]


def test_one_workspace_for_calls_of_other_sizes():
    """A workspace serves calls of all smaller sizes in any order, again and again."""
    _say("workspace")
    data = [(_x(m, k).cuda(), _gw(_w(n, k))) for m, n, k in CALLS]
    want = [nv.int8_gemm_w8a8(x, w) for x, w in data]
    ws = torch.zeros(max(nv.int8_workspace(x.shape[0], w).numel() for x, w in data), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for (x, w), y in zip(data, want):
            assert torch.equal(nv.int8_gemm_w8a8(x, w, workspace=ws), y)
    hidden, inter = 256, 768
    W = [_gw(_w(inter, hidden, 1)), _gw(_w(inter, hidden, 2)), _gw(_w(hidden, inter, 3))]
    x = _x(300, hidden).cuda()
    want = nv.dense_ffn_forward_int8(x, *W)
    ws = nv.int8_workspace(300, *W)
    for m in (300, 1, 40, 129, 300):
        assert torch.equal(nv.dense_ffn_forward_int8(x[:m], *W, workspace=ws), want[:m])


def test_two_streams_with_workspaces_of_their_own():
    _say("streams")
    data = [(_x(m, k).cuda(), _gw(_w(n, k))) for m, n, k in CALLS]
    want = [nv.int8_gemm_w8a8(x, w) for x, w in data]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [[nv.int8_workspace(x.shape[0], w) for x, w in data] for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for st, ws in zip(streams, spaces):
            for (x, w), space in zip(data, ws):
                got.append(nv.int8_gemm_w8a8(x, w, workspace=space, stream=st))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % len(CALLS)]), i


@pytest.mark.parametrize("m", [1, 40, 300])
def test_block_in_two_graphs(m):
    """The block as it is used -- norm to int8, FFN, norm with gate and residual, next norm to int8 and a product --
    captured into two graphs that are replayed in turn with eager work between, each with a workspace of its own."""
    _say("graphs", m)
    hidden, inter = 1024, 2816
    W = [_gw(_w(inter, hidden, 1)), _gw(_w(inter, hidden, 2)), _gw(_w(hidden, inter, 3))]
    proj = _gw(_w(640, hidden, 4))
    g = _gen(9)
    w1, w2, w3 = ((1 + 0.2 * torch.randn(hidden, generator=g)).to(BF).cuda() for _ in range(3))
    gate = torch.randn(hidden, generator=g).to(BF).cuda()

    def block(x, ws, ws1):
        n = nv.rms_norm(x, w1, int8=True)
        y = nv.dense_ffn_forward_int8(n, *W, workspace=ws)
        h, n = nv.rms_norm_residual(x, y, post=w2, gate=gate, scale=0.5, norm=w3, int8=True)
        return h, nv.int8_gemm_w8a8(n, proj, workspace=ws1)

    graphs = []
    for i in range(2):
        x = _x(m, hidden, i).cuda()
        ws, ws1 = nv.int8_workspace(m, *W), nv.int8_workspace(m, proj)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block(x, ws, ws1)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = block(x, ws, ws1)
        graphs.append((graph, x, out, ws, ws1))  # (what a graph uses lives as long as it)
    for turn in range(4):
        for i, (graph, x, out, *_) in enumerate(graphs):
            x.copy_(_x(m, hidden, 10 * turn + i).cuda())
            want = block(x, None, None)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), (turn, i)


def test_a_captured_call_needs_a_workspace():
    _say("capture")
    x, w = _x(4, 256).cuda(), _gw(_w(64, 256))
    nv.int8_gemm_w8a8(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = torch.zeros(1, device="cuda")
    with torch.cuda.graph(graph):
        keep += 1
        with pytest.raises(nv.Nvfp4Error, match="workspace"):
            nv.int8_gemm_w8a8(x, w, y=torch.empty(4, 64, dtype=BF, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert float(keep) == 1
