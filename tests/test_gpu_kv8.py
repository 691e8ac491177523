"""The 8-bit paged KV cache on the GPU against the 64-bit reference: codes, scales and kept positions exactly,
attention, log-sums and accumulated weights within the bounds that kv8_ref counts from their roundings."""

import math

import pytest
import torch

import kv8_ref as ref
import nvfp4_weight_dense_amd as nv

pytestmark = pytest.mark.gpu
NEG = -math.inf


def _say(*a):
    print(*a, flush=True)


def _gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


def _filled(pages, heads, dim, page, seed, weights=False, spread=6):
    """A pool whose every byte is set: random finite codes (or normal ones), scales over 2 * spread binades."""
    g = _gen(seed)
    c = nv.kv8_cache(pages, heads, dim, page, weights=weights, device="cpu")
    for t in (c.k_codes, c.v_codes):
        x = torch.randn(t.shape, generator=g) * 60
        t.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.randint(122 - spread, 122 + spread, t.shape, generator=g).to(torch.uint8))
    if weights:
        c.weights.copy_(torch.exp(2 * torch.randn(c.weights.shape, generator=g) - 3))
    return c


def _gpu(c):
    f = lambda t: None if t is None else t.cuda()  # noqa: E731
    return nv.KV8Cache(f(c.k_codes), f(c.v_codes), f(c.k_scales), f(c.v_scales), f(c.weights))


def _table(lens, page, pages, seed, cols=None, spare=0):
    """A table of distinct pages in random order; `spare` further pages of the pool stay unused."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(pages - spare, generator=_gen(seed))
    t = torch.full((len(lens), cols or max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    return t


def _starts(rows):
    return torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _same(pool, c):
    for isv, (codes, scales) in enumerate(((c.k_codes, c.k_scales), (c.v_codes, c.v_scales))):
        assert torch.equal(scales.cpu(), pool.scales[isv]), "v scales" if isv else "k scales"
        assert torch.equal(codes.cpu(), pool.raw(isv)), "v codes" if isv else "k codes"
    if pool.weights is not None:
        assert torch.equal(c.weights.cpu().view(torch.int32), pool.weights.view(torch.int32)), "weights"


def _within(got, want, bound, what):
    got, want = got.cpu().double(), want
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    ok = ~nan & ~inf
    over = ((got - want).abs() / bound.clamp(min=1e-300))[ok]
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of its bound"
    return worst


# ---- append ------------------------------------------------------------------------------------------

APPENDS = [  # dim, page, heads, lens, rows
    (128, 64, 2, [1, 64, 65, 200], [1, 1, 1, 1]),
    (128, 64, 2, [1, 63, 64, 130, 7], [1, 63, 64, 130, 7]),
    (64, 16, 3, [100, 17, 33, 16], [37, 2, 33, 0]),
    (256, 32, 1, [90, 31], [70, 5]),
    (128, 128, 2, [300, 129], [299, 3]),
    (64, 32, 1, [5, 0, 40], [9, 3, 2]),       # more rows than tokens: the first are dropped
]


@pytest.mark.parametrize("dim,page,heads,lens,rows", APPENDS)
def test_append(dim, page, heads, lens, rows):
    _say("append", dim, page, heads, lens, rows)
    pages = sum(-(-n // page) for n in lens) + 2
    c = _filled(pages, heads, dim, page, 1, weights=True)
    pool, dev = ref.Pool(c), _gpu(c)
    table = _table(lens, page, pages, 2)
    g = _gen(3)
    # a part of a projection's output; magnitudes that need other scales from token to token
    qkv = torch.randn(sum(rows), 4 + 2 * heads, dim, generator=g) * torch.exp(2 * torch.randn(sum(rows), 1, 1, generator=g))
    qkv = qkv.bfloat16()
    pool.append(qkv[:, 4:4 + heads], qkv[:, 4 + heads:], table, lens, rows)
    d = qkv.cuda()
    nv.kv8_append(d[:, 4:4 + heads], d[:, 4 + heads:], dev, table.cuda(), _i32(lens).cuda(),
                  _starts(rows).cuda(), max_rows=max(rows))
    _same(pool, dev)


def test_append_token_by_token_and_in_parts():
    _say("append in parts")
    dim, page, heads = 128, 32, 2
    c = _filled(8, heads, dim, page, 4, weights=True)
    pool, dev = ref.Pool(c), _gpu(c)
    g, n = _gen(5), 0
    table = _table([200], page, 8, 6)
    for r in (1, 1, 1, 30, 2, 1, 60, 17, 1, 1, 64):
        x = (torch.randn(r, 2 * heads, dim, generator=g) * math.exp(0.4 * n ** 0.5 - 2)).bfloat16()
        n += r
        pool.append(x[:, :heads], x[:, heads:], table, [n], [r])
        d = x.cuda()
        nv.kv8_append(d[:, :heads], d[:, heads:], dev, table.cuda(), _i32([n]).cuda())
        _same(pool, dev)


def test_append_values_at_the_edges():
    _say("append edges")
    dim, page, heads = 64, 16, 1
    rows = []
    big = 3.3895313892515355e38                       # the largest bf16
    for vals in ([0.0], [-0.0, 0.0], [math.inf, 1.0, -2.0], [math.nan, 3.0], [-math.inf, math.nan], [big, 1.0],
                 [9.2e-41, 0.0], [2.0 ** -126, 2.0 ** -120], [448.0, 449.0, 464.0], [1.75, 1.7578125], [1e-30, 1e30]):
        rows.append((vals * dim)[:dim])
    x = torch.tensor(rows).bfloat16()[:, None]
    lens, each = [1] * len(rows), [1] * len(rows)
    c = _filled(len(rows), heads, dim, page, 7)
    pool, dev = ref.Pool(c), _gpu(c)
    table = _table(lens, page, len(rows), 8)
    pool.append(x, x, table, lens, each)
    nv.kv8_append(x.cuda(), x.cuda(), dev, table.cuda(), _i32(lens).cuda())
    _same(pool, dev)
    # each then follows one of 1.0 in the page
    two = torch.ones_like(x)
    for y, n in ((two, 1), (x, 2)):
        pool.append(y, y, table, [n] * len(rows), each)
        nv.kv8_append(y.cuda(), y.cuda(), dev, table.cuda(), _i32([n] * len(rows)).cuda())
    _same(pool, dev)


def test_append_leaves_unnamed_pages_alone():
    _say("append bad pages")
    dim, page, heads = 64, 16, 2
    c = _filled(6, heads, dim, page, 9, weights=True)
    pool, dev = ref.Pool(c), _gpu(c)
    table = _i32([[0, -1, 2, 6], [2 ** 31 - 1, 4, -2 ** 31, 5]])
    x = torch.randn(120, heads, dim, generator=_gen(10)).bfloat16()
    pool.append(x, -x, table, [60, 64], [60, 60])
    nv.kv8_append(x.cuda(), -x.cuda(), dev, table.cuda(), _i32([60, 64]).cuda())
    _same(pool, dev)


# ---- attention ---------------------------------------------------------------------------------------

CASES = [  # dim, page, heads, q_heads, lens, rows, window
    (128, 64, 2, 8, [1], [1], 0),
    (128, 64, 1, 1, [77], [1], 0),
    (128, 64, 2, 8, [513, 64, 65, 1, 0, 250], [1] * 6, 0),
    (128, 64, 2, 10, [300, 1000], [1, 1], 0),
    (64, 16, 2, 4, [100, 33, 16], [4, 3, 1], 0),
    (64, 32, 1, 3, [190, 70], [2, 2], 50),
    (256, 128, 1, 4, [140, 400], [1, 3], 0),
    (128, 16, 1, 16, [90], [5], 7),
    (128, 64, 1, 4, [130], [130], 0),
    (128, 32, 2, 4, [200, 97, 64], [150, 97, 1], 0),
    (64, 64, 1, 8, [260, 129], [100, 129], 33),
    (256, 64, 1, 2, [150], [150], 0),
    (256, 16, 1, 3, [300], [77], 100),
    (128, 64, 1, 2, [40, 3], [60, 5], 0),      # rows before the first token see nothing
    (128, 128, 1, 5, [700], [321], 1),
    (128, 64, 1, 32, [2100], [9], 0),
]


def _problem(dim, page, heads, q_heads, lens, rows, window, seed=11, weights=True):
    pages = sum(-(-n // page) for n in lens) + 3
    c = _filled(pages, heads, dim, page, seed, weights=weights)
    table = _table(lens, page, pages, seed + 1, cols=-(-max(max(lens), 1) // page) + 1, spare=1)
    q = torch.randn(sum(rows), q_heads + 3, dim, generator=_gen(seed + 2)).bfloat16()
    return c, table, q


def _check(c, table, q, q_heads, lens, rows, window=0, accumulate=True, max_len=None, factor=0.02, **kw):
    """Runs the call and compares out, lse and the weights; returns them."""
    dim = c.k_codes.shape[3]
    pool, dev = ref.Pool(c), _gpu(c)
    scale = factor / math.sqrt(dim)
    out, lse, b_out, b_lse, w = pool.attention(q[:, 1:1 + q_heads], table, lens, rows, scale, window, max_len)
    got = nv.kv8_attention(q.cuda()[:, 1:1 + q_heads], dev, table.cuda(), _i32(lens).cuda(), _starts(rows).cuda(),
                           scale=scale, window=window, max_rows=max(rows), lse=True, accumulate=accumulate,
                           max_len=max_len, **kw)
    worst = _within(got[0], out, b_out, "out"), _within(got[1], lse, b_lse, "lse")
    if accumulate:
        want, bound = pool.weights.double(), pool.weights.double() * 2.0 ** -23
        for b, (x, bx) in enumerate(w):
            page, slot = pool.where(table, b, torch.arange(len(x)))
            ok = page >= 0
            want[page[ok], slot[ok]] += x[ok]
            bound[page[ok], slot[ok]] += bx[ok]
        worst += (_within(dev.weights, want, bound + 1e-30, "weights"),)
    _say("  of the bounds:", ["%.2f" % x for x in worst])
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert torch.equal(getattr(dev, name).cpu(), getattr(c, name))
    return got[0], got[1], dev.weights


@pytest.mark.parametrize("dim,page,heads,q_heads,lens,rows,window", CASES)
def test_attention(dim, page, heads, q_heads, lens, rows, window):
    _say("attention", dim, page, heads, q_heads, lens, rows, window)
    c, table, q = _problem(dim, page, heads, q_heads, lens, rows, window)
    _check(c, table, q, q_heads, lens, rows, window)


COLUMNS = [  # as CASES; rows times query heads of a KV head around what one workgroup takes, up to the wide kernel
    (128, 64, 1, 4, [300, 64, 9], [5, 8, 1], 0),
    (128, 64, 2, 8, [700, 130], [10, 3], 0),
    (128, 32, 1, 3, [513], [17], 0),
    (128, 16, 1, 10, [250, 1000], [12, 7], 60),
    (64, 64, 2, 2, [400, 33], [33, 33], 0),
    (64, 128, 1, 8, [1500], [16], 200),
    (64, 16, 1, 3, [90, 50], [43, 2], 0),
    (64, 32, 1, 16, [4000], [8], 0),
    (256, 64, 1, 4, [600, 70], [8, 4], 0),
    (256, 16, 1, 1, [333], [33], 50),
    (256, 128, 2, 8, [1025, 100], [16, 9], 0),
    (256, 32, 1, 5, [777], [13], 0),
    (128, 64, 1, 1, [129], [128], 0),
    (128, 64, 1, 1, [129], [129], 0),
    (256, 64, 1, 2, [2000, 1900], [300, 257], 0),
    (64, 64, 1, 1, [9000], [600], 0),
    (128, 128, 1, 1, [5000, 64], [400, 64], 1500),
    (128, 16, 1, 1, [1, 0, 17, 255, 256, 257], [1, 0, 17, 255, 256, 257], 0),
    (128, 64, 2, 2, [3, 1500, 0, 1100], [200, 400, 0, 129], 0),   # long enough to be dealt, some rows see nothing
    (64, 32, 3, 3, [1300, 1024, 1], [300, 129, 1], 100),
    (256, 16, 1, 1, [1030, 17], [260, 17], 0),
]


@pytest.mark.parametrize("dim,page,heads,q_heads,lens,rows,window", COLUMNS)
def test_attention_columns(dim, page, heads, q_heads, lens, rows, window):
    _say("attention", dim, page, heads, q_heads, lens, rows, window)
    c, table, q = _problem(dim, page, heads, q_heads, lens, rows, window, seed=90)
    _check(c, table, q, q_heads, lens, rows, window)


@pytest.mark.parametrize("factor", [-0.02, 0.0, -1e-30, 1.0])
@pytest.mark.parametrize("dim,rows", [(128, [1, 3]), (64, [20, 9]), (256, [12, 16]), (128, [100, 60])])
def test_attention_scales(dim, rows, factor):
    """Negative scales, and 0: every token counts alike; 1: each row sees little but its largest score."""
    _say("attention, scale", dim, rows, factor)
    c, table, q = _problem(dim, 64, 1, 4, [200, 131], rows, 0, seed=100)
    _, lse, _ = _check(c, table, q, 4, [200, 131], rows, factor=factor)
    if factor == 0.0:
        seen = torch.tensor([n - r + 1 + i for n, r in zip([200, 131], rows) for i in range(r)]).double()
        assert float((lse.cpu().double() - seen.log()[:, None]).abs().max()) <= 2.0 ** -20


@pytest.mark.parametrize("dim,rows", [(128, [20, 12]), (64, [9, 31]), (256, [13, 16])])
def test_attention_columns_with_unnamed_pages_and_far_from_zero(dim, rows):
    _say("attention, bad pages and large scores", dim, rows)
    c, table, q = _problem(dim, 16, 1, 4, [150, 90], rows, 0, seed=110)
    table[0, 2], table[0, 7], table[1, 0] = -1, 2 ** 30, c.k_codes.shape[0]
    _check(c, table, q * 40, 4, [150, 90], rows)
    _check(c, table, q, 4, [150, 90], rows, max_len=37)
    table[:] = -1
    out, lse, _ = _check(c, table, q, 4, [150, 90], rows)
    assert not out.any() and bool((lse == NEG).all())


@pytest.mark.parametrize("rows", [[1, 1], [6, 5], [50, 70]])
def test_strides(rows):
    """K and V of one head shared by several (a head stride of 0), q with its heads outermost, rows far apart."""
    _say("strides", rows)
    lens, dim, page = [100, 77], 128, 16
    c = _filled(12, 3, dim, page, 120, weights=True)
    pool, dev = ref.Pool(c), _gpu(c)
    table = _table(lens, page, 12, 121)
    g = _gen(122)
    k = torch.randn(sum(rows), 1, dim, generator=g).bfloat16().expand(-1, 3, -1)
    v = torch.randn(3, sum(rows), dim, generator=g).bfloat16().transpose(0, 1)
    pool.append(k, v, table, lens, rows)
    kd = k[:, :1].cuda().expand(-1, 3, -1)
    vd = v.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    assert kd.stride(1) == 0 and vd.stride(0) == dim
    nv.kv8_append(kd, vd, dev, table.cuda(), _i32(lens).cuda(), _starts(rows).cuda(), max_rows=max(rows))
    _same(pool, dev)
    q = torch.randn(6, sum(rows), 3 * dim, generator=g).bfloat16()
    qd = q.cuda().transpose(0, 1)[:, :, dim:2 * dim]
    out, lse, b_out, b_lse, _ = pool.attention(q.transpose(0, 1)[:, :, dim:2 * dim], table, lens, rows, dim ** -0.5)
    got = nv.kv8_attention(qd, dev, table.cuda(), _i32(lens).cuda(), _starts(rows).cuda(), max_rows=max(rows), lse=True)
    _within(got[0], out, b_out, "out")
    _within(got[1], lse, b_lse, "lse")


@pytest.mark.parametrize("rows", [[1, 1], [4, 4], [100, 60]])
def test_attention_far_from_zero(rows):
    """Scores of some hundreds, so that whole tiles lie far below the maximum and maxima keep rising."""
    _say("attention, large scores", rows)
    c, table, q = _problem(128, 64, 1, 4, [500, 300], rows, 0)
    _check(c, table, q * 40, 4, [500, 300], rows)


@pytest.mark.parametrize("rows", [[1, 1], [40, 70]])
def test_attention_skips_unnamed_pages(rows):
    _say("attention, bad pages", rows)
    c, table, q = _problem(64, 16, 2, 4, [150, 90], rows, 0)
    table[0, 2], table[0, 7], table[1, 0] = -1, 2 ** 30, c.k_codes.shape[0]
    _check(c, table, q, 4, [150, 90], rows)
    table[:] = -1                                     # no page at all: nothing is seen
    out, lse, _ = _check(c, table, q, 4, [150, 90], rows)
    assert not out.any() and bool((lse == NEG).all())


@pytest.mark.parametrize("dim,page,rows,window", [(128, 64, [1, 1, 1], 0), (128, 64, [4, 2, 1], 0), (64, 16, [70, 30, 9], 0),
                                                  (256, 32, [5, 90, 33], 40), (128, 32, [3, 1, 2], 21)])
def test_unseen_tokens_have_no_influence(dim, page, rows, window):
    """NaN codes beyond each length, before the window and in later rows' own tokens reach no row that does not
    see them; a row that sees one gets NaN there and nowhere else."""
    _say("NaN in unseen places", dim, page, rows, window)
    lens = [90, 130, 35]
    c, table, q = _problem(dim, page, 1, 4, lens, rows, window)
    at = {isv: ref.order(page, dim, isv) for isv in (0, 1)}
    for isv, codes in ((0, c.k_codes), (1, c.v_codes)):
        flat = codes.view(codes.shape[0], 1, -1)
        flat[table[0, -2:].clamp(min=0).long(), 0, 0] = 0x7F   # not in use
        for b, n in enumerate(lens):
            for t in range(n, -(-n // page) * page):            # beyond the length
                flat[int(table[b, t // page]), 0, at[isv][t % page]] = 0x7F + 128 * (t % 2)
        if isv:                                                  # the last token's V, two channels
            for b, n in enumerate(lens):
                flat[int(table[b, (n - 1) // page]), 0, at[1][(n - 1) % page, [3, dim - 1]]] = 0xFF
            if window:                                           # and one that only the first rows see
                flat[int(table[1, (130 - 90 - window + 2) // page]), 0,
                     at[1][(130 - 90 - window + 2) % page, 7]] = 0x7F
    _check(c, table, q, 4, lens, rows, window)


@pytest.mark.parametrize("dim,page,rows,window", [(128, 64, [1, 1, 1], 0), (128, 64, [4, 2, 1], 0), (64, 16, [70, 30, 9], 0),
                                                  (256, 32, [5, 90, 33], 40), (128, 32, [3, 1, 2], 21),
                                                  (128, 128, [90, 130, 35], 0), (128, 64, [20, 12, 8], 0),
                                                  (64, 16, [30, 9, 2], 40), (256, 64, [13, 9, 16], 0)])
def test_finite_where_only_unseen_places_hold_nan(dim, page, rows, window):
    """The same with NaN in every code that no row sees, and in the last token's V, which only the last row sees:
    every other row's result is finite."""
    _say("NaN in every unseen place", dim, page, rows, window)
    lens = [90, 130, 35]
    c, table, q = _problem(dim, page, 1, 4, lens, rows, window, seed=70)
    free = torch.ones(c.k_codes.shape[0], dtype=torch.bool)
    free[table[table >= 0].long()] = False
    at = {isv: ref.order(page, dim, isv) for isv in (0, 1)}
    for isv, codes in ((0, c.k_codes), (1, c.v_codes)):
        flat = codes.view(codes.shape[0], 1, -1)
        flat[free] = 0x7F
        for b, (n, r) in enumerate(zip(lens, rows)):
            gone = [t for t in range(-(-n // page) * page) if t >= n or (window and t <= n - r - window)]
            for t in gone:
                flat[int(table[b, t // page]), 0, at[isv][t % page]] = 0x7F + 128 * (t % 2)
        if isv:
            for b, n in enumerate(lens):
                flat[int(table[b, (n - 1) // page]), 0, at[1][(n - 1) % page, [3, dim - 1]]] = 0xFF
    out, lse, _ = _check(c, table, q, 4, lens, rows, window)
    last = [sum(rows[:b + 1]) - 1 for b in range(3)]
    bad = torch.isnan(out).any(2).any(1).cpu()
    assert bad.nonzero().reshape(-1).tolist() == last and bool(torch.isfinite(lse).all())


def test_nan_in_q_and_k_stays_in_its_row():
    _say("NaN in q and K")
    lens, rows = [90, 60], [8, 50]
    c, table, q = _problem(128, 64, 1, 4, lens, rows, 0)
    q[3, 2] = math.nan
    c.k_codes.view(c.k_codes.shape[0], 1, -1)[int(table[1, 0]), 0, int(ref.k_at(40, 5, 128))] = 0x7F
    _check(c, table, q, 4, lens, rows, accumulate=False)


@pytest.mark.parametrize("rows", [[1, 1], [9, 100]])
def test_max_len_leaves_the_rest_out(rows):
    _say("max_len", rows)
    c, table, q = _problem(128, 64, 1, 4, [300, 200], rows, 0)
    _check(c, table, q, 4, [300, 200], rows, max_len=150)


def test_lengths_beyond_the_table_and_rows_beyond_the_arrays_are_held():
    _say("lengths and starts out of range")
    c, table, q = _problem(64, 16, 1, 2, [60, 40], [2, 2], 0)
    table = table[:, :3].contiguous()                 # 48 tokens
    dev = _gpu(c)
    starts = _i32([-5, 2, 2 ** 30]).cuda()
    out, lse = nv.kv8_attention(q.cuda()[:, :2], dev, table.cuda(), _i32([2 ** 30, -7]).cuda(), starts, lse=True)
    want, wl, b_out, b_lse, _ = ref.Pool(c).attention(q[:, :2], table, [48, 0], [2, 2], 64 ** -0.5)
    _within(out, want, b_out, "out")
    _within(lse, wl, b_lse, "lse")


def test_long_cache_of_one_sequence():
    _say("long cache")
    c, table, q = _problem(128, 128, 1, 8, [40000], [2], 0)
    _check(c, table, q, 8, [40000], [2])


def test_rows_and_streams_and_workspaces():
    """Rows without starts, a caller's out, lse and workspace, another stream, and the same bits each time."""
    _say("streams and workspaces")
    lens, rows = [900, 333, 64, 1], [2, 2, 2, 2]
    c, table, q = _problem(128, 64, 2, 8, lens, rows, 0)
    first = _check(c, table, q, 8, lens, rows)
    dev, t, n = _gpu(c), table.cuda(), _i32(lens).cuda()
    qd = q.cuda()[:, 1:9]
    ws = nv.kv8_workspace(8, dev, t, n, 8)
    out, lse = torch.full_like(first[0], 7.0), torch.full_like(first[1], 7.0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        out.fill_(7.0)
        torch.cuda.synchronize()
        got = nv.kv8_attention(qd, dev, t, n, scale=0.02 / math.sqrt(128), out=out, lse=lse, workspace=ws,
                               stream=s)
        s.synchronize()
        assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == lse.data_ptr()
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])
    again = _gpu(c)
    nv.kv8_attention(qd, again, t, n, scale=0.02 / math.sqrt(128), accumulate=True)
    assert torch.equal(again.weights.view(torch.int32), first[2].view(torch.int32))


def test_rows_outside_the_sequences_are_not_written():
    _say("rows outside")
    c, table, q = _problem(128, 64, 1, 4, [90, 70], [3, 2], 0)
    dev = _gpu(c)
    qd = torch.cat([q[:1], q, q[:2]]).cuda()[:, :4]
    out = torch.full((8, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 4), 7.0, device="cuda")
    nv.kv8_attention(qd, dev, table.cuda(), _i32([90, 70]).cuda(), _i32([1, 4, 6]).cuda(), out=out, lse=lse)
    assert bool((out[[0, 6, 7]] == 7.0).all()) and bool((lse[[0, 6, 7]] == 7.0).all())
    assert not bool((lse[1:6] == 7.0).any())


@pytest.mark.parametrize("rows", [1, 130])
def test_pool_beyond_four_gib(rows):
    """Pages whose byte offsets pass 2^32."""
    _say("pool beyond 4 GiB", rows)
    dim, page, heads, lens = 128, 64, 4, [200]
    c, table, q = _problem(dim, page, heads, 8, lens, [rows], 0)
    n = c.k_codes.shape[0]
    first = 2 ** 32 // (heads * page * dim) + 5
    big = nv.kv8_cache(first + n, heads, dim, page, weights=True)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "weights"):
        getattr(big, name)[first:] = getattr(c, name).cuda()
    pool = ref.Pool(c)
    x = torch.randn(rows, 2 * heads, dim, generator=_gen(21)).bfloat16()
    pool.append(x[:, :heads], x[:, heads:], table, lens, [rows])
    far = torch.where(table >= 0, table + first, -1).cuda()
    d = x.cuda()
    nv.kv8_append(d[:, :heads], d[:, heads:], big, far, _i32(lens).cuda())
    view = nv.KV8Cache(*(getattr(big, s)[first:] for s in ("k_codes", "v_codes", "k_scales", "v_scales", "weights")))
    _same(pool, view)
    out, lse, b_out, b_lse, _ = pool.attention(q[:, :8], table, lens, [rows], 0.002)
    got = nv.kv8_attention(q.cuda()[:, :8], big, far, _i32(lens).cuda(), scale=0.002, lse=True)
    _within(got[0], out, b_out, "out")
    _within(got[1], lse, b_lse, "lse")
    assert not bool(big.k_codes[:first].any())


def test_step_in_a_graph():
    """append, attention with accumulation, eviction: captured once, replayed on other inputs."""
    _say("graph")
    lens, page, heads, dim = [130, 77], 64, 2, 128
    c, table, q = _problem(dim, page, heads, 8, lens, [1, 1], 0)
    t, n = table.cuda(), _i32(lens).cuda()
    dev = _gpu(c)
    spare = [i for i in range(c.k_codes.shape[0]) if i not in set(table.reshape(-1).tolist())]
    new_table = _i32([[spare[0]], [spare[1]]]).cuda()
    qd, x = q.cuda()[:, :8], torch.empty(2, 2 * heads, dim, dtype=torch.bfloat16, device="cuda")
    ws = nv.kv8_workspace(8, dev, t, n, 2)
    names = ("k_codes", "v_codes", "k_scales", "v_scales", "weights")

    def step(dev):
        nv.kv8_append(x[:, :heads], x[:, heads:], dev, t, n)
        out = nv.kv8_attention(qd, dev, t, n, scale=0.002, accumulate=True, workspace=ws)
        return (out,) + nv.kv8_evict(dev, t, n, new_table, 50, recent=9, sink=2)

    inputs = [torch.randn(x.shape, generator=_gen(30 + i)).bfloat16() for i in range(4)]
    want = []
    for y in inputs:                                  # eager, on pools of their own
        x.copy_(y)
        e = _gpu(c)
        want.append([r.clone() for r in step(e)] + [getattr(e, s) for s in names])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(dev)
    for y, w in zip(inputs, want):
        for s in names:
            getattr(dev, s).copy_(getattr(c, s))
        x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(list(got) + [getattr(dev, s) for s in names], w):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---- eviction ----------------------------------------------------------------------------------------

EVICTS = [  # dim, page, heads, lens, keep, recent, sink, kind
    (128, 64, 2, [300, 100, 64, 0, 101], 100, 10, 4, "random"),
    (64, 16, 1, [500, 33], 32, 0, 0, "random"),
    (256, 32, 1, [90], 70, 70, 0, "random"),           # only the last
    (128, 128, 2, [1000, 700], 300, 20, 280, "random"),  # only the ends
    (64, 32, 2, [200, 77], 50, 3, 1, "equal"),
    (64, 16, 1, [400], 111, 7, 2, "steps"),
    (64, 16, 1, [300], 1, 0, 0, "odd"),
    (128, 64, 1, [5000], 1234, 100, 4, "steps"),
    (64, 64, 1, [260, 90], 80, 5, 2, "odd"),
]


@pytest.mark.parametrize("dim,page,heads,lens,keep,recent,sink,kind", EVICTS)
def test_evict(dim, page, heads, lens, keep, recent, sink, kind):
    _say("evict", dim, page, heads, lens, keep, recent, sink, kind)
    per = -(-keep // page)
    pages = sum(-(-n // page) for n in lens) + len(lens) * per + 1
    c = _filled(pages, heads, dim, page, 40, weights=True)
    g = _gen(41)
    if kind == "equal":
        c.weights.fill_(0.25)
    elif kind == "steps":                              # few values: ties everywhere
        c.weights.copy_(torch.randint(0, 3, c.weights.shape, generator=g) * 0.125)
    elif kind == "odd":
        few = torch.tensor([0.0, -0.0, math.inf, math.nan, -1.0, 1e-42, 3.0, -math.inf])
        c.weights.copy_(few[torch.randint(0, 8, c.weights.shape, generator=g)])
    table = _table(lens, page, pages, 42, spare=len(lens) * per)
    first = pages - len(lens) * per
    new_table = (first + torch.randperm(len(lens) * per, generator=g)).to(torch.int32).reshape(len(lens), per)
    pool, dev = ref.Pool(c), _gpu(c)
    news, kept = pool.evict(table, lens, new_table, keep, recent, sink)
    got = nv.kv8_evict(dev, table.cuda(), _i32(lens).cuda(), new_table.cuda(), keep, recent=recent, sink=sink)
    assert torch.equal(got[0].cpu(), news) and torch.equal(got[1].cpu(), kept)
    _same(pool, dev)


def test_evict_with_unnamed_pages():
    _say("evict, bad pages")
    page = 16
    c = _filled(40, 2, 64, page, 50, weights=True)
    table = _table([150, 200], page, 40, 51, spare=10)
    table[0, 3], table[1, 0] = -1, 40                 # their tokens come last, and as zeros if kept
    new_table = _i32([[30, 31, 99], [32, -1, 33]])
    pool, dev = ref.Pool(c), _gpu(c)
    news, kept = pool.evict(table, [150, 200], new_table, 45, 5, 3)
    got = nv.kv8_evict(dev, table.cuda(), _i32([150, 200]).cuda(), new_table.cuda(), 45, recent=5, sink=3)
    assert torch.equal(got[0].cpu(), news) and torch.equal(got[1].cpu(), kept)
    _same(pool, dev)


def test_evict_then_attend():
    """Attention over what an eviction kept is attention over those tokens."""
    _say("evict, then attend")
    c, table, q = _problem(128, 64, 1, 4, [400], [1], 0)
    c2 = _filled(c.k_codes.shape[0] + 2, 1, 128, 64, 60, weights=True)
    for s in ("k_codes", "v_codes", "k_scales", "v_scales", "weights"):
        getattr(c2, s)[:c.k_codes.shape[0]] = getattr(c, s)
    first = c.k_codes.shape[0]
    new_table = _i32([[first + 1, first]])
    dev, pool = _gpu(c2), ref.Pool(c2)
    pool.evict(table, [400], new_table, 100, 16, 4)
    n, _ = nv.kv8_evict(dev, table.cuda(), _i32([400]).cuda(), new_table.cuda(), 100, recent=16, sink=4)
    out, lse, b_out, b_lse, _ = pool.attention(q[:, :4], new_table, [100], [1], 0.002)
    got = nv.kv8_attention(q.cuda()[:, :4], dev, new_table.cuda(), n, scale=0.002, lse=True)
    _within(got[0], out, b_out, "out")
    _within(got[1], lse, b_lse, "lse")


def test_many_rounds_of_a_very_long_cache():
    """More tokens than one launch's pieces hold at a time (pages named again and again, so that the pool stays
    small: the reference sees the same tokens)."""
    _say("very long cache")
    dim, page, heads, q_heads, n = 64, 128, 1, 2, 700000
    c = _filled(9, heads, dim, page, 80)
    table = torch.randint(0, 9, (1, -(-n // page)), generator=_gen(81), dtype=torch.int32)
    q = torch.randn(1, q_heads + 3, dim, generator=_gen(82)).bfloat16()
    _check(c, table, q, q_heads, [n], [1], accumulate=False)


@pytest.mark.parametrize("kind", ["random", "equal", "steps", "odd"])
def test_evict_long(kind):
    """More tokens than one workgroup selects from, next to a sequence that is kept whole and one that is not."""
    _say("evict long", kind)
    dim, page, heads, lens, keep, recent, sink = 64, 128, 1, [41003, 900, 33000], 1500, 130, 5
    test_evict(dim, page, heads, lens, keep, recent, sink, kind)
    test_evict(dim, page, heads, [36000], 4200, 4000, 200, kind)


def test_evict_holds_a_length_to_max_len():
    _say("evict, max_len")
    c = _filled(12, 1, 64, 64, 90, weights=True)
    table, new_table = _table([400], 64, 12, 91, spare=3), _i32([[9, 10]])
    pool, dev = ref.Pool(c), _gpu(c)
    news, kept = pool.evict(table, [333], new_table, 100, 7, 3)
    got = nv.kv8_evict(dev, table.cuda(), _i32([400]).cuda(), new_table.cuda(), 100, recent=7, sink=3, max_len=333)
    assert torch.equal(got[0].cpu(), news) and torch.equal(got[1].cpu(), kept)
    _same(pool, dev)
