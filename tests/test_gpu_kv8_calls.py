"""Calls of the 8-bit paged KV cache as programs make them, on the GPU against the 64-bit reference: their own
workspaces, and what test_gpu_kv8.py's cases of one kernel each do not combine."""

import math

import pytest
import torch

import kv8_ref as ref
import nvfp4_weight_dense_amd as nv
from test_gpu_kv8 import _check, _filled, _gen, _gpu, _i32, _problem, _same, _say, _starts, _table, _within

pytestmark = pytest.mark.gpu


# ---- workspaces --------------------------------------------------------------------------------------

@pytest.mark.parametrize("cols,lens,rows,window", [(4096, [3969, 64, 4100, 3970, 1, 4090, 129, 4001], 1, 454351),
                                                   (4096, [3969, 300, 3970], 4, 0), (31, [3968, 200], 8, 4096),
                                                   (4000, [4000, 777], 150, 3000)])
def test_workspace_of_exactly_the_given_size(cols, lens, rows, window):
    """A table far wider than its sequences, so that a few tokens are many pieces: the bytes past the workspace
    keep what they hold, and the workspace is ready for the next call."""
    _say("workspace", cols, lens, rows, window)
    dim, page, heads, q_heads = 128, 128, 2, 8
    c, _, q = _problem(dim, page, heads, q_heads, lens, [rows] * len(lens), window, weights=False)
    table = _table(lens, page, c.k_codes.shape[0], 12, cols=cols)
    pool, dev, t, n = ref.Pool(c), _gpu(c), table.cuda(), _i32(lens).cuda()
    size = nv.kv8_workspace(q_heads, dev, t, n, rows * len(lens)).numel()
    room = torch.full((size + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    assert room.data_ptr() % 256 == 0
    ws = room[:size]
    ws.zero_()
    want = pool.attention(q[:, :q_heads], table, lens, [rows] * len(lens), 0.002, window)
    for _ in range(2):
        out, lse = nv.kv8_attention(q.cuda()[:, :q_heads], dev, t, n, scale=0.002, window=window, lse=True, workspace=ws)
        _within(out, want[0], want[2], "out")
        _within(lse, want[1], want[3], "lse")
        assert bool((room[size:] == 0x5A).all())


def test_one_workspace_for_calls_of_other_sizes():
    """What one call leaves in a workspace is no other's trouble: caches of other pools, with and without weights,
    few rows and many, in turn on one workspace."""
    _say("one workspace, many sizes")
    jobs = []
    for i, (dim, page, heads, q_heads, lens, rows, weights) in enumerate([
            (128, 64, 2, 8, [700, 64, 300], [1, 1, 1], True), (64, 16, 1, 2, [900, 50], [200, 50], True),
            (256, 32, 1, 4, [1200], [3], False), (128, 16, 1, 1, [2000, 1999, 5], [1, 2, 3], True),
            (64, 128, 4, 4, [1500], [400], False)]):
        c, table, q = _problem(dim, page, heads, q_heads, lens, rows, 0, seed=280 + 5 * i, weights=weights)
        jobs.append((c, table, q, q_heads, lens, rows, weights))
    ws = max((nv.kv8_workspace(h, _gpu(c), t.cuda(), _i32(lens).cuda(), sum(rows), _starts(rows).cuda(),
                               max_rows=max(rows)) for c, t, _, h, lens, rows, _ in jobs), key=lambda x: x.numel())
    for _ in range(3):
        for c, table, q, q_heads, lens, rows, weights in jobs:
            _check(c, table, q, q_heads, lens, rows, accumulate=weights, workspace=ws)


# ---- rows beyond max_rows ----------------------------------------------------------------------------

@pytest.mark.parametrize("dim,page,max_rows", [(128, 64, 1), (128, 64, 8), (64, 16, 1), (64, 16, 8), (256, 32, 1),
                                               (256, 32, 8), (128, 128, 20), (64, 128, 40)])
def test_append_leaves_rows_beyond_max_rows_out(dim, page, max_rows):
    """starts that give a sequence more rows than max_rows: its first max_rows rows are written, at their own
    places, and nothing else changes."""
    _say("append, max_rows", dim, page, max_rows)
    heads, lens, rows = 2, [200, 33, 90, 5, 1], [50, 33, 7, 9, 1]
    c = _filled(sum(-(-n // page) for n in lens) + 2, heads, dim, page, 130, weights=True)
    pool, dev = ref.Pool(c), _gpu(c)
    table = _table(lens, page, c.k_codes.shape[0], 131)
    x = torch.randn(sum(rows), 2 * heads, dim, generator=_gen(132))
    x = (x * torch.exp(2 * torch.randn(sum(rows), 1, 1, generator=_gen(133)))).bfloat16()
    held, most, at = [], [], 0
    for n, r in zip(lens, rows):
        m = min(r, max_rows)
        held.append(x[at:at + m])
        most.append(m)
        at += r
    y = torch.cat(held)
    pool.append(y[:, :heads], y[:, heads:], table, [n - r + m for n, r, m in zip(lens, rows, most)], most)
    d = x.cuda()
    nv.kv8_append(d[:, :heads], d[:, heads:], dev, table.cuda(), _i32(lens).cuda(), _starts(rows).cuda(), max_rows=max_rows)
    _same(pool, dev)


# ---- windows -----------------------------------------------------------------------------------------

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 2 ** 30, 2 ** 63 - 1, 10 ** 5])
@pytest.mark.parametrize("dim,page,q_heads,lens,rows", [
    (128, 64, 4, [300, 77], [1, 1]), (128, 32, 4, [40, 3], [12, 9]), (64, 16, 4, [700, 600], [690, 600]),
    (128, 64, 2, [40, 3], [60, 150]), (256, 16, 1, [1100, 5], [300, 280]), (64, 64, 8, [20, 700], [16, 16])])
def test_windows_wider_than_any_cache(dim, page, q_heads, lens, rows, window):
    """A window past every length is none, also for rows before position 0 (which see nothing) and for weights."""
    _say("wide window", dim, page, q_heads, lens, rows, window)
    c, table, q = _problem(dim, page, 1, q_heads, lens, rows, 0, seed=140)
    got = _check(c, table, q, q_heads, lens, rows, window=window)
    want = _check(c, table, q, q_heads, lens, rows, window=10 ** 6)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---- shared pages ------------------------------------------------------------------------------------

def _shared(kind, lens, page, pages, seed):
    """A table whose sequences share pages: all of a common prefix; at other blocks; within one sequence too."""
    table = _table(lens, page, pages, seed)
    g = _gen(seed + 1)
    if kind == "prefix":
        for b in range(1, len(lens)):
            most = min(lens[0], lens[b]) // page
            table[b, :most] = table[0, :most]
    elif kind == "anywhere":
        for b, n in enumerate(lens):
            for c in range(-(-n // page)):
                if float(torch.rand((), generator=g)) < 0.5:
                    table[b, c] = int(torch.randint(0, 3, (), generator=g))
    else:                                              # every block names one of two pages
        for b, n in enumerate(lens):
            table[b, :-(-n // page)] = torch.randint(0, 2, (-(-n // page),), generator=g, dtype=torch.int32)
    return table


SHARED = [  # dim, page, heads, q_heads, lens, rows, window
    (128, 64, 2, 8, [700, 641, 130, 64, 65, 1, 0, 400], [1, 1, 1, 1, 1, 1, 1, 0], 0),
    (128, 16, 1, 4, [300, 290, 17, 260, 33], [1, 4, 2, 4, 3], 0),
    (64, 128, 2, 2, [500, 384, 129], [7, 1, 5], 200),
    (256, 32, 1, 1, [330, 290, 64], [16, 3, 9], 0),
    (128, 64, 2, 4, [300, 280, 90], [30, 25, 1], 0),            # more columns than the attention leaves scores for
    (64, 32, 1, 2, [700, 650, 333, 65], [300, 222, 100, 65], 0),
    (256, 16, 1, 4, [210, 199, 40], [90, 60, 2], 70),
    (64, 64, 1, 1, [129 + i for i in range(150)], [1] * 150, 0),  # more sequences than are looked up at a time
]


@pytest.mark.parametrize("kind", ["prefix", "anywhere", "two"])
@pytest.mark.parametrize("dim,page,heads,q_heads,lens,rows,window", SHARED)
def test_weights_of_shared_pages(dim, page, heads, q_heads, lens, rows, window, kind):
    """A page's weights get what the rows of every sequence that names it give, with the same bits each time."""
    _say("shared pages", kind, dim, page, heads, q_heads, len(lens), max(lens), max(rows), window)
    pages = sum(-(-n // page) for n in lens) + 3
    c = _filled(pages, heads, dim, page, 150, weights=True)
    table = _shared(kind, lens, page, pages, 151)
    q = torch.randn(sum(rows), q_heads, dim, generator=_gen(152)).bfloat16()
    pool = ref.Pool(c)
    out, lse, b_out, b_lse, w = pool.attention(q, table, lens, rows, 0.002, window)
    want, bound = pool.weights.double(), pool.weights.double() * 2.0 ** -23
    uses = torch.zeros_like(want)
    for b, (x, bx) in enumerate(w):
        at = pool.where(table, b, torch.arange(len(x)))
        assert bool((at[0] >= 0).all())
        want.index_put_(at, x, accumulate=True)
        bound.index_put_(at, bx, accumulate=True)
        uses.index_put_(at, torch.ones_like(x), accumulate=True)
    bound += uses * want * 2.0 ** -24                   # one addition for each use
    first = None
    for _ in range(4):
        dev = _gpu(c)
        got = nv.kv8_attention(q.cuda(), dev, table.cuda(), _i32(lens).cuda(), _starts(rows).cuda(), scale=0.002,
                               window=window, max_rows=max(rows), lse=True, accumulate=True)
        _within(got[0], out, b_out, "out")
        _within(got[1], lse, b_lse, "lse")
        _within(dev.weights, want, bound + 1e-30, "weights")
        bits = dev.weights.view(torch.int32).clone()
        assert first is None or torch.equal(first, bits)
        first = bits


def test_weights_of_a_page_that_every_block_names():
    """More blocks on one page than are listed at a time."""
    _say("one page")
    dim, page, lens = 64, 16, [40000, 17, 20000]
    c = _filled(3, 1, dim, page, 160, weights=True)
    table = torch.full((3, 2500), 1, dtype=torch.int32)
    q = torch.randn(3, 2, dim, generator=_gen(161)).bfloat16()
    pool = ref.Pool(c)
    *_, w = pool.attention(q, table, lens, [1, 1, 1], 0.002)
    want = pool.weights.double()
    for x, _ in w:
        want[1] += torch.nn.functional.pad(x, (0, -len(x) % page)).reshape(-1, page).sum(0)
    dev = _gpu(c)
    nv.kv8_attention(q.cuda(), dev, table.cuda(), _i32(lens).cuda(), scale=0.002, accumulate=True)
    # each weight is the sum of some thousand, each of which is off by some 2^-20 of itself
    _within(dev.weights, want, want * (5000 * 2.0 ** -24 + 2.0 ** -18), "weights")


def test_lengths_of_a_table_wider_than_its_sequences():
    """Weights where the table names pages beyond the lengths: those get none."""
    _say("wide table")
    c, table, q = _problem(128, 64, 1, 4, [100, 64, 1], [1, 1, 1], 0, seed=170)
    wide = torch.randint(0, c.k_codes.shape[0], (3, 700), generator=_gen(171), dtype=torch.int32)
    wide[:, :2] = table[:, :2].clamp(min=0)
    _check(c, wide, q, 4, [100, 64, 1], [1, 1, 1])


# ---- streams -----------------------------------------------------------------------------------------

def _others(like):
    """Takes memory of these tensors' sizes for other work of the current stream, and fills it."""
    got = [torch.empty_like(x) for x in like for _ in range(8)]
    for x in got:
        x.view(torch.uint8).fill_(0xFF)
    return got


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("rows", [[1, 1, 1, 1], [30, 5, 64, 1]])
def test_tensors_of_a_call_on_another_stream(rows, handle):
    """The call's own tensors are not handed out again before its kernels have run: its stream is held up while
    the current one asks for tensors of the same sizes."""
    _say("another stream", rows, handle)
    lens = [900, 333, 64, 1]
    c, table, q = _problem(128, 64, 2, 8, lens, rows, 0, seed=180)
    pages = c.k_codes.shape[0]
    more = _filled(pages + 8, 2, 128, 64, 181, weights=True)
    for x in ("k_codes", "v_codes", "k_scales", "v_scales", "weights"):
        getattr(more, x)[:pages] = getattr(c, x)
    new_table = (pages + torch.randperm(8, generator=_gen(182))).to(torch.int32).reshape(4, 2).cuda()
    t, n, at, qd = table.cuda(), _i32(lens).cuda(), _starts(rows).cuda(), q.cuda()[:, 1:9]
    kw = dict(max_rows=max(rows), scale=0.002, accumulate=True)
    here, there = _gpu(more), _gpu(more)
    want = nv.kv8_attention(qd, here, t, n, at, **kw), nv.kv8_evict(here, t, n, new_table, 100, recent=9, sink=2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)                   # about a tenth of a second
    to = s.cuda_stream if handle else s
    out = nv.kv8_attention(qd, there, t, n, at, stream=to, **kw)
    nv.kv8_evict(there, t, n, new_table, 100, recent=9, sink=2, stream=to)      # (what it returns is dropped)
    held = _others([torch.empty(sum(rows), 8, device="cuda"), *want[1]])
    assert not s.query()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want[0].view(torch.int16))
    for x in ("k_codes", "v_codes", "k_scales", "v_scales", "weights"):
        assert torch.equal(getattr(there, x).view(torch.uint8), getattr(here, x).view(torch.uint8)), x
    assert all(bool((x.view(torch.uint8) == 0xFF).all()) for x in held)


# ---- scales ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("byte", [246, 247, 250, 254, 255, 0])
@pytest.mark.parametrize("dim,rows", [(128, [3, 1]), (64, [12, 9]), (256, [9, 16]), (128, [70, 40])])
def test_scale_bytes_beyond_those_that_append_writes(dim, rows, byte):
    """A byte above 246 acts as 246, whose largest code is still a bf16 number, and 0 as 1: rows that do not see
    such a page's tokens keep their results, and those that do get the values these bytes stand for."""
    _say("scale bytes", dim, rows, byte)
    lens, page = [100, 75], 16
    c, table, q = _problem(dim, page, 1, 4, lens, rows, 0, seed=190)
    last = [int(table[b, (n - 1) // page]) for b, n in enumerate(lens)]
    c.v_scales[last] = byte                               # seen by the last rows only
    c.k_scales[int(table[0, 2])] = 0                      # scores of next to nothing
    held = nv.KV8Cache(c.k_codes, c.v_codes, c.k_scales.clamp(1, 246), c.v_scales.clamp(1, 246), c.weights)
    pool, dev = ref.Pool(held), _gpu(c)
    want = pool.attention(q[:, 1:5], table, lens, rows, 0.002)
    got = nv.kv8_attention(q.cuda()[:, 1:5], dev, table.cuda(), _i32(lens).cuda(), _starts(rows).cuda(), scale=0.002,
                           max_rows=max(rows), lse=True)
    at = 0
    for n, r in zip(lens, rows):                          # rows at positions before the last page
        some = slice(at, at + max(r - (n - (n - 1) // page * page), 0))
        assert bool(torch.isfinite(got[0][some].float()).all())
        _within(got[0][some], want[0][some], want[2][some], "out")
        at += r
    _within(got[1], want[1], want[3], "lse")
    _within(got[0], want[0], want[2], "out") if byte < 240 else None


@pytest.mark.parametrize("byte", [250, 255])
def test_append_after_a_scale_byte_beyond_those_it_writes(byte):
    """Tokens that join a page with such a scale keep their values; the page's byte becomes the one it acted as."""
    _say("append, scale byte", byte)
    c, table, _ = _problem(64, 16, 1, 1, [20], [1], 0, seed=200)
    c.k_scales[:], c.v_scales[:] = byte, byte
    held = nv.KV8Cache(c.k_codes, c.v_codes, c.k_scales.clamp(1, 246), c.v_scales.clamp(1, 246), c.weights)
    for x in (torch.full((1, 1, 64), 2.0 ** 120), torch.full((1, 1, 64), -3.0e38)):
        pool, dev = ref.Pool(held), _gpu(c)
        x = x.bfloat16()
        pool.append(x, x, table, [20], [1])
        nv.kv8_append(x.cuda(), x.cuda(), dev, table.cuda(), _i32([20]).cuda())
        page = int(table[0, 1])
        assert int(dev.k_scales[page]) == int(dev.v_scales[page]) == 246
        for isv, codes in ((0, dev.k_codes), (1, dev.v_codes)):
            assert torch.equal(codes[page].cpu(), pool.raw(isv)[page])


# ---- eviction with its own workspace -----------------------------------------------------------------

def _long(seed, lens=(41003, 900, 33000), keep=1500):
    dim, page = 64, 128
    per = -(-keep // page)
    pages = sum(-(-n // page) for n in lens) + len(lens) * per
    c = _filled(pages, 1, dim, page, seed, weights=True)
    table = _table(list(lens), page, pages, seed + 1, spare=len(lens) * per)
    new_table = (pages - len(lens) * per + torch.arange(len(lens) * per)).to(torch.int32).reshape(len(lens), per)
    pool = ref.Pool(c)
    news, kept = pool.evict(table, list(lens), new_table, keep, 130, 5)
    return c, pool, news, kept, (table.cuda(), _i32(list(lens)).cuda(), new_table.cuda(), keep)


def test_evictions_that_overlap():
    """Two streams with a workspace each, of any contents and used again for fewer sequences and tokens."""
    _say("evictions on two streams")
    jobs = [_long(210), _long(220, lens=(36000, 40000), keep=3000)]
    streams, spaces = [torch.cuda.Stream() for _ in jobs], []
    for c, *_, (t, n, nt, keep) in jobs:
        ws = nv.kv8_evict_workspace(_gpu(c), t, n)
        spaces.append(ws.random_(0, 256))
    for again in range(2):
        devs = [_gpu(c) for c, *_ in jobs]
        torch.cuda.synchronize()
        got = []
        for (c, *_, (t, n, nt, keep)), dev, s, ws in zip(jobs, devs, streams, spaces):
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)
            got.append(nv.kv8_evict(dev, t, n, nt, keep, recent=130, sink=5, workspace=ws, stream=s))
        torch.cuda.synchronize()
        for (c, pool, news, kept, _), dev, g in zip(jobs, devs, got):
            assert torch.equal(g[0].cpu(), news) and torch.equal(g[1].cpu(), kept)
            _same(pool, dev)
    c, pool, news, kept, (t, n, nt, keep) = _long(230, lens=(33000,), keep=200)
    dev = _gpu(c)
    got = nv.kv8_evict(dev, t, n, nt, keep, recent=130, sink=5, workspace=spaces[0])
    assert torch.equal(got[0].cpu(), news) and torch.equal(got[1].cpu(), kept)
    _same(pool, dev)


def test_eviction_in_a_graph_after_the_arena_has_grown():
    """A captured eviction of a long cache keeps its results when a later call takes a larger arena."""
    _say("eviction in a graph")
    c, pool, news, kept, (t, n, nt, keep) = _long(240)
    dev = _gpu(c)
    ws = nv.kv8_evict_workspace(dev, t, n)
    nv.kv8_evict(dev, t, n, nt, keep, recent=130, sink=5, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = nv.kv8_evict(dev, t, n, nt, keep, recent=130, sink=5, workspace=ws)
    big = _long(250, lens=(200000, 200000, 200000, 200000))
    for again in range(3):
        for x in ("k_codes", "v_codes", "k_scales", "v_scales", "weights"):
            getattr(dev, x).copy_(getattr(c, x))
        got[0].zero_()
        got[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0].cpu(), news) and torch.equal(got[1].cpu(), kept)
        _same(pool, dev)
        other = _gpu(big[0])                                # eager work between the replays
        r = nv.kv8_evict(other, *big[4], recent=130, sink=5)
        torch.cuda.synchronize()
        assert torch.equal(r[1].cpu(), big[3])


# ---- precision ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dim,heads,q_heads,lens,rows", [(128, 2, 8, [3000, 517], [1, 1]), (128, 1, 4, [900, 77], [16, 5]),
                                                         (128, 1, 2, [700], [64]), (64, 2, 8, [2100, 64], [1, 1]),
                                                         (64, 1, 4, [600, 300], [8, 7]), (256, 1, 8, [1500], [1]),
                                                         (256, 1, 4, [800, 90], [16, 3])])
def test_few_rows_lose_nothing_but_the_rounding_of_their_results(dim, heads, q_heads, lens, rows):
    """The probabilities' share of the bound is two bf16 (2^-16), not one (2^-8)."""
    _say("precision", dim, heads, q_heads, lens, rows)
    c, table, q = _problem(dim, 64, heads, q_heads, lens, rows, 0, seed=260, weights=False)
    q = q[:, :q_heads]
    pool, size = ref.Pool(c), ref.Pool(c)
    size.codes[1] = size.codes[1] & 0x7F                   # |v|
    want, _, bound, _, _ = pool.attention(q, table, lens, rows, 0.002)
    mass = size.attention(q, table, lens, rows, 0.002)[0]
    got = nv.kv8_attention(q.cuda(), _gpu(c), table.cuda(), _i32(lens).cuda(), _starts(rows).cuda(), scale=0.002,
                           max_rows=max(rows))
    _say("  %.2f of the bound" % _within(got, want, bound - mass * (2.0 ** -8 - 2.0 ** -16), "out"))


# ---- infinite scores ---------------------------------------------------------------------------------

@pytest.mark.parametrize("dim,rows", [(128, [1, 3]), (128, [12, 9]), (64, [100, 60]), (256, [30, 41])])
def test_rows_whose_scores_are_all_minus_infinity(dim, rows):
    """Such a row gives no token any weight, and leaves those of the other rows as they are."""
    _say("scores of -inf", dim, rows)
    lens = [200, 131]
    c, table, q = _problem(dim, 64, 1, 4, lens, rows, 0, seed=270)
    flat = c.k_codes.view(c.k_codes.shape[0], -1)
    flat[:, ref.k_at(torch.arange(64), 5, dim)] = 0x38     # 1.0 in every token's channel 5
    q = q[:, :4].clone()
    clean = q.clone()
    q[0, 1, 5], q[rows[0], 2, 5] = -math.inf, -math.inf
    t, n, at = table.cuda(), _i32(lens).cuda(), _starts(rows).cuda()
    devs = [_gpu(c) for _ in range(2)]
    (out, lse), (ref_out, ref_lse) = (nv.kv8_attention(x.cuda(), dev, t, n, at, scale=0.002, max_rows=max(rows), lse=True,
                                                       accumulate=True) for x, dev in zip((q, clean), devs))
    gone = torch.zeros(sum(rows), 4, dtype=torch.bool)
    gone[0, 1] = gone[rows[0], 2] = True
    assert not out.cpu()[gone].any() and bool((lse.cpu()[gone] == -math.inf).all())
    assert torch.equal(out.cpu()[~gone].view(torch.int16), ref_out.cpu()[~gone].view(torch.int16))
    given = [(d.weights.cpu().double() - c.weights.double()).sum().item() for d in devs]
    assert abs(given[1] - sum(rows) * 4) < 1e-3 and abs(given[0] - (sum(rows) * 4 - 2)) < 1e-3
