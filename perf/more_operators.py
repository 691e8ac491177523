"""The operators of an FFN block in 8-bit integers, as measured: quantizing rows, the matrix product with a scale
for each token and channel, the SwiGLU FFN built of it, and the norms before and after the block.

`run` computes a case either in its plain form (elementary torch operations in 32 bits) or, where `own` is
true, through the package's entry points.  The definitions:

* rows in int8: s = amax / 127 in fp32 (1 for a row of zeros), code = x / s in fp32, rounded to the nearest
  whole number, ties to the even one.  (A row with an infinity or a NaN has s = NaN and codes of 0.)
* product: y[r][c] = bf16(s_row[r] * s_col[c] * sum_k x[r][k] * w[c][k]), the sum of whole numbers;
* FFN: gate, up and act = silu(gate) * up are rounded to bf16, x and act are quantized by rows;
* norm: n = x / sqrt(mean(x^2) + eps) * (offset + weight), rounded to bf16 and, where asked for, quantized;
* residual: h = bf16(residual + scale * gate * norm(y)), then the next block's norm of h.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # a few decode rows enter an int8 projection
        dict(name="quantize step", op="quantize", m=37, k=4096),
        # a whole up projection is quantized by output channels when a model is loaded
        dict(name="quantize weight", op="quantize", m=17408, k=5120),
        # one token: the projection to 32 query, 8 key and 8 value heads of 128
        dict(name="project one", op="product", m=1, n=6144, k=4096, rows=False),
        # a batch of uneven prompts' last pieces; an odd number of channels
        dict(name="project ragged", op="product", m=333, n=7001, k=4128, rows=False),
        # a prompt whose rows the norm before has quantized
        dict(name="project prompt", op="product", m=2048, n=17408, k=5120, rows=True),
        # the FFN of one token
        dict(name="ffn one", op="ffn", m=1, n=12288, k=4096, rows=False),
        # the FFN of a serving batch
        dict(name="ffn batch", op="ffn", m=64, n=17408, k=5120, rows=False),
        # the FFN of a prompt
        dict(name="ffn prompt", op="ffn", m=2048, n=17408, k=5120, rows=False),
        # the norm before a block at a decode step, straight to int8
        dict(name="norm step", op="norm", m=4, k=4096, int8=True, weight=True, offset=0.0),
        # the norm before a block for a batch of prompts
        dict(name="norm prompt", op="norm", m=8192, k=5120, int8=False, weight=True, offset=1.0),
        # the end of a block at a decode step: norm after it, a gate for each channel, residual, next norm to int8
        dict(name="residual step", op="residual", m=64, k=5120, int8=True, post=True, gates=1, scale=0.5, next=True,
             offset=1.0),
        # the end of a block for prompts, with a gate for each row and channel
        dict(name="residual prompt", op="residual", m=4099, k=4096, int8=False, post=True, gates=4099, scale=1.0,
             next=True, offset=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "ffn", "ffn", "norm", "residual", "residual"])
    c = dict(op=op, m=_log(rng, 1, 8192), k=32 * _log(rng, 8, 544))
    if op in ("product", "ffn"):
        c["rows"] = rng.random() < 0.5
        # any number of output channels; the FFN's inner width is the down projection's k
        c["n"] = _log(rng, 17, 17408) if op == "product" else 32 * _log(rng, 8, 544)
        while c["m"] * c["n"] * c["k"] > 2048 * 17408 * 5120:
            c["m"] = c["m"] * 2 // 3
    else:
        if op == "quantize":
            c["m"] = _log(rng, 1, 17408)
        while c["m"] * c["k"] > 2 ** 25:
            c["m"] = c["m"] * 2 // 3
    if op in ("norm", "residual"):
        c["int8"] = rng.random() < 0.5
        c["offset"] = rng.choice([0.0, 1.0])
    if op == "norm":
        c["weight"] = rng.random() < 0.8
    if op == "residual":
        c["post"], c["next"] = rng.random() < 0.7, rng.random() < 0.8
        c["scale"] = rng.choice([1.0, 0.5, 0.22])
        c["gates"] = rng.choice([0, 1, c["m"], max(g for g in range(1, min(c["m"], 64) + 1) if c["m"] % g == 0)])
        c["int8"] = c["int8"] and c["next"]
    return c


def work(case):
    c = case
    m, k, op = c["m"], c["k"], c["op"]
    rows8, rows16 = m * (k + 4), 2 * m * k
    if op == "quantize":
        return {"bytes": rows16 + rows8, "flops": 0}
    if op == "product":
        return {"bytes": (rows8 if c["rows"] else rows16) + c["n"] * (k + 4) + 2 * m * c["n"], "flops": 2 * m * c["n"] * k}
    if op == "ffn":
        return {"bytes": (rows8 if c["rows"] else rows16) + 3 * c["n"] * k + 8 * c["n"] + 4 * k + rows16,
                "flops": 6 * m * c["n"] * k}
    out = rows8 if c["int8"] else rows16
    if op == "norm":
        return {"bytes": rows16 + out + 2 * k * c["weight"], "flops": 0}
    return {"bytes": 3 * rows16 + (out if c["next"] else 0) + 2 * k * (c["gates"] + c["post"] + c["next"]), "flops": 0}


# ---- what a program has in hand -------------------------------------------------------------------

def _activations(g, m, k):
    """Rows of unit size, one value in a hundred twenty times as large."""
    x = torch.randn(m, k, generator=g, device=DEV)
    far = torch.rand(m, k, generator=g, device=DEV) < 0.01
    return torch.where(far, 20 * x, x).to(torch.bfloat16)


def _weight(g, n, k):
    """Codes and channel scales of a weight that keeps a product near its input's size."""
    codes = torch.empty(n, k, dtype=torch.int8, device=DEV)
    step = max(1, 2 ** 26 // k)
    for i in range(0, n, step):
        part = torch.randn(min(step, n - i), k, generator=g, device=DEV)
        codes[i:i + step] = (32 * part).round_().clamp_(-127, 127).to(torch.int8)
    return codes, (0.5 + torch.rand(n, generator=g, device=DEV)) * (k ** -0.5 / 32)


def _vector(g, k, offset):
    return (1 - offset + 0.2 * torch.randn(k, generator=g, device=DEV)).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    m, k = c["m"], c["k"]
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case=dict(c))
    if c["op"] in ("quantize", "product", "ffn"):
        s["x"] = _activations(g, m, k)
        if c.get("rows"):
            s["x8"] = _quantize(s["x"])
        if c["op"] == "product":
            s["w"] = _weight(g, c["n"], k)
        if c["op"] == "ffn":
            s["wg"], s["wu"], s["wd"] = _weight(g, c["n"], k), _weight(g, c["n"], k), _weight(g, k, c["n"])
        return s
    # a residual stream: some channels are much larger than the others
    size = torch.exp(0.7 * torch.randn(k, generator=g, device=DEV))
    s["x"] = (4 * size * torch.randn(m, k, generator=g, device=DEV)).to(torch.bfloat16)
    if c["op"] == "norm":
        s["weight"] = _vector(g, k, c["offset"]) if c["weight"] else None
        return s
    s["y"] = _activations(g, m, k)
    s["post"] = _vector(g, k, c["offset"]) if c["post"] else None
    s["next"] = _vector(g, k, c["offset"]) if c["next"] else None
    s["gate"] = torch.tanh(torch.randn(c["gates"], k, generator=g, device=DEV)).to(torch.bfloat16) if c["gates"] else None
    return s


# ---- the framework's kernels -----------------------------------------------------------------------

def _run_own(s):
    import nvfp4_weight_dense_amd as nv
    c = s["case"]
    if c["op"] == "quantize":
        return list(nv.int8_quantize_rows(s["x"]))
    if c["op"] == "norm":
        return _rows_out(c, nv.rms_norm(s["x"], s["weight"], eps=EPS, weight_offset=c["offset"], int8=c["int8"]))
    if c["op"] == "residual":
        h, n = nv.rms_norm_residual(s["x"], s["y"], post=s["post"], gate=s["gate"], scale=c["scale"], norm=s["next"],
                                    eps=EPS, weight_offset=c["offset"], int8=c["int8"])
        return [h] + ([] if n is None else _rows_out(c, n))
    x = nv.Int8Rows(*s["x8"]) if c["rows"] else s["x"]
    if c["op"] == "product":
        return nv.int8_gemm_w8a8(x, nv.Int8Weight(*s["w"]))
    return nv.dense_ffn_forward_int8(x, *(nv.Int8Weight(*s[w]) for w in ("wg", "wu", "wd")))


def _rows_out(c, n):
    """A norm's result: bf16 rows, or int8 rows as the values they stand for, with their scales."""
    return [_values(*n), n[1]] if c["int8"] else [n]


def _values(codes, scale):
    return (codes.float() * scale[:, None]).to(torch.bfloat16)


# ---- the plain forms ------------------------------------------------------------------------------

def _quantize(x):
    """int8 rows: codes and scales.  The divisions are done in 64 bits and rounded to 32, which is the
    correctly rounded quotient in 32 bits."""
    x = x.float()
    amax = x.abs().amax(1, keepdim=True)
    scale = (amax.double() / torch.full_like(amax, 127.0).double()).float()
    scale = torch.where(amax == 0, 1.0, scale)
    scale = torch.where(torch.isfinite(amax), scale, math.nan)
    q = (x.double() / scale.double()).float().round_().clamp_(-127, 127)
    return torch.nan_to_num_(q, nan=0.0).to(torch.int8), scale[:, 0]


def _product(x8, w):
    acc = torch.matmul(x8[0].float(), w[0].float().t())
    return (acc * x8[1][:, None] * w[1]).to(torch.bfloat16)


def _norm(x, weight, offset):
    n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    return n if weight is None else n * (offset + weight.float())


def _norm_out(c, n):
    n = n.to(torch.bfloat16)
    return _rows_out(c, _quantize(n) if c["int8"] else n)


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s)
    if c["op"] == "quantize":
        return list(_quantize(s["x"]))
    if c["op"] == "norm":
        return _norm_out(c, _norm(s["x"].float(), s["weight"], c["offset"]))
    if c["op"] == "residual":
        y = s["y"].float()
        if c["post"]:
            y = _norm(y, s["post"], c["offset"])
        if s["gate"] is not None:
            y = (y.view(c["gates"], -1, c["k"]) * s["gate"].float()[:, None]).view(c["m"], c["k"])
        h = (s["x"].float() + c["scale"] * y).to(torch.bfloat16)
        return [h] + (_norm_out(c, _norm(h.float(), s["next"], c["offset"])) if c["next"] else [])
    x8 = s["x8"] if c["rows"] else _quantize(s["x"])
    if c["op"] == "product":
        return _product(x8, s["w"])
    gate, up = _product(x8, s["wg"]).float(), _product(x8, s["wu"]).float()
    act = (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    return _product(_quantize(act), s["wd"])


# ---- in 64 bits, from the definitions --------------------------------------------------------------

def _nearest_bf16(x):
    """x (64 bits) rounded once to 8 significant bits, half to even."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 8).clamp(min=-133))
    return torch.round(x / step) * step


def _by_rows(x):
    """The whole numbers (as numbers) and the scale of each row of x (64 bits, finite)."""
    top = x.abs().max(1, keepdim=True).values
    s = (top / torch.tensor(127.0, dtype=torch.float64, device=x.device)).float().double()
    s[top == 0] = 1.0
    return torch.round((x / s).float().double()), s


def _exact_norm(x, weight, offset):
    n = x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS)
    return n if weight is None else n * (weight.double() + offset)


def _exact_out(c, n):
    if not c["int8"]:
        return [n]
    q, s = _by_rows(_nearest_bf16(n))
    return [q * s, s[:, 0]]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    x = s["x"].double()
    if c["op"] == "quantize":
        q, scale = _by_rows(x)
        return [q.to(torch.int8), scale[:, 0]]
    if c["op"] == "norm":
        return _exact_out(c, _exact_norm(x, s["weight"], c["offset"]))
    if c["op"] == "residual":
        y = s["y"].double()
        if c["post"]:
            y = _exact_norm(y, s["post"], c["offset"])
        if c["gates"]:
            y = y * s["gate"].double().repeat_interleave(c["m"] // c["gates"], 0)
        h = x + c["scale"] * y
        return [h] + (_exact_out(c, _exact_norm(_nearest_bf16(h), s["next"], c["offset"])) if c["next"] else [])

    def times(q, scale, w):
        return (q @ w[0].double().t()) * (scale * w[1].double())

    q, scale = (s["x8"][0].double(), s["x8"][1].double()[:, None]) if c["rows"] else _by_rows(x)
    if c["op"] == "product":
        return times(q, scale, s["w"])
    gate, up = _nearest_bf16(times(q, scale, s["wg"])), _nearest_bf16(times(q, scale, s["wu"]))
    return times(*_by_rows(_nearest_bf16(gate * torch.sigmoid(gate) * up)), s["wd"])
