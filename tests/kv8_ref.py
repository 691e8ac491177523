"""A plain 64-bit reference of the 8-bit paged KV cache, on the CPU: the cache
as numbers (values and scale exponents per token), written from the
definitions in include/nvfp4ffn.h, and the order of the codes in a page.

Error bounds count roundings: half a step relative to the value is
``torch.finfo(t).eps / 2`` (bf16 2^-8, fp32 2^-24)."""

from __future__ import annotations

import math

import torch

MIN_E, MAX_E = -117, 119
BF, F32 = 2.0 ** -8, 2.0 ** -24


def e4m3_values() -> torch.Tensor:
    """The number of each E4M3FN byte, from its fields."""
    v = torch.empty(256, dtype=torch.float64)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9)
        v[b] = math.nan if (b & 0x7F) == 0x7F else math.copysign(x, -1 if b & 128 else 1)
    return v


VALUES = e4m3_values()


def encode(x: torch.Tensor) -> torch.Tensor:
    """fp64 -> E4M3 bytes: nearest, ties to the even code, saturating, NaN kept."""
    mag = VALUES[:127]
    a = x.abs().clamp(max=448.0).nan_to_num(0.0)
    hi = torch.searchsorted(mag, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - mag[lo], mag[hi] - a
    code = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = torch.where(torch.isnan(x), 127, code)
    return (code + 128 * torch.signbit(x).long()).to(torch.uint8)


def exponent(amax: float) -> int:
    e = MIN_E
    while e < MAX_E and amax > math.ldexp(448.0, e):
        e += 1
    return e


def k_at(slot, d, dim):
    return (slot // 16) * 16 * dim + (d // 16) * 256 + (slot % 16) * 16 + d % 16


def v_at(slot, d, dim):
    return (slot // 16) * 16 * dim + (d // 64) * 1024 + (slot % 16 // 4) * 256 + (d % 16) * 16 + \
        (d % 64 // 16) * 4 + slot % 4


def order(page, dim, isv):
    """[page, dim] -> offset of each code in a page of one head."""
    t, d = torch.arange(page)[:, None], torch.arange(dim)[None, :]
    return (v_at if isv else k_at)(t, d, dim)


class Pool:
    """Codes per token [pages, heads, page, dim] (bytes) and scale bytes, for K and V."""

    def __init__(self, cache):
        self.pages, self.heads, self.page, self.dim = cache.k_codes.shape
        self.codes, self.scales = [], []
        for isv, (c, s) in enumerate(((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))):
            flat = c.cpu().reshape(self.pages, self.heads, -1)
            self.codes.append(flat[:, :, order(self.page, self.dim, isv)])
            self.scales.append(s.cpu().clone())
        self.weights = None if cache.weights is None else cache.weights.cpu().clone()

    def raw(self, isv):
        """Codes in the order of the cache's buffers."""
        flat = torch.empty(self.pages, self.heads, self.page * self.dim, dtype=torch.uint8)
        flat[:, :, order(self.page, self.dim, isv).reshape(-1)] = \
            self.codes[isv].reshape(self.pages, self.heads, -1)
        return flat.reshape(self.pages, self.heads, self.page, self.dim)

    def value(self, isv, page, slot):
        """fp64 values [n, heads, dim] of tokens; zero where page is -1."""
        ok = page >= 0
        p = page.clamp(min=0)
        x = VALUES[self.codes[isv][p, :, slot].long()]
        x = x * torch.ldexp(torch.ones(1, dtype=torch.float64), self.scales[isv][p].int() - 127)[..., None]
        x[~ok] = 0.0
        return x

    def append(self, k, v, table, lens, rows):
        """rows: new tokens per sequence; k, v in order."""
        at = 0
        for b, r in enumerate(rows):
            n = min(max(int(lens[b]), 0), table.shape[1] * self.page)
            for i in range(r):
                pos = n - r + i
                if pos < 0 or (i and pos % self.page):
                    continue                      # dropped, or written with the first token of its page's part
                m = min(n, (pos // self.page + 1) * self.page) - pos
                page = int(table[b, pos // self.page])
                if not 0 <= page < self.pages:
                    continue
                for isv, x in enumerate((k, v)):
                    self._write(isv, page, pos % self.page, x[at + i:at + i + m].double())
                if self.weights is not None:
                    self.weights[page, pos % self.page:pos % self.page + m] = 0
            at += r

    def _write(self, isv, page, slot, x):
        for h in range(self.heads):
            y = x[:, h]
            fin = y[torch.isfinite(y)].abs()
            e = exponent(float(fin.max()) if fin.numel() else 0.0)
            if slot:
                was = int(self.scales[isv][page, h]) - 127
                e = max(e, was)
                old = self.codes[isv][page, h, :slot]
                self.codes[isv][page, h, :slot] = encode(VALUES[old.long()] * math.ldexp(1.0, was - e))
            self.codes[isv][page, h, slot:slot + len(y)] = encode(y * math.ldexp(1.0, -e))
            self.scales[isv][page, h] = e + 127

    def where(self, table, b, t):
        page = table[b].long()[t // self.page]
        page = torch.where((page >= 0) & (page < self.pages), page, -1)
        return page, t % self.page

    def attention(self, q, table, lens, rows, scale, window=0, max_len=None):
        """out, lse, their error bounds, and per sequence the weights each token receives with their bounds."""
        hq, d = q.shape[1], self.dim
        group = hq // self.heads
        out = torch.zeros(q.shape, dtype=torch.float64)
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
        b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
        got, at = [], 0
        for b, r in enumerate(rows):
            n = min(max(int(lens[b]), 0), table.shape[1] * self.page)
            t = torch.arange(n)
            page, slot = self.where(table, b, t)
            k, v = self.value(0, page, slot), self.value(1, page, slot)
            w, bw = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
            pos = torch.arange(n - r, n)[:, None]
            seen = (t <= pos) & (page >= 0)
            if window:
                seen = seen & (t > pos - window)
            if max_len is not None:
                seen = seen & (t < max_len)
            for u in range(hq if n and r else 0):
                x = q[at:at + r, u].double()
                s = x @ k[:, u // group].t() * scale
                size = (x.abs() @ k[:, u // group].abs().t() * abs(scale)).masked_fill(~seen, 0.0).amax(1)
                s = s.masked_fill(~seen, -math.inf)
                z = torch.logsumexp(s, 1)
                p = torch.where(seen, torch.exp(s - z[:, None]), 0.0)
                # a score is a sum of d products, scaled, made a power of two and shifted: each fp32
                delta = F32 * ((d + 8) * size + 2 * z.abs().nan_to_num(posinf=0.0) + 16) * 2
                vv = v[:, u // group]
                # a row's own tokens only: a NaN elsewhere does not reach it
                o = torch.stack([p[i, seen[i]] @ vv[seen[i]] for i in range(r)])
                a = torch.stack([p[i, seen[i]] @ vv[seen[i]].abs() for i in range(r)])
                out[at:at + r, u], lse[at:at + r, u] = o, z
                b_lse[at:at + r, u] = delta + F32 * (n + 4 + z.abs().nan_to_num(posinf=0.0))
                b_out[at:at + r, u] = BF * o.abs() + a * (BF + 2 * delta + n * F32)[:, None] * (1 + BF)
                w += p.sum(0)
                bw += (p.nan_to_num(0.0) * (2 * delta.nan_to_num(0.0) + F32 * (n + 8))[:, None]).sum(0)  # NaN weights have no bound
            got.append((w, bw + w * F32 * (r * hq + 4)))
            at += r
        return out, lse, b_out, b_lse, got

    def evict(self, table, lens, new_table, keep, recent, sink):
        kept, news = [], []
        for b in range(table.shape[0]):
            n = min(max(int(lens[b]), 0), table.shape[1] * self.page)
            t = torch.arange(n)
            page, slot = self.where(table, b, t)
            w = torch.where(page >= 0, self.weights[page.clamp(min=0), slot].double(), -math.inf)
            w = torch.where(torch.isnan(w), math.inf, w).tolist()
            nan = torch.isnan(self.weights[page.clamp(min=0), slot]).tolist()
            if n <= keep:
                mine = list(range(n))
            else:
                rest = sorted(range(sink, n - recent), key=lambda i: (not (nan[i] and page[i] >= 0), -w[i], i))
                mine = sorted(list(range(sink)) + rest[:keep - sink - recent] + list(range(n - recent, n)))
            kept.append(mine + [-1] * (keep - len(mine)))
            news.append(len(mine))
            own = torch.tensor(mine, dtype=torch.long)
            page, slot = page[own], slot[own]
            x = [self.value(i, page, slot) for i in (0, 1)]
            for c in range(-(-len(mine) // self.page)):
                part = slice(c * self.page, min((c + 1) * self.page, len(mine)))
                to = int(new_table[b, c])
                if not 0 <= to < self.pages:
                    continue
                for i in (0, 1):
                    self._write(i, to, 0, x[i][part])
                m = part.stop - part.start
                got = self.weights[page[part].clamp(min=0), slot[part]]
                self.weights[to, :m] = torch.where(page[part] >= 0, got, torch.zeros(()))
        return torch.tensor(news, dtype=torch.int32), torch.tensor(kept, dtype=torch.int32)
