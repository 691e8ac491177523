"""One decoder layer with NVFP4 weights, generating over the 8-bit KV cache.

    python examples/decode_layer.py [--steps N] [--budget TOKENS]

A batch of prompts of different lengths is run through the layer, then one
token per sequence and step.  Each call of the layer is

    x += Wo . attention(q, cache)      [q k v] = Wqkv . norm(x); k, v appended
    x += FFN(norm(x))

with nvfp4_gemm_w4a16 for the projections, kv8_append and kv8_attention for
the cache, and dense_ffn_forward for the FFN.  kv8_attention also keeps the
attention weight that each token has received; a sequence that reaches the
budget is cut by kv8_evict to its first, its last and its most attended
tokens, and its old pages are free again.  Weights are random, position
encodings are left out, and the layer's output stands in for the next token's
embedding.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import nvfp4_weight_dense_amd as nv  # noqa: E402


def _weight(n: int, k: int, g: torch.Generator) -> nv.NVFP4Weight:
    """Random codes and block scales of 1; the tensor scale keeps a product near its input's size."""
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = torch.full((n, k // 16), 0x38, dtype=torch.uint8)  # 1.0
    return nv.NVFP4Weight(codes.cuda(), scales.cuda(), 0.35 * k ** -0.5)


def _norm(x: torch.Tensor) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Layer:
    def __init__(self, hidden=1024, inter=2816, q_heads=8, kv_heads=2, dim=128, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        self.wqkv = _weight((q_heads + 2 * kv_heads) * dim, hidden, g)
        self.wo = _weight(hidden, q_heads * dim, g)
        self.wg, self.wu = _weight(inter, hidden, g), _weight(inter, hidden, g)
        self.wd = _weight(hidden, inter, g)

    def __call__(self, x, cache, table, lens, starts=None, max_rows=None, max_len=None, workspace=None):
        qkv = nv.nvfp4_gemm_w4a16(_norm(x), self.wqkv).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split((self.q_heads, self.kv_heads, self.kv_heads), 1)
        nv.kv8_append(k, v, cache, table, lens, starts, max_rows=max_rows)
        a = nv.kv8_attention(q, cache, table, lens, starts, max_rows=max_rows, max_len=max_len,
                             accumulate=cache.weights is not None, workspace=workspace)
        self.last = q, a
        x = x + nv.nvfp4_gemm_w4a16(a.view(x.shape[0], -1), self.wo)
        return x + nv.dense_ffn_forward(_norm(x), self.wg, self.wu, self.wd)


class Pages:
    """The pool's free pages, and a table of each sequence's own."""

    def __init__(self, pages: int, seqs: int, cols: int, page: int):
        self.page, self.free = page, list(range(pages))
        self.own = [[] for _ in range(seqs)]
        self.host = torch.full((seqs, cols), -1, dtype=torch.int32)

    def take(self, tokens: int) -> list:
        n = -(-tokens // self.page)
        if n > len(self.free):
            raise MemoryError(f"{n} pages wanted, {len(self.free)} free")
        return [self.free.pop() for _ in range(n)]

    def grow(self, lens) -> torch.Tensor:
        """The table, with pages for lens tokens of each sequence."""
        for b, n in enumerate(lens):
            self.own[b] += self.take(max(n - len(self.own[b]) * self.page, 0))
            self.host[b, :len(self.own[b])] = torch.tensor(self.own[b], dtype=torch.int32)
        return self.host.cuda()

    def swap(self, b: int, new: list) -> None:
        self.free += self.own[b]
        self.own[b] = new
        self.host[b] = -1
        self.host[b, :len(new)] = torch.tensor(new, dtype=torch.int32)


def generate(layer: Layer, prompts, steps: int, budget: int, page: int = 64, sink: int = 4, recent: int = 64):
    """Runs the prompts (bf16 [tokens, hidden] each) and `steps` tokens more of each sequence; a sequence that has
    `budget` tokens is cut to half of them.  Returns the last outputs, the cache, its pages, the table and the
    lengths (as Python and as device integers)."""
    seqs, keep = len(prompts), budget // 2
    if keep < sink + recent:
        raise ValueError(f"half of a budget of {budget} tokens is below sink + recent = {sink + recent}")
    lens = [len(p) for p in prompts]
    top = max(budget, max(lens) + 1)
    cols = -(-top // page)
    pages = Pages((seqs + 1) * cols, seqs, cols, page)
    cache = nv.kv8_cache((seqs + 1) * cols, layer.kv_heads, layer.dim, page, weights=True)

    # the prompts, of unequal lengths, in one call
    starts = torch.tensor([sum(lens[:b]) for b in range(seqs + 1)], dtype=torch.int32, device="cuda")
    table, n = pages.grow(lens), torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = layer(torch.cat(prompts), cache, table, n, starts, max_rows=max(lens), max_len=top)
    x = x[starts[1:].long() - 1]

    workspace = nv.kv8_workspace(layer.q_heads, cache, table, n, seqs, max_len=top)
    for _ in range(steps):
        for b in range(seqs):
            if lens[b] < budget:
                continue
            new = pages.take(keep)
            cut, kept = nv.kv8_evict(cache, table[b:b + 1], n[b:b + 1],
                                     torch.tensor([new], dtype=torch.int32, device="cuda"), keep,
                                     recent=recent, sink=sink)
            n[b:b + 1] = cut
            pages.swap(b, new)
            lens[b] = keep
        lens = [m + 1 for m in lens]
        n += 1
        table = pages.grow(lens)
        x = layer(_norm(x), cache, table, n, max_len=top, workspace=workspace)
    return x, cache, pages, table, lens, n


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--budget", type=int, default=512)
    args = ap.parse_args()
    layer = Layer()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randn(n, 1024, generator=g).bfloat16().cuda() for n in (500, 37, 256, 1)]
    x, cache, pages, _, lens, _ = generate(layer, prompts, args.steps, args.budget)
    torch.cuda.synchronize()
    size = sum(t.numel() * t.element_size() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales))
    print(f"{len(prompts)} sequences, prompts of {[len(p) for p in prompts]} tokens, {args.steps} steps: "
          f"{lens} tokens kept, {len(pages.free)} pages free, pool of {size / 1e6:.1f} MB; "
          f"output rms {x.float().square().mean().sqrt().item():.3f}", flush=True)


if __name__ == "__main__":
    main()
