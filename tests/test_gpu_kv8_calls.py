"""Calls of the 8-bit paged KV cache as programs make them, on the GPU against the 64-bit reference: their own
workspaces, and what test_gpu_kv8.py's cases of one kernel each do not combine."""

import math

import pytest
import torch

import kv8_ref as ref
import nvfp4_weight_dense_amd as nv
from test_gpu_kv8 import _gpu, _i32, _problem, _say, _table, _within

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
