"""The 64-bit reference of the KV cache against hand-worked values and torch's own casts (CPU)."""

import math

import torch

import kv8_ref as ref
import nvfp4_weight_dense_amd as nv


def _cache(pages=4, heads=1, dim=64, page=16, weights=True):
    return nv.kv8_cache(pages, heads, dim, page, weights=weights, device="cpu")


def test_encode_is_torchs_cast_and_keeps_nan():
    x = torch.randn(4096, dtype=torch.float64).float() * torch.exp(3 * torch.randn(4096))
    x = torch.cat([x.clamp(-448, 448), torch.tensor([0.0, -0.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 448.0])])
    assert torch.equal(ref.encode(x.double()), x.to(torch.float8_e4m3fn).view(torch.uint8))
    assert ref.encode(torch.tensor([math.inf, -math.inf, 1e9, math.nan], dtype=torch.float64)).tolist() == \
        [0x7E, 0xFE, 0x7E, 0x7F]


def test_exponent_is_the_smallest_that_holds():
    assert [ref.exponent(a) for a in (448.0, 448.5, 224.0, 1.75, 0.0, 3e38)] == [0, 1, -1, -8, -117, 119]


def test_layouts_are_permutations_and_the_documented_ones():
    for dim in (64, 128, 256):
        for page in (16, 64):
            for isv in (0, 1):
                o = ref.order(page, dim, isv).reshape(-1)
                assert torch.equal(o.sort().values, torch.arange(page * dim))
    # V, dim 128, token 4*2+3 of unit 1, channel 64*1 + 16*2 + 5
    assert int(ref.v_at(16 + 11, 101, 128)) == 2048 + 1024 + 2 * 256 + 5 * 16 + 2 * 4 + 3
    assert int(ref.k_at(16 + 11, 101, 128)) == 2048 + 6 * 256 + 11 * 16 + 5


def test_a_rising_scale_moves_whole_exponents():
    c = ref.Pool(_cache())
    table, one = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, 1, 64)
    c.append(one, one, table, torch.tensor([1]), [1])
    assert int(c.scales[0][0, 0]) == 127 - 8        # 1 <= 448 * 2^-8 = 1.75
    c.append(100 * one, one, table, torch.tensor([2]), [1])
    assert int(c.scales[0][0, 0]) == 127 - 2
    # 100 / 2^-2 = 400, halfway between 384 (the even code) and 416
    assert c.value(0, torch.tensor([0, 0]), torch.tensor([0, 1]))[:, 0, 0].tolist() == [1.0, 96.0]


def test_attention_of_two_tokens_by_hand():
    c = ref.Pool(_cache())
    k, v = torch.zeros(2, 1, 64), torch.zeros(2, 1, 64)
    k[1, 0, 0], v[0, 0, 3], v[1, 0, 3] = 1.0, 1.0, 3.0
    table = torch.zeros(1, 1, dtype=torch.int32)
    c.append(k, v, table, torch.tensor([2]), [2])
    q = torch.zeros(2, 1, 64)
    q[:, 0, 0] = math.log(3.0)
    out, lse, *_, w = c.attention(q, table, torch.tensor([2]), [2], 1.0)
    assert float(out[0, 0, 3]) == 1.0 and abs(float(out[1, 0, 3]) - 2.5) < 1e-7
    assert float(lse[0, 0]) == 0.0 and abs(float(lse[1, 0]) - math.log(4.0)) < 1e-7
    assert torch.allclose(w[0][0], torch.tensor([1.25, 0.75], dtype=torch.float64), atol=1e-7)
    out, lse, *_ = c.attention(q, table, torch.tensor([1]), [2], 1.0)   # the first row is before the sequence
    assert float(lse[0, 0]) == -math.inf and not out[0].any()


def test_evict_keeps_the_ends_and_the_largest_first_of_equals():
    c = ref.Pool(_cache())
    c.weights[0, :10] = torch.tensor([0.0, 5, 1, 1, 1, 9, 1, 0, 0, 0])
    news, kept = c.evict(torch.zeros(1, 1, dtype=torch.int32), torch.tensor([10]), torch.tensor([[1]]), 6, 2, 1)
    assert news.tolist() == [6] and kept.tolist() == [[0, 1, 2, 5, 8, 9]]
