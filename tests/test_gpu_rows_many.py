"""Many rows through the int8 quantizer: each of its widths of a wave's row, and where rows go to waves or to workgroups,
against the same rows in small batches (whose own tests hold them to the definition), on the GPU."""

import pytest
import torch

import nvfp4_weight_dense_amd as nv

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _same(got, want):
    return torch.equal(got.codes, want.codes) and torch.equal(got.row_scale.view(torch.int32), want.row_scale.view(torch.int32))


@pytest.mark.parametrize("m,k", [(2047, 2048), (2048, 2048), (2048, 2056), (2051, 1024), (4099, 1032), (16383, 5120), (16384, 2056),
                                 *((16385, 512 * p + d) for p in range(2, 13) for d in (-8, 0, 8))])
def test_rows_in_any_number(m, k):
    print("quantize", m, k, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + k)
    x = torch.randn(m, k, generator=g, device="cuda").to(BF)
    x[:: 97] *= torch.tensor(2.0 ** 40, dtype=BF, device="cuda")
    x[5], x[m - 2, k - 1] = 0.0, float("inf")
    got = nv.int8_quantize_rows(x)
    for r in range(0, m, 1023):
        assert _same(nv.Int8Rows(got.codes[r:r + 1023], got.row_scale[r:r + 1023]), nv.int8_quantize_rows(x[r:r + 1023])), r
    assert bool(got.row_scale[m - 2].isnan()) and float(got.row_scale[5]) == 1.0 and int(got.row_scale.isnan().sum()) == 1
