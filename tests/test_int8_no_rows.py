"""A batch without rows takes a gate for each of its rows (CPU: past the shapes, these tensors are on no GPU)."""

import pytest
import torch

import nvfp4_weight_dense_amd as nv

BF = torch.bfloat16


def test_a_gate_for_each_of_no_rows():
    nv.load_library()
    x = torch.zeros(0, 64, dtype=BF)
    for gate in (torch.zeros(0, 64, dtype=BF), torch.zeros(64, dtype=BF), torch.zeros(3, 64, dtype=BF)):
        with pytest.raises(ValueError, match="GPU"):
            nv.rms_norm_residual(x, x, gate=gate, norm=True)
    with pytest.raises(ValueError, match="divide"):
        nv.rms_norm_residual(torch.zeros(2, 64, dtype=BF), torch.zeros(2, 64, dtype=BF), gate=torch.zeros(0, 64, dtype=BF))


@pytest.mark.gpu
def test_no_rows_come_back():
    print("no rows", flush=True)
    x = torch.zeros(0, 64, dtype=BF, device="cuda")
    h, n = nv.rms_norm_residual(x, x, gate=x, norm=True)
    assert h.shape == n.shape == (0, 64)
