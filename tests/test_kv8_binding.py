"""What the KV cache's binding asks of its arguments beyond their shapes (CPU)."""

import pytest
import torch

import nvfp4_weight_dense_amd as nv


@pytest.mark.parametrize("current,tensors", [(0, 1), (1, 0), (3, 2)])
def test_another_current_device_is_refused(monkeypatch, current, tensors):
    """The library's scratch and its launches are the current device's."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    with pytest.raises(ValueError, match=f"cuda:{tensors}.*cuda:{current}"):
        nv._kv8_on(tensors)
    nv._kv8_on(current)
