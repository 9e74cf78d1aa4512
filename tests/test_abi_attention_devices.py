"""The attention layers' calls take tensors of one device (checked on devices that need no
GPU: the binding's own comparison)."""
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import _lib
from gated_deltanet_linear_recurrence_gb300.build import build


def test_tensors_of_one_device():
    build()
    one_device = _lib.binding().one_device
    cpu, meta = torch.zeros(3), torch.zeros(3, device="meta")
    assert one_device(cpu, cpu) is None and one_device(meta, torch.zeros(5, device="meta")) is None
    with pytest.raises(ValueError):
        one_device(cpu, meta)
    with pytest.raises(ValueError):
        one_device(meta, cpu)
    with pytest.raises(TypeError):
        one_device(cpu, 3)
