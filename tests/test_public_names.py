"""The 8-bit operators' binding asks torch by its public names."""
import inspect

import torch

import top_routing_expert_moe_gb300 as moe


def test_the_current_device_by_its_public_name(monkeypatch):
    assert moe.mx8._current_device is torch.cuda.current_device
    assert "torch._C" not in inspect.getsource(moe.mx8)
