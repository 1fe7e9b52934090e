"""The binding's own helpers."""
from types import SimpleNamespace

import torch

import top_routing_expert_moe_gb300 as moe


def test_the_current_stream_without_torchs_private_names(monkeypatch):
    """The quick look-up uses names that torch does not promise; without them its public
    call serves."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=4711))
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        with monkeypatch.context() as m:
            m.delattr(torch._C, name, raising=False)
            assert moe._s(None) == 4711
    assert moe._s(SimpleNamespace(cuda_stream=7)) == 7
