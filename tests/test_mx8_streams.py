"""The 8-bit operators where a call leaves the beaten track: streams that are given, memory off the
current device, and first calls that a graph captures."""
import subprocess
import sys

import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests.test_streams import STREAM, bf, follow  # noqa: F401  (the fixture)


@pytest.fixture
def follow8(follow, monkeypatch):  # noqa: F811
    for name, f in (("_p", lambda t: t if t is None else t.data_ptr()), ("_s", lambda s: 0), ("_call", lambda *a: None)):
        monkeypatch.setattr(moe.mx8, name, f)
    monkeypatch.setattr(moe.mx8._Numbers, "ptrs", property(lambda self: (0, 0)))
    monkeypatch.setattr(moe.mx8, "mx8_weight_bytes", lambda E, K, N: (16384, 512))
    monkeypatch.setattr(moe.mx8, "mx8_rows_capacity", lambda c: 16)
    monkeypatch.setattr(moe, "mx8_rows_capacity", lambda c: 16)
    monkeypatch.setattr(moe, "rows_capacity", lambda c: 16)
    monkeypatch.setattr(moe.mx8, "permute_mx8_workspace_size", lambda c: 4096)
    return follow


def cases():
    def quantize(s):
        moe.mx8_quantize(bf(4, 64), stream=s)

    def values(s):
        q = moe.MX8Tensor((4, 64), "cpu")
        return lambda: q.dequantize(stream=s)

    def weight(s):
        moe.mx8_quantize_weight(bf(2, 64, 8), stream=s)

    def weight_values(s):
        q = moe.MX8Weight((2, 8, 64), "cpu")
        return lambda: q.dequantize(stream=s)

    def experts(s):
        moe.MX8Experts(bf(2, 64, 32), bf(2, 32, 64), bf(2, 64, 32), stream=s)

    def norm(s):
        n = moe.BlockNorm(moe.NormConfig(T=4, d=64, leave=0), "cpu")
        return lambda: n.forward_mx8(bf(4, 64), w_pre=torch.ones(64), stream=s)

    def layer(s):
        L = moe.MoELayer(moe.MoEConfig(T=8, d=128, f=128, E=2, k=1), "cpu")
        ex = moe.MX8Experts(bf(2, 128, 128), bf(2, 128, 128))
        return lambda: L.forward_mx8(bf(8, 128), bf(128, 2), ex, stream=s)

    def checkpointed(s):
        cfg = moe.MoEConfig(T=8, d=128, f=128, E=2, k=1)
        L, ck, W = moe.MoELayer(cfg, "cpu"), moe.MoECheckpoint(cfg, "cpu"), bf(2, 128, 128)
        L.forward(bf(8, 128), bf(128, 2), W, W, stream=s, checkpoint=ck)
        return lambda: L.backward(bf(8, 128), stream=s, checkpoint=ck)

    return {f.__name__: f for f in (quantize, values, weight, weight_values, experts, norm, layer, checkpointed)}


@pytest.mark.parametrize("name", list(cases()))
def test_memory_belongs_to_the_given_stream(follow8, name):
    call = cases()[name](STREAM)
    if call is not None:
        follow8.clear()
        call()
    assert follow8 and all(s is STREAM for s, _ in follow8), follow8


def test_numbers_off_the_current_device_are_refused(monkeypatch):
    q = moe.MX8Tensor((4, 64), "cpu")
    with pytest.raises(ValueError, match="must live on the GPU"):
        q.ptrs
    q._ptrs, q._device = (0x10000, 0x20000), torch.device("cuda", 1)
    monkeypatch.setattr(moe.mx8, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="not the current device"):
        q.dequantize()
    monkeypatch.setattr(moe.mx8, "_current_device", lambda: 1)
    assert q.ptrs == (0x10000, 0x20000)


FIRST = """
import torch
import top_routing_expert_moe_gb300 as moe
x = torch.randn(300, 256, device="cuda").bfloat16()
cfg = moe.MoEConfig(T=300, d=256, f=256, E=4, k=2, ffn=moe.SWIGLU)
W = [torch.randn(s, device="cuda").bfloat16() * 0.05 for s in ((4, 256, 256), (4, 256, 256), (4, 256, 256), (256, 4))]
b, ck = moe.MoEBlock(cfg), moe.MoECheckpoint(cfg)
w = dict(w_in=torch.ones(256, device="cuda"), W_r=W[3], W_up=W[0], W_down=W[1], W_gate=W[2])
moe.load_library()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
def go():
    ex = moe.MX8Experts(W[0], W[1], W[2])
    a = b.forward_mx8(x, w, ex).clone()
    c = b.layer.forward(x, W[3], W[0], W[1], W[2], checkpoint=ck).clone()
    return [a, c] + [t.clone() for t in b.layer.backward(x, checkpoint=ck).values() if t is not None]
with torch.cuda.graph(g):
    got = go()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, c) for a, c in zip(got, go())) and moe.last_device_status() == 0
print("same")
"""


@pytest.mark.gpu
def test_a_first_call_under_capture():
    """Nothing of a process' first call needs to happen outside of a graph."""
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.gpu
def test_two_graphs_of_one_block_in_turn():
    """Graphs that share a block's buffers, replayed one after the other."""
    cfg = moe.MoEConfig(T=40, d=128, f=256, E=4, k=2)
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    b = moe.MoEBlock(cfg, post_norm=1)
    Wu, Wd = r(4, 128, 256).bfloat16() / 12, r(4, 256, 128).bfloat16() / 16
    w = dict(w_in=torch.ones(128, device="cuda"), w_out=torch.ones(128, device="cuda"), W_r=r(128, 4).bfloat16())
    ex, xs = moe.MX8Experts(Wu, Wd), [r(40, 128).bfloat16() for _ in range(2)]
    want = [b.forward_mx8(x, w, ex).clone() for x in xs]
    graphs, outs = [], []
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(b.forward_mx8(x, w, ex).clone())
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])
