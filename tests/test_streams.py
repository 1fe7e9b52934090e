"""Memory of calls that are given a stream.  The allocator orders reuse of a block by
the stream it was taken under, so what a call allocates for work on a given stream is
taken under that stream: under another, the block may still be in use by queued work
there, and it goes back there while the given stream still reads it.

On the CPU the binding is followed without its launches; on the GPU the allocator is
asked which stream a result's segment belongs to.
"""
import contextlib

import pytest
import torch

import top_routing_expert_moe_gb300 as moe

STREAM = object()


@pytest.fixture
def follow(monkeypatch):
    """List of (stream that an allocation was made under, its bytes)."""
    under, made, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        under.append(s)
        try:
            yield
        finally:
            under.pop()

    def recorded(*a, **kw):
        t = empty(*a, **kw)
        made.append((under[-1], t.numel() * t.element_size()))
        return t

    for m in (moe, moe.block):
        monkeypatch.setattr(m, "_p", lambda t: t if t is None else t.data_ptr())
        monkeypatch.setattr(m, "_s", lambda s: 0)
        monkeypatch.setattr(m, "_call", lambda *a: None)
    monkeypatch.setattr(moe.block, "norm_workspace_size", lambda c: 4096)
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    return made


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def cases():
    def quantize(s):
        moe.mx4_quantize(bf(4, 64), stream=s)

    def dequantize(s):
        q = moe.MX4Tensor((4, 64), "cpu")
        return lambda: q.dequantize(stream=s)

    def weight(s):
        moe.mx4_quantize_weight(bf(2, 64, 8), stream=s)

    def experts(s):
        moe.MX4Experts(bf(2, 64, 32), bf(2, 32, 64), bf(2, 64, 32), stream=s)

    def norm_grads(s):
        n = moe.BlockNorm(moe.NormConfig(T=4, d=64), "cpu")
        return lambda: n.backward(bf(4, 64), dx_out=bf(4, 64), dz=bf(4, 64), w_pre=torch.ones(64), stream=s)

    def layer_mx4(s):
        L = moe.MoELayer(moe.MoEConfig(T=8, d=128, f=128, E=2, k=1), "cpu")
        e = moe.MX4Experts(bf(2, 128, 128), bf(2, 128, 128))
        return lambda: L.forward_mx4(bf(8, 128), bf(128, 2), e, stream=s)

    def layer_grads(s):
        L = moe.MoELayer(moe.MoEConfig(T=8, d=128, f=128, E=2, k=1), "cpu")
        L.forward(bf(8, 128), bf(128, 2), bf(2, 128, 128), bf(2, 128, 128))
        return lambda: L.backward(bf(8, 128), stream=s)

    def block(s):
        b = moe.MoEBlock(moe.MoEConfig(T=8, d=128, f=128, E=2, k=1), device="cpu")
        w = dict(w_in=torch.ones(128), W_r=bf(128, 2), W_up=bf(2, 128, 128), W_down=bf(2, 128, 128))

        def go():
            b.forward(bf(8, 128), w, stream=s)
            b.backward(bf(8, 128), stream=s)
        return go
    return [quantize, dequantize, weight, experts, norm_grads, layer_mx4, layer_grads, block]


@pytest.mark.parametrize("case", cases(), ids=lambda c: c.__name__)
def test_what_a_call_allocates_is_the_given_streams(case, follow):
    for s in (STREAM, None):
        follow.clear()
        rest = case(s)
        if rest is not None:                   # set up first, then the call that is looked at
            follow.clear()
            rest()
        assert follow, "nothing was allocated"
        assert all(u is s for u, _ in follow), follow


@pytest.mark.gpu
def test_the_allocators_stream():
    s = torch.cuda.Stream()
    x = torch.randn(300, 256, device="cuda").bfloat16()
    W = torch.randn(2, 256, 64, device="cuda").bfloat16()
    want, want_w = moe.mx4_quantize(x).dequantize(), moe.mx4_quantize_weight(W).dequantize()
    s.wait_stream(torch.cuda.current_stream())
    q, w = moe.mx4_quantize(x, stream=s), moe.mx4_quantize_weight(W, stream=s)
    a, b = q.dequantize(stream=s), w.dequantize(stream=s)
    n = moe.BlockNorm(moe.NormConfig(T=300, d=256, leave=0))
    s.wait_stream(torch.cuda.current_stream())
    g = n.backward(x, dz=x, w_pre=torch.ones(256, device="cuda"), stream=s)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want_w)
    segments = [(e["address"], e["address"] + e["total_size"], e["stream"]) for e in torch.cuda.memory_snapshot()]
    for t in (q.codes, q.scales, w.codes, w.scales, a, b, g["dx"], g["dw_pre"]):
        (owner,) = [st for lo, hi, st in segments if lo <= t.data_ptr() < hi]
        assert owner == s.cuda_stream
    del q, w, a, b                             # to the stream's own pool
    assert moe.last_device_status() == 0
