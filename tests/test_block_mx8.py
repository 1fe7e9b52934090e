"""Norm, routing, dispatch, both products and the combine in 8 bits, together as a server
runs them, and the checkpointed layer beside them."""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests.test_block import EPS, weights
from tests.test_mx8 import quantize64


def test_refusals():
    cfg = moe.MoEConfig(T=8, d=128, f=128, E=2, k=1)
    layer = moe.MoELayer(cfg, "cpu")
    x = torch.zeros(8, 128, dtype=torch.bfloat16)

    class Experts:
        def __init__(self, up, down, gate=None):
            self.up, self.down, self.gate = (moe.MX8Weight(s, "cpu") if s else None for s in (up, down, gate))

    with pytest.raises(ValueError, match="gate matrix"):
        layer.forward_mx8(x, x, Experts((2, 128, 128), (2, 128, 128), (2, 128, 128)))
    with pytest.raises(ValueError, match="shapes"):
        layer.forward_mx8(x, x, Experts((1, 128, 128), (2, 128, 128)))
    for bad in (moe.MoEConfig(T=8, d=128, f=128, E=2, k=1, dtype=moe.F32),
                moe.MoEConfig(T=8, d=128, f=128, E=2, k=1, f_shared=128)):
        with pytest.raises(ValueError, match="bf16 layer"):
            moe.MoELayer(bad, "cpu").forward_mx8(x, x, Experts((2, 128, 128), (2, 128, 128)))


@pytest.mark.gpu
@pytest.mark.parametrize("T,swiglu,cf", [(1, True, 0.0), (3, False, 0.0), (300, True, 0.0), (700, True, 0.8), (1100, False, 0.0)])
def test_experts_in_eight_bits(T, swiglu, cf):
    """The block with 8-bit experts against the same steps in 64 bits on the values that its
    8-bit numbers stand for (the layer's bf16 parity bound)."""
    d, f, E, k = 256, 384, 5, 2
    x, w, _ = weights(T, d, f, E, torch.bfloat16, swiglu, moe.GATE_NONE, seed=T)
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU if swiglu else moe.SILU, capacity_factor=cf)
    b = moe.MoEBlock(cfg, post_norm=1, eps=EPS)
    wc = {n: t.cuda() for n, t in w.items()}
    mask = (torch.arange(T) % 5 != 2).to(torch.uint8) if T == 1100 else None
    ex = moe.MX8Experts(wc["W_up"], wc["W_down"], wc.get("W_gate"))
    x_out = b.forward_mx8(x.cuda(), wc, ex, token_mask=None if mask is None else mask.cuda()).cpu()
    assert moe.last_device_status() == 0
    L = b.layer
    zq = b.enter.z8.dequantize(torch.float32).cpu().double()
    slot, gate, topk = L._mx8[0].slot_of.cpu(), L.gate.cpu().double(), L.topk_idx.cpu()
    q = lambda W: torch.stack([quantize64(W[e].t())[1].t() for e in range(E)])  # noqa: E731
    Wu, Wd, Wg = q(w["W_up"]), q(w["W_down"]), q(w["W_gate"]) if swiglu else None
    u, dropped = torch.zeros(T, d).double(), 0
    for e in range(E):
        t, j = torch.nonzero((topk == e) & (slot >= 0), as_tuple=True)
        dropped += int(((topk == e) & (slot < 0)).sum())
        if not len(t):
            continue
        h = zq[t] @ Wu[e]
        g = zq[t] @ Wg[e] if swiglu else h
        a = quantize64(g / (1 + torch.exp(-g)) * (h if swiglu else 1))[1]
        u.index_add_(0, t, gate[t, j][:, None] * (a @ Wd[e]))
    assert L.stats[moe.STAT_DROPPED] == dropped and (cf == 0) == (dropped == 0)
    got = L.out.cpu().double()
    assert ((got - u).norm() / u.norm()).item() <= 2e-2
    if mask is not None:
        assert (got[mask == 0] == 0).all()
    want = x.double() + got / torch.sqrt((got * got).mean(-1, keepdim=True) + EPS) * w["w_out"].double()
    assert ((x_out.double() - want).norm() / want.norm()).item() <= 2e-2
    # rows quantised by the layer itself: the same but for z's rounding to 16 bits
    out = L.out.clone()
    again = L.forward_mx8(b.enter.z, wc["W_r"], ex, wc["bias"], token_mask=None if mask is None else mask.cuda())
    assert ((again.double() - out.double()).norm() / out.double().norm()).item() <= 2.0 ** -3
    with pytest.raises(RuntimeError, match="forward"):
        L.backward(x.cuda())


@pytest.mark.gpu
def test_block_in_a_graph_repeats_the_eager_pass():
    """Decoding: the same captured pass for new tokens, which go to other experts."""
    T, d, f, E, k = 2, 256, 512, 8, 2
    x, w, _ = weights(T, d, f, E, torch.bfloat16, True, moe.GATE_CHANNEL)
    b = moe.MoEBlock(moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU), post_norm=1, gate=moe.GATE_CHANNEL)
    wc, xc = {n: t.cuda() for n, t in w.items()}, x.cuda()
    ex = moe.MX8Experts(wc["W_up"], wc["W_down"], wc["W_gate"])
    b.forward_mx8(xc, wc, ex)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = b.forward_mx8(xc, wc, ex)
    seen = set()
    for seed in range(6):
        xc.copy_(torch.randn(T, d, generator=torch.Generator().manual_seed(seed)).to(xc))
        graph.replay()
        out = got.clone()
        seen.add(tuple(b.layer.topk_idx.flatten().tolist()))
        assert torch.equal(out, b.forward_mx8(xc, wc, ex))
    assert len(seen) > 1 and moe.last_device_status() == 0
