"""The layer in its place on the residual stream: norms, experts, balance loss and
their gradients together, and the same block with its experts in 4 bits."""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests.test_mx4 import quantize64

pytestmark = pytest.mark.gpu
EPS, RA, OB, BC, ZC = 1e-6, 0.9, 0.7, 3.0, 0.2


def weights(T, d, f, E, dt, swiglu, gate, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean  # noqa: E731
    w = dict(w_in=r(d, std=0.1, mean=1), w_out=r(d, std=0.1, mean=1), W_r=r(d, E, std=0.2).to(dt),
             W_up=r(E, d, f, std=d ** -0.5).to(dt), W_down=r(E, f, d, std=f ** -0.5).to(dt),
             bias=r(E, std=0.1))
    if swiglu:
        w["W_gate"] = r(E, d, f, std=d ** -0.5).to(dt)
    if gate == moe.GATE_CHANNEL:
        w["gate"] = r(d, std=0.3, mean=0.5)
    elif gate == moe.GATE_TOKEN:
        w["gate"] = r(T, std=0.3, mean=0.5)
    return r(T, d).to(dt), w, r(T, d).to(dt)


def block64(x, w, topk, offs, k, swiglu, gate):
    """x' and the losses by the definitions in 64 bits, with the routing given."""
    def unit(v):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    T, E = x.shape[0], w["W_r"].shape[1]
    z = unit(x) * w["w_in"]
    logits = z @ w["W_r"] + w["bias"]
    gates = torch.softmax(logits.gather(1, topk), 1)
    u = torch.zeros_like(x)
    for e in range(E):
        h = z @ w["W_up"][e]
        if swiglu:
            gt = z @ w["W_gate"][e]
            a = gt / (1 + torch.exp(-gt)) * h
        else:
            a = h / (1 + torch.exp(-h))
        u = u + (gates * (topk == e)).sum(1, keepdim=True) * (a @ w["W_down"][e])
    n = unit(u) * w["w_out"]
    if gate != moe.GATE_NONE:
        n = n * (w["gate"][:, None] if gate == moe.GATE_TOKEN else w["gate"])
    p, lse = torch.softmax(logits, 1), torch.logsumexp(logits, 1)
    bal = 0.0
    for s in range(len(offs) - 1):
        lo, hi = offs[s], offs[s + 1]
        c = torch.bincount(topk[lo:hi].reshape(-1), minlength=E).double()
        bal = bal + (E * c / (k * (hi - lo)) * p[lo:hi].mean(0)).sum() / (len(offs) - 1)
    return RA * x + OB * n, BC * bal, ZC * (lse ** 2).mean()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("swiglu,gate", [(False, moe.GATE_NONE), (True, moe.GATE_CHANNEL),
                                         (True, moe.GATE_TOKEN)])
def test_block_forward_and_backward(dt, swiglu, gate):
    T, d, f, E, k = 200, 128, 256, 4, 2
    x, w, dout = weights(T, d, f, E, dt, swiglu, gate)
    offs = [0, 90, 200]
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU if swiglu else moe.SILU,
                        dtype=moe.F32 if dt == torch.float32 else moe.BF16)
    b = moe.MoEBlock(cfg, post_norm=1, gate=gate, eps=EPS, res_scale=RA, out_scale=OB, sequences=2,
                     balance_coef=BC, z_coef=ZC)
    wc = {n: t.cuda() for n, t in w.items()}
    o = torch.tensor(offs, dtype=torch.int32).cuda()
    x_out, loss = b.forward(x.cuda(), wc, o)
    g = b.backward(dout.cuda(), dloss=torch.full((1,), 2.0, device="cuda"))
    assert moe.last_device_status() == 0
    topk = b.layer.topk_idx.cpu().long()
    x64 = x.double().requires_grad_()
    w64 = {n: t.double().requires_grad_() for n, t in w.items()}
    want, bal, zl = block64(x64, w64, topk, offs, k, swiglu, gate)
    grads = torch.autograd.grad((want * dout.double()).sum() + 2 * (bal + zl), [x64] + list(w64.values()))
    # the layer's parity bounds (its tests derive them); the losses see bf16 z and W_r
    tol = 2e-5 if dt == torch.float32 else 2e-2
    rel = lambda a, t: ((a.double().cpu() - t).norm() / t.norm()).item()  # noqa: E731
    assert rel(x_out, want.detach()) <= tol
    assert rel(loss, torch.stack([bal + zl, bal, zl]).detach()) <= tol
    for n, t in zip(["dx"] + ["d" + n for n in w64], grads):
        assert rel(g[n], t) <= tol, (n, rel(g[n], t))
    with pytest.raises(RuntimeError, match="forward"):
        moe.MoEBlock(cfg).backward(dout.cuda())


def test_block_in_a_graph_repeats_the_eager_pass():
    T, d, f, E, k = 512, 256, 256, 8, 2
    x, w, dout = weights(T, d, f, E, torch.bfloat16, True, moe.GATE_CHANNEL)
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU)
    b = moe.MoEBlock(cfg, post_norm=1, gate=moe.GATE_CHANNEL)
    wc, xc, dc = {n: t.cuda() for n, t in w.items()}, x.cuda(), dout.cuda()

    def go():
        x_out, loss = b.forward(xc, wc)
        return {"x_out": x_out, "loss": loss, **b.backward(dc)}

    want = {n: t.clone() for n, t in go().items() if t is not None}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = go()
    for t in got.values():
        if t is not None:
            t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for n, t in want.items():
        assert torch.equal(t, got[n]), n


@pytest.mark.parametrize("T,swiglu,cf", [(1, True, 0.0), (3, False, 0.0), (300, True, 0.0), (700, True, 0.8)])
def test_experts_in_four_bits(T, swiglu, cf):
    """The layer with 4-bit experts against the same steps in 64 bits on the values its
    4-bit numbers stand for (the layer's bf16 parity bound)."""
    d, f, E, k = 256, 384, 5, 2
    x, w, _ = weights(T, d, f, E, torch.bfloat16, swiglu, moe.GATE_NONE, seed=T)
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU if swiglu else moe.SILU, capacity_factor=cf)
    b = moe.MoEBlock(cfg, post_norm=1, eps=EPS)
    wc = {n: t.cuda() for n, t in w.items()}
    ex = moe.MX4Experts(wc["W_up"], wc["W_down"], wc.get("W_gate"))
    x_out = b.forward_mx4(x.cuda(), wc, ex).cpu()
    assert moe.last_device_status() == 0
    L = b.layer
    z = b.enter.z.cpu()
    slot, gate, topk = L.slot_of.cpu(), L.gate.cpu().double(), L.topk_idx.cpu()
    zq = quantize64(z)[0]
    u = torch.zeros(T, d).double()
    q = lambda W: torch.stack([quantize64(W[e].t())[0].t() for e in range(E)])  # noqa: E731
    Wu, Wd, Wg = q(w["W_up"]), q(w["W_down"]), q(w["W_gate"]) if swiglu else None
    for t in range(T):
        for j in range(k):
            if slot[t, j] < 0:
                continue
            e = int(topk[t, j])
            h = zq[t] @ Wu[e]
            gt = zq[t] @ Wg[e] if swiglu else h
            a = gt / (1 + torch.exp(-gt)) * (h if swiglu else 1)
            a = quantize64(a.to(torch.bfloat16)[None])[0][0]
            u[t] += gate[t, j] * (a @ Wd[e])
    rel = ((L.out.cpu().double() - u).norm() / u.norm()).item()
    assert rel <= 2e-2, rel
    n = L.out.cpu().double()
    want = x.double() + n / torch.sqrt((n * n).mean(-1, keepdim=True) + EPS) * w["w_out"].double()
    assert ((x_out.double() - want).norm() / want.norm()).item() <= 2e-2
    with pytest.raises(RuntimeError, match="forward"):
        L.backward(x.cuda())


def test_four_bit_refusals():
    layer = moe.MoELayer(moe.MoEConfig(T=8, d=128, f=128, E=2, k=1))
    W = torch.zeros(2, 128, 128, dtype=torch.bfloat16, device="cuda")
    x, Wr = torch.zeros(8, 128, dtype=torch.bfloat16, device="cuda"), W[0, :, :2].contiguous()
    with pytest.raises(ValueError, match="gate matrix"):
        layer.forward_mx4(x, Wr, moe.MX4Experts(W, W, W))
    with pytest.raises(ValueError, match="shapes"):
        layer.forward_mx4(x, Wr, moe.MX4Experts(W[:1].contiguous(), W))
    f32 = moe.MoELayer(moe.MoEConfig(T=8, d=128, f=128, E=2, k=1, dtype=moe.F32))
    with pytest.raises(ValueError, match="bf16 layer"):
        f32.forward_mx4(x, Wr, moe.MX4Experts(W, W))
