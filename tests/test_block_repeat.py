"""A block that is run on its own output, as a weight-tied stack does, and one whose
forward did not come to its end."""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests import test_block as base

CFG = dict(T=200, d=128, f=256, E=4, k=2)


def on_cpu(monkeypatch):
    """The binding without its launches, so that which buffers it passes can be followed."""
    for m in (moe, moe.block):
        monkeypatch.setattr(m, "_p", lambda t: t)
        monkeypatch.setattr(m, "_s", lambda s: 0)
        monkeypatch.setattr(m, "_call", lambda name, *a: calls.append((name, a)))
    calls = []
    return calls


def cpu_block(monkeypatch, **kw):
    cfg = moe.MoEConfig(**CFG)
    b = moe.MoEBlock(cfg, device="cpu", **kw)
    calls = on_cpu(monkeypatch)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    w = dict(w_in=torch.ones(128), W_r=z(128, 4), W_up=z(4, 128, 256), W_down=z(4, 256, 128))
    return b, w, calls


def test_the_saved_stream_is_not_written(monkeypatch):
    b, w, calls = cpu_block(monkeypatch)
    x = torch.zeros(200, 128, dtype=torch.bfloat16)
    seen = []
    for _ in range(4):
        calls.clear()
        out, _ = b.forward(x, w)
        (leave,) = [a for n, a in calls if n == "moe_block_norm" and a[2] is not None]
        assert leave[1] is x and leave[6] is out
        assert out.data_ptr() != x.data_ptr()
        seen.append(out.data_ptr())
        x = out
    assert len(set(seen)) == 2                 # two buffers take turns
    fresh = torch.zeros_like(x)
    assert b.forward(fresh, w)[0].data_ptr() == b.forward(fresh, w)[0].data_ptr()


def test_a_forward_that_raised_leaves_no_backward(monkeypatch):
    b, w, _ = cpu_block(monkeypatch, post_norm=1)
    x = torch.zeros(200, 128, dtype=torch.bfloat16)
    w["w_out"] = torch.ones(128)
    b.forward(x, w)
    b.backward(x)
    with pytest.raises(ValueError, match="w_post"):
        b.forward(x, {**w, "w_out": torch.ones(127)})
    with pytest.raises(RuntimeError, match="forward"):
        b.backward(x)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gradients_of_a_block_on_its_own_output(dt):
    T, d, f, E, k = (CFG[n] for n in "TdfEk")
    x, w, dout = base.weights(T, d, f, E, dt, True, moe.GATE_CHANNEL)
    offs = [0, 90, 200]
    cfg = moe.MoEConfig(**CFG, ffn=moe.SWIGLU, dtype=moe.F32 if dt == torch.float32 else moe.BF16)
    b = moe.MoEBlock(cfg, post_norm=1, gate=moe.GATE_CHANNEL, eps=base.EPS, res_scale=base.RA,
                     out_scale=base.OB, sequences=2, balance_coef=base.BC, z_coef=base.ZC)
    wc = {n: t.cuda() for n, t in w.items()}
    o = torch.tensor(offs, dtype=torch.int32).cuda()
    x1 = b.forward(x.cuda(), wc, o)[0]
    x1_host = x1.cpu()
    x2 = b.forward(x1, wc, o)[0]
    g = b.backward(dout.cuda())
    assert torch.equal(x1.cpu(), x1_host)
    topk = b.layer.topk_idx.cpu().long()
    x64 = x1_host.double().requires_grad_()
    w64 = {n: t.double().requires_grad_() for n, t in w.items()}
    want, bal, zl = base.block64(x64, w64, topk, offs, k, True, moe.GATE_CHANNEL)
    grads = torch.autograd.grad((want * dout.double()).sum() + bal + zl, [x64] + list(w64.values()))
    tol = 2e-5 if dt == torch.float32 else 2e-2          # the layer's parity bounds, as in test_block.py
    rel = lambda a, t: ((a.double().cpu() - t).norm() / t.norm()).item()  # noqa: E731
    assert rel(x2, want.detach()) <= tol
    for n, t in zip(["dx"] + ["d" + n for n in w64], grads):
        assert rel(g[n], t) <= tol, (n, rel(g[n], t))
