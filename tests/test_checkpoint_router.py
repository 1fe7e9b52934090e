"""What the checkpointed layer's backward gives the router: its gradients step by step, the balance
loss's share of them, and the outputs y in 8 bits that dgate is formed from.

With e = 2^-24 and HALF half a bf16 step: dgate is a sum of d products, off by d e sum |dout y|.
dx and dW_r take dlogits in bf16: off by HALF of each term's magnitude and by the sums' own
(terms + 1) e, then rounded to bf16 themselves.  dbias is a sum of fp32 numbers.
"""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests.test_checkpoint import E24, HALF, layer_case
from tests.test_mx8 import quantize64


def steps(cfg, ck, x, w, dout):
    """The backward's entry points one by one, from what the checkpoint holds: no balance loss."""
    R, bf = moe.rows_capacity(cfg), torch.bfloat16
    e = lambda *s, dt=bf: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    ws = e(max(moe.workspace_size(cfg), 256), dt=torch.uint8)
    t = dict(x_perm=e(R, cfg.d), act=e(R, cfg.f), dy=e(R, cfg.d), dgate=e(cfg.T, cfg.k, dt=torch.float32),
             dh=e(cfg.nh, R, cfg.f), dx_perm=e(R, cfg.d), dlogits=e(cfg.T, cfg.E, dt=torch.float32))
    g = dict(dx=e(cfg.T, cfg.d), dW_r=e(cfg.d, cfg.E), dbias=e(cfg.E, dt=torch.float32), dW_up=e(*w["W_up"].shape),
             dW_gate=e(*w["W_gate"].shape) if w["W_gate"] is not None else None, dW_down=e(*w["W_down"].shape))
    y = ck.y.dequantize(bf)
    token, slot, kept, offs = (v.clone() for v in (ck.perm_token, ck.slot_of, ck.kept, ck.offsets))
    moe.moe_permute(cfg, x, ck.topk_idx, t["x_perm"], token, slot, kept, offs, None, ws)
    moe.moe_combine_backward(cfg, dout, y, ck.gate, slot, token, offs, t["dy"], t["dgate"])
    moe.moe_grouped_ffn_backward_mx8(cfg, t["x_perm"], offs, w["W_up"], w["W_gate"], w["W_down"], ck.h.codes, ck.h.scales,
                                     t["act"], t["dy"], t["dh"], t["dx_perm"], g["dW_up"], g["dW_gate"], g["dW_down"], ws)
    moe.moe_router_backward(cfg, x, w["W_r"], ck.logits, ck.topk_idx, ck.gate, slot, t["dgate"], t["dx_perm"], ck.stats,
                            g["dx"], g["dW_r"], g["dbias"], t["dlogits"], ws)
    return g, t, y


def near(got, want, terms, what):
    err, tol = (got.double() - want).abs(), HALF * want.abs() + terms
    assert (err <= tol).all(), (what, (err / tol.clamp(min=1e-300)).max().item())


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,swiglu,cf", [(600, 4, 2, True, 0.0), (333, 7, 3, False, 0.8), (1, 2, 1, True, 0.0)])
def test_router_gradients_of_a_checkpointed_forward(T, E, k, swiglu, cf):
    d, f = 256, 384
    x, w, dout = layer_case(T, d, f, E, k, swiglu, T)
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU if swiglu else moe.SILU, capacity_factor=cf, aux_coef=0.01)
    layer, ck = moe.MoELayer(cfg), moe.MoECheckpoint(cfg)
    layer.forward(x, **w, checkpoint=ck)
    n = int(ck.offsets[-1])
    # y in 8 bits: quantised from the second product's bf16 rows
    y16 = layer.y_perm[:n].double().cpu()
    assert torch.equal(ck.y.dequantize(torch.float32)[:n].double().cpu(), quantize64(y16)[1])

    plain = {m: t.clone() for m, t in layer.backward(dout, checkpoint=ck).items() if t is not None}
    want, t, y = steps(cfg, ck, x, w, dout)
    for m, v in plain.items():
        assert torch.equal(v, want[m]), m

    # dgate of the kept y
    slot, rows = ck.slot_of.long(), y.double()
    d64, here = dout.double(), slot >= 0
    picked = rows[slot.clamp(min=0)] * here[..., None]
    dot = (d64[:, None] * picked).sum(-1)
    assert ((t["dgate"].double() - dot).abs() <= d * E24 * (d64[:, None] * picked).abs().sum(-1)).all()

    # a balance loss's gradient on the logits, as large as the router's own
    dl = torch.randn(T, E, generator=torch.Generator().manual_seed(7)).cuda() * t["dlogits"].abs().mean().clamp(min=1e-3)
    g = {m: v.clone() for m, v in layer.backward(dout, checkpoint=ck, dlogits_aux=dl).items() if v is not None}
    for m in ("dW_up", "dW_down", "dW_gate"):
        assert m not in g or torch.equal(g[m], plain[m]), m
    both, mag = t["dlogits"].double() + dl.double(), t["dlogits"].double().abs() + dl.double().abs()
    x64, Wr = x.double(), w["W_r"].double()
    near(g["dW_r"], x64.t() @ both, (HALF + (T + 2) * E24) * (x64.abs().t() @ mag), "dW_r")
    sums = (t["dx_perm"].double()[slot.clamp(min=0)] * here[..., None]).sum(1)
    size = (t["dx_perm"].double()[slot.clamp(min=0)] * here[..., None]).abs().sum(1)
    near(g["dx"], sums + both @ Wr.t(), (HALF + (E + 2) * E24) * (mag @ Wr.abs().t()) + (k + E + 1) * E24 * size, "dx")
    assert ((g["dbias"].double() - both.sum(0)).abs() <= (T + 2) * E24 * mag.sum(0)).all()
    # and the share is there: none of the three would hold without it
    assert ((both.sum(0) - t["dlogits"].double().sum(0)).abs() > (T + 2) * E24 * mag.sum(0)).any()
    for m in ("dW_r", "dx", "dbias"):
        assert not torch.equal(g[m], plain[m]), m
    with pytest.raises(ValueError, match="dlogits_aux"):
        layer.backward(dout, checkpoint=ck, dlogits_aux=dl[:, :1])
    assert moe.last_device_status() == 0
