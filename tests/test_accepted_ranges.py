"""Calls inside the documented ranges that take a path of their own: many sequences,
outputs written over inputs and an absent stream gradient in batches of the ring,
channel sums held so that one row of thousands would be missed, segments without
padding, deep and wide products, tensors of more than 2^32 elements.

Channel sums of data of one sign: a CTA adds its rows in order, a lane the CTAs'
partials in order, then 32 lanes, so T / 152 + 32 + 32 roundings and 64 for the terms,
each 2^-24 of the sum; a row that is left out is about 1 / T of it, several times that.
"""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests import test_balance_loss as bal
from tests import test_block_norm as norm
from tests import test_mx4 as mx4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,S", [(9000, 2049), (9000, 5000), (3000, 65536)])
def test_many_sequences(T, S):
    bal.check(*bal.make(T, 8, 2, S, seed=S))


@pytest.mark.parametrize("T,d,dt", [(20600, 520, torch.bfloat16), (1237, 1001, torch.bfloat16), (1237, 1001, torch.float32),
                                    (2700, 4104, torch.bfloat16), (2700, 4104, torch.float32), (333, 7, torch.bfloat16)])
@pytest.mark.parametrize("form", [(1, 1, 1, "channel"), (1, 0, 1, "none"), (1, 1, 0, "token"), (1, 1, 1, "full")])
def test_outputs_over_inputs_in_long_batches(T, d, dt, form):
    v = norm.make(T, d, dt, *form, seed=d)
    c = {k: t.cuda() for k, t in v.items()}
    cfg = norm.config(T, d, dt, *form)
    n = moe.BlockNorm(cfg)
    args = {k: c[k] for k in ("u", "w_pre", "w_post", "gate") if k in c}
    x1, z1 = n.forward(c["x"], **args)
    for _ in range(3):
        x, u = c["x"].clone(), c["u"].clone()
        moe.moe_block_norm(cfg, x, u, c.get("w_post"), c.get("gate"), c.get("w_pre"), x, u if form[2] else None)
        assert torch.equal(x, x1)
        assert torch.equal(u, z1 if form[2] else c["u"])


@pytest.mark.parametrize("T,d", [(1303, 1024), (5000, 264), (1237, 1001), (400, 8191), (40, 1024)])
@pytest.mark.parametrize("form", [(1, 1, 1, "none"), (1, 0, 1, "none"), (0, 0, 1, "none"), (1, 1, 1, "full")])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_absent_stream_gradient_is_zero_in_long_batches(T, d, form, dt):
    v = norm.make(T, d, dt, *form, seed=T)
    v["dx_out"] = torch.zeros_like(v["dx_out"])
    n = moe.BlockNorm(norm.config(T, d, dt, *form))
    c = {k: t.cuda() for k, t in v.items()}
    args = {k: c[k] for k in ("u", "w_pre", "w_post", "gate") if k in c}
    g = n.backward(c["x"], dz=c["dz"], **args)
    g64, m64 = norm.backward64(v, v["x"], *form)
    for k in g64:
        norm.near(g[k], g64[k], m64[k], 64 + (T if g64[k].shape == (d,) else 0), k)
    assert moe.last_device_status() == 0


@pytest.mark.parametrize("T,d", [(20600, 520), (2700, 4104), (5000, 264), (1237, 1001), (20011, 31), (3000, 9000), (6000, 40)])
@pytest.mark.parametrize("form", [(0, 0, 1, "none"), (1, 1, 0, "channel")])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_no_row_is_missing_from_the_channel_sums(T, d, form, dt):
    v = {k: t.abs() + 0.125 for k, t in norm.make(T, d, torch.float32, *form, seed=d).items()}
    for k in ("x", "u", "dx_out", "dz"):
        if k in v:
            v[k] = v[k].clamp(max=4.0).to(dt)
    n = moe.BlockNorm(norm.config(T, d, dt, *form))
    c = {k: t.cuda() for k, t in v.items()}
    args = {k: c[k] for k in ("u", "w_pre", "w_post", "gate") if k in c}
    g = n.backward(c["x"], dx_out=c["dx_out"], dz=c.get("dz"), **args)
    g64, _ = norm.backward64(c, c["x"], *form)
    for k in ("dw_pre",) if form[2] else ("dw_post", "dgate"):
        rel = ((g[k].double() - g64[k]).abs() / g64[k]).max().item()
        assert rel <= (T / 152 + 128) * 2.0 ** -24, (k, rel)
    assert moe.last_device_status() == 0


@pytest.mark.parametrize("E,K,N,act", [(64, 256, 128, "none"), (8, 4096, 136, "none"), (3, 2048, 64, "swiglu")])
def test_segments_without_padding(E, K, N, act):
    """A bound with fewer than 127 rows an expert to spare, all of it real rows: more tiles
    than the bound less 127 rows an expert would make."""
    mx4.product_case([128] * E, K, N, act, torch.bfloat16, seed=E, slack=0)
    mx4.product_case([128] * (E - 1) + [0], K, N, act, torch.float32, seed=E, slack=0)


@pytest.mark.parametrize("K,N", [(2 ** 17, 40), (65536 + 32, 8), (64, 2 ** 15 + 8)])
def test_deep_and_wide_products(K, N):
    mx4.product_case([130, 0, 5], K, N, "none", torch.float32, seed=N)


def test_rows_of_the_largest_width():
    K = 2 ** 24
    x = mx4.rows_of(2, K, torch.bfloat16, seed=1)
    v, byte = mx4.quantize64(x)
    q = moe.mx4_quantize(x.cuda())
    assert torch.equal(q.scales.cpu(), mx4.tiles(byte, 2, K))
    assert mx4.same(q.dequantize().cpu().double(), v)


def test_tensors_of_more_than_two_to_the_32_elements():
    T, d = 2 ** 20 + 135, 4128
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    part = torch.randn(1024, d, generator=g, device="cuda").bfloat16()
    for i in range(0, T, 1024):
        x[i:i + 1024] = part[:min(1024, T - i)]
    x[T - 135:] = torch.randn(135, d, generator=g, device="cuda").bfloat16()
    some = torch.cat([torch.arange(0, 5), torch.arange(2 ** 19 - 3, 2 ** 19 + 3), torch.arange(T - 135, T)]).cuda()
    n = moe.BlockNorm(moe.NormConfig(T=T, d=d, leave=0, eps=norm.EPS))
    w = torch.ones(d, device="cuda")
    z = n.forward(x, w_pre=w)[1]
    v = {"x": x[some].cpu(), "w_pre": w.cpu()}
    _, _, z64, mz = norm.forward64(v, 0, 0, 1, "none")
    norm.near(z[some], z64, mz, 64, "z")
    dx = n.backward(x, dz=x, w_pre=w)["dx"]
    v["dz"], v["dx_out"] = v["x"], torch.zeros_like(v["x"])
    g64, m64 = norm.backward64(v, v["x"], 0, 0, 1, "none")
    norm.near(dx[some], g64["dx"], m64["dx"], 64, "dx")
    q = moe.mx4_quantize(x)
    got = q.dequantize()
    want, _ = mx4.quantize64(x[some].cpu())
    assert mx4.same(got[some].cpu().double(), want)
    assert moe.last_device_status() == 0
