"""The fp32 product's silu far below zero, where e^-z leaves fp32's range before silu(z) does.

z is one product and one of small numbers, exact in fp32.  The tolerance: a few units of fp32 (as
the other products' tests), e^-|z| off by half of fp32's last denormal 2^-149 times |z| < 128, and
the result's own half of it.
"""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 1000])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_silu_where_its_divisor_would_leave_the_range(rows, act):
    K, N = 32, 256
    x, W = torch.zeros(rows, K), torch.zeros(1, K, N)
    x[:, 0], x[:, 1] = -80.0, -1.0
    x[1::2] = -x[1::2]                                       # and the other side
    W[0, 0] = 1.0
    W[0, 1] = torch.linspace(0, 30, N)                       # to the nearest e4m3
    xq, w = moe.mx8_quantize(x.cuda()), moe.mx8_quantize_weight(W.cuda())
    z = xq.dequantize(torch.float32).cpu().double() @ w.dequantize(torch.float32).cpu().double()[0].t()
    assert len(set(z[0].tolist())) > 20 and z.min() < -108 and ((z < -87.4) & (z > -103)).any()
    o = torch.tensor([0, rows], dtype=torch.int32).cuda()
    want = z / (1 + torch.exp(-z))
    up = torch.ones_like(z)
    args = ()
    if act == "swiglu":
        wu = moe.mx8_quantize_weight(torch.full((1, K, N), 0.125).cuda())
        up = xq.dequantize(torch.float32).cpu().double() @ torch.full((K, N), 0.125).double()
        want, args = want * up, (w,)
        w = wu
    code = moe.MX8_ACT_SILU if act == "silu" else moe.MX8_ACT_SWIGLU
    m = moe.MX8Product(moe.MX8ProductConfig(rows=rows, K=K, N=N, E=1, act=code, out_dtype=moe.F32))
    got = m.forward(xq, o, w, *args).cpu().double()
    tol = 16 * 2.0 ** -22 * want.abs() + (128 * 2.0 ** -150 + 2.0 ** -149) * up.abs().clamp(min=1)
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max().item()
