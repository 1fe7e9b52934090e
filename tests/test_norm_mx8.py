"""The residual stream's norms with the next block's input in 8 bits.

In fp32 the stored z is the very value that is quantised, so the codes are held to those of
``mx8_quantize(z)`` bit for bit, and x' and z to the plain call's.  In bf16 a row's sums run in
another order than the plain call's (16 elements a thread), so x', z and the codes are all held to
the definition in 64 bits.  With e = 2^-24:
  x' = a x + b g n is off by  ty = (d / 2 + 16) e (|a x| + |b g n|)   (n's sum of d squares)
  z  = w x' r       is off by  t  = r |w| ty + |z| ((d / 2 + 8) e + |ty| / |x'|)   (2-norms)
both and half a bf16 step where they are stored, and a value t off is stored within t + 2^-4 (|z| + t) + 2^-10 s of it, where s < (amax + t) / 224
is the scale: half a step of its code, or of the smallest codes.
"""
import ctypes

import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests.test_mx8 import quantize64

EPS, RA, OB = 1e-6, 0.9, 0.7
GATES = {"none": moe.GATE_NONE, "channel": moe.GATE_CHANNEL, "token": moe.GATE_TOKEN, "full": moe.GATE_FULL}


def inputs(T, d, dt, gate, leave, post, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean  # noqa: E731
    c = dict(x=(r(T, d) * torch.exp(r(T, 1))).to(dt), w_pre=r(d, std=0.2, mean=1.0))
    if leave:
        c["u"] = r(T, d).to(dt)
    if post:
        c["w_post"] = r(d, std=0.2, mean=1.0)
    if gate == "channel":
        c["gate"] = r(d, std=0.3, mean=0.5)
    elif gate == "token":
        c["gate"] = r(T, std=0.3, mean=0.5)
    elif gate == "full":
        c["gate"] = r(T, d, std=0.3, mean=0.5).to(dt)
    return c


def config(T, d, dt, gate, leave, post):
    return moe.NormConfig(T=T, d=d, dtype=moe.BF16 if dt == torch.bfloat16 else moe.F32, leave=leave, post_norm=post,
                          enter=1, gate=GATES[gate], eps=EPS, res_scale=RA, out_scale=OB)


def exact(c, gate, leave, post):
    """x' and z, and how far fp32 may be from each."""
    d, e = c["x"].shape[1], 2.0 ** -24
    v = {k: t.double() for k, t in c.items()}
    y, ty = v["x"], torch.zeros_like(v["x"])
    if leave:
        n = v["u"]
        if post:
            n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + EPS) * v["w_post"]
        if gate != "none":
            n = n * (v["gate"][:, None] if gate == "token" else v["gate"])
        ty = (d / 2 + 16) * e * ((RA * y).abs() + (OB * n).abs())
        y = RA * y + OB * n
    r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
    z = y * r * v["w_pre"]
    off = ty.norm(dim=-1, keepdim=True) / y.norm(dim=-1, keepdim=True).clamp(min=1e-300)
    return y, ty, z, r * v["w_pre"].abs() * ty + z.abs() * ((d / 2 + 8) * e + off)


def near(got, want, off):
    """Stored in bf16."""
    return ((got.cpu().double() - want).abs() <= off + 2.0 ** -8 * (want.abs() + off)).all()


def check(T, d, dt, gate, leave, post, keep_z=True, seed=0):
    c = inputs(T, d, dt, gate, leave, post, seed)
    cuda = {k: t.cuda() for k, t in c.items()}
    cfg = config(T, d, dt, gate, leave, post)
    plain, n = moe.BlockNorm(cfg), moe.BlockNorm(cfg)
    x1, z1 = plain.forward(**cuda)
    n.z.fill_(7.0)
    x2, z8, z2 = n.forward_mx8(**cuda, keep_z=keep_z)
    assert moe.last_device_status() == 0
    if keep_z:
        assert z2 is n.z
    else:
        assert z2 is None and (n.z == 7.0).all()
    if dt == torch.float32:
        assert torch.equal(x1, x2) and (not keep_z or torch.equal(z1, z2))
        q = moe.mx8_quantize(z1)
        assert torch.equal(q.codes, z8.codes)
        assert torch.equal(q.scales[:, :d // 32], z8.scales[:, :d // 32])
        return
    y, ty, z, t = exact(c, gate, leave, post)
    assert near(x2, y, ty) if leave else x2 is cuda["x"]
    assert not keep_z or near(z2, z, t)
    got = z8.dequantize(torch.float32).cpu().double()
    amax = (z.abs() + t).reshape(T, -1, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(T, d)
    tol = t + 2.0 ** -4 * (z.abs() + t) + 2.0 ** -10 * amax / 224
    assert ((got - z).abs() <= tol).all(), ((got - z).abs() / tol).max()
    # and most values are the very ones that the exact z rounds to
    if d <= 4096:
        assert (got != quantize64(z)[1]).float().mean() < 0.01


# ----------------------------------------------------------------- CPU
def test_refusals():
    lib, p, bad = moe.load_library(), ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    cfg = config(4, 64, torch.bfloat16, "channel", 1, 1)
    for i in range(9):
        args = [p] * 9
        args[i] = bad
        assert lib.moe_block_norm_mx8(ctypes.byref(cfg), *args, None) == moe.ERR_INVALID_ARG, i
        args[i] = None
        if i != 6:                                        # z may be absent
            assert lib.moe_block_norm_mx8(ctypes.byref(cfg), *args, None) == moe.ERR_INVALID_ARG, i
    odd = config(4, 40, torch.bfloat16, "channel", 1, 1)
    assert lib.moe_block_norm_mx8(ctypes.byref(odd), *[p] * 9, None) == moe.ERR_UNSUPPORTED
    leave = moe.NormConfig(T=4, d=64, enter=0)
    assert lib.moe_block_norm_mx8(ctypes.byref(leave), p, p, None, None, p, p, None, p, p, None) == moe.ERR_INVALID_ARG
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="enters"):
        moe.BlockNorm(leave, "cpu").forward_mx8(x, x)
    n = moe.BlockNorm(config(4, 64, torch.bfloat16, "none", 0, 0), "cpu")
    with pytest.raises(ValueError, match="x: expected"):
        n.forward_mx8(x[:3], w_pre=torch.ones(64))
    with pytest.raises(ValueError, match="w_pre: expected"):
        n.forward_mx8(x, w_pre=torch.ones(65))
    with pytest.raises(moe.MoEError):
        moe.BlockNorm(odd, "cpu").forward_mx8(x[:, :40], x[:, :40], gate=torch.ones(40), w_post=torch.ones(40))


# ----------------------------------------------------------------- GPU
FORMS = [("none", 0, 0), ("none", 1, 0), ("none", 1, 1), ("channel", 1, 1), ("token", 1, 1), ("full", 1, 1), ("token", 1, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate,leave,post", FORMS)
@pytest.mark.parametrize("T,d", [(1, 32), (5, 64), (33, 96), (7, 1056), (3, 4096), (151, 8192), (2, 8224), (3, 16384)])
def test_short_batches(T, d, dt, gate, leave, post):
    check(T, d, dt, gate, leave, post, seed=T + d)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate,leave,post", FORMS)
@pytest.mark.parametrize("T,d", [(9000, 1184), (4000, 4096), (1700, 6176), (165000, 64)])
def test_long_batches(T, d, dt, gate, leave, post):
    """Rows through the ring of shared memory."""
    check(T, d, dt, gate, leave, post, keep_z=T % 3 == 0, seed=T + d)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(40, 96), (11000, 1024)])
def test_rows_of_zeros_and_nans(T, d):
    c = inputs(T, d, torch.float32, "none", 0, 0)
    c["x"][3] = 0
    c["x"][4, 70], c["x"][5, 7] = float("nan"), float("inf")
    n = moe.BlockNorm(config(T, d, torch.float32, "none", 0, 0))
    z8, z = n.forward_mx8(c["x"].cuda(), w_pre=c["w_pre"].cuda())[1:]
    q = moe.mx8_quantize(z)
    assert torch.equal(q.codes, z8.codes) and torch.equal(q.scales[:, :d // 32], z8.scales[:, :d // 32])
    assert (z8.codes[3] & 127 == 0).all() and (z8.scales[4, :d // 32] == 255).all() and z8.scales[5, 0] == 255


@pytest.mark.gpu
def test_in_place_on_another_stream():
    T, d = 3000, 4096
    c = {k: t.cuda() for k, t in inputs(T, d, torch.bfloat16, "channel", 1, 1).items()}
    cfg = config(T, d, torch.bfloat16, "channel", 1, 1)
    n = moe.BlockNorm(cfg)
    want, z8, z = n.forward_mx8(**c)
    want, codes, z = want.clone(), z8.codes.clone(), z.clone()
    s = torch.cuda.Stream()
    z8.codes.zero_()
    s.wait_stream(torch.cuda.current_stream())
    # x' over x and z over u
    moe.moe_block_norm_mx8(cfg, c["x"], c["u"], c["w_post"], c["gate"], c["w_pre"], c["x"], c["u"], z8.codes, z8.scales, s)
    s.synchronize()
    assert torch.equal(c["x"], want) and torch.equal(c["u"], z) and torch.equal(z8.codes, codes)
