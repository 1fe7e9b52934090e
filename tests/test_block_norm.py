"""The residual stream's norms around a block against the formulas in 64 bits.

Tolerances.  A stored value is rounded once: half a step of its type relative to
the value (bf16 2^-8, fp32 2^-24, times 1 + 2^-6 for the arithmetic before it).
fp32 arithmetic adds C 2^-24 of the sum of the magnitudes of the terms that form
the value: a row's sums run over 16 elements a thread in order, then 5 shuffles
and at most 32 warps, so 64 covers them with the few products around them; sums
over T rows add up to T more.
"""
import ctypes

import pytest
import torch

import top_routing_expert_moe_gb300 as moe

EPS, RA, OB = 1e-6, 0.75, 0.5
GATES = {"none": moe.GATE_NONE, "channel": moe.GATE_CHANNEL, "token": moe.GATE_TOKEN,
         "full": moe.GATE_FULL}


def half_step(dt):
    return torch.finfo(dt).eps / 2 * (1 + 2.0 ** -6)


def make(T, d, dt, leave, post, enter, gate, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    v = {"x": (r(T, d) * torch.exp(r(T, 1))).to(dt)}
    if leave:
        v["u"] = r(T, d).to(dt)
    if post:
        v["w_post"] = 1 + 0.1 * r(d)
    if enter:
        v["w_pre"] = 1 + 0.1 * r(d)
    if gate != "none":
        shape = {"channel": (d,), "token": (T,), "full": (T, d)}[gate]
        v["gate"] = 0.5 + 0.3 * r(*shape)
        if gate == "full":
            v["gate"] = v["gate"].to(dt)
    if T > 2:
        v["x"][1] = 0                      # a zero row of the stream, and of the block's output
        if leave:
            v["u"][1] = 0
    v["dx_out"] = r(T, d).to(dt)
    if enter:
        v["dz"] = r(T, d).to(dt)
    return v


def forward64(v, leave, post, enter, gate):
    """x', z and for each the sum of the magnitudes of its terms."""
    f = {k: t.double() for k, t in v.items()}
    x = f["x"]
    if leave:
        n = f["u"]
        if post:
            n = f["w_post"] * n / torch.sqrt((n * n).mean(-1, keepdim=True) + EPS)
        if gate != "none":
            n = n * (f["gate"][:, None] if gate == "token" else f["gate"])
        y, m = RA * x + OB * n, (RA * x).abs() + (OB * n).abs()
    else:
        y, m = x, x.abs()
    if not enter:
        return y, m, None, None
    r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
    return y, m, f["w_pre"] * y * r, (f["w_pre"] * r).abs() * m


def loss64(f, leave, post, enter, gate):
    """A scalar whose gradients are those of the block norm: f holds doubles, x' among them."""
    def unit(v):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    y = f["x"]
    if leave:
        n = unit(f["u"]) * f["w_post"] if post else f["u"]
        if gate != "none":
            n = n * (f["gate"][:, None] if gate == "token" else f["gate"])
        y = RA * y + OB * n
    out = (y * f["dx_out"]).sum()
    if enter:
        out = out + (unit(y) * f["w_pre"] * f["dz"]).sum()
    return out


def backward64(v, y, leave, post, enter, gate):
    """Gradients by the formulas at the stream y, and the magnitudes of their terms."""
    f = {k: t.double() for k, t in v.items()}
    d = y.shape[1]
    y, G = y.double(), f["dx_out"]
    mG, g, m = G.abs(), {}, {}
    if enter:
        r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
        a = f["w_pre"] * f["dz"]
        A = (a * y).sum(-1, keepdim=True)
        mG = mG + (r * a).abs() + (y * r ** 3 / d).abs() * (a * y).abs().sum(-1, keepdim=True)
        G = G + r * a - y * r ** 3 / d * A
        g["dw_pre"] = (f["dz"] * y * r).sum(0)
        m["dw_pre"] = (f["dz"] * y * r).abs().sum(0)
    if not leave:
        g["dx"], m["dx"] = G, mG
        return g, m
    g["dx"], m["dx"] = RA * G, RA * mG
    u = f["u"]
    ru = 1 / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS) if post else torch.ones(1, 1, device=u.device).double()
    n = u * ru * (f["w_post"] if post else 1)
    gt = 1 if gate == "none" else f["gate"][:, None] if gate == "token" else f["gate"]
    dn, mdn = OB * gt * G, (OB * gt * mG).abs() if gate != "none" else OB * mG
    if gate != "none":
        dims = {"channel": 0, "token": 1, "full": ()}[gate]
        dg, mdg = OB * G * n, (OB * mG * n).abs()
        g["dgate"] = dg if gate == "full" else dg.sum(dims)
        m["dgate"] = mdg if gate == "full" else mdg.sum(dims)
    if post:
        b, mb = dn * f["w_post"], mdn * f["w_post"].abs()
        g["du"] = ru * b - u * ru ** 3 / d * (b * u).sum(-1, keepdim=True)
        m["du"] = ru * mb + (u * ru ** 3 / d).abs() * (mb * u.abs()).sum(-1, keepdim=True)
        g["dw_post"], m["dw_post"] = (dn * u * ru).sum(0), (mdn * (u * ru).abs()).sum(0)
    else:
        g["du"], m["du"] = dn, mdn
    return g, m


def near(got, want, terms, c, name):
    tol = half_step(got.dtype) * want.abs() + c * 2.0 ** -24 * terms
    err = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all(), name
    assert (err <= tol).all(), (name, (err / tol.clamp(min=1e-300)).max().item())


def config(T, d, dt, leave, post, enter, gate):
    return moe.NormConfig(T=T, d=d, dtype=moe.BF16 if dt == torch.bfloat16 else moe.F32,
                          leave=leave, post_norm=post, enter=enter, gate=GATES[gate], eps=EPS,
                          res_scale=RA, out_scale=OB)


FORMS = [(0, 0, 1, "none"), (1, 0, 1, "none"), (1, 1, 1, "none"), (1, 0, 0, "token"),
         (1, 1, 0, "channel"), (1, 1, 1, "channel"), (1, 1, 1, "token"), (1, 1, 1, "full"),
         (1, 0, 1, "full"), (1, 0, 1, "channel")]


# ----------------------------------------------------------------- CPU
@pytest.mark.parametrize("form", FORMS)
def test_formulas_against_differences(form):
    """The 64-bit gradients the kernels are held to, against central differences."""
    v = make(3, 5, torch.float64, *form, seed=4)
    v["x"][1] += 0.3                       # differences need a smooth point
    if form[0]:
        v["u"][1] += 0.2
    y, _, _, _ = forward64(v, *form)
    g, _ = backward64(v, y, *form)
    names = {"dx": "x", "du": "u", "dw_pre": "w_pre", "dw_post": "w_post", "dgate": "gate"}
    h = 1e-6
    for gn, gt in g.items():
        p = v[names[gn]].double()
        for idx in [tuple(int(i) for i in j) for j in torch.ones(p.shape).nonzero()]:
            lo, hi = p.clone(), p.clone()
            lo[idx] -= h
            hi[idx] += h
            f = {k: t.double() for k, t in v.items()}
            num = (loss64({**f, names[gn]: hi}, *form) - loss64({**f, names[gn]: lo}, *form)) / (2 * h)
            assert abs(num - gt[idx]) <= 1e-6 * (1 + abs(gt[idx])), (gn, idx)


def test_config_refusals():
    ok = dict(T=4, d=64)
    assert moe.check_norm_config(moe.NormConfig(**ok)) == moe.OK
    assert moe.check_norm_config(moe.NormConfig(T=1, d=1, dtype=moe.F32)) == moe.OK
    for b in (dict(T=0), dict(d=0), dict(dtype=2), dict(leave=2), dict(post_norm=-1), dict(enter=3),
              dict(gate=4), dict(gate=-1), dict(eps=0.0), dict(eps=float("nan")), dict(eps=-1e-6),
              dict(res_scale=float("inf")), dict(out_scale=float("nan")),
              dict(leave=0, post_norm=1), dict(leave=0, gate=moe.GATE_TOKEN),
              dict(leave=0, enter=0)):
        assert moe.check_norm_config(moe.NormConfig(**{**ok, **b})) == moe.ERR_INVALID_ARG, b
    assert moe.check_norm_config(moe.NormConfig(T=4, d=16385)) == moe.ERR_UNSUPPORTED
    assert moe.load_library().moe_check_norm_config(None) == moe.ERR_INVALID_ARG
    with pytest.raises(moe.MoEError):
        moe.norm_workspace_size(moe.NormConfig(T=0, d=8))
    with pytest.raises(moe.MoEError):
        moe.BlockNorm(moe.NormConfig(T=0, d=8), device="cpu")


def test_pointer_refusals_before_launch():
    lib = moe.load_library()
    p, bad = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    c = moe.NormConfig(T=4, d=64, post_norm=1, gate=moe.GATE_CHANNEL)
    for i in range(7):                     # each tensor missing, then misaligned
        for v in (None, bad):
            args = [p] * 7
            args[i] = v
            assert lib.moe_block_norm(ctypes.byref(c), *args, None) == moe.ERR_INVALID_ARG, i
    plain = moe.NormConfig(T=4, d=64, leave=0)
    assert lib.moe_block_norm(ctypes.byref(plain), p, p, None, None, p, None, p, None) == \
        moe.ERR_INVALID_ARG                # u given, but nothing leaves a block
    for i in range(13):
        if i == 5:
            continue                       # dx_out may be missing
        args = [p] * 13
        args[i] = None
        assert lib.moe_block_norm_backward(ctypes.byref(c), *args, None) == moe.ERR_INVALID_ARG, i
    stop = moe.NormConfig(T=4, d=64, enter=0)
    args = [p, p, None, None, None, None, None, p, p, None, None, None, p]
    assert lib.moe_block_norm_backward(ctypes.byref(stop), *args, None) == moe.ERR_INVALID_ARG


def test_binding_refuses_other_shapes_and_types():
    n = moe.BlockNorm(moe.NormConfig(T=4, d=64), device="cpu")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="u: expected"):
        n.forward(x, u=x[:3], w_pre=w)
    with pytest.raises(ValueError, match="w_pre: expected"):
        n.forward(x, u=x, w_pre=w.bfloat16())
    with pytest.raises(ValueError, match="gate given"):
        n.forward(x, u=x, w_pre=w, gate=w)
    with pytest.raises(ValueError, match="must live on the GPU"):
        n.forward(x, u=x, w_pre=w)


# ----------------------------------------------------------------- GPU
def check(T, d, dt, form, seed=0):
    v = make(T, d, dt, *form, seed=seed)
    n = moe.BlockNorm(config(T, d, dt, *form))
    c = {k: t.cuda() for k, t in v.items()}
    args = {k: c[k] for k in ("u", "w_pre", "w_post", "gate") if k in c}
    x_out, z = n.forward(c["x"], **args)
    y, my, z64, mz = forward64(v, *form)
    if form[0]:
        near(x_out, y, my, 64, "x_out")
    if form[2]:
        near(z, z64, mz, 64, "z")
    g = n.backward(x_out, dx_out=c["dx_out"], dz=c.get("dz"), **args)
    g64, m64 = backward64(v, x_out.cpu(), *form)
    assert {k for k, t in g.items() if t is not None} == set(g64)
    for k in g64:
        near(g[k], g64[k], m64[k], 64 + (T if g64[k].shape == (d,) else 0), k)
    assert moe.last_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(5, 256), (3, 77), (37, 1000)])
def test_forms(T, d, dt, form):
    check(T, d, dt, form)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1, 2, 7, 8, 31, 40, 127, 512, 513, 520, 1001, 2816, 4096, 4100, 6000,
                               8192, 8200, 16377, 16384])
def test_widths(d, dt):
    check(6, d, dt, (1, 1, 1, "channel"), seed=d)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(1, 4096), (1, 9), (2, 64), (1237, 64), (4001, 24), (2500, 1024),
                                 (3001, 333)])
def test_lengths(T, d):
    check(T, d, torch.bfloat16, (1, 1, 1, "channel"), seed=T)
    check(T, d, torch.float32, (1, 1, 1, "token"), seed=T)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_long_batches_of_every_form(form, dt):
    """Batches that go through the shared-memory ring (several rows a CTA)."""
    check(1303, 520, dt, form, seed=11)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(304, 8), (3000, 16), (5000, 264), (303, 1024), (305, 2816),
                                 (700, 4096), (640, 4104), (700, 8192), (320, 16384), (305, 1),
                                 (311, 3), (333, 7), (1001, 33), (1237, 1001), (400, 4097), (305, 8191)])
def test_long_batches_of_every_width(T, d, dt):
    check(T, d, dt, (1, 1, 1, "channel"), seed=d)
    check(T, d, dt, (1, 1, 1, "full"), seed=d)


@pytest.mark.gpu
@pytest.mark.parametrize("form", [(0, 0, 1, "none"), (1, 0, 0, "token"), (1, 1, 0, "channel"), (1, 0, 1, "full"),
                                  (1, 1, 1, "channel"), (1, 1, 1, "full"), (1, 1, 1, "token")])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(20600, 520), (2700, 4104), (1300, 8192)])
def test_batches_of_more_than_ten_million_elements(T, d, dt, form):
    """Both passes of aligned rows through the ring, against the formulas in 64 bits on the GPU."""
    v = make(T, d, dt, *form, seed=T)
    n = moe.BlockNorm(config(T, d, dt, *form))
    c = {k: t.cuda() for k, t in v.items()}
    args = {k: c[k] for k in ("u", "w_pre", "w_post", "gate") if k in c}
    x_out, z = n.forward(c["x"], **args)
    y, my, z64, mz = (None if t is None else t.cpu() for t in forward64(c, *form))
    if form[0]:
        near(x_out, y, my, 64, "x_out")
    if form[2]:
        near(z, z64, mz, 64, "z")
    g = n.backward(x_out, dx_out=c["dx_out"], dz=c.get("dz"), **args)
    g64, m64 = backward64(c, x_out, *form)
    for k in g64:
        near(g[k], g64[k].cpu(), m64[k].cpu(), 64 + (T if g64[k].shape == (d,) else 0), k)
    assert moe.last_device_status() == 0


@pytest.mark.gpu
def test_stream_gradient_absent_is_zero():
    form = (1, 1, 1, "none")
    v = make(9, 128, torch.float32, *form)
    n = moe.BlockNorm(config(9, 128, torch.float32, *form))
    c = {k: t.cuda() for k, t in v.items()}
    args = dict(u=c["u"], w_pre=c["w_pre"], w_post=c["w_post"])
    a = {k: t.clone() for k, t in n.backward(c["x"], dz=c["dz"], **args).items() if t is not None}
    b = n.backward(c["x"], dx_out=torch.zeros_like(c["x"]), dz=c["dz"], **args)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.gpu
def test_in_place_repeatable_and_on_another_stream():
    form = (1, 1, 1, "channel")
    T, d = 300, 1024
    v = make(T, d, torch.bfloat16, *form)
    c = {k: t.cuda() for k, t in v.items()}
    cfg = config(T, d, torch.bfloat16, *form)
    n = moe.BlockNorm(cfg)
    x1, z1 = n.forward(c["x"], u=c["u"], w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"])
    x, u = c["x"].clone(), c["u"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_block_norm(cfg, x, u, c["w_post"], c["gate"], c["w_pre"], x, u, stream=s)
    s.synchronize()
    assert torch.equal(x, x1) and torch.equal(u, z1)
    g = n.backward(x1, dx_out=c["dx_out"], dz=c["dz"], u=c["u"], w_pre=c["w_pre"],
                   w_post=c["w_post"], gate=c["gate"])
    first = {k: t.clone() for k, t in g.items() if t is not None}
    g = n.backward(x1, dx_out=c["dx_out"], dz=c["dz"], u=c["u"], w_pre=c["w_pre"],
                   w_post=c["w_post"], gate=c["gate"])
    for k, t in first.items():
        assert torch.equal(t, g[k]), k
