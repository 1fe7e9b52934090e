"""The experts' activations kept in 8 bits between forward and backward.

The forward's outputs are moe_grouped_ffn's bit for bit.  With e = 2^-24 and the terms' sums of
magnitudes:
  the kept h is Q8 of a sum of d products, off by t = d e sum |x W|, so that its value lies within
    t + 2^-4 (|h| + t) + 2^-10 s of h, where the scale s < (amax + t) / 224
  act, formed from the kept values, is off by 16 2^-22 of it and half a bf16 step
  dh = dact f(h) with dact a sum of d products: d e sum |dy W| |f| + 16 2^-22 |dh| (and of the
    derivative's two terms, which may cancel) and half a bf16 step
  dW and dx are sums of bf16 products, off by n e sum |a b| and half a bf16 step
each held against 64 bits with the tensors that its kernel reads as inputs.
"""
import ctypes

import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests.test_mx8 import quantize64

E24, HALF = 2.0 ** -24, 2.0 ** -8 * (1 + 2.0 ** -6)      # a unit of fp32, half a bf16 step


def sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def act_of(g, u):
    return g * sigmoid(g) * (1 if u is None else u)


def dh_of(dact, g, u):
    """(dh, None) or (dg, du), as the header states them."""
    s = sigmoid(g)
    if u is None:
        return dact * (s * (1 + g * (1 - s))), None
    return dact * u * (s * (1 + g * (1 - s))), dact * g * s


# ----------------------------------------------------------------- CPU
@pytest.mark.parametrize("swiglu", [False, True])
def test_the_formulas_are_the_derivatives_at_the_kept_values(swiglu):
    """Central differences of <dy, act(h^ + (h(x, W) - h0)) W_down> in x and every weight."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, Wu, Wg, Wd, dy = r(5, 32), r(32, 32) / 6, r(32, 32) / 6, r(32, 4), r(5, 4)
    ug0 = [x @ Wu] + ([x @ Wg] if swiglu else [])
    kept = [quantize64(h)[1] for h in ug0]

    def loss(x, Wu, Wg, Wd):
        u = kept[0] + x @ Wu - ug0[0]
        if not swiglu:
            return (act_of(u, None) @ Wd * dy).sum()
        return (act_of(kept[1] + x @ Wg - ug0[1], u) @ Wd * dy).sum()

    gate, up = (kept[1], kept[0]) if swiglu else (kept[0], None)
    dh, du = dh_of(dy @ Wd.t(), gate, up)
    grads = {3: act_of(gate, up).t() @ dy}
    if swiglu:
        grads.update({0: du @ Wu.t() + dh @ Wg.t(), 1: x.t() @ du, 2: x.t() @ dh})
    else:
        grads.update({0: dh @ Wu.t(), 1: x.t() @ dh})
    at, h = [x, Wu, Wg, Wd], 1e-5
    for k, want in grads.items():
        for _ in range(6):
            i = tuple(int(torch.randint(0, n, (1,), generator=g)) for n in at[k].shape)
            d = []
            for sgn in (1, -1):
                moved = [t.clone() for t in at]
                moved[k][i] += sgn * h
                d.append(loss(*moved))
            # the third derivative's part, and 64-bit rounding over 2 h
            assert abs((d[0] - d[1]) / (2 * h) - want[i]) <= 1e-7 * (1 + abs(want[i])), (k, i)


def test_refusals():
    lib, p, bad = moe.load_library(), ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    cfg = moe.MoEConfig(T=8, d=128, f=128, E=2, k=1, ffn=moe.SWIGLU)
    for i in range(9):
        for v in (None, bad):
            args = [p] * 9
            args[i] = v
            assert lib.moe_grouped_ffn_mx8(ctypes.byref(cfg), *args, p, None) == moe.ERR_INVALID_ARG, i
    for i in range(14):
        for v in (None, bad):
            args = [p] * 14
            args[i] = v
            assert lib.moe_grouped_ffn_backward_mx8(ctypes.byref(cfg), *args, p, None) == moe.ERR_INVALID_ARG, i
    half = ctypes.c_void_p(0x10010)                          # 16-byte aligned
    for i in (5, 7):
        args = [p] * 9
        args[i] = half
        assert lib.moe_grouped_ffn_mx8(ctypes.byref(cfg), *args, p, None) == moe.ERR_INVALID_ARG, i
    for i in (5, 7, 9):
        args = [p] * 14
        args[i] = half
        assert lib.moe_grouped_ffn_backward_mx8(ctypes.byref(cfg), *args, p, None) == moe.ERR_INVALID_ARG, i
    for i in (12, 14, 25):
        args = [p] * 26
        args[i] = half
        assert lib.moe_backward_mx8(ctypes.byref(cfg), *args, None) == moe.ERR_INVALID_ARG, i
    for c in (moe.MoEConfig(T=8, d=128, f=128, E=2, k=1, dtype=moe.F32),
              moe.MoEConfig(T=8, d=128, f=128, E=2, k=1, f_shared=128)):
        assert lib.moe_grouped_ffn_mx8(ctypes.byref(c), *[p] * 10, None) == moe.ERR_UNSUPPORTED
        assert lib.moe_grouped_ffn_backward_mx8(ctypes.byref(c), *[p] * 15, None) == moe.ERR_UNSUPPORTED
        assert lib.moe_backward_mx8(ctypes.byref(c), *[p] * 26, None) == moe.ERR_UNSUPPORTED
        with pytest.raises(ValueError, match="bf16 layer without shared"):
            moe.MoECheckpoint(c, "cpu")
    assert lib.moe_backward_mx8(ctypes.byref(cfg), *[p] * 25, None, None) == moe.ERR_INVALID_ARG
    with pytest.raises(moe.MoEError):
        moe.MoECheckpoint(moe.MoEConfig(T=8, d=100, f=128, E=2, k=1), "cpu")
    layer, other = moe.MoELayer(cfg, "cpu"), moe.MoECheckpoint(moe.MoEConfig(T=9, d=128, f=128, E=2, k=1), "cpu")
    x = torch.zeros(8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="another layer"):
        layer.forward(x, x, x, x, x, checkpoint=other)
    with pytest.raises(ValueError, match="another layer"):
        layer.backward(x, checkpoint=other)
    with pytest.raises(ValueError, match="no shared experts"):
        layer.forward(x, x, x, x, x, shared=(x, x), checkpoint=moe.MoECheckpoint(cfg, "cpu"))
    with pytest.raises(ValueError, match="must live on the GPU"):
        layer.forward(x, x, x, x, x, checkpoint=moe.MoECheckpoint(cfg, "cpu"))
    with pytest.raises(RuntimeError, match="needs a forward"):
        layer.backward(x, checkpoint=moe.MoECheckpoint(cfg, "cpu"))


# ----------------------------------------------------------------- GPU
def ffn_case(T, d, f, E, k, swiglu, seed=0, cf=0.0, empty=()):
    """Rows as moe_permute leaves them, and their gradients."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU if swiglu else moe.SILU, capacity_factor=cf)
    R = moe.rows_capacity(cfg)
    left, offs, x, dy = T * k, [0], torch.zeros(R, d), torch.zeros(R, d)
    for e in range(E):
        n = 0 if e in empty else left if e == E - 1 else int(torch.randint(0, left + 1, (1,), generator=g)) if left else 0
        n = min(n, T)
        a = offs[-1]
        x[a:a + n], dy[a:a + n] = r(n, d), r(n, d)
        offs.append(a + (n + 127) // 128 * 128)
        left -= n
    c = dict(x=x, dy=dy, W_up=r(E, d, f, std=d ** -0.5), W_down=r(E, f, d, std=f ** -0.5))
    if swiglu:
        c["W_gate"] = r(E, d, f, std=d ** -0.5)
    return cfg, R, offs, {n: t.to(torch.bfloat16) for n, t in c.items()}


def run_ffn(cfg, R, offs, c):
    cu = {n: t.cuda() for n, t in c.items()}
    o = torch.tensor(offs, dtype=torch.int32).cuda()
    W = cu["W_up"], cu.get("W_gate"), cu["W_down"]
    b = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h = moe.MX8Tensor((cfg.nh, R, cfg.f))
    h.codes.fill_(7)
    h.scales.fill_(9)
    t = dict(y=b(R, cfg.d), act1=b(R, cfg.f), act2=b(R, cfg.f), dh=b(cfg.nh, R, cfg.f), dx=b(R, cfg.d),
             dW_up=torch.empty_like(cu["W_up"]), dW_down=torch.empty_like(cu["W_down"]),
             dW_gate=torch.empty_like(cu["W_gate"]) if "W_gate" in cu else None)
    ws = torch.empty(max(moe.workspace_size(cfg), 256), dtype=torch.uint8, device="cuda")
    moe.moe_grouped_ffn_mx8(cfg, cu["x"], o, *W, h.codes, h.scales, t["act1"], t["y"], ws)
    moe.moe_grouped_ffn_backward_mx8(cfg, cu["x"], o, *W, h.codes, h.scales, t["act2"], cu["dy"], t["dh"], t["dx"],
                                     t["dW_up"], t["dW_gate"], t["dW_down"], ws)
    y, act, hs = b(R, cfg.d), b(R, cfg.f), b(cfg.nh, R, cfg.f)
    moe.moe_grouped_ffn(cfg, cu["x"], o, *W, hs, act, y, ws)
    assert moe.last_device_status() == 0
    n = offs[-1]
    assert torch.equal(t["y"][:n], y[:n]) and torch.equal(t["act1"][:n], act[:n])
    for v in (t["y"], t["act1"], t["act2"], t["dx"]):
        assert (v[n:] == 7.0).all()
    assert (t["dh"][:, n:] == 7.0).all() and (h.codes[:, n:] == 7).all() and (h.scales[:, n:] == 9).all()
    return t, h


def near(got, want, terms, what):
    err = (got.double().cpu() - want).abs()
    tol = HALF * want.abs() + terms
    assert (err <= tol).all(), (what, (err / tol.clamp(min=1e-300)).max().item())


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("T,d,f,E,k", [(1, 128, 128, 1, 1), (2, 128, 256, 4, 2), (300, 256, 384, 3, 1), (700, 384, 256, 5, 2),
                                       (1000, 128, 640, 2, 2)])
def test_grouped_ffn(T, d, f, E, k, swiglu):
    cfg, R, offs, c = ffn_case(T, d, f, E, k, swiglu, seed=T)
    t, h = run_ffn(cfg, R, offs, c)
    kept = [v.cpu().double() for v in h.dequantize(torch.float32)]           # h, or g then u
    v = {n: w.double() for n, w in c.items()}
    act2, dh = t["act2"].cpu().double(), t["dh"].cpu().double()
    for e in range(E):
        a, b = offs[e], offs[e + 1]
        dW = {n: t["d" + n][e] for n in v if n[0] == "W"}
        if a == b:
            assert all((w == 0).all() for w in dW.values())
            continue
        x, dy, W = v["x"][a:b], v["dy"][a:b], {n: w[e] for n, w in v.items() if n[0] == "W"}
        for i, n in enumerate(["W_gate", "W_up"] if swiglu else ["W_up"]):
            want, to = x @ W[n], d * E24 * (x.abs() @ W[n].abs())
            block = lambda q: q.reshape(b - a, -1, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(b - a, f)  # noqa: E731
            tol = to + 2.0 ** -4 * (want.abs() + to) + 2.0 ** -10 * (block(want.abs()) + block(to)) / 224
            assert ((kept[i][a:b] - want).abs() <= tol).all(), n
            assert (kept[i][a:b] != quantize64(want)[1]).float().mean() < 0.01
        g, u = kept[0][a:b], kept[1][a:b] if swiglu else None
        want = act_of(g, u)
        near(t["act2"][a:b], want, 16 * 2.0 ** -22 * want.abs(), "act")
        dact, td = dy @ W["W_down"].t(), d * E24 * (dy.abs() @ W["W_down"].abs().t())
        s = sigmoid(g)
        fac = (s * (1 + g.abs() * (1 - s))) * (1 if u is None else u.abs())   # both terms' magnitudes
        want, wu = dh_of(dact, g, u)
        near(t["dh"][0, a:b], want, td * fac + 16 * 2.0 ** -22 * dact.abs() * fac, "dh")
        if swiglu:
            near(t["dh"][1, a:b], wu, td * (g * s).abs() + 16 * 2.0 ** -22 * wu.abs(), "du")
        # the products, of the stored tensors
        at, dg, du = act2[a:b], dh[0, a:b], dh[1, a:b] if swiglu else None
        n = b - a
        near(dW["W_down"], at.t() @ dy, n * E24 * (at.abs().t() @ dy.abs()), "dW_down")
        near(dW["W_up"], x.t() @ (du if swiglu else dg), n * E24 * (x.abs().t() @ (du if swiglu else dg).abs()), "dW_up")
        want, to = (du if swiglu else dg) @ W["W_up"].t(), (du if swiglu else dg).abs() @ W["W_up"].abs().t()
        if swiglu:
            near(dW["W_gate"], x.t() @ dg, n * E24 * (x.abs().t() @ dg.abs()), "dW_gate")
            want, to = want + dg @ W["W_gate"].t(), to + dg.abs() @ W["W_gate"].abs().t()
        near(t["dx"][a:b], want, cfg.nh * f * E24 * to, "dx")


@pytest.mark.gpu
def test_empty_experts_and_no_rows_at_all():
    cfg, R, offs, c = ffn_case(200, 128, 128, 4, 1, True, empty=(0, 2))
    t, _ = run_ffn(cfg, R, offs, c)
    assert (t["dW_up"][0] == 0).all() and (t["dW_gate"][2] == 0).all() and (t["dW_down"][0] == 0).all()
    t, _ = run_ffn(cfg, R, [0] * 5, c)
    assert all((t[n] == 0).all() for n in ("dW_up", "dW_gate", "dW_down"))


def layer_case(T, d, f, E, k, swiglu, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std)  # noqa: E731
    bf = torch.bfloat16
    w = dict(W_r=r(d, E, std=0.2).to(bf), W_up=r(E, d, f, std=d ** -0.5).to(bf), W_down=r(E, f, d, std=f ** -0.5).to(bf),
             W_gate=r(E, d, f, std=d ** -0.5).to(bf) if swiglu else None, bias=r(E, std=0.1))
    return r(T, d).to(bf).cuda(), {n: None if t is None else t.cuda() for n, t in w.items()}, r(T, d).to(bf).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu,cf,mask", [(True, 0.0, False), (False, 0.8, False), (True, 1.2, True)])
def test_layer_forward_is_the_plain_one_and_gradients_are_near_its(swiglu, cf, mask):
    T, d, f, E, k = 600, 256, 384, 4, 2
    x, w, dout = layer_case(T, d, f, E, k, swiglu)
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU if swiglu else moe.SILU, capacity_factor=cf, aux_coef=0.01)
    token_mask = (torch.arange(T) % 7 != 3).to(torch.uint8).cuda() if mask else None
    plain, layer, ck = moe.MoELayer(cfg), moe.MoELayer(cfg), moe.MoECheckpoint(cfg)
    want = plain.forward(x, **w, token_mask=token_mask).clone()
    gw = plain.backward(dout)
    assert torch.equal(layer.forward(x, **w, token_mask=token_mask, checkpoint=ck), want)
    with pytest.raises(RuntimeError, match="needs a forward"):
        layer.backward(dout)                       # nothing of it is in the layer itself
    dl = torch.zeros(T, E, device="cuda")
    g = layer.backward(dout, checkpoint=ck, dlogits_aux=dl)
    assert moe.last_device_status() == 0
    for n in ("logits", "topk_idx", "gate", "slot_of", "offsets", "kept", "counts", "stats"):
        assert torch.equal(getattr(ck, n), getattr(plain, n)), n
    for n, t in gw.items():
        if t is None:
            assert g[n] is None
            continue
        # an e4m3 number is within 2^-4 of what it stands for, evenly spread: a relative 2-norm of
        # 2^-4 / sqrt 3 at most, and through act and its derivative (h, u: twice) below 2^-3
        rel = ((g[n].double() - t.double()).norm() / t.double().norm()).item()
        assert rel <= 2.0 ** -3, (n, rel)
        assert n == "dbias" or rel > 0


@pytest.mark.gpu
def test_one_layer_serves_two_depths():
    T, d, f, E, k = 500, 128, 256, 4, 2
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU)
    x, w0, dout = layer_case(T, d, f, E, k, True, 1)
    _, w1, _ = layer_case(T, d, f, E, k, True, 2)

    def depths(layers, checkpoints):
        h = layers[0].forward(x, **w0, checkpoint=checkpoints[0]).clone()
        out = layers[1].forward(h, **w1, checkpoint=checkpoints[1]).clone()
        g1 = {n: t.clone() for n, t in layers[1].backward(dout, checkpoint=checkpoints[1]).items()}
        g0 = {n: t.clone() for n, t in layers[0].backward(g1["dx"], checkpoint=checkpoints[0]).items()}
        return [out] + list(g1.values()) + list(g0.values())

    two = depths([moe.MoELayer(cfg), moe.MoELayer(cfg)], [moe.MoECheckpoint(cfg), moe.MoECheckpoint(cfg)])
    one = moe.MoELayer(cfg)
    cks = [moe.MoECheckpoint(cfg), moe.MoECheckpoint(cfg)]
    for t in (one.act, one.y_perm, one.x_perm):
        t.fill_(float("nan"))
    for a, b in zip(two, depths([one, one], cks)):
        assert torch.equal(a, b)
    # captured, and replayed with other inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = depths([one, one], cks)
    x.copy_(torch.randn(T, d, generator=torch.Generator().manual_seed(9)).to(x))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(depths([one, one], [moe.MoECheckpoint(cfg), moe.MoECheckpoint(cfg)]), got):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_checkpoint_is_used_again_and_on_another_stream():
    T, d, f, E, k = 300, 128, 128, 2, 1
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k)
    x, w, dout = layer_case(T, d, f, E, k, False)
    layer, ck = moe.MoELayer(cfg), moe.MoECheckpoint(cfg)
    layer.forward(x, **w, checkpoint=ck)
    a = {n: t.clone() for n, t in layer.backward(dout, checkpoint=ck).items() if t is not None}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer.forward(-x, **w, checkpoint=ck, stream=s)
    layer.forward(x, **w, checkpoint=ck, stream=s)
    b = layer.backward(dout, checkpoint=ck, stream=s)
    s.synchronize()
    for n, t in a.items():
        assert torch.equal(t, b[n]), n
