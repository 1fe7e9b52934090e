"""The per-sequence balance and z losses against the formulas in 64 bits.

Tolerances.  An fp32 softmax probability carries the errors of one product, the
subtraction of the maximum (2^-24 of the logits' magnitude, at most 40 here, as
an absolute error of the exponent), expf (2 ulp), up to 8 + 5 additions and a
division: C = (2 * 40 + 24) 2^-24 relative.  Means of up to T of them stay
within that plus the sums' 2^-24 per term a lane adds in order (at most 64).
A gradient p (w - <w,p> + c lse) has that C on p and about the same on the
bracket, so 4 C of the magnitudes of its terms; lse has 2^-24 * 50 relative
where it is away from 0, taken on the magnitudes of max and log.
"""
import ctypes

import pytest
import torch

import top_routing_expert_moe_gb300 as moe

C = (2 * 40 + 24) * 2.0 ** -24
BC, ZC = 0.02, 1e-3


def make(T, E, k, S, seed=0, masked=True):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * 2 + torch.linspace(1, -1, E)
    topk = torch.topk(logits, k).indices.to(torch.int32)
    if masked:
        topk[torch.rand(T, generator=g) < 0.25] = -1
    offs = [0] + sorted(torch.randint(0, T + 1, (S - 1,), generator=g).tolist()) + [T]
    return logits, topk, torch.tensor(offs, dtype=torch.int32)


def formulas(logits, topk, offs, tau=1.0):
    """loss [3], counts, pbar, dlogits and the magnitudes of dlogits' terms, in 64 bits."""
    T, E = logits.shape
    k, S = topk.shape[1], len(offs) - 1
    a = logits.double() / tau
    on = topk[:, 0] >= 0
    m = a.max(1, keepdim=True).values
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    ex = torch.exp(a - m)
    z = ex.sum(1, keepdim=True)
    p = torch.where(z > 0, ex / z.clamp(min=1e-300), torch.zeros_like(ex)) * on[:, None]
    lse = torch.where(z > 0, m + torch.log(z.clamp(min=1e-300)), torch.zeros_like(z))[:, 0] * on
    mag = (m.abs()[:, 0] + torch.log(z.clamp(min=1e-300)).abs()[:, 0]) * on
    counts = torch.zeros(S, E, dtype=torch.int64)
    pbar, f, n = torch.zeros(S, E).double(), torch.zeros(S, E).double(), torch.zeros(S).double()
    for s in range(S):
        lo, hi = int(offs[s]), int(offs[s + 1])
        n[s] = on[lo:hi].sum()
        if n[s] == 0:
            continue
        pk = topk[lo:hi][on[lo:hi]]
        counts[s] = torch.bincount(pk[pk >= 0].long(), minlength=E)
        pbar[s] = p[lo:hi].sum(0) / n[s]
        f[s] = E * counts[s] / (k * n[s])
    live, total = max(int((n > 0).sum()), 1), max(float(n.sum()), 1.0)
    bal, zl = BC * (f * pbar).sum() / live, ZC * (lse ** 2).sum() / total
    dl, terms = torch.zeros_like(p), torch.zeros_like(p)
    for s in range(S):
        lo, hi = int(offs[s]), int(offs[s + 1])
        if n[s] == 0:
            continue
        w, q = BC / live * f[s] / n[s], p[lo:hi]
        dot, cz = (q * w).sum(1, keepdim=True), 2 * ZC / total
        dl[lo:hi] = q * (w - dot + cz * lse[lo:hi, None]) / tau
        terms[lo:hi] = q * (w + dot + cz * mag[lo:hi, None]) / tau
    return torch.stack([bal + zl, bal, zl]), counts, pbar, dl, terms


def run(logits, topk, offs, tau=1.0, dloss=None, S=None):
    T, E = logits.shape
    cfg = moe.BalanceConfig(T=T, E=E, k=topk.shape[1], S=S or (len(offs) - 1 if offs is not None else 1),
                            balance_coef=BC, z_coef=ZC, temperature=tau)
    b = moe.BalanceLoss(cfg)
    loss = b.forward(logits.cuda(), topk.cuda(), None if offs is None else offs.cuda())
    dl = b.backward(dloss)
    return loss.cpu().double(), b.counts.cpu(), b.pbar.cpu().double(), dl.cpu().double()


def check(logits, topk, offs, tau=1.0):
    loss, counts, pbar, dl, terms = formulas(logits, topk, offs, tau)
    l, c, p, d = run(logits, topk, offs, tau)
    assert torch.equal(c.long(), counts)
    assert ((p - pbar).abs() <= (C + 64 * 2.0 ** -24) * pbar + 1e-37).all()
    assert ((l - loss).abs() <= 4 * (C + 64 * 2.0 ** -24) * loss.abs() + 1e-12).all()
    assert ((d - dl).abs() <= 4 * C * terms + 1e-30).all()
    assert moe.last_device_status() == 0


# ----------------------------------------------------------------- CPU
def test_formulas_against_differences():
    logits, topk, offs = make(7, 5, 2, 3, seed=3)
    _, _, _, dl, _ = formulas(logits, topk, offs, tau=0.7)
    h = 1e-6
    for t in range(7):
        for e in range(5):
            a, b = logits.double().clone(), logits.double().clone()
            a[t, e] -= h
            b[t, e] += h
            num = (formulas(b, topk, offs, 0.7)[0][0] - formulas(a, topk, offs, 0.7)[0][0]) / (2 * h)
            assert abs(num - dl[t, e]) <= 1e-8 + 1e-6 * abs(dl[t, e])


def test_uniform_router_has_the_closed_form():
    """Equal logits and equal counts: sum_e f P = 1 for each sequence, lse = ln E."""
    topk = torch.arange(8, dtype=torch.int32)[:, None] % 4
    loss, _, pbar, _, _ = formulas(torch.zeros(8, 4), topk, torch.tensor([0, 4, 8]))
    assert abs(loss[1] - BC) < 1e-15 and abs(loss[2] - ZC * torch.log(torch.tensor(4.0).double()) ** 2) < 1e-15
    assert (pbar == 0.25).all()


def test_refusals():
    ok = dict(T=8, E=4, k=2)
    assert moe.check_balance_config(moe.BalanceConfig(**ok)) == moe.OK
    for b in (dict(T=0), dict(E=0), dict(k=0), dict(k=5), dict(S=0), dict(balance_coef=float("nan")),
              dict(z_coef=float("inf")), dict(temperature=-1.0), dict(temperature=float("nan"))):
        assert moe.check_balance_config(moe.BalanceConfig(**{**ok, **b})) == moe.ERR_INVALID_ARG, b
    for b in (dict(E=257), dict(E=64, k=17), dict(S=65537)):
        assert moe.check_balance_config(moe.BalanceConfig(**{**ok, **b})) == moe.ERR_UNSUPPORTED, b
    lib, p = moe.load_library(), ctypes.c_void_p(0x10000)
    c = moe.BalanceConfig(**ok)
    for i in range(8):
        if i == 2:
            continue                       # offsets may be missing where S = 1
        args = [p] * 8
        args[i] = None
        assert lib.moe_balance_loss(ctypes.byref(c), *args, None) == moe.ERR_INVALID_ARG, i
    two = moe.BalanceConfig(S=2, **ok)
    assert lib.moe_balance_loss(ctypes.byref(two), p, p, None, p, p, p, p, p, None) == moe.ERR_INVALID_ARG
    assert lib.moe_balance_loss_backward(ctypes.byref(two), p, p, None, p, None, p, None) == \
        moe.ERR_INVALID_ARG
    b = moe.BalanceLoss(c, device="cpu")
    with pytest.raises(ValueError, match="logits: expected"):
        b.forward(torch.zeros(8, 5), torch.zeros(8, 2, dtype=torch.int32))
    with pytest.raises(RuntimeError, match="forward"):
        b.backward()


# ----------------------------------------------------------------- GPU
@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (4, 2), (5, 3), (8, 8), (13, 2), (16, 2), (31, 4),
                                 (32, 8), (64, 8), (65, 16), (128, 8), (200, 6), (256, 16)])
def test_expert_counts(E, k):
    check(*make(777, E, k, 5, seed=E))


@pytest.mark.gpu
@pytest.mark.parametrize("T,S", [(1, 1), (2, 1), (255, 1), (256, 1), (257, 3), (511, 40), (4096, 16),
                                 (5000, 300), (20011, 7)])
def test_lengths_and_sequences(T, S):
    check(*make(T, 8, 2, S, seed=T), tau=1.0 if T % 2 else 0.5)


@pytest.mark.gpu
def test_whole_batch_needs_no_offsets():
    logits, topk, offs = make(1000, 8, 2, 1, masked=False)
    a, b = run(logits, topk, offs), run(logits, topk, None)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    check(logits, topk, offs)


@pytest.mark.gpu
def test_empty_sequences_and_batches_without_tokens():
    logits, topk, _ = make(600, 6, 2, 1, seed=9)
    check(logits, topk, torch.tensor([0, 0, 0, 300, 300, 600, 600], dtype=torch.int32))
    topk[:300] = -1                        # a sequence of padding only
    check(logits, topk, torch.tensor([0, 300, 600], dtype=torch.int32))
    topk[:] = -1
    l, c, p, d = run(logits, topk, torch.tensor([0, 300, 600], dtype=torch.int32))
    assert not l.any() and not c.any() and not p.any() and not d.any()


@pytest.mark.gpu
def test_masked_experts_and_garbage_in_masked_tokens():
    logits, topk, offs = make(500, 8, 2, 4, seed=2)
    logits[::3, 5] = float("-inf")
    topk[:, 1] = -1                        # one pick only
    on = (topk[:, 0] >= 0).nonzero()[:, 0]
    logits[on[3]] = float("-inf")          # a routed token whose experts are all masked
    check(logits, topk, offs)
    a = run(logits, topk, offs)
    off = topk[:, 0] < 0
    logits[off] = float("nan")             # masked tokens are not looked at
    b = run(logits, topk, offs)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    logits[off] = torch.finfo(torch.float32).min
    check(logits, topk, offs)
    assert moe.last_device_status() == 0


@pytest.mark.gpu
def test_nonfinite_logits_and_bad_indices_are_recorded():
    logits, topk, offs = make(300, 8, 2, 2, masked=False)
    logits[7, 3] = float("inf")
    run(logits, topk, offs)
    assert moe.last_device_status() == moe.ERR_NONFINITE
    logits[7, 3] = 0.0
    ref = run(logits, topk, offs)
    topk[11, 1] = 8                        # no such expert: left out
    got = run(logits, topk, offs)
    assert moe.last_device_status() == moe.ERR_DEVICE_BOUNDS
    assert int((ref[1] - got[1]).abs().sum()) == 1
    topk[11, 1] = 0
    for bad in ([0, 400, 300], [-5, 100, 300], [0, 100, 299], [3, 100, 300]):
        run(logits, topk, torch.tensor(bad, dtype=torch.int32))
        assert moe.last_device_status() == moe.ERR_DEVICE_BOUNDS, bad


@pytest.mark.gpu
def test_upstream_gradient_and_repeats():
    logits, topk, offs = make(3000, 16, 2, 5)
    one = run(logits, topk, offs)
    assert all(torch.equal(a, b) for a, b in zip(one, run(logits, topk, offs)))
    half = run(logits, topk, offs, dloss=torch.tensor([0.5], device="cuda"))
    assert torch.equal(half[3], 0.5 * one[3])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_layer_takes_the_gradient(dtype):
    """The layer's backward with this gradient equals its backward without it plus
    dlogits' own contributions dl W_r^T, x^T dl (the layer's parity bounds)."""
    T, d, f, E, k = 256, 256, 256, 8, 2
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    g = torch.Generator().manual_seed(5)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dt).cuda()  # noqa: E731
    x, Wr = r(T, d), r(d, E, std=0.05)
    Wu, Wd, dout = r(E, d, f, std=0.05), r(E, f, d, std=0.05), r(T, d)
    layer = moe.MoELayer(moe.MoEConfig(T=T, d=d, f=f, E=E, k=k,
                                       dtype=moe.F32 if dtype == "fp32" else moe.BF16))
    bias = torch.zeros(E, device="cuda")
    layer.forward(x, Wr, Wu, Wd, bias=bias)
    b = moe.BalanceLoss(moe.BalanceConfig(T=T, E=E, k=k, S=2, balance_coef=50.0, z_coef=1.0))
    b.forward(layer.logits, layer.topk_idx, torch.tensor([0, 100, T], dtype=torch.int32).cuda())
    dl = b.backward(dloss=torch.full((1,), 100.0, device="cuda"))   # as large as the task's
    base = {n: t.double() for n, t in layer.backward(dout).items() if t is not None}
    got = {n: t.double() for n, t in layer.backward(dout, dlogits_aux=dl).items() if t is not None}
    want = dict(base)
    want["dx"] = base["dx"] + dl.double() @ Wr.double().t()
    want["dW_r"] = base["dW_r"] + x.double().t() @ dl.double()
    want["dbias"] = base["dbias"] + dl.double().sum(0)
    assert (want["dW_r"] - base["dW_r"]).norm() > 0.1 * base["dW_r"].norm()
    for n in want:
        rel = ((got[n] - want[n]).norm() / want[n].norm()).item()
        assert rel <= (1e-5 if dtype == "fp32" else 2e-2), (n, rel)
    with pytest.raises(ValueError, match="dlogits_aux"):
        layer.backward(dout, dlogits_aux=dl[:5])
