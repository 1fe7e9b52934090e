"""The residual stream's norms at the ends of fp32's range: a row's result must not
depend on the kernel that its batch takes, nor lose its gradient where r^3 leaves
the range that r itself is well inside.

Rows whose squares overflow have an infinite sum, so r = 0 in every kernel: their
finite elements give exactly 0 (z, n) or pass the rest through (x', dx).  The other
tolerances are those of test_block_norm.py.
"""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests import test_block_norm as base

pytestmark = pytest.mark.gpu
SIZES = [(10500, 1000), (3700, 2880), (2600, 4104)]     # no multiple of 256 columns: idle threads


def norm_of(v, T, d, dt, form):
    n = moe.BlockNorm(base.config(T, d, dt, *form))
    c = {k: t.cuda() for k, t in v.items()}
    return n, c, {k: c[k] for k in ("u", "w_pre", "w_post", "gate") if k in c}


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SIZES + [(7, 1000), (7, 4104)])
def test_overflowing_and_infinite_rows_entering(T, d, dt):
    form = (0, 0, 1, "none")
    v = base.make(T, d, dt, *form, seed=d)
    v["x"][3, d - 2] = float("inf")                     # in the row's last 16 bytes
    v["x"][4, d - 1] = 1e25                             # its square overflows
    v["x"][5, d // 2] = 1e25
    n, c, args = norm_of(v, T, d, dt, form)
    z = n.forward(c["x"], **args)[1].cpu()
    keep = torch.ones(T, dtype=torch.bool)
    keep[3:6] = False
    y, my, z64, mz = base.forward64(v, *form)
    base.near(z[keep], z64[keep], mz[keep], 64, "z")
    fin = torch.ones(d, dtype=torch.bool)
    fin[d - 2] = False
    assert (z[3, fin] == 0).all() and z[3, d - 2].isnan()
    assert (z[4:6] == 0).all()
    v["x"][3] = 1.0                                     # (an infinity's gradient has no value)
    n, c, args = norm_of(v, T, d, dt, form)
    g = n.backward(c["x"], dx_out=c["dx_out"], dz=c["dz"], **args)
    assert torch.equal(g["dx"][4:6].cpu(), v["dx_out"][4:6])
    w = {k: t[[i for i in range(T) if i not in (4, 5)]] if t.dim() == 2 else t for k, t in v.items()}
    g64, m64 = base.backward64(w, w["x"], *form)
    keep[3] = True
    base.near(g["dx"][keep.cuda()], g64["dx"], m64["dx"], 64, "dx")
    base.near(g["dw_pre"], g64["dw_pre"], m64["dw_pre"], 64 + T, "dw_pre")
    assert moe.last_device_status() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SIZES + [(7, 1000), (7, 4104)])
def test_overflowing_and_infinite_rows_leaving(T, d, dt):
    form = (1, 1, 0, "none")
    v = base.make(T, d, dt, *form, seed=d + 1)
    v["u"][3, d - 3] = float("-inf")
    v["u"][4, d - 1] = -1e25
    n, c, args = norm_of(v, T, d, dt, form)
    x = n.forward(c["x"], **args)[0].cpu()
    fin = torch.ones(d, dtype=torch.bool)
    fin[d - 3] = False
    want = (base.RA * v["x"].float()).to(dt)            # 0.75 x is exact in 32 bits
    assert torch.equal(x[3, fin], want[3, fin]) and x[3, d - 3].isnan()
    assert torch.equal(x[4], want[4])
    v["u"][3] = 1.0
    n, c, args = norm_of(v, T, d, dt, form)
    g = n.backward(c["x"], dx_out=c["dx_out"], **args)
    assert (g["du"][4] == 0).all()
    w = {k: t[[i for i in range(T) if i != 4]] if t.dim() == 2 else t for k, t in v.items()}
    g64, m64 = base.backward64(w, w["x"], *form)
    keep = torch.arange(T) != 4
    base.near(g["du"][keep.cuda()], g64["du"], m64["du"], 64, "du")
    base.near(g["dw_post"], g64["dw_post"], m64["dw_post"], 64 + T, "dw_post")
    assert moe.last_device_status() == 0


@pytest.mark.parametrize("form", [(0, 0, 1, "none"), (1, 0, 1, "none"), (1, 1, 0, "channel"),
                                  (1, 1, 1, "token"), (1, 1, 1, "full")])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(9, 256), (4400, 1000), (400, 1001)])
def test_gradients_where_the_cube_of_r_leaves_the_range(T, d, dt, form, monkeypatch):
    """Zero and tiny rows under a tiny eps (r = 1e15), rows of size 1e15."""
    monkeypatch.setattr(base, "EPS", 1e-30)
    v = base.make(T, d, dt, *form, seed=T)              # row 1 is zero
    for t in (v[n] for n in ("x", "u") if n in v):
        t[3] = (t[3].float() * 1e-16).to(dt)
        t[4] = (t[4].float() * 1e15).to(dt)
    n, c, args = norm_of(v, T, d, dt, form)
    x_out, z = n.forward(c["x"], **args)
    y, my, z64, mz = base.forward64(v, *form)
    if form[0]:
        base.near(x_out, y, my, 64, "x_out")
    if form[2]:
        base.near(z, z64, mz, 64, "z")
    g = n.backward(x_out, dx_out=c["dx_out"], dz=c.get("dz"), **args)
    g64, m64 = base.backward64(v, x_out.cpu(), *form)
    for k in g64:
        base.near(g[k], g64[k], m64[k], 64 + (T if g64[k].shape == (d,) else 0), k)
    assert moe.last_device_status() == 0
