"""The routing that MoELayer.forward_mx8 leaves in the layer is that of its own call."""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests.test_depths import calls  # noqa: F401  (the fixture)

PLACES = ("slot_of", "perm_token", "kept", "offsets")


class Experts:
    def __init__(self, up, down, gate=None):
        self.up, self.down, self.gate = (moe.MX8Weight(s, "cpu") if s else None for s in (up, down, gate))


def test_the_places_are_the_layers(calls):  # noqa: F811
    cfg = moe.MoEConfig(T=8, d=128, f=128, E=2, k=1)
    layer, x = moe.MoELayer(cfg, "cpu"), torch.zeros(8, 128, dtype=torch.bfloat16)
    layer.forward_mx8(x, torch.zeros(128, 2, dtype=torch.bfloat16), Experts((2, 128, 128), (2, 128, 128)))
    (a,) = [a for n, a in calls if n == "moe_permute_mx8"]
    perm_token, slot_of, kept, offsets = a[6:10]
    for n, t in zip(PLACES, (slot_of, perm_token, kept, offsets)):
        assert t.data_ptr() == getattr(layer, n).data_ptr(), n
    assert perm_token.numel() == 8
    (combine,) = [a for n, a in calls if n == "moe_combine"]
    assert combine[2] is layer.slot_of


def test_rows_of_another_shape_or_type_are_refused():
    """The router reads x itself, also where its rows come in 8 bits beside it."""
    layer = moe.MoELayer(moe.MoEConfig(T=8, d=128, f=128, E=2, k=1), "cpu")
    ex, x8 = Experts((2, 128, 128), (2, 128, 128)), moe.MX8Tensor((8, 128), "cpu")
    W_r = torch.zeros(128, 2, dtype=torch.bfloat16)
    for x in (torch.zeros(8, 128), torch.zeros(7, 128, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)):
        for rows in (None, x8):
            with pytest.raises(ValueError, match="^x: expected"):
                layer.forward_mx8(x, W_r, ex, x8=rows)


def test_rows_that_the_call_itself_writes_are_refused(calls):  # noqa: F811
    """Square products one after the other: their tiles would be read and written at once."""
    m = moe.MX8Product(moe.MX8ProductConfig(rows=16, K=64, N=64, E=2, out_dtype=moe.MX8), "cpu")
    w, o = moe.MX8Weight((2, 64, 64), "cpu"), torch.zeros(3, dtype=torch.int32)
    y = m.forward(moe.MX8Tensor((16, 64), "cpu"), o, w)
    with pytest.raises(ValueError, match="writes"):
        m.forward(y, o, w)
    d = moe.MX8Dispatch(moe.MoEConfig(T=16, d=128, f=128, E=2, k=1), "cpu")
    rows = d.forward(moe.MX8Tensor((16, 128), "cpu"), torch.zeros(16, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="writes"):
        d.forward(rows, torch.zeros(16, 1, dtype=torch.int32))
    assert len(calls) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("T,cf", [(40, 0.0), (500, 0.0), (500, 0.7)])
def test_places_after_other_forwards(T, cf):
    d, f, E, k = 128, 256, 4, 2
    g = torch.Generator().manual_seed(T)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, capacity_factor=cf)
    layer, W_r, Wu, Wd = moe.MoELayer(cfg), r(d, E, std=0.3), r(E, d, f, std=0.1), r(E, f, d, std=0.1)
    ex, C = moe.MX8Experts(Wu, Wd), moe.capacity(cfg)
    for i in range(3):
        layer.forward(r(T, d), W_r, Wu, Wd)                  # leaves places of its own, padded
        layer.forward_mx8(r(T, d), W_r, ex)
        topk = layer.topk_idx.cpu().tolist()
        left, kept = [0] * E, [0] * E
        for row in topk:
            for e in row:
                kept[e] += left[e] < C
                left[e] += 1
        offs = [sum(kept[:e]) for e in range(E + 1)]
        slots, tokens, seen = [], [None] * offs[-1], [0] * E
        for t, row in enumerate(topk):
            for e in row:
                slots.append(offs[e] + seen[e] if seen[e] < C else -1)
                if seen[e] < C:
                    tokens[slots[-1]] = t
                seen[e] += 1
        assert layer.kept.tolist() == kept and layer.offsets.tolist() == offs
        assert layer.slot_of.flatten().tolist() == slots and layer.perm_token[:offs[-1]].tolist() == tokens
        assert layer.stats[moe.STAT_DROPPED] == sum(seen) - offs[-1]
    assert moe.last_device_status() == 0
