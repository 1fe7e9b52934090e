"""The balance loss where logits are far from zero or at the ends of fp32's range.

A softmax depends on the logits' differences only, so its error may not grow with
their common part: the bounds of test_balance_loss.py hold at any offset.  At a small
temperature the exponent x = (l - max) / tau is as long as p stays normal, |x| <= 88,
and carries five roundings (the difference, 1 / tau, log2 e, their product, the
exponent): (5 * 88 + 24) 2^-24 in place of C.
"""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests import test_balance_loss as base

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("E,k", [(4, 2), (13, 2), (64, 8), (200, 6)])
@pytest.mark.parametrize("offset", [200.0, -1000.0, 1e4])
def test_a_common_offset_cancels(E, k, offset):
    logits, topk, offs = base.make(777, E, k, 5, seed=E)
    base.check(logits + offset, topk, offs)


@pytest.mark.parametrize("E", [4, 64])
def test_small_temperatures(E, monkeypatch):
    monkeypatch.setattr(base, "C", (5 * 88 + 24) * 2.0 ** -24)
    logits, topk, offs = base.make(777, E, 2, 5, seed=E)
    base.check(logits + 30.0, topk, offs, tau=torch.tensor(0.01).item())   # as fp32 holds it


@pytest.mark.parametrize("E", [4, 5, 64])
def test_routed_tokens_of_the_lowest_and_largest_values(E, monkeypatch):
    """Equal logits of any size are a uniform softmax; 3e38 is a number."""
    monkeypatch.setattr(base, "ZC", 0.0)
    logits, topk, offs = base.make(600, E, 2, 4, seed=E, masked=False)
    logits[5] = LOWEST
    logits[6] = LOWEST
    logits[6, 1] = 0.0
    logits[7, 2] = 3e38
    logits[8] = 3e38
    logits[9, 0], logits[9, 1] = 3e38, LOWEST
    logits[10] = float("-inf")
    base.check(logits, topk, offs)
    base.check(logits, topk, offs, tau=0.5)


def test_the_z_loss_of_the_lowest_values_is_infinite_not_a_masked_row():
    logits, topk, offs = base.make(300, 8, 2, 2, masked=False)
    clean = base.formulas(logits, topk, offs)
    logits[5] = LOWEST
    want = base.formulas(logits, topk, offs)
    loss, counts, pbar, dl = base.run(logits, topk, offs)
    assert torch.isinf(loss[2]) and loss[2] > 0
    assert ((loss[1] - want[0][1]).abs() <= 4 * (base.C + 64 * 2.0 ** -24) * want[0][1])
    assert ((pbar - want[2]).abs() <= (base.C + 64 * 2.0 ** -24) * want[2]).all()
    assert ((dl - want[3]).abs() <= 4 * base.C * want[4] + 1e-30).all()
    assert not torch.equal(want[2], clean[2])           # the row counts in P
    assert moe.last_device_status() == 0


@pytest.mark.parametrize("offs", [[0, 200, 100, 300], [0, 250, 20, 260, 300], [0, 300, 0, 300]])
def test_descending_offsets_leave_every_output_zero(offs):
    """Recorded, and nothing of what the workspace held before shows."""
    logits, topk, _ = base.make(300, 8, 2, 1, masked=False)
    o = torch.tensor(offs, dtype=torch.int32)
    for fill in (0, 63, 127):
        b = moe.BalanceLoss(moe.BalanceConfig(T=300, E=8, k=2, S=len(offs) - 1, balance_coef=1.0, z_coef=1.0))
        b.ws.fill_(fill)
        loss = b.forward(logits.cuda(), topk.cuda(), o.cuda())
        dl = b.backward()
        for t in (loss, b.counts, b.pbar, dl):
            assert not t.any()
        assert moe.last_device_status() == moe.ERR_DEVICE_BOUNDS
