"""The expert FFN over offsets that are not moe_permute's: its lanes store h in 8 bits, act and dh
by themselves, where no tensor map bounds them, so such offsets are recorded and nothing is written."""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe

# T = 300, two experts: rows_cap = 300 + 2 x 127 = 554
BAD = ([0, 128, 640], [0, 256, 128], [-128, 0, 128], [0, 100, 300], [0, 128, 1 << 20], [0, 555, 555], [128, 0, 256])


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("kept", [True, False])
def test_bad_offsets_write_nothing(swiglu, kept):
    T, d, f, E = 300, 128, 256, 2
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=1, ffn=moe.SWIGLU if swiglu else moe.SILU)
    R, nh = moe.rows_capacity(cfg), cfg.nh
    assert R == 554
    full = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    W = full(E, d, f), full(E, d, f) if swiglu else None, full(E, f, d)
    x, dy, h8 = full(R, d), full(R, d), moe.MX8Tensor((nh, R, f))
    h8.codes.fill_(7)
    h8.scales.fill_(9)
    h, act, y, dh, dx = full(nh, R, f), full(R, f), full(R, d), full(nh, R, f), full(R, d)
    dW = full(E, d, f), full(E, d, f) if swiglu else None, full(E, f, d)
    ws = torch.empty(max(moe.workspace_size(cfg), 256), dtype=torch.uint8, device="cuda")

    def run(offs):
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")
        if kept:
            moe.moe_grouped_ffn_mx8(cfg, x, o, *W, h8.codes, h8.scales, act, y, ws)
            first = moe.last_device_status()
            moe.moe_grouped_ffn_backward_mx8(cfg, x, o, *W, h8.codes, h8.scales, act, dy, dh, dx, dW[0], dW[1], dW[2], ws)
        else:
            moe.moe_grouped_ffn(cfg, x, o, *W, h, act, y, ws)
            first = moe.last_device_status()
            moe.moe_grouped_ffn_backward(cfg, x, o, *W, h, act, dy, dh, dx, dW[0], dW[1], dW[2], ws)
        return first, moe.last_device_status()

    for bad in BAD:
        assert run(bad) == (moe.ERR_DEVICE_BOUNDS,) * 2, bad
    for t in (h, act, y, dh, dx, *dW):
        assert t is None or (t == 7.0).all()
    assert (h8.codes == 7).all() and (h8.scales == 9).all()
    # segments that moe_permute can make, up to the last row that it may use
    for good in ([0, 0, 0], [0, 256, 512], [0, 512, 512], [0, 0, 512]):
        assert run(good) == (0, 0), good
        assert (y[good[-1]:] == 7.0).all() and not (y[:good[-1]] == 7.0).all() or good[-1] == 0
