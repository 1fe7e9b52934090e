"""Microscaled 8-bit numbers, and the permutation of rows held in them.

Quantisation is exact but for its rounding to a code, so codes and scales are held to
the definition in 64 bits, bit for bit; the permutation moves bytes.
"""
import ctypes

import pytest
import torch

import top_routing_expert_moe_gb300 as moe

# magnitudes of the codes 0..126 (127 is NaN)
GRID = torch.tensor([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)][:127],
                    dtype=torch.float64)


def quantize64(x):
    """x [rows, K]: the codes, the values they stand for, and the scale bytes."""
    b = x.double().reshape(x.shape[0], -1, 32)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    amax = b.abs().amax(-1)
    byte = torch.zeros_like(amax, dtype=torch.int64)
    for s in range(255):                              # the smallest scale that holds amax
        byte += (amax > 448 * 2.0 ** (s - 127)).long()
    a = b.abs() * torch.exp2((127 - byte).double())[..., None]
    hi = torch.searchsorted(GRID, a.contiguous()).clamp(max=126)   # GRID[hi] >= a
    lo = (hi - 1).clamp(min=0)
    up, down = GRID[hi] - a, a - GRID[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    neg = torch.signbit(b) & ~bad[..., None]
    v = GRID[code] * torch.where(neg, -1.0, 1.0) * torch.exp2((byte - 127).double())[..., None]
    v = torch.where(bad[..., None], torch.full_like(v, float("nan")), v)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    code = (code + 128 * neg.long()).to(torch.uint8)
    return code.reshape(x.shape), v.reshape(x.shape), byte.to(torch.uint8)


def rows_of(T, K, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g) * torch.exp(3 * torch.randn(T, 1, generator=g))
    x[:, :32] = torch.randint(-40, 41, (T, 32), generator=g) / 4.0   # ties
    x[:, 0] = 448.0 / 4
    if T > 2:
        x[1] = 0
        x[2, 32:64] *= 2.0 ** -130                                   # subnormal amax
    return x.to(dt)


def weight_blocks(code, byte):
    """Codes [N, K] and scale bytes [N, K / 32] in the blocks' order (include/moe.h)."""
    N, K = code.shape
    nt, kt = (N + 127) // 128, (K + 127) // 128
    c, s = torch.zeros(nt * 128, kt * 128, dtype=torch.uint8), torch.zeros(nt * 128, kt * 4, dtype=torch.uint8)
    c[:N, :K], s[:N, :K // 32] = code, byte
    # [nt, n, kt, k] -> [nt, kt, n, k];  [nt, n / 32, n % 32, kt, block] -> [nt, kt, n % 32, n / 32, block]
    return (c.reshape(nt, 128, kt, 128).permute(0, 2, 1, 3).reshape(-1),
            s.reshape(nt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1))


def same(a, b):
    return torch.equal(a.nan_to_num(nan=12345.0), b.nan_to_num(nan=12345.0))


# ----------------------------------------------------------------- CPU
def test_the_definition_on_hand_worked_blocks():
    x = torch.zeros(6, 32)
    x[0, :7] = torch.tensor([448.0, 1.0, 17.0, 19.0, 18.0, -0.0009765625, 0.0029296875])   # scale 1
    x[1, :2] = torch.tensor([450.0, 1.0])               # above 448: the next scale
    x[2, :2] = torch.tensor([224.0, 223.0])             # 448 of scale 1/2
    x[3, 0] = 2.0 ** -140
    x[4, 0] = float("inf")
    x[5, 0] = 3.4e38
    code, v, byte = quantize64(x)
    # 17 and 19 lie half way between 16, 18 and 20 (even: 16, 20); 2^-10 half way to 2^-9
    assert v[0, :7].tolist() == [448.0, 1.0, 16.0, 20.0, 18.0, 0.0, 0.00390625]
    assert code[0, 0] == 126 and code[0, 1] == 56 and code[0, 5] == 128
    assert v[1, :2].tolist() == [448.0, 1.0] and v[2, :2].tolist() == [224.0, 224.0]
    assert byte[:, 0].tolist() == [127, 128, 126, 0, 255, 247]
    assert v[3, 0] == 0 and v[4].isnan().all() and torch.isfinite(v[5]).all()


def test_pitch():
    for K, p in ((32, 16), (512, 16), (544, 32), (4096, 128), (14336, 448)):
        assert moe.mx8_scale_pitch(K) == p
        assert moe.MX8Tensor((3, K), "cpu").scales.shape == (3, p)
        assert moe.MX8Tensor((2, 3, K), "cpu").scales.shape == (2, 3, p)


def test_weight_blocks():
    N, K = 200, 160
    byte = (torch.arange(N * 5).reshape(N, 5) % 251).to(torch.uint8)
    code = (torch.arange(N * K).reshape(N, K) % 253).to(torch.uint8)
    c, s = weight_blocks(code, byte)
    assert (c.numel(), s.numel()) == moe.mx8_weight_bytes(1, K, N) == (4 * 16384, 4 * 512)
    assert moe.mx8_weight_bytes(3, K, N) == (12 * 16384, 12 * 512)
    for n, k in ((0, 0), (31, 100), (32, 127), (127, 128), (128, 31), (199, 159)):
        b = n // 128 * 2 + k // 128
        assert c[b * 16384 + n % 128 * 128 + k % 128] == code[n, k]
        assert s[b * 512 + n % 32 * 16 + n % 128 // 32 * 4 + k % 128 // 32] == byte[n, k // 32]


def test_refusals():
    lib, p, bad = moe.load_library(), ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    n = ctypes.c_int32()
    assert lib.moe_mx8_scale_pitch(0, ctypes.byref(n)) == moe.ERR_INVALID_ARG
    assert lib.moe_mx8_scale_pitch(48, ctypes.byref(n)) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx8_scale_pitch(2 ** 24 + 32, ctypes.byref(n)) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx8_quantize(moe.BF16, 4, 33, p, None, p, p, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx8_quantize(moe.BF16, 2 ** 31, 32, p, None, p, p, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx8_quantize(5, 4, 32, p, None, p, p, None) == moe.ERR_INVALID_ARG
    for i in (0, 2, 3):
        for v in (None, bad):
            args = [p, None, p, p]
            args[i] = v
            assert lib.moe_mx8_quantize(moe.BF16, 4, 32, *args, None) == moe.ERR_INVALID_ARG
    assert lib.moe_mx8_quantize(moe.BF16, 4, 32, p, ctypes.c_void_p(0x10002), p, p, None) == moe.ERR_INVALID_ARG
    assert lib.moe_mx8_quantize_weight(moe.F32, 2, 32, 12, p, p, p, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx8_quantize_weight(moe.F32, 1, 32, 2 ** 21 + 8, p, p, p, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx8_quantize_weight(moe.F32, 0, 32, 16, p, p, p, None) == moe.ERR_INVALID_ARG
    assert lib.moe_mx8_quantize_weight(moe.F32, 2 ** 12, 2 ** 14, 2 ** 12, p, p, p, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx8_dequantize(moe.F32, 4, 32, p, None, p, None) == moe.ERR_INVALID_ARG
    assert lib.moe_mx8_dequantize_weight(moe.F32, 1, 32, 8, p, None, p, None) == moe.ERR_INVALID_ARG
    assert lib.moe_mx8_dequantize_weight(7, 1, 32, 8, p, p, p, None) == moe.ERR_INVALID_ARG
    assert lib.moe_mx8_dequantize_weight(moe.F32, 1, 32, 12, p, p, p, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx8_weight_bytes(1, 32, 8, None, None) == moe.ERR_INVALID_ARG
    assert lib.moe_mx8_weight_bytes(0, 32, 8, p, p) == moe.ERR_INVALID_ARG
    cfg = moe.MoEConfig(T=8, d=128, f=128, E=2, k=1)
    for i in range(10):
        for v in (None, bad):
            args = [p] * 9 + [None, p]
            args[i if i < 9 else 10] = v
            assert lib.moe_permute_mx8(ctypes.byref(cfg), *args, None) == moe.ERR_INVALID_ARG, i
    assert lib.moe_permute_mx8(ctypes.byref(cfg), *[p] * 9, bad, p, None) == moe.ERR_INVALID_ARG
    odd = moe.MoEConfig(T=8, d=40, f=128, E=2, k=1, dtype=moe.F32)
    assert lib.moe_permute_mx8(ctypes.byref(odd), *[p] * 9, None, p, None) == moe.ERR_UNSUPPORTED
    with pytest.raises(moe.MoEError):
        moe.MX8Dispatch(odd, "cpu")
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        moe.mx8_quantize(torch.zeros(4, 32, dtype=torch.float16))
    with pytest.raises(moe.MoEError):
        moe.mx8_quantize(torch.zeros(4, 40))
    for shape in ((0, 32), (2, 0, 32)):
        with pytest.raises(ValueError, match="1 or more"):
            moe.MX8Tensor(shape, "cpu")
    with pytest.raises(ValueError, match="rows, K"):
        moe.MX8Tensor((32,), "cpu")
    d = moe.MX8Dispatch(cfg, "cpu")
    x, topk = moe.MX8Tensor((8, 128), "cpu"), torch.zeros(8, 1, dtype=torch.int32)
    with pytest.raises(TypeError, match="MX8Tensor"):
        d.forward(torch.zeros(8, 128), topk)
    with pytest.raises(ValueError, match="x: expected"):
        d.forward(moe.MX8Tensor((7, 128), "cpu"), topk)
    with pytest.raises(ValueError, match="topk_idx: expected"):
        d.forward(x, topk.long())
    with pytest.raises(ValueError, match="must live on the GPU"):
        d.forward(x, topk)


# ----------------------------------------------------------------- GPU
@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K", [(1, 32), (3, 64), (7, 96), (31, 128), (33, 160), (128, 256), (129, 288),
                                 (257, 1056), (1000, 512), (130, 4096), (5, 8192), (3, 8224), (2, 20000)])
def test_rows(T, K, dt):
    x = rows_of(T, K, dt, seed=T)
    code, v, byte = quantize64(x)
    q = moe.mx8_quantize(x.cuda())
    assert torch.equal(q.codes.cpu(), code)
    assert torch.equal(q.scales.cpu()[:, :K // 32], byte)
    for out in (torch.bfloat16, torch.float32):
        assert torch.equal(q.dequantize(out).cpu(), v.to(out))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,K,N", [(1, 32, 8), (2, 64, 40), (3, 160, 72), (1, 128, 128), (2, 288, 136), (1, 1056, 200),
                                   (5, 96, 320)])
def test_weights(E, K, N, dt):
    W = torch.stack([rows_of(N, K, dt, seed=e).t() for e in range(E)]).contiguous()
    q = moe.mx8_quantize_weight(W.cuda())
    assert q.shape == (E, N, K)
    codes, scales = q.codes.cpu().reshape(E, -1), q.scales.cpu().reshape(E, -1)
    for e in range(E):
        code, v, byte = quantize64(W[e].t())
        c, s = weight_blocks(code, byte)
        assert torch.equal(codes[e], c) and torch.equal(scales[e], s)
        for out in (torch.bfloat16, torch.float32):
            assert torch.equal(q.dequantize(out)[e].cpu(), v.to(out))


@pytest.mark.gpu
def test_infinities_and_nans_make_their_block_nan():
    x = rows_of(40, 128, torch.float32)
    x[3, 5], x[4, 70], x[5, 127], x[6, 0] = float("nan"), float("inf"), float("-inf"), 3.4e38
    code, v, byte = quantize64(x)
    q = moe.mx8_quantize(x.cuda())
    assert torch.equal(q.scales.cpu()[:, :4], byte) and torch.equal(q.codes.cpu(), code)
    # (3.4e38 stands for 2^128, which fp32 has no number for)
    assert same(q.dequantize(torch.float32).cpu(), v.float())
    W = moe.mx8_quantize_weight(x.t()[None].contiguous().cuda())
    c, s = weight_blocks(code, byte)
    assert torch.equal(W.scales.cpu(), s) and torch.equal(W.codes.cpu(), c)
    assert same(W.dequantize(torch.float32)[0].cpu(), v.float())


@pytest.mark.gpu
def test_rows_used_leaves_the_rest():
    x = rows_of(400, 96, torch.bfloat16).cuda()
    code, _, byte = quantize64(x.cpu())
    for used in (0, 1, 128, 200, 400, 1000, -3):
        q = moe.MX8Tensor((400, 96))
        q.codes.fill_(7)
        q.scales.fill_(9)
        moe.mx8_quantize(x, torch.tensor([used], dtype=torch.int32).cuda(), q)
        n = min(max(used, 0), 400)
        assert (q.codes[n:] == 7).all() and (q.scales[n:] == 9).all()
        assert torch.equal(q.codes[:n].cpu(), code[:n]) and torch.equal(q.scales[:n, :3].cpu(), byte[:n])


def dispatch_reference(topk, E, C):
    """Rows by expert in token order, the first C of each: (perm_token, slot_of, kept, offsets)."""
    token, slot, kept, offs = [], torch.full(topk.shape, -1, dtype=torch.int32), [], [0]
    for e in range(E):
        at = [(t, j) for t in range(topk.shape[0]) for j in range(topk.shape[1]) if topk[t, j] == e][:C]
        for t, j in at:
            slot[t, j] = len(token)
            token.append(t)
        kept.append(len(at))
        offs.append(len(token))
    return token, slot, kept, offs


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,k,cf", [(1, 128, 1, 1, 0.0), (2, 256, 8, 2, 0.0), (17, 1024, 4, 2, 0.0), (255, 128, 3, 3, 0.0),
                                        (256, 256, 64, 8, 0.0), (256, 128, 64, 8, 0.5), (33, 2176, 64, 1, 0.0),
                                        (200, 128, 5, 2, 0.6), (257, 128, 5, 2, 0.6), (700, 384, 7, 3, 1.0),
                                        (1500, 2176, 6, 4, 0.0)])
def test_dispatch(T, d, E, k, cf):
    g = torch.Generator().manual_seed(T)
    topk = torch.topk(torch.randn(T, E, generator=g) + torch.linspace(1, -1, E), k, dim=1).indices.int()
    if T > 10:
        topk[torch.rand(T, generator=g) < 0.1] = -1            # tokens that take part in nothing
    cfg = moe.MoEConfig(T=T, d=d, f=128, E=E, k=k, capacity_factor=cf)
    x = moe.mx8_quantize(rows_of(T, d, torch.bfloat16, T).cuda())
    D = moe.MX8Dispatch(cfg)
    D.rows.codes.fill_(7)
    D.rows.scales.fill_(9)
    D.perm_token.fill_(-5)
    stats = torch.zeros(9 + E, device="cuda")
    rows = D.forward(x, topk.cuda(), stats)
    assert moe.last_device_status() == 0
    token, slot, kept, offs = dispatch_reference(topk, E, moe.capacity(cfg))
    n = offs[-1]
    assert n <= D.rows_cap and D.rows_cap == moe.mx8_rows_capacity(cfg)
    assert D.offsets.tolist() == offs and D.kept.tolist() == kept and torch.equal(D.slot_of.cpu(), slot)
    assert D.perm_token[:n].tolist() == token and (D.perm_token[n:] == -5).all()
    at = torch.tensor(token, dtype=torch.long).cuda()
    assert torch.equal(rows.codes[:n], x.codes[at])
    assert torch.equal(rows.scales[:n, :d // 32], x.scales[at][:, :d // 32])
    assert (rows.codes[n:] == 7).all() and (rows.scales[n:] == 9).all()
    assert stats[moe.STAT_DROPPED] == (topk >= 0).sum() - n


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 300])
def test_dispatch_of_an_expert_that_a_token_names_twice(T):
    """The token takes one row of the expert, and both of its slots point there."""
    topk = torch.tensor([[0, 0], [1, 0], [1, 1], [0, 1]] + [[-1, -1]] * (T - 4), dtype=torch.int32)
    D = moe.MX8Dispatch(moe.MoEConfig(T=T, d=128, f=128, E=2, k=2))
    x = moe.mx8_quantize(rows_of(T, 128, torch.bfloat16).cuda())
    rows = D.forward(x, topk.cuda())
    assert D.slot_of[:4].tolist() == [[0, 0], [3, 1], [4, 4], [2, 5]]
    token = D.perm_token.tolist()
    assert (token[0], token[1], token[2], token[3], token[4], token[5]) == (0, 1, 3, 1, 2, 3)
    assert torch.equal(rows.codes[:6], x.codes[torch.tensor(token[:6]).cuda()])
    # and so does moe_permute, to segments of whole 128s
    L = moe.MoELayer(moe.MoEConfig(T=T, d=128, f=128, E=2, k=2))
    xb = x.dequantize()
    L.perm_token.fill_(2 ** 30)
    moe.moe_permute(L.cfg, xb, topk.cuda(), L.x_perm, L.perm_token, L.slot_of, L.kept, L.offsets, None, L.ws)
    assert L.slot_of[:4].tolist() == [[0, 0], [128, 1], [129, 129], [2, 130]] and L.kept.tolist() == [3, 3]
    assert L.perm_token[:4].tolist() == [0, 1, 3, -1] and L.perm_token[128:132].tolist() == [1, 2, 3, -1]
    assert torch.equal(L.x_perm[:3], xb[[0, 1, 3]]) and (L.x_perm[3:128] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("more", [0, 300])
def test_dispatch_reports_and_drops_an_expert_out_of_range(more):
    topk = torch.tensor([[0], [5], [1], [-7], [1]] + [[-1]] * more, dtype=torch.int32)
    cfg = moe.MoEConfig(T=5 + more, d=128, f=128, E=2, k=1)
    D = moe.MX8Dispatch(cfg)
    D.forward(moe.mx8_quantize(rows_of(5 + more, 128, torch.bfloat16).cuda()), topk.cuda())
    assert moe.last_device_status() == moe.ERR_DEVICE_BOUNDS
    assert D.slot_of[:5].flatten().tolist() == [0, -1, 1, -1, 2] and D.offsets.tolist() == [0, 1, 3]
    assert (D.slot_of[5:] == -1).all()
