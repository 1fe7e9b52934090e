"""Microscaled 4-bit numbers and the experts' grouped product in them.

Quantisation is exact but for its rounding to a code, so codes and scales are
held to the definition in 64 bits, bit for bit.

Tolerance of the product: codes times scales are exact in fp32 and so are their
products; a sum of K of them in fp32 is off by at most K 2^-24 of the sum of the
magnitudes (any order), the activation by a few 2^-22 of its value (and twice
that through the product of two), and the stored value by half a step.
"""
import ctypes

import pytest
import torch

import top_routing_expert_moe_gb300 as moe

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantize64(x):
    """x [rows, K]: the values its 4-bit numbers stand for and the scale bytes."""
    b = x.double().reshape(x.shape[0], -1, 32)
    bad = ~torch.isfinite(b).all(-1)
    amax = torch.where(bad[..., None], torch.zeros_like(b), b).abs().amax(-1)
    _, ex = torch.frexp(amax)                       # amax in [2^(ex-1), 2^ex)
    byte = torch.where(amax > 0, (ex - 1 + 127 - 2).clamp(min=0), torch.zeros_like(ex))
    a = torch.where(bad[..., None], torch.zeros_like(b), b) * torch.exp2((127 - byte).double())[..., None]
    dist = (a.abs()[..., None] - GRID).abs()        # nearest of the eight, ties to the even index
    near = dist == dist.min(-1, keepdim=True).values
    idx = torch.arange(8)
    code = torch.where(near, torch.where(idx % 2 == 0, idx, idx + 100), 1000).min(-1).values % 100
    v = GRID[code] * torch.sign(a) * torch.exp2((byte - 127).double())[..., None]
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    v = torch.where(bad[..., None], torch.full_like(v, float("nan")), v)
    return v.reshape(x.shape), byte


def tiles(byte, rows, K):
    """Scale bytes [rows, K / 32] in the tiles' order (include/moe.h)."""
    rt, kt = (rows + 127) // 128, (K + 127) // 128
    full = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8)
    full[:rows, :K // 32] = byte.to(torch.uint8)
    # [rt, r / 32, r % 32, kt, block] -> [rt, kt, r % 32, r / 32, block]
    return full.reshape(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def rows_of(T, K, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g) * torch.exp(3 * torch.randn(T, 1, generator=g))
    x[:, :32] = torch.randint(-16, 17, (T, 32), generator=g) / 4.0   # ties and saturation
    if T > 2:
        x[1] = 0
        x[2, 32:64] *= 2.0 ** -130                                   # subnormal amax
    return x.to(dt)


# ----------------------------------------------------------------- CPU
def test_the_definition_on_hand_worked_blocks():
    x = torch.zeros(5, 32)
    x[0, :9] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.3, -5.0])   # scale 1
    x[1, :3] = torch.tensor([7.9, 0.1, -6.0])        # scale 1, above the largest code
    x[2, :2] = torch.tensor([1024.0, 100.0])         # scale 2^8
    x[3, 0] = 2.0 ** -140                            # below the smallest scale's grid
    x[4, 0] = float("inf")
    v, byte = quantize64(x)
    assert v[0, :9].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -0.5, -4.0]
    assert v[1, :3].tolist() == [6.0, 0.0, -6.0]
    assert v[2, :2].tolist() == [1024.0, 128.0]
    assert byte[:, 0].tolist() == [127, 127, 135, 0, 255] and v[3].abs().max() == 0 and v[4].isnan().all()


def test_scale_tiles():
    byte = torch.arange(200 * 5).reshape(200, 5) % 251
    t = tiles(byte, 200, 160)
    assert t.numel() == moe.mx4_scale_bytes(200, 160) == 2 * 2 * 512
    for r, b in ((0, 0), (31, 3), (32, 1), (127, 2), (128, 0), (199, 4)):
        i = ((r // 128) * 2 + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
        assert t[i] == byte[r, b]


def test_refusals():
    lib, p, bad = moe.load_library(), ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    n = ctypes.c_size_t()
    assert lib.moe_mx4_scale_bytes(0, 32, ctypes.byref(n)) == moe.ERR_INVALID_ARG
    assert lib.moe_mx4_scale_bytes(4, 48, ctypes.byref(n)) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx4_quantize(moe.BF16, 4, 33, p, None, p, p, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx4_quantize(5, 4, 32, p, None, p, p, None) == moe.ERR_INVALID_ARG
    for i in (0, 2, 3):
        for v in (None, bad):
            args = [p, None, p, p]
            args[i] = v
            assert lib.moe_mx4_quantize(moe.BF16, 4, 32, *args, None) == moe.ERR_INVALID_ARG
    assert lib.moe_mx4_quantize(moe.BF16, 4, 32, p, ctypes.c_void_p(0x10002), p, p, None) == \
        moe.ERR_INVALID_ARG
    assert lib.moe_mx4_quantize_weight(moe.F32, 2, 32, 12, p, p, p, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx4_quantize_weight(moe.F32, 0, 32, 16, p, p, p, None) == moe.ERR_INVALID_ARG
    assert lib.moe_mx4_dequantize(moe.F32, 1, 4, 32, p, None, p, None) == moe.ERR_INVALID_ARG
    ok = dict(rows=256, K=64, N=16, E=2)
    assert moe.check_mx4_product_config(moe.MX4ProductConfig(**ok)) == moe.OK
    for b in (dict(rows=0), dict(K=0), dict(N=0), dict(E=0), dict(act=3), dict(out_dtype=2)):
        assert moe.check_mx4_product_config(moe.MX4ProductConfig(**{**ok, **b})) == moe.ERR_INVALID_ARG, b
    assert lib.moe_mx4_quantize_weight(moe.F32, 1, 32, 2 ** 21 + 8, p, p, p, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_mx4_dequantize(moe.F32, 2 ** 20, 2 ** 20, 32, p, p, p, None) == moe.ERR_UNSUPPORTED
    for b in (dict(K=40), dict(N=12), dict(E=65), dict(N=2 ** 21 + 8), dict(rows=2 ** 30, N=2 ** 15)):
        assert moe.check_mx4_product_config(moe.MX4ProductConfig(**{**ok, **b})) == moe.ERR_UNSUPPORTED, b
    plain, dual = moe.MX4ProductConfig(**ok), moe.MX4ProductConfig(act=moe.MX4_ACT_SWIGLU, **ok)
    for i in range(8):
        args = [p, p, p, p, p, None, None, p]
        args[i] = bad if i in (5, 6) else None
        assert lib.moe_mx4_grouped_product(ctypes.byref(plain), *args, None) == moe.ERR_INVALID_ARG, i
        args = [p] * 8
        args[i] = None
        assert lib.moe_mx4_grouped_product(ctypes.byref(dual), *args, None) == moe.ERR_INVALID_ARG, i
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        moe.mx4_quantize(torch.zeros(4, 32, dtype=torch.float16))
    with pytest.raises(moe.MoEError):
        moe.mx4_quantize(torch.zeros(4, 40))
    m = moe.MX4Product(plain, device="cpu")
    w = moe.MX4Tensor((2, 16, 64), device="cpu")
    offs = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="x: expected"):
        m.forward(torch.zeros(255, 64), offs, w)
    with pytest.raises(ValueError, match="wg is required"):
        m.forward(torch.zeros(256, 64), offs, w, w)
    with pytest.raises(ValueError, match="w: expected"):
        m.forward(torch.zeros(256, 64), offs, moe.MX4Tensor((2, 32, 64), device="cpu"))


# ----------------------------------------------------------------- GPU
def same(a, b):
    return torch.equal(a.nan_to_num(nan=12345.0), b.nan_to_num(nan=12345.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K", [(1, 32), (3, 64), (7, 96), (31, 128), (33, 160), (128, 256),
                                 (129, 288), (257, 1056), (1000, 512), (130, 4096)])
def test_rows(T, K, dt):
    x = rows_of(T, K, dt, seed=T)
    v, byte = quantize64(x)
    q = moe.mx4_quantize(x.cuda())
    assert torch.equal(q.scales.cpu(), tiles(byte, T, K))
    for out in (torch.bfloat16, torch.float32):
        assert same(q.dequantize(out).cpu().double(), v)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,K,N", [(1, 32, 8), (2, 64, 40), (3, 160, 72), (1, 128, 128), (2, 288, 136),
                                   (1, 1056, 200), (5, 96, 320)])
def test_weights(E, K, N, dt):
    W = torch.stack([rows_of(N, K, dt, seed=e).t() for e in range(E)]).contiguous()
    q = moe.mx4_quantize_weight(W.cuda())
    n = moe.mx4_scale_bytes(N, K)
    for e in range(E):
        v, byte = quantize64(W[e].t())
        assert torch.equal(q.scales[e * n:(e + 1) * n].cpu(), tiles(byte, N, K))
        assert same(q.dequantize(torch.float32)[e].cpu().double(), v)


@pytest.mark.gpu
def test_infinities_and_nans_make_their_block_nan():
    x = rows_of(40, 128, torch.float32)
    x[3, 5], x[4, 70], x[5, 127], x[6, 0] = float("nan"), float("inf"), float("-inf"), 3.4e38
    v, byte = quantize64(x)
    q = moe.mx4_quantize(x.cuda())
    assert torch.equal(q.scales.cpu(), tiles(byte, 40, 128))
    assert same(q.dequantize(torch.float32).cpu().double(), v)


@pytest.mark.gpu
def test_rows_used_leaves_the_rest():
    x = rows_of(400, 96, torch.bfloat16).cuda()
    for used in (0, 1, 128, 200, 400, 1000, -3):
        q = moe.MX4Tensor((400, 96))
        q.codes.fill_(7)
        q.scales.fill_(9)
        moe.mx4_quantize(x, torch.tensor([used], dtype=torch.int32).cuda(), q)
        n = min(max(used, 0), 400)
        v, byte = quantize64(x[:n].cpu()) if n else (None, None)
        assert (q.codes[n:] == 7).all()
        up = (n + 127) // 128 * 128
        assert (q.scales[moe.mx4_scale_bytes(max(up, 1), 96) if up else 0:] == 9).all()
        if n:
            full = torch.zeros(up, 3, dtype=torch.int64)
            full[:n] = byte
            assert torch.equal(q.scales[:moe.mx4_scale_bytes(up, 96)].cpu(), tiles(full, up, 96))


def product64(x, W, Wg, offs, act):
    """out and its tolerance's terms for the rows of the segments."""
    N, K = W.shape[2], W.shape[1]
    out, terms = torch.zeros(offs[-1], N).double(), torch.zeros(offs[-1], N).double()
    for e in range(W.shape[0]):
        a, b = offs[e], offs[e + 1]
        if a == b:
            continue
        xv = quantize64(x[a:b])[0]
        def mul(M):
            w = quantize64(M[e].t())[0].t()
            return xv @ w, K * 2.0 ** -24 * (xv.abs() @ w.abs())
        u, tu = mul(W)
        if act == "none":
            out[a:b], terms[a:b] = u, tu
        elif act == "silu":
            s = 1 / (1 + torch.exp(-u))
            out[a:b], terms[a:b] = u * s, 1.1 * tu + 8 * 2.0 ** -22 * (u * s).abs()
        else:
            g, tg = mul(Wg)
            s = g / (1 + torch.exp(-g))
            out[a:b] = s * u
            terms[a:b] = 1.1 * (tg * u.abs() + s.abs() * tu + 1.1 * tg * tu) + 16 * 2.0 ** -22 * (s * u).abs()
    return out, terms


def product_case(counts, K, N, act, out_dt, seed=0, dt=torch.bfloat16, slack=130):
    E = len(counts)
    g = torch.Generator().manual_seed(seed)
    offs = [0]
    for c in counts:
        offs.append(offs[-1] + (c + 127) // 128 * 128)
    x = torch.zeros(offs[-1] + slack, K)
    for e, c in enumerate(counts):
        x[offs[e]:offs[e] + c] = torch.randn(c, K, generator=g)
    x[offs[-1]:] = float("nan")                    # nothing past the segments is looked at
    x = x.to(dt)
    W = (torch.randn(E, K, N, generator=g) * 0.05).to(dt)
    Wg = (torch.randn(E, K, N, generator=g) * 0.05).to(dt) if act == "swiglu" else None
    cfg = moe.MX4ProductConfig(rows=x.shape[0], K=K, N=N, E=E,
                               act=["none", "silu", "swiglu"].index(act),
                               out_dtype=moe.BF16 if out_dt == torch.bfloat16 else moe.F32)
    m = moe.MX4Product(cfg)
    m.out.fill_(77.0)
    o = torch.tensor(offs, dtype=torch.int32).cuda()
    out = m.forward(x.cuda(), o, moe.mx4_quantize_weight(W.cuda()),
                    moe.mx4_quantize_weight(Wg.cuda()) if Wg is not None else None)
    got = out.cpu().double()
    assert moe.last_device_status() == 0
    assert (got[offs[-1]:] == 77.0).all()
    want, terms = product64(x, W, Wg, offs, act)
    tol = torch.finfo(out_dt).eps / 2 * (1 + 2.0 ** -6) * want.abs() + terms
    err = (got[:offs[-1]] - want).abs()
    assert (err <= tol).all(), ((err / tol.clamp(min=1e-300)).max().item(), (err > tol).float().mean().item())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
@pytest.mark.parametrize("out_dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K,N", [(64, 256), (256, 256), (512, 128), (1024, 512)])
def test_product(K, N, act, out_dt):
    product_case([100, 0, 300], K, N, act, out_dt, seed=K + N)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [32, 96, 128, 160, 224, 288, 384, 1056])
def test_product_depths(K):
    product_case([3, 129], K, 136, "none", torch.float32, seed=K)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [8, 16, 40, 120, 128, 136, 248, 264, 392, 1000])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_product_widths(N, act):
    product_case([1, 0, 200, 5], 288, N, act, torch.bfloat16, seed=N)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[1], [0, 0, 1], [128], [129], [0, 512, 0, 640, 1], [5000],
                                    [1] * 64, [300] * 7])
def test_product_segments(counts):
    product_case(counts, 192, 520, "silu", torch.bfloat16, seed=len(counts))


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[1], [2, 0, 1], [0, 0, 0, 5], [3, 1]])
@pytest.mark.parametrize("K,N", [(2048, 64), (2080, 136), (4096, 640), (4128, 128), (6048, 1000)])
@pytest.mark.parametrize("act,out_dt", [("none", torch.float32), ("silu", torch.bfloat16),
                                        ("swiglu", torch.bfloat16), ("swiglu", torch.float32)])
def test_product_of_few_rows_over_long_depths(K, N, counts, act, out_dt):
    """Few tiles: clusters of two or four CTAs share a tile's depth."""
    product_case(counts, K, N, act, out_dt, seed=K + N, slack=127 * len(counts) - sum(-c % 128 for c in counts))


@pytest.mark.gpu
def test_product_many_tiles_of_each_unit():
    """More tiles than the GPU holds at once, so that accumulators alternate."""
    product_case([4000, 3000], 320, 2560, "none", torch.float32)
    product_case([4000, 3000], 320, 1288, "swiglu", torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [32, 96, 224, 288, 1056])
@pytest.mark.parametrize("N,act,out_dt", [(136, "none", torch.float32), (392, "silu", torch.bfloat16),
                                          (1000, "swiglu", torch.bfloat16), (264, "swiglu", torch.float32)])
def test_product_long_segments_at_odd_sizes(K, N, act, out_dt):
    """Segments of two row blocks or more go to CTA pairs; odd numbers of blocks leave one idle."""
    product_case([700, 0, 130, 1500], K, N, act, out_dt, seed=K + N)


@pytest.mark.gpu
def test_product_no_rows_writes_nothing():
    cfg = moe.MX4ProductConfig(rows=256, K=64, N=64, E=2)
    m = moe.MX4Product(cfg)
    m.out.fill_(5.0)
    w = moe.mx4_quantize_weight(torch.ones(2, 64, 64, device="cuda"))
    m.forward(torch.ones(256, 64, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), w)
    assert (m.out == 5.0).all() and moe.last_device_status() == 0


@pytest.mark.gpu
def test_product_with_bad_offsets_computes_nothing():
    cfg = moe.MX4ProductConfig(rows=256, K=64, N=64, E=2)
    m = moe.MX4Product(cfg)
    w = moe.mx4_quantize_weight(torch.ones(2, 64, 64, device="cuda"))
    x = torch.ones(256, 64, device="cuda")
    for bad in ([0, 128, 384], [0, 100, 256], [128, 0, 128], [-128, 0, 128]):
        m.out.fill_(5.0)
        m.forward(x, torch.tensor(bad, dtype=torch.int32, device="cuda"), w)
        assert (m.out == 5.0).all()
        assert moe.last_device_status() == moe.ERR_DEVICE_BOUNDS, bad


@pytest.mark.gpu
def test_product_nan_rows_stay_in_their_rows():
    x = torch.randn(256, 128, generator=torch.Generator().manual_seed(1))
    W = torch.randn(1, 128, 64, generator=torch.Generator().manual_seed(2))
    m = moe.MX4Product(moe.MX4ProductConfig(rows=256, K=128, N=64, E=1, out_dtype=moe.F32))
    w, o = moe.mx4_quantize_weight(W.cuda()), torch.tensor([0, 256], dtype=torch.int32).cuda()
    clean = m.forward(x.cuda(), o, w).clone()
    x[17, 40], x[200, 3] = float("nan"), float("inf")
    got = m.forward(x.cuda(), o, w)
    assert got[[17, 200]].isnan().all()
    keep = [i for i in range(256) if i not in (17, 200)]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.gpu
def test_repeats_are_identical_and_other_streams_work():
    x = torch.randn(384, 256, generator=torch.Generator().manual_seed(1)).cuda()
    w = moe.mx4_quantize_weight(torch.randn(3, 256, 264, generator=torch.Generator().manual_seed(2)).cuda())
    o = torch.tensor([0, 128, 128, 384], dtype=torch.int32).cuda()
    m = moe.MX4Product(moe.MX4ProductConfig(rows=384, K=256, N=264, E=3))
    a = m.forward(x, o, w).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.out.zero_()
        b = m.forward(x, o, w).clone()
    s.synchronize()
    assert torch.equal(a, b)
