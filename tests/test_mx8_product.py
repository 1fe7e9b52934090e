"""The experts' grouped product in microscaled 8-bit numbers, over segments of any length.

Tolerance: codes times scales are exact in fp32 and so are their products; a sum of K of
them in fp32 is off by at most K 2^-24 of the sum of the magnitudes (any order), the
activation by a few 2^-22 of its value (and twice that through the product of two), and
the stored value by half a step.  Where the output is in 8 bits again, a value t off is
stored within t + 2^-4 (|v| + t) + 2^-10 s: half a step of its code, or of the smallest
codes at the scale s, which is below (amax + t) / 224.
"""
import ctypes

import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests.test_mx8 import quantize64

ACTS = ["none", "silu", "swiglu"]
OUTS = {"bf16": (moe.BF16, torch.bfloat16), "fp32": (moe.F32, torch.float32), "mx8": (moe.MX8, torch.float32)}


def product64(x, W, Wg, offs, act):
    """Values and the tolerance's terms for the rows of the segments."""
    N, K = W.shape[2], W.shape[1]
    out, terms = torch.zeros(x.shape[0], N).double(), torch.zeros(x.shape[0], N).double()
    for e in range(W.shape[0]):
        a, b = offs[e], offs[e + 1]
        if a == b:
            continue
        xv = quantize64(x[a:b])[1]
        def mul(M):
            w = quantize64(M[e].t())[1].t()
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


def product_case(counts, K, N, act, out, seed=0, slack=5, first=0):
    """``first`` rows before the segments and ``slack`` behind them are of none."""
    E = len(counts)
    g = torch.Generator().manual_seed(seed)
    offs = [first]
    for c in counts:
        offs.append(offs[-1] + c)
    x = torch.randn(offs[-1] + slack, K, generator=g)
    x[:first] = x[offs[-1]:] = float("nan")        # nothing around the segments is looked at
    x = x.to(torch.bfloat16)
    W = (torch.randn(E, K, N, generator=g) * 0.05).to(torch.bfloat16)
    Wg = (torch.randn(E, K, N, generator=g) * 0.05).to(torch.bfloat16) if act == "swiglu" else None
    code, dt = OUTS[out]
    m = moe.MX8Product(moe.MX8ProductConfig(rows=x.shape[0], K=K, N=N, E=E, act=ACTS.index(act), out_dtype=code))
    for t in (m.out.codes, m.out.scales) if out == "mx8" else (m.out,):
        t.fill_(77)
    o = torch.tensor(offs, dtype=torch.int32).cuda()
    res = m.forward(moe.mx8_quantize(x.cuda()), o, moe.mx8_quantize_weight(W.cuda()),
                    moe.mx8_quantize_weight(Wg.cuda()) if Wg is not None else None)
    assert moe.last_device_status() == 0
    for t in (res.codes, res.scales) if out == "mx8" else (res,):
        assert (t[:first] == 77).all() and (t[offs[-1]:] == 77).all()
    if offs[-1] == first:
        return
    got = (res.dequantize(dt) if out == "mx8" else res).cpu().double()[first:offs[-1]]
    want, terms = (t[first:offs[-1]] for t in product64(x, W, Wg, offs, act))
    if out == "mx8":
        block = lambda t: t.reshape(t.shape[0], -1, 32)  # noqa: E731
        s = (block(want).abs().amax(-1, keepdim=True) + block(terms).amax(-1, keepdim=True)) / 224
        s = s.expand(-1, -1, 32).reshape(want.shape)
        tol = terms + 2.0 ** -4 * (want.abs() + terms) + 2.0 ** -10 * s
        # and most values are the very ones that the exact sums round to
        assert (got != quantize64(want)[1]).float().mean() < 0.01
    else:
        tol = torch.finfo(dt).eps / 2 * (1 + 2.0 ** -6) * want.abs() + terms
    err = (got - want).abs()
    assert (err <= tol).all(), ((err / tol.clamp(min=1e-300)).max().item(), (err > tol).float().mean().item())


# ----------------------------------------------------------------- CPU
def test_refusals():
    lib, p, bad = moe.load_library(), ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    ok = dict(rows=256, K=64, N=16, E=2)
    assert moe.check_mx8_product_config(moe.MX8ProductConfig(**ok)) == moe.OK
    for b in (dict(rows=0), dict(K=0), dict(N=0), dict(E=0), dict(act=3), dict(act=-1), dict(out_dtype=3)):
        assert moe.check_mx8_product_config(moe.MX8ProductConfig(**{**ok, **b})) == moe.ERR_INVALID_ARG, b
    for b in (dict(K=40), dict(N=12), dict(E=65), dict(N=2 ** 21 + 8), dict(rows=2 ** 30, N=2 ** 15),
              dict(rows=2 ** 30 + 1), dict(out_dtype=moe.MX8), dict(K=2 ** 20, N=2 ** 20)):
        assert moe.check_mx8_product_config(moe.MX8ProductConfig(**{**ok, **b})) == moe.ERR_UNSUPPORTED, b
    with pytest.raises(moe.MoEError):
        moe.MX8Product(moe.MX8ProductConfig(rows=4, K=33, N=8, E=1), "cpu")
    plain, dual = moe.MX8ProductConfig(**ok), moe.MX8ProductConfig(act=moe.MX8_ACT_SWIGLU, **ok)
    eight = moe.MX8ProductConfig(rows=256, K=64, N=32, E=2, out_dtype=moe.MX8)
    for i in range(9):
        args = [p, p, p, p, p, None, None, p, None]
        args[i] = p if i in (5, 6, 8) else None          # gate weights or output scales that have no place
        assert lib.moe_mx8_grouped_product(ctypes.byref(plain), *args, None) == moe.ERR_INVALID_ARG, i
        args[i] = bad
        assert lib.moe_mx8_grouped_product(ctypes.byref(plain), *args, None) == moe.ERR_INVALID_ARG, i
    for i in range(8):
        args = [p] * 8 + [None]
        args[i] = None
        assert lib.moe_mx8_grouped_product(ctypes.byref(dual), *args, None) == moe.ERR_INVALID_ARG, i
    assert lib.moe_mx8_grouped_product(ctypes.byref(eight), p, p, p, p, p, None, None, p, None, None) == \
        moe.ERR_INVALID_ARG
    m = moe.MX8Product(plain, device="cpu")
    x, w = moe.MX8Tensor((256, 64), "cpu"), moe.MX8Weight((2, 16, 64), "cpu")
    offs = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="x: expected an MX8Tensor"):
        m.forward(torch.zeros(256, 64), offs, w)
    with pytest.raises(ValueError, match="x: expected"):
        m.forward(moe.MX8Tensor((255, 64), "cpu"), offs, w)
    with pytest.raises(ValueError, match="offsets: expected"):
        m.forward(x, offs.long(), w)
    with pytest.raises(ValueError, match="wg is required"):
        m.forward(x, offs, w, w)
    with pytest.raises(ValueError, match="w: expected"):
        m.forward(x, offs, moe.MX8Weight((2, 32, 64), "cpu"))
    with pytest.raises(TypeError, match="w: expected an MX8Weight"):
        m.forward(x, offs, moe.MX8Tensor((2, 16, 64), "cpu"))
    with pytest.raises(ValueError, match="wg: expected"):
        moe.MX8Product(dual, device="cpu").forward(x, offs, w, moe.MX8Weight((2, 32, 64), "cpu"))


# ----------------------------------------------------------------- GPU
@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", list(OUTS))
@pytest.mark.parametrize("K,N", [(32, 128), (128, 256), (512, 128), (1024, 512)])
def test_product(K, N, act, out):
    product_case([100, 0, 301], K, N, act, out, seed=K + N)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 224, 288, 384, 544, 1056])
def test_product_depths(K):
    product_case([3, 129], K, 136, "none", "fp32", seed=K)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [8, 16, 40, 120, 128, 136, 248, 264, 392, 1000])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_product_widths(N, act):
    product_case([1, 0, 200, 5], 288, N, act, "bf16", seed=N)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [32, 64, 96, 160, 224, 288, 1056])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("counts", [[1, 0, 200, 5], [700, 331]])
def test_product_widths_in_8_bits(N, act, counts):
    product_case(counts, 160, N, act, "mx8", seed=N)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[1], [0, 0, 1], [128], [129], [127, 1, 31, 33], [0, 512, 0, 640, 1], [5000], [1] * 64,
                                    [300] * 7, [257] * 3, list(range(64))])
@pytest.mark.parametrize("out", ["bf16", "mx8"])
def test_product_segments(counts, out):
    product_case(counts, 192, 544, "silu", out, seed=len(counts))


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[1], [2, 0, 1], [0, 0, 0, 5], [3, 1]])
@pytest.mark.parametrize("K,N", [(1024, 64), (1056, 136), (2048, 640), (2080, 128), (6048, 1000)])
@pytest.mark.parametrize("act,out", [("none", "fp32"), ("silu", "bf16"), ("swiglu", "bf16"), ("swiglu", "fp32")])
def test_product_of_few_rows_over_long_depths(K, N, counts, act, out):
    """Few tiles: clusters of two or four CTAs share a tile's depth."""
    product_case(counts, K, N, act, out, seed=K + N, slack=0)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[1], [3, 1], [0, 5, 0]])
@pytest.mark.parametrize("K,N", [(8192, 136), (8224, 40), (9056, 520)])
@pytest.mark.parametrize("act,out", [("none", "fp32"), ("swiglu", "bf16")])
def test_product_of_few_rows_over_the_longest_depths(K, N, counts, act, out):
    """Four CTAs a tile, whose shares differ in length."""
    product_case(counts, K, N, act, out, seed=K + N, slack=0)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [4, 0, 0, 0], [2, 0, 1, 1]])
def test_product_that_shares_a_depth_or_not_by_what_rows_name(counts):
    """The launch is sized for four experts of 20 tiles: 80 do not fit the GPU in pairs of CTAs,
    which take them in turn then, fewer do."""
    product_case(counts, 3200, 2560, "none", "bf16", seed=sum(counts) + counts[0], slack=0)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [1024, 4096])
@pytest.mark.parametrize("act", ACTS)
def test_product_of_few_rows_in_8_bits(K, act):
    product_case([3, 1, 0, 2], K, 416, act, "mx8", seed=K, slack=0)


@pytest.mark.gpu
def test_product_many_tiles_of_each_unit():
    """More tiles than the GPU holds at once, so that accumulators alternate."""
    product_case([4001, 2999], 320, 2560, "none", "fp32")
    product_case([4001, 2999], 320, 1312, "swiglu", "mx8")


@pytest.mark.gpu
@pytest.mark.parametrize("K", [32, 96, 224, 288, 1056])
@pytest.mark.parametrize("N,act,out", [(136, "none", "fp32"), (392, "silu", "bf16"), (1000, "swiglu", "bf16"),
                                       (264, "swiglu", "fp32")])
def test_product_long_segments_at_odd_sizes(K, N, act, out):
    """CTA pairs: segments that end in either half of a tile, and in any box of it."""
    product_case([703, 0, 130, 1501, 37], K, N, act, out, seed=K + N)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[40, 50], [900, 811]])
@pytest.mark.parametrize("out", list(OUTS))
def test_product_of_segments_inside_the_rows(counts, out):
    product_case(counts, 96, 96, "none", out, slack=200, first=33)


@pytest.mark.gpu
@pytest.mark.parametrize("first", [0, 100, 256])
def test_product_no_rows_writes_nothing(first):
    product_case([0, 0], 64, 64, "none", "mx8", first=first, slack=256 - first + (first == 256))


@pytest.mark.gpu
def test_product_with_bad_offsets_computes_nothing():
    m = moe.MX8Product(moe.MX8ProductConfig(rows=256, K=64, N=64, E=2))
    w = moe.mx8_quantize_weight(torch.ones(2, 64, 64, device="cuda"))
    x = moe.mx8_quantize(torch.ones(256, 64, device="cuda"))
    for bad in ([0, 128, 257], [128, 0, 128], [-1, 0, 128], [0, 200, 100]):
        m.out.fill_(5.0)
        m.forward(x, torch.tensor(bad, dtype=torch.int32, device="cuda"), w)
        assert (m.out == 5.0).all()
        assert moe.last_device_status() == moe.ERR_DEVICE_BOUNDS, bad


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [200, 1000])
def test_product_nan_rows_stay_in_their_rows(rows):
    """Also where a tile holds rows of the next segment."""
    x = torch.randn(rows, 128, generator=torch.Generator().manual_seed(1))
    W = torch.randn(3, 128, 64, generator=torch.Generator().manual_seed(2))
    W[2, 3, 5] = float("nan")
    m = moe.MX8Product(moe.MX8ProductConfig(rows=rows, K=128, N=64, E=3, out_dtype=moe.F32))
    w, o = moe.mx8_quantize_weight(W.cuda()), torch.tensor([0, 18, rows - 50, rows], dtype=torch.int32).cuda()
    clean = m.forward(moe.mx8_quantize(x.cuda()), o, w).clone()
    assert clean[rows - 50:, 5].isnan().all() and not clean[:rows - 50].isnan().any()
    assert not clean[:, 6:].isnan().any()
    x[17, 40], x[18, 3], x[rows - 50, 0] = float("nan"), float("inf"), float("-inf")
    got = m.forward(moe.mx8_quantize(x.cuda()), o, w)
    bad = [17, 18, rows - 50]
    assert got[bad].isnan().all()
    keep = [i for i in range(rows) if i not in bad]
    assert torch.equal(got[keep].nan_to_num(nan=1e9), clean[keep].nan_to_num(nan=1e9))


@pytest.mark.gpu
def test_repeats_are_identical_on_other_streams_and_in_graphs():
    x = moe.mx8_quantize(torch.randn(384, 256, generator=torch.Generator().manual_seed(1)).cuda())
    w = moe.mx8_quantize_weight(torch.randn(3, 256, 288, generator=torch.Generator().manual_seed(2)).cuda())
    o = torch.tensor([0, 128, 129, 384], dtype=torch.int32).cuda()
    m = moe.MX8Product(moe.MX8ProductConfig(rows=384, K=256, N=288, E=3, out_dtype=moe.MX8))
    a = m.forward(x, o, w).dequantize(torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.out.codes.zero_()
    s.wait_stream(torch.cuda.current_stream())
    b = m.forward(x, o, w, stream=s).dequantize(torch.float32, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(x, o, w)
    # the segments of a later replay are read then
    o.copy_(torch.tensor([0, 0, 300, 384], dtype=torch.int32))
    graph.replay()
    c = m.out.dequantize(torch.float32).clone()
    assert torch.equal(c, m.forward(x, o, w).dequantize(torch.float32)) and not torch.equal(a, c)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 1000])
def test_product_nan_rows_in_8_bits(rows):
    """A row that is no number makes its own blocks so, and nothing else."""
    g = torch.Generator().manual_seed(1)
    x, W = torch.randn(rows, 96, generator=g), torch.randn(2, 96, 160, generator=g)
    m = moe.MX8Product(moe.MX8ProductConfig(rows=rows, K=96, N=160, E=2, act=moe.MX8_ACT_SILU, out_dtype=moe.MX8))
    w, o = moe.mx8_quantize_weight(W.cuda()), torch.tensor([0, 7, rows], dtype=torch.int32).cuda()
    clean = m.forward(moe.mx8_quantize(x.cuda()), o, w).dequantize(torch.float32)
    x[6, 1], x[7, 95] = float("nan"), float("inf")
    out = m.forward(moe.mx8_quantize(x.cuda()), o, w)
    got = out.dequantize(torch.float32)
    assert (out.scales[6:8, :5] == 255).all() and (out.codes[6:8] == 0).all()
    assert got[6:8].isnan().all()
    keep = [i for i in range(rows) if i not in (6, 7)]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "swiglu"])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [64, 700])
def test_activations_far_from_zero(act, out, rows):
    """Gates of up to some thousands, where e^-z leaves fp32's range on either side."""
    K, N = 64, 64
    g = torch.Generator().manual_seed(5)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-8, 9, (rows, 1), generator=g).float())
    W, Wg = torch.randn(1, K, N, generator=g), torch.randn(1, K, N, generator=g)
    code, dt = OUTS[out]
    m = moe.MX8Product(moe.MX8ProductConfig(rows=rows, K=K, N=N, E=1, act=ACTS.index(act), out_dtype=code))
    o = torch.tensor([0, rows], dtype=torch.int32).cuda()
    got = m.forward(moe.mx8_quantize(x.cuda()), o, moe.mx8_quantize_weight(W.cuda()),
                    moe.mx8_quantize_weight(Wg.cuda()) if act == "swiglu" else None).cpu().double()
    want, terms = product64(x, W, Wg, [0, rows], act)
    assert want.abs().max() > 1000 and torch.isfinite(got).all()
    # the quick form (bf16) has e^-z off by up to |z| 2^-24 of it, where |z| stays below 128 (0 beyond)
    tol = torch.finfo(dt).eps / 2 * (1 + 2.0 ** -6) * want.abs() + terms + (128 * 2.0 ** -24 * want.abs() if out == "bf16" else 0)
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol.clamp(min=1e-300)).max()


@pytest.mark.gpu
@pytest.mark.parametrize("out,N", [("fp32", 72), ("bf16", 48), ("bf16", 40), ("mx8", 96)])
@pytest.mark.parametrize("rows", [70, 700])
def test_product_into_memory_of_16_byte_alignment(out, N, rows):
    """An output that is no whole, aligned pieces of 32 bytes is stored in pieces of 16."""
    K, E = 96, 2
    g = torch.Generator().manual_seed(rows)
    x = moe.mx8_quantize(torch.randn(rows, K, generator=g).cuda())
    w = moe.mx8_quantize_weight(torch.randn(E, K, N, generator=g).cuda())
    o = torch.tensor([0, 33, rows], dtype=torch.int32).cuda()
    code, _ = OUTS[out]
    m = moe.MX8Product(moe.MX8ProductConfig(rows=rows, K=K, N=N, E=E, out_dtype=code))
    want = m.forward(x, o, w)
    want = want.codes if out == "mx8" else want
    es = want.element_size()
    raw = torch.full((rows * N + 32 // es,), 7, dtype=want.dtype, device="cuda")
    at = 16 // es                                          # 16 bytes on
    got = raw[at:at + rows * N].view(rows, N)
    assert got.data_ptr() % 32 == 16
    moe.moe_mx8_grouped_product(m.cfg, x.codes, x.scales, o, w.codes, w.scales, None, None, got,
                                m.out.scales if out == "mx8" else None)
    assert torch.equal(got, want) and (raw[:at] == 7).all() and (raw[at + rows * N:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "swiglu"])
@pytest.mark.parametrize("out", ["fp32", "bf16", "mx8"])
@pytest.mark.parametrize("rows,N", [(64, 64), (1000, 2560)])
def test_activations_at_infinity(act, out, rows, N):
    """Sums past fp32's range on either side, and far inside it: silu(inf) is inf,
    silu(-inf) by z / (1 + e^-z) no number, silu(+-2^30) 2^30 and 0, all exactly."""
    K, n = 64, 2.0 ** 70
    a = torch.tensor([n, -n, n ** -1 * 2.0 ** 24, -n ** -1 * 2.0 ** 24]).repeat(rows // 4)
    x = moe.mx8_quantize(a[:, None].expand(rows, K).contiguous().cuda())
    o = torch.tensor([0, rows], dtype=torch.int32).cuda()
    big = moe.mx8_quantize_weight(torch.full((1, K, N), n).cuda())
    up = moe.mx8_quantize_weight(torch.full((1, K, N), 2.0 ** 20).cuda())
    run = lambda act, code, *w: moe.MX8Product(moe.MX8ProductConfig(  # noqa: E731
        rows=rows, K=K, N=N, E=1, act=act, out_dtype=code)).forward(x, o, *w)
    z = run(moe.MX8_ACT_NONE, moe.F32, big).cpu().double()
    assert (z[0::4] == float("inf")).all() and (z[1::4] == -float("inf")).all()
    assert (z[2::4] == 2.0 ** 30).all() and (z[3::4] == -2.0 ** 30).all()
    want = z / (1 + torch.exp(-z))
    if act == "swiglu":
        want = want * (a.double() * K * 2.0 ** 20)[:, None]
    got = run(ACTS.index(act), OUTS[out][0], *((up, big) if act == "swiglu" else (big,)))
    if out == "mx8":                                        # (no block is infinite)
        got, want = got.dequantize(torch.float32), torch.where(want.isinf(), float("nan"), want)
    assert torch.equal(got.cpu().double().nan_to_num(nan=-7.0), want.nan_to_num(nan=-7.0))
