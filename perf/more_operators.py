"""What is measured of the experts in 8 bits.

Four families, each as a user's program calls it.  Their 8-bit numbers are e4m3
codes with one power-of-two scale for 32 of them along a row:

  norm        the residual stream's norms around a block, with the next block's
              normalised input in 8 bits
  dispatch    rows in 8 bits sorted by the experts that they go to, without padding
  product     the experts' grouped product over such segments, both operands in 8
              bits, its activation in the same pass, its output in 8 bits again or not
  checkpoint  the experts' feed-forward layer and all of its gradients, with what is
              kept in between in 8 bits

``own`` False computes them with elementary torch operations in 32 bits;
``own`` True makes the framework's calls.
"""
import math

import torch

own = False

EPS = 1e-6
RES_SCALE, OUT_SCALE = 1.0, 0.5

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token being decoded: the latency of a stream update between two blocks
        dict(name="norm_decode", op="norm", T=1, d=4096, dtype="bf16", gate="none", leave=1, post=0,
             z=1),
        # a batch of prompts of the widest layer, sandwich norms with a learned channel gate; the
        # 16-bit copy beside the 8-bit one is the router's
        dict(name="norm_prompt", op="norm", T=16384, d=4096, dtype="bf16", gate="channel", leave=1,
             post=1, z=1),
        # a ragged batch in 32 bits, gated per token, at a width of no whole 128
        dict(name="norm_ragged", op="norm", T=1237, d=1056, dtype="fp32", gate="token", leave=1,
             post=1, z=0),
        # a few tokens being decoded
        dict(name="dispatch_decode", op="dispatch", T=17, d=1024, E=4, k=2),
        # a large batch over many experts
        dict(name="dispatch_large", op="dispatch", T=32768, d=2048, E=64, k=8),
        # two tokens being decoded: gate and up of the widest experts, their output ready for down
        dict(name="product_decode", op="product", T=2, E=8, k=2, K=4096, N=14336, act="swiglu",
             out="mx8"),
        # a short prompt at odd sizes, an expert without rows
        dict(name="product_odd", op="product", T=333, E=5, k=2, K=1056, N=1000, act="none",
             out="fp32"),
        # the middle layer's up product for a batch of prompts, its output ready for down
        dict(name="product_prompt", op="product", T=16384, E=8, k=2, K=2048, N=4096, act="silu",
             out="mx8"),
        # the widest layer's down product for a prompt
        dict(name="product_down", op="product", T=4096, E=8, k=2, K=14336, N=4096, act="none",
             out="bf16"),
        # the widest layer's gate and up products for a batch of prompts
        dict(name="product_large", op="product", T=16384, E=8, k=2, K=4096, N=14336, act="swiglu",
             out="bf16"),
        # a small training batch
        dict(name="checkpoint_small", op="checkpoint", T=2048, d=1024, f=2048, E=4, k=2,
             act="silu"),
        # the middle layer's training batch
        dict(name="checkpoint_train", op="checkpoint", T=16384, d=2048, f=4096, E=8, k=2,
             act="swiglu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "dispatch", "product", "product", "checkpoint"])
    if op == "norm":
        d = 32 * _log(rng, 2, 256)
        leave = rng.choice([0, 1, 1, 1])
        return dict(op=op, T=min(_log(rng, 1, 65536), 2 ** 26 // d), d=d,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    gate=rng.choice(["none", "channel", "token", "full"]) if leave else "none",
                    leave=leave, post=rng.choice([0, 1, 1]) if leave else 0, z=rng.choice([0, 1]))
    if op == "dispatch":
        E = _log(rng, 1, 64)
        k, d = rng.randint(1, min(E, 8)), 128 * _log(rng, 1, 64)
        return dict(op=op, T=min(_log(rng, 1, 65536), 2 ** 29 // (d * k)), d=d, E=E, k=k)
    if op == "product":
        out = rng.choice(["bf16", "mx8", "mx8", "fp32"])
        K = 32 * _log(rng, 2, 256)
        N = 32 * _log(rng, 1, 250) if out == "mx8" else 8 * _log(rng, 4, 1000)
        E = _log(rng, 1, 64)
        k = rng.randint(1, min(E, 2))
        E = max(k, min(E, 2 ** 28 // (K * N)))
        T = min(_log(rng, 1, 16384), max(1, 2 ** 39 // (K * N * k)))
        return dict(op=op, T=T, E=E, k=k, K=K, N=N, act=rng.choice(["none", "silu", "swiglu"]), out=out)
    d, f, E = 128 * _log(rng, 1, 16), 128 * _log(rng, 1, 32), _log(rng, 1, 16)
    k = rng.randint(1, min(E, 2))
    return dict(op=op, T=min(_log(rng, 1, 16384), 2 ** 37 // (d * f * k)), d=d, f=f, E=E, k=k,
                act=rng.choice(["silu", "swiglu"]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2 + 1)


def _randn(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def _norm_inputs(case, seed):
    g, T, d, dt = _gen(seed), case["T"], case["d"], _DT[case["dtype"]]
    # the stream's rows differ in size by token, as they do in a deep model
    size = torch.exp(_randn(g, T, 1, std=0.7))
    s = {"x": (_randn(g, T, d) * size).to(dt), "w_pre": _randn(g, d, std=0.1, mean=1.0)}
    if case["leave"]:
        s["u"] = _randn(g, T, d, std=0.8).to(dt)
    if case["post"]:
        s["w_post"] = _randn(g, d, std=0.1, mean=1.0)
    if case["gate"] == "channel":
        s["gate"] = _randn(g, d, std=0.3, mean=0.5)
    elif case["gate"] == "token":
        s["gate"] = torch.rand(T, generator=g, device="cuda")
    elif case["gate"] == "full":
        s["gate"] = torch.rand(T, d, generator=g, device="cuda").to(dt)
    return s


def _dispatch_inputs(case, seed):
    g, T, E = _gen(seed), case["T"], case["E"]
    # some experts are preferred, as in a router that is not balanced yet
    score = _randn(g, T, E, std=1.5) + torch.linspace(1.0, -1.0, E, device="cuda")
    topk = torch.topk(score, case["k"], dim=1).indices.to(torch.int32)
    return {"x": _randn(g, T, case["d"], dtype=torch.bfloat16), "topk": topk.contiguous()}


def _counts(case):
    """Rows of each expert: a skewed share of the T k assignments (the same for every seed of a
    case, so that the outputs keep their shapes)."""
    g, E = _gen(case["T"]), case["E"]
    pref = torch.rand(E, generator=g, device="cuda") + 0.2
    if E > 4:
        pref[E // 2] = 0.0                       # an expert that no token picks
    pick = torch.multinomial(pref, case["T"] * case["k"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=E).tolist()


def _segments(counts, pad):
    offs = [0]
    for c in counts:
        offs.append(offs[-1] + (c + pad - 1) // pad * pad)
    return offs


def _product_inputs(case, seed):
    g = _gen(seed)
    E, K, N = case["E"], case["K"], case["N"]
    offs = _segments(_counts(case), 1)
    s = {"x": _randn(g, offs[-1], K, dtype=torch.bfloat16), "offs": offs,
         "W": _randn(g, E, K, N, std=0.02, dtype=torch.bfloat16)}
    if case["act"] == "swiglu":
        s["Wg"] = _randn(g, E, K, N, std=0.02, dtype=torch.bfloat16)
    return s


def _checkpoint_inputs(case, seed):
    """Rows as the layer's permutation leaves them: segments padded to 128 with zeros."""
    g, E, d, f = _gen(seed), case["E"], case["d"], case["f"]
    counts = _counts(case)
    offs = _segments(counts, 128)
    bound = case["T"] * case["k"] + 127 * E
    real = torch.zeros(bound, 1, dtype=torch.bool, device="cuda")
    for e in range(E):
        real[offs[e]:offs[e] + counts[e]] = True
    s = {"offs": offs, "x": torch.where(real, _randn(g, bound, d), 0.0).to(torch.bfloat16),
         "dy": torch.where(real, _randn(g, bound, d, std=0.5), 0.0).to(torch.bfloat16),
         "W_up": _randn(g, E, d, f, std=0.02, dtype=torch.bfloat16),
         "W_down": _randn(g, E, f, d, std=0.02, dtype=torch.bfloat16)}
    if case["act"] == "swiglu":
        s["W_gate"] = _randn(g, E, d, f, std=0.02, dtype=torch.bfloat16)
    return s


def _offsets(offs):
    return torch.tensor(offs, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    op = case["op"]
    if own:
        import top_routing_expert_moe_gb300 as moe
    if op == "norm":
        s = _norm_inputs(case, seed)
        if own:
            gates = {"none": moe.GATE_NONE, "channel": moe.GATE_CHANNEL, "token": moe.GATE_TOKEN,
                     "full": moe.GATE_FULL}
            s["norm"] = moe.BlockNorm(moe.NormConfig(
                T=case["T"], d=case["d"], dtype=moe.BF16 if case["dtype"] == "bf16" else moe.F32,
                leave=case["leave"], post_norm=case["post"], enter=1, gate=gates[case["gate"]], eps=EPS,
                res_scale=RES_SCALE, out_scale=OUT_SCALE))
    elif op == "dispatch":
        s = _dispatch_inputs(case, seed)
        # the rows are in 8 bits before they are sorted
        x = s.pop("x")
        if own:
            s["x"] = moe.mx8_quantize(x)
            s["dispatch"] = moe.MX8Dispatch(moe.MoEConfig(T=case["T"], d=case["d"], f=128, E=case["E"],
                                                          k=case["k"]))
        else:
            s["x"] = _plain_pack(x)
    elif op == "product":
        s = _product_inputs(case, seed)
        x, W, Wg = s.pop("x"), s.pop("W"), s.pop("Wg", None)
        # rows come in 8 bits, and the weights are quantised once, when a model is loaded
        if own:
            s["x"], s["w"] = moe.mx8_quantize(x), moe.mx8_quantize_weight(W)
            s["wg"] = None if Wg is None else moe.mx8_quantize_weight(Wg)
            s["offsets"] = _offsets(s["offs"])
            s["product"] = moe.MX8Product(moe.MX8ProductConfig(
                rows=x.shape[0], K=case["K"], N=case["N"], E=case["E"],
                act={"none": moe.MX8_ACT_NONE, "silu": moe.MX8_ACT_SILU,
                     "swiglu": moe.MX8_ACT_SWIGLU}[case["act"]],
                out_dtype={"bf16": moe.BF16, "fp32": moe.F32, "mx8": moe.MX8}[case["out"]]))
        else:
            s["x"], s["w"] = _plain_pack(x), _plain_pack(W.transpose(1, 2))
            s["wg"] = None if Wg is None else _plain_pack(Wg.transpose(1, 2))
    else:
        s = _checkpoint_inputs(case, seed)
        if own:
            swiglu = case["act"] == "swiglu"
            cfg = moe.MoEConfig(T=case["T"], d=case["d"], f=case["f"], E=case["E"], k=case["k"],
                                ffn=moe.SWIGLU if swiglu else moe.SILU)
            rows, d, f = s["x"].shape[0], case["d"], case["f"]
            s["cfg"], s["offsets"] = cfg, _offsets(s["offs"])
            s["h"] = moe.MX8Tensor((cfg.nh, rows, f))
            for name, like in (("y", "x"), ("dx", "x"), ("dW_up", "W_up"), ("dW_gate", "W_gate"),
                               ("dW_down", "W_down")):
                s[name] = torch.empty_like(s[like]) if like in s else None
            # the memory of one pass, which all layers of a model share
            s["act"] = torch.empty(rows, f, dtype=torch.bfloat16, device="cuda")
            s["dh"] = torch.empty(cfg.nh, rows, f, dtype=torch.bfloat16, device="cuda")
            s["ws"] = torch.empty(max(moe.workspace_size(cfg), 256), dtype=torch.uint8, device="cuda")
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _plain_pack(x):
    """x [.., K]: e4m3 codes, and one byte b for 32 of them: the scale 2^(b - 127) is the smallest
    that takes the largest magnitude to 448 or below."""
    b = x.float().unflatten(-1, (-1, 32))
    bits = b.abs().amax(-1).contiguous().view(torch.int32)
    byte = torch.clamp(((bits + 0x1FFFFF) >> 23) - 8, min=0)
    code = torch.ldexp(b, (127 - byte)[..., None]).to(torch.float8_e4m3fn)
    return code.flatten(-2), byte.to(torch.uint8)


def _plain_unpack(packed):
    code, byte = packed
    return torch.ldexp(code.float().unflatten(-1, (-1, 32)), (byte.int() - 127)[..., None]).flatten(-2)


def _plain_norm(case, s):
    x = s["x"].float()
    if case["leave"]:
        n = s["u"].float()
        if case["post"]:
            n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + EPS) * s["w_post"]
        if case["gate"] != "none":
            g = s["gate"].float()
            n = n * (g[:, None] if case["gate"] == "token" else g)
        x = RES_SCALE * x + OUT_SCALE * n
    z = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w_pre"]
    dt = s["x"].dtype
    out = {"z8": _plain_unpack(_plain_pack(z)).to(torch.bfloat16)}
    if case["leave"]:
        out["x_out"] = x.to(dt)
    if case["z"]:
        out["z"] = z.to(dt)
    return out


def _plain_dispatch(case, s):
    T, E, k = case["T"], case["E"], case["k"]
    flat = s["topk"].reshape(-1).long()
    order = torch.sort(flat, stable=True).indices          # by expert, tokens ascending
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * k, device=order.device)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    token = order // k
    code, byte = s["x"]
    rows = code.view(torch.uint8)[token].view(torch.float8_e4m3fn), byte[token]
    return {"rows": _plain_unpack(rows).to(torch.bfloat16), "token": token.to(torch.int32),
            "slot": slot.to(torch.int32).view(T, k), "kept": counts.to(torch.int32),
            "offsets": offsets.to(torch.int32)}


def _plain_product(case, s):
    offs, K = s["offs"], case["K"]
    x = _plain_unpack(s["x"])
    out = torch.empty(offs[-1], case["N"], device=x.device)
    for e in range(case["E"]):
        rows = x[offs[e]:offs[e + 1]]
        if not len(rows):
            continue
        u = rows @ _plain_unpack((s["w"][0][e], s["w"][1][e])).t()
        if case["act"] == "silu":
            u = u * torch.sigmoid(u)
        elif case["act"] == "swiglu":
            g = rows @ _plain_unpack((s["wg"][0][e], s["wg"][1][e])).t()
            u = g * torch.sigmoid(g) * u
        out[offs[e]:offs[e + 1]] = u
    if case["out"] == "mx8":
        return _plain_unpack(_plain_pack(out)).to(torch.bfloat16)
    return out.to(_DT[case["out"]])


def _plain_checkpoint(case, s):
    offs, swiglu = s["offs"], case["act"] == "swiglu"
    x, dy = s["x"][:offs[-1]].float(), s["dy"][:offs[-1]].float()
    out = {"y": torch.empty_like(x), "dx": torch.empty_like(x)}
    for name in ("W_up", "W_gate", "W_down"):
        if name in s:
            out["d" + name] = torch.zeros(s[name].shape, device=x.device)
    for e in range(case["E"]):
        a, b = offs[e], offs[e + 1]
        if a == b:
            continue
        xe, dye = x[a:b], dy[a:b]
        Wu, Wd = s["W_up"][e].float(), s["W_down"][e].float()
        u = xe @ Wu
        g = xe @ s["W_gate"][e].float() if swiglu else u
        act = g * torch.sigmoid(g) * (u if swiglu else 1.0)
        out["y"][a:b] = act @ Wd
        # the backward sees what was kept in 8 bits
        g = _plain_unpack(_plain_pack(g))
        u = _plain_unpack(_plain_pack(u)) if swiglu else 1.0
        sg = torch.sigmoid(g)
        out["dW_down"][e] = (g * sg * u).t() @ dye
        dact = dye @ Wd.t()
        dg = dact * u * (sg * (1 + g * (1 - sg)))
        if swiglu:
            du = dact * (g * sg)
            out["dW_gate"][e], out["dW_up"][e] = xe.t() @ dg, xe.t() @ du
            out["dx"][a:b] = du @ Wu.t() + dg @ s["W_gate"][e].float().t()
        else:
            out["dW_up"][e], out["dx"][a:b] = xe.t() @ dg, dg @ Wu.t()
    return {n: t.to(torch.bfloat16) for n, t in out.items()}


# ------------------------------------------------------------------ one pass
def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "dispatch": _plain_dispatch, "product": _plain_product,
                "checkpoint": _plain_checkpoint}[op](case, s)
    import top_routing_expert_moe_gb300 as moe
    if op == "norm":
        y, z8, z = s["norm"].forward_mx8(s["x"], u=s.get("u"), w_pre=s["w_pre"], w_post=s.get("w_post"),
                                         gate=s.get("gate"), keep_z=bool(case["z"]))
        out = {"z8": z8.dequantize(torch.bfloat16)}
        if case["leave"]:
            out["x_out"] = y
        if case["z"]:
            out["z"] = z
        return out
    if op == "dispatch":
        d, n = s["dispatch"], case["T"] * case["k"]
        rows = d.forward(s["x"], s["topk"])
        return {"rows": rows.dequantize(torch.bfloat16)[:n], "token": d.perm_token[:n], "slot": d.slot_of,
                "kept": d.kept, "offsets": d.offsets}
    if op == "product":
        out = s["product"].forward(s["x"], s["offsets"], s["w"], s["wg"])
        return out.dequantize(torch.bfloat16) if case["out"] == "mx8" else out
    n, h = s["offs"][-1], s["h"]
    W = s["W_up"], s.get("W_gate"), s["W_down"]
    moe.moe_grouped_ffn_mx8(s["cfg"], s["x"], s["offsets"], *W, h.codes, h.scales, s["act"], s["y"],
                            s["ws"])
    moe.moe_grouped_ffn_backward_mx8(s["cfg"], s["x"], s["offsets"], *W, h.codes, h.scales, s["act"],
                                     s["dy"], s["dh"], s["dx"], s["dW_up"], s["dW_gate"], s["dW_down"],
                                     s["ws"])
    out = {"y": s["y"][:n], "dx": s["dx"][:n], "dW_up": s["dW_up"], "dW_down": s["dW_down"]}
    if s["dW_gate"] is not None:
        out["dW_gate"] = s["dW_gate"]
    return out


def work(case):
    op = case["op"]
    q = 1 + 1 / 32                                   # bytes of a number in 8 bits with its share of the scale
    if op == "norm":
        es, n = (2 if case["dtype"] == "bf16" else 4), case["T"] * case["d"]
        rows = 1 + 2 * case["leave"] + (case["gate"] == "full") + case["z"]
        b = rows * n * es + (1 + case["post"] + (case["gate"] == "channel")) * case["d"] * 4
        if case["gate"] == "token":
            b += 4 * case["T"]
        # 8-bit numbers written and read again, their values written
        return {"bytes": int(b + n * (2 * q + 2)), "flops": 18 * n}
    if op == "dispatch":
        T, d, r = case["T"], case["d"], case["T"] * case["k"]
        return {"bytes": int(T * d * q + r * d * (2 * q + 2) + 12 * r), "flops": 2 * r * d}
    n = case["T"] * case["k"]
    nw = 2 if case["act"] == "swiglu" else 1
    if op == "product":
        # as many experts' weights are read as the rows can name
        b = n * case["K"] * q + nw * min(case["E"], n) * case["K"] * case["N"] * q
        b += n * case["N"] * {"bf16": 2, "fp32": 4, "mx8": 2 * q + 2}[case["out"]]
        return {"bytes": int(b), "flops": 2 * nw * n * case["K"] * case["N"]}
    d, f, e = case["d"], case["f"], min(case["E"], n)
    # x, dy, y, dx; the weights and their gradients; what is kept, written and read
    b = 8 * n * d + 4 * (nw + 1) * e * d * f + 2 * nw * n * f * q
    return {"bytes": int(b), "flops": 6 * (nw + 1) * n * d * f}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_grid(x):
    """Nearest e4m3 values at each block's scale, ties to the even code."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    m, ex = torch.frexp(top)                          # top = m 2^ex with m in [1/2, 1); 448 = 7/8 2^9
    scale = torch.exp2(torch.clamp(ex.double() - 9 + (m > 0.875).double(), min=-127.0))
    a = b.abs() / scale
    _, ea = torch.frexp(a)                            # spacing 2^(floor(log2 a) - 3), 2^-9 below 2^-6
    step = torch.exp2(torch.clamp(ea.double() - 4, min=-9.0))
    q = torch.round(a / step) * step                  # round() takes ties to even
    return (q * torch.sign(b) * scale).reshape(x.shape)


def _exact_act(case, u, g):
    if case["act"] == "none":
        return u
    return g / (1 + torch.exp(-g)) * (u if case["act"] == "swiglu" else 1.0)


def exact(case, seed):
    op = case["op"]
    if op == "norm":
        return _exact_norm(case, _norm_inputs(case, seed))
    if op == "dispatch":
        return _exact_dispatch(case, _dispatch_inputs(case, seed))
    if op == "checkpoint":
        return _exact_checkpoint(case, _checkpoint_inputs(case, seed))
    s, parts = _product_inputs(case, seed), []
    for e in range(case["E"]):
        x = s["x"][s["offs"][e]:s["offs"][e + 1]]
        if not len(x):
            continue
        x = _exact_grid(x)
        u = x @ _exact_grid(s["W"][e].t()).t()
        g = x @ _exact_grid(s["Wg"][e].t()).t() if case["act"] == "swiglu" else u
        v = _exact_act(case, u, g)
        parts.append(_exact_grid(v) if case["out"] == "mx8" else v)
    return torch.cat(parts)


def _exact_norm(case, s):
    def unit(v):
        return v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS)

    v = {k: t.double() for k, t in s.items()}
    y, out = v["x"], {}
    if case["leave"]:
        b = unit(v["u"]) * v["w_post"] if case["post"] else v["u"]
        if "gate" in v:
            b = b * (v["gate"].unsqueeze(1) if case["gate"] == "token" else v["gate"])
        y = out["x_out"] = RES_SCALE * y + OUT_SCALE * b
    z = unit(y) * v["w_pre"]
    out["z8"] = _exact_grid(z)
    if case["z"]:
        out["z"] = z
    return out


def _exact_dispatch(case, s):
    T, E, k = case["T"], case["E"], case["k"]
    topk, ranks, at = s["topk"].long(), [], 0
    slot = torch.zeros(T, k, dtype=torch.int64, device="cuda")
    offsets = [0]
    for e in range(E):                                # each expert's tokens in their order
        t, j = torch.nonzero(topk == e, as_tuple=True)
        slot[t, j] = at + torch.arange(len(t), device="cuda")
        ranks.append(t)
        at += len(t)
        offsets.append(at)
    token = torch.cat(ranks)
    kept = torch.tensor([b - a for a, b in zip(offsets, offsets[1:])], device="cuda")
    return {"rows": _exact_grid(s["x"])[token], "token": token.to(torch.int32), "slot": slot.to(torch.int32),
            "kept": kept.to(torch.int32), "offsets": _offsets(offsets)}


def _exact_checkpoint(case, s):
    """Gradients by differentiating the layer at the kept values of its hidden rows."""
    swiglu, offs = case["act"] == "swiglu", s["offs"]
    names = ["W_up"] + (["W_gate"] if swiglu else []) + ["W_down"]
    out = {"y": [], "dx": []}
    out.update({"d" + n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in names})
    for e in range(case["E"]):
        a, b = offs[e], offs[e + 1]
        if a == b:
            continue
        x = s["x"][a:b].double().requires_grad_()
        w = {n: s[n][e].double().requires_grad_() for n in names}
        u = x @ w["W_up"]
        g = x @ w["W_gate"] if swiglu else u
        out["y"].append((_exact_act(case, u, g) @ w["W_down"]).detach())
        # values of the kept numbers, with the hidden rows' own dependence on x and W
        u = u + (_exact_grid(u.detach()) - u.detach())
        g = g + (_exact_grid(g.detach()) - g.detach()) if swiglu else u
        total = ((_exact_act(case, u, g) @ w["W_down"]) * s["dy"][a:b].double()).sum()
        grads = torch.autograd.grad(total, [x] + [w[n] for n in names])
        out["dx"].append(grads[0])
        for n, t in zip(names, grads[1:]):
            out["d" + n][e] = t
    return {n: torch.cat(t) if isinstance(t, list) else t for n, t in out.items()}
