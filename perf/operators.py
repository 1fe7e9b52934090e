"""What is measured of the operators around the expert layer.

Three families, each as a user's program calls it:

  norm      the residual stream's norms around a block: the block's output is
            normalised, gated, scaled and added to the stream, and the next
            block's input is normalised, in one pass; and its gradients
  balance   the router's balance and z losses with per-expert counts, per
            sequence, forward and backward
  mx4       microscaled 4-bit numbers (e2m1 codes, one power-of-two scale for
            32 of them): quantisation of activations and expert weights, and
            the grouped product of the experts with both operands in 4 bits

``own`` False computes them with elementary torch operations in 32 bits;
``own`` True makes the framework's calls.
"""
import math

import torch

own = False

EPS = 1e-6
RES_SCALE, OUT_SCALE = 1.0, 0.5
BALANCE_COEF, Z_COEF = 0.01, 1e-3

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token being decoded: the latency of a stream update between two blocks
        dict(name="norm_decode", op="norm_fwd", T=1, d=4096, dtype="bf16", gate="none", leave=1,
             post=0, enter=1),
        # a training batch of the widest layer, sandwich norms with a learned channel gate
        dict(name="norm_train", op="norm_fwd", T=65536, d=4096, dtype="bf16", gate="channel",
             leave=1, post=1, enter=1),
        # its gradients
        dict(name="norm_train_grad", op="norm_bwd", T=65536, d=4096, dtype="bf16", gate="channel",
             leave=1, post=1, enter=1),
        # a ragged batch in 32 bits at an odd width (no 16-byte rows), gated per token
        dict(name="norm_ragged_grad", op="norm_bwd", T=1237, d=1001, dtype="fp32", gate="token",
             leave=1, post=1, enter=1),
        # a small training batch, one sequence, four experts
        dict(name="balance_small", op="balance", T=2048, E=4, k=2, S=1, masked=0),
        # a large batch of ragged sequences with padding tokens and many experts
        dict(name="balance_large", op="balance", T=65536, E=64, k=8, S=37, masked=1),
        # a prompt's activations before a product in 4 bits
        dict(name="quantize_rows", op="quantize", form="rows", rows=5003, K=4096, dtype="bf16"),
        # the experts' weights when a model is loaded
        dict(name="quantize_weights", op="quantize", form="weights", E=8, K=2048, N=4096,
             dtype="bf16"),
        # two tokens being decoded: the gate and up products of the widest experts
        dict(name="product_decode", op="product", T=2, E=8, k=2, K=4096, N=14336, act="swiglu",
             out="bf16"),
        # a short prompt at odd sizes, an expert without rows
        dict(name="product_odd", op="product", T=333, E=5, k=2, K=1056, N=1000, act="none",
             out="fp32"),
        # the middle layer's up product for a batch of prompts
        dict(name="product_prompt", op="product", T=16384, E=8, k=2, K=2048, N=4096, act="silu",
             out="bf16"),
        # the widest layer's gate and up products for a batch of prompts
        dict(name="product_large", op="product", T=16384, E=8, k=2, K=4096, N=14336, act="swiglu",
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "balance", "quantize", "product"])
    if op in ("norm_fwd", "norm_bwd"):
        d = _log(rng, 40, 8192)
        if rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        T = min(_log(rng, 1, 65536), 65536 * 2048 // d)
        leave = rng.choice([0, 1, 1, 1])
        return dict(op=op, T=T, d=d, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    gate=rng.choice(["none", "channel", "token", "full"]) if leave else "none",
                    leave=leave, post=rng.choice([0, 1, 1]) if leave else 0,
                    enter=rng.choice([0, 1, 1]) if leave else 1)
    if op == "balance":
        E = _log(rng, 2, 256)
        k = rng.randint(1, min(E, 8))
        T = min(_log(rng, 1, 100000), 65536 * 64 // E)
        return dict(op=op, T=T, E=E, k=k, S=min(T, _log(rng, 1, 64)), masked=rng.choice([0, 1]))
    if op == "quantize":
        K = 32 * _log(rng, 1, 300)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        if rng.random() < 0.5:
            return dict(op=op, form="rows", rows=min(_log(rng, 1, 20000), 2 ** 25 // K), K=K,
                        dtype=dtype)
        N = 8 * _log(rng, 1, 800)
        return dict(op=op, form="weights", E=max(1, min(rng.randint(1, 16), 2 ** 26 // (K * N))),
                    K=K, N=N, dtype=dtype)
    K, N = 32 * _log(rng, 2, 256), 8 * _log(rng, 4, 1000)
    E = rng.randint(1, 12)
    k = rng.randint(1, min(E, 2))
    T = min(_log(rng, 1, 16384), max(1, 2 ** 39 // (K * N * k)))
    act = rng.choice(["none", "silu", "swiglu"])
    return dict(op=op, T=T, E=E, k=k, K=K, N=N, act=act, out=rng.choice(["bf16", "bf16", "fp32"]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2 + 1)


def _randn(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def _norm_inputs(case, seed):
    g, T, d, dt = _gen(seed), case["T"], case["d"], _DT[case["dtype"]]
    # the stream's rows differ in size by token, as they do in a deep model
    size = torch.exp(_randn(g, T, 1, std=0.7))
    s = {"x": (_randn(g, T, d) * size).to(dt)}
    if case["leave"]:
        s["u"] = _randn(g, T, d, std=0.8).to(dt)
    if case["post"]:
        s["w_post"] = _randn(g, d, std=0.1, mean=1.0)
    if case["enter"]:
        s["w_pre"] = _randn(g, d, std=0.1, mean=1.0)
    if case["gate"] == "channel":
        s["gate"] = _randn(g, d, std=0.3, mean=0.5)
    elif case["gate"] == "token":
        s["gate"] = torch.rand(T, generator=g, device="cuda")
    elif case["gate"] == "full":
        s["gate"] = torch.rand(T, d, generator=g, device="cuda").to(dt)
    if case["op"] == "norm_bwd":
        s["dx_out"] = _randn(g, T, d).to(dt)
        if case["enter"]:
            s["dz"] = _randn(g, T, d).to(dt)
        # the stream after the block, as the forward pass stored it
        s["x_out"] = _norm_plain_forward(case, s)[0].to(dt) if case["leave"] else s["x"]
    return s


def _balance_inputs(case, seed):
    g, T, E, k, S = _gen(seed), case["T"], case["E"], case["k"], case["S"]
    # some experts are preferred, as in a router that is not balanced yet
    logits = _randn(g, T, E, std=1.5) + torch.linspace(1.0, -1.0, E, device="cuda")
    topk = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    if case["masked"]:
        topk[torch.rand(T, generator=g, device="cuda") < 0.2] = -1   # padding tokens
    cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda")).values
    offs = torch.cat([torch.zeros(1, device="cuda"), cuts, torch.full((1,), T, device="cuda")])
    return {"logits": logits.contiguous(), "topk": topk.contiguous(),
            "seq_offsets": offs.to(torch.int32)}


def _quantize_inputs(case, seed):
    g, dt = _gen(seed), _DT[case["dtype"]]
    if case["form"] == "rows":
        size = torch.exp(_randn(g, case["rows"], 1))
        return {"x": (_randn(g, case["rows"], case["K"]) * size).to(dt)}
    return {"W": _randn(g, case["E"], case["K"], case["N"], std=0.02).to(dt)}


def _segments(case):
    """Rows of each expert: a skewed share of the T k assignments, padded to 128 (the same for
    every seed of a case, so that the output keeps its shape)."""
    g = _gen(case["T"])
    E, n = case["E"], case["T"] * case["k"]
    pref = torch.rand(E, generator=g, device="cuda") + 0.2
    if E > 4:
        pref[E // 2] = 0.0                       # an expert that no token picks
    pick = torch.multinomial(pref, n, replacement=True, generator=g)
    counts = torch.bincount(pick, minlength=E).tolist()
    offs = [0]
    for c in counts:
        offs.append(offs[-1] + (c + 127) // 128 * 128)
    return counts, offs


def _product_inputs(case, seed):
    g = _gen(seed)
    E, K, N = case["E"], case["K"], case["N"]
    counts, offs = _segments(case)
    x = torch.zeros(case["T"] * case["k"] + 127 * E, K, dtype=torch.bfloat16, device="cuda")
    for e in range(E):                            # rows past an expert's count are zeros
        x[offs[e]:offs[e] + counts[e]] = _randn(g, counts[e], K).to(torch.bfloat16)
    s = {"x": x, "offs": offs, "offsets": torch.tensor(offs, dtype=torch.int32, device="cuda")}
    s["W"] = _randn(g, E, K, N, std=0.02).to(torch.bfloat16)
    if case["act"] == "swiglu":
        s["Wg"] = _randn(g, E, K, N, std=0.02).to(torch.bfloat16)
    return s


def prepare(case, seed):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        s = _norm_inputs(case, seed)
        if own:
            import top_routing_expert_moe_gb300 as moe
            gates = {"none": moe.GATE_NONE, "channel": moe.GATE_CHANNEL, "token": moe.GATE_TOKEN,
                     "full": moe.GATE_FULL}
            s["norm"] = moe.BlockNorm(moe.NormConfig(
                T=case["T"], d=case["d"], dtype=moe.BF16 if case["dtype"] == "bf16" else moe.F32,
                leave=case["leave"], post_norm=case["post"], enter=case["enter"],
                gate=gates[case["gate"]], eps=EPS, res_scale=RES_SCALE, out_scale=OUT_SCALE))
    elif op == "balance":
        s = _balance_inputs(case, seed)
        if own:
            import top_routing_expert_moe_gb300 as moe
            s["loss"] = moe.BalanceLoss(moe.BalanceConfig(
                T=case["T"], E=case["E"], k=case["k"], S=case["S"], balance_coef=BALANCE_COEF,
                z_coef=Z_COEF))
    elif op == "quantize":
        s = _quantize_inputs(case, seed)
    else:
        s = _product_inputs(case, seed)
        if own:
            import top_routing_expert_moe_gb300 as moe
            # the weights are quantised once, when a model is loaded
            s["w"] = moe.mx4_quantize_weight(s.pop("W"))
            s["wg"] = moe.mx4_quantize_weight(s.pop("Wg")) if "Wg" in s else None
            s["product"] = moe.MX4Product(moe.MX4ProductConfig(
                rows=s["x"].shape[0], K=case["K"], N=case["N"], E=case["E"],
                act={"none": moe.MX4_ACT_NONE, "silu": moe.MX4_ACT_SILU,
                     "swiglu": moe.MX4_ACT_SWIGLU}[case["act"]],
                out_dtype=moe.BF16 if case["out"] == "bf16" else moe.F32))
        else:
            for name in ("W", "Wg"):
                if name in s:
                    s[name] = _plain_pack(s[name].transpose(1, 2))
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _norm_plain_forward(case, s):
    x = s["x"].float()
    if case["leave"]:
        n = s["u"].float()
        if case["post"]:
            n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + EPS) * s["w_post"]
        y = RES_SCALE * x + OUT_SCALE * _gated(case, s, n)
    else:
        y = x
    z = None
    if case["enter"]:
        z = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["w_pre"]
    return y, z


def _gated(case, s, n):
    if case["gate"] == "none":
        return n
    g = s["gate"].float()
    return n * (g[:, None] if case["gate"] == "token" else g)


def _norm_plain_backward(case, s):
    out, dt = {}, s["x"].dtype
    y, G = s["x_out"].float(), s["dx_out"].float()
    d = case["d"]
    if case["enter"]:
        dz = s["dz"].float()
        r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        a = dz * s["w_pre"]
        G = G + r * a - y * (r ** 3 / d) * (a * y).sum(-1, keepdim=True)
        out["dw_pre"] = (dz * (y * r)).sum(0)
    if not case["leave"]:
        out["dx"] = G.to(dt)
        return out
    out["dx"] = (RES_SCALE * G).to(dt)
    u = s["u"].float()
    if case["post"]:
        ru = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
        n = u * ru * s["w_post"]
    else:
        n = u
    dn = _gated(case, s, OUT_SCALE * G)
    dg = OUT_SCALE * G * n
    if case["gate"] == "channel":
        out["dgate"] = dg.sum(0)
    elif case["gate"] == "token":
        out["dgate"] = dg.sum(1)
    elif case["gate"] == "full":
        out["dgate"] = dg.to(dt)
    if case["post"]:
        b = dn * s["w_post"]
        out["du"] = (ru * b - u * (ru ** 3 / d) * (b * u).sum(-1, keepdim=True)).to(dt)
        out["dw_post"] = (dn * (u * ru)).sum(0)
    else:
        out["du"] = dn.to(dt)
    return out


def _balance_plain(case, s):
    l, topk, offs = s["logits"], s["topk"].long(), s["seq_offsets"].long()
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    valid = topk[:, 0] >= 0
    seq = torch.searchsorted(offs[1:], torch.arange(T, device=l.device), right=True)
    m = l.max(1, keepdim=True).values
    ex = torch.exp(l - m)
    z = ex.sum(1, keepdim=True)
    p = ex / z * valid[:, None]
    lse = (m + torch.log(z))[:, 0] * valid
    # sums over tokens in 64 bits (long sums)
    one = torch.zeros(S, T, dtype=torch.float64, device=l.device) if S * T <= 2 ** 24 else None
    if one is not None:
        one[seq, torch.arange(T, device=l.device)] = 1.0
        n, psum = one @ valid.double(), one @ p.double()
    else:
        n = torch.zeros(S, dtype=torch.float64, device=l.device).index_add_(0, seq, valid.double())
        psum = torch.zeros(S, E, dtype=torch.float64, device=l.device).index_add_(0, seq, p.double())
    flat = (seq[:, None] * E + topk)[topk >= 0]
    counts = torch.bincount(flat, minlength=S * E).view(S, E)
    live = n > 0
    nseq = torch.clamp(live.sum(), min=1)
    ns = torch.clamp(n, min=1.0)
    pbar = psum / ns[:, None]
    f = counts * (E / (k * ns))[:, None]
    bal = BALANCE_COEF * (f * pbar).sum() / nseq
    n_all = torch.clamp(n.sum(), min=1.0)
    zl = Z_COEF * (lse.double() ** 2).sum() / n_all
    w = (BALANCE_COEF / nseq * f / ns[:, None]).float()[seq]      # d balance / d p
    dl = p * (w - (w * p).sum(1, keepdim=True)) + (2 * Z_COEF / n_all).float() * lse[:, None] * p
    return {"loss": torch.stack([bal + zl, bal, zl]).float(), "counts": counts.to(torch.int32),
            "pbar": pbar.float(), "dlogits": dl}


def _plain_codes(x):
    """x [.., K]: codes 0..15 (sign, then the magnitude's index) and scale bytes."""
    b = x.float().unflatten(-1, (-1, 32))
    e = b.abs().amax(-1).contiguous().view(torch.int32) >> 23
    byte = torch.where(e == 255, e, torch.clamp(e - 2, min=0))
    m = torch.ldexp(b, (127 - byte)[..., None])
    a = m.abs()
    mag = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
           + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    code = torch.where(m < 0, mag + 8, mag)
    return code.flatten(-2), byte.to(torch.uint8)


def _plain_values(code, byte):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    v = torch.cat([grid, -grid])[code.int()].unflatten(-1, (-1, 32))
    e = byte.int()
    v = torch.ldexp(v, (e - 127)[..., None])
    return torch.where((e == 255)[..., None], float("nan"), v).flatten(-2)


def _plain_pack(x):
    code, byte = _plain_codes(x)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte


def _plain_unpack(packed, byte):
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    return _plain_values(code, byte)


def _product_plain(case, s):
    offs = s["offs"]
    out = torch.empty(offs[-1], case["N"], dtype=_DT[case["out"]], device="cuda")
    for e in range(case["E"]):
        a, b = offs[e], offs[e + 1]
        if a == b:
            continue
        x = _plain_values(*_plain_codes(s["x"][a:b]))
        u = x @ _plain_unpack(s["W"][0][e], s["W"][1][e]).t()
        if case["act"] == "silu":
            u = u * torch.sigmoid(u)
        elif case["act"] == "swiglu":
            g = x @ _plain_unpack(s["Wg"][0][e], s["Wg"][1][e]).t()
            u = g * torch.sigmoid(g) * u
        out[a:b] = u.to(out.dtype)
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if op == "norm_fwd":
        if own:
            y, z = s["norm"].forward(s["x"], u=s.get("u"), w_pre=s.get("w_pre"),
                                     w_post=s.get("w_post"), gate=s.get("gate"))
        else:
            y, z = _norm_plain_forward(case, s)
            y, z = y.to(s["x"].dtype), None if z is None else z.to(s["x"].dtype)
        out = {}
        if case["leave"]:
            out["x_out"] = y
        if case["enter"]:
            out["z"] = z
        return out
    if op == "norm_bwd":
        if not own:
            return _norm_plain_backward(case, s)
        g = s["norm"].backward(s["x_out"], dx_out=s["dx_out"], dz=s.get("dz"), u=s.get("u"),
                               w_pre=s.get("w_pre"), w_post=s.get("w_post"), gate=s.get("gate"))
        return {k: v for k, v in g.items() if v is not None}
    if op == "balance":
        if not own:
            return _balance_plain(case, s)
        bl = s["loss"]
        loss = bl.forward(s["logits"], s["topk"], s["seq_offsets"])
        dl = bl.backward()
        return {"loss": loss, "counts": bl.counts, "pbar": bl.pbar, "dlogits": dl}
    if op == "quantize":
        if not own:
            if case["form"] == "rows":
                return _plain_unpack(*_plain_pack(s["x"])).to(s["x"].dtype)
            return _plain_unpack(*_plain_pack(s["W"].transpose(1, 2))).to(s["W"].dtype)
        import top_routing_expert_moe_gb300 as moe
        if case["form"] == "rows":
            return moe.mx4_quantize(s["x"]).dequantize(s["x"].dtype)
        return moe.mx4_quantize_weight(s["W"]).dequantize(s["W"].dtype)
    if not own:
        return _product_plain(case, s)
    out = s["product"].forward(s["x"], s["offsets"], s["w"], s["wg"])
    return out[:s["offs"][-1]]


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        es, n = (2 if case["dtype"] == "bf16" else 4), case["T"] * case["d"]
        vecs = case["post"] + case["enter"] + (case["gate"] == "channel")
        full = case["gate"] == "full"
        if op == "norm_fwd":
            rows = 1 + 2 * case["leave"] + case["enter"] + full
            b = rows * n * es + vecs * case["d"] * 4
        else:
            # x_out only where it is normalised, u only where the gate or the norm needs it
            need_u = case["leave"] and (case["post"] or case["gate"] != "none")
            rows = 1 + 2 * case["enter"] + 1 + case["leave"] + bool(need_u) + 2 * full
            b = rows * n * es + 2 * vecs * case["d"] * 4
        if case["gate"] == "token":
            b += 4 * case["T"] * (1 if op == "norm_fwd" else 2)
        return {"bytes": b, "flops": n * (12 if op == "norm_fwd" else 24)}
    if op == "balance":
        T, E = case["T"], case["E"]
        return {"bytes": 8 * T * E + 4 * T * case["k"] + 8 * case["S"] * E, "flops": 12 * T * E}
    if op == "quantize":
        n = case["rows"] * case["K"] if case["form"] == "rows" else case["E"] * case["K"] * case["N"]
        es = 2 if case["dtype"] == "bf16" else 4
        # read, codes and scales written and read again, values written
        return {"bytes": int(n * (2 * es + 2 * (0.5 + 1 / 32))), "flops": 6 * n}
    n = case["T"] * case["k"]
    nw = 2 if case["act"] == "swiglu" else 1
    # as many experts' weights are read as the rows can name
    e = min(case["E"], n)
    b = n * case["K"] * 2 + nw * e * case["K"] * case["N"] * (0.5 + 1 / 32)
    b += n * case["N"] * (2 if case["out"] == "bf16" else 4)
    return {"bytes": int(b), "flops": 2 * nw * n * case["K"] * case["N"]}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        return _exact_norm(case, _norm_inputs(case, seed))
    if op == "balance":
        return _exact_balance(case, _balance_inputs(case, seed))
    if op == "quantize":
        s = _quantize_inputs(case, seed)
        return _exact_grid(s["x"] if case["form"] == "rows" else s["W"].transpose(1, 2))
    if 2 * case["T"] * case["k"] * case["K"] * case["N"] > 4e12:
        return None
    s = _product_inputs(case, seed)
    parts = []
    for e in range(case["E"]):
        if s["offs"][e] == s["offs"][e + 1]:
            continue
        x = _exact_grid(s["x"][s["offs"][e]:s["offs"][e + 1]])
        u = x @ _exact_grid(s["W"][e].t()).t()
        if case["act"] == "silu":
            u = u / (1 + torch.exp(-u))
        elif case["act"] == "swiglu":
            g = x @ _exact_grid(s["Wg"][e].t()).t()
            u = u * g / (1 + torch.exp(-g))
        parts.append(u)
    return torch.cat(parts)


def _exact_norm(case, s):
    """Values by the formula; gradients by differentiating it at the stored stream."""
    def unit(v):
        return v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS)

    v = {k: t.double().requires_grad_(case["op"] == "norm_bwd") for k, t in s.items()}

    def branch():
        b = unit(v["u"]) * v["w_post"] if case["post"] else v["u"]
        if "gate" in v:
            b = b * (v["gate"].unsqueeze(1) if case["gate"] == "token" else v["gate"])
        return OUT_SCALE * b

    if case["op"] == "norm_fwd":
        y = RES_SCALE * v["x"] + branch() if case["leave"] else v["x"]
        out = {}
        if case["leave"]:
            out["x_out"] = y
        if case["enter"]:
            out["z"] = unit(y) * v["w_pre"]
        return out
    y = v["x_out"]
    total = (y * v["dx_out"].detach()).sum()
    if case["enter"]:
        total = total + (unit(y) * v["w_pre"] * v["dz"].detach()).sum()
    names = {"dw_pre": "w_pre"} if case["enter"] else {}
    grads = torch.autograd.grad(total, [y] + [v[n] for n in names.values()])
    out = dict(zip(names, grads[1:]))
    if not case["leave"]:
        out["dx"] = grads[0]
        return out
    out["dx"] = RES_SCALE * grads[0]
    names = {"du": "u"}
    if case["post"]:
        names["dw_post"] = "w_post"
    if "gate" in v:
        names["dgate"] = "gate"
    out.update(zip(names, torch.autograd.grad((branch() * grads[0]).sum(),
                                              [v[n] for n in names.values()])))
    return out


def _exact_balance(case, s):
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    l = s["logits"].double().requires_grad_()
    offs = s["seq_offsets"].tolist()
    balance, zsum, tokens, live = 0.0, 0.0, 0, 0
    counts = torch.zeros(S, E, dtype=torch.int64, device="cuda")
    pbar = torch.zeros(S, E, dtype=torch.float64, device="cuda")
    for i in range(S):
        idx = s["topk"][offs[i]:offs[i + 1]]
        keep = idx[:, 0] >= 0
        n = int(keep.sum())
        if n == 0:
            continue
        rows = l[offs[i]:offs[i + 1]][keep]
        lse = torch.logsumexp(rows, 1)
        mean_p = torch.exp(rows - lse[:, None]).mean(0)
        c = torch.stack([(idx[keep] == e).sum() for e in range(E)])
        counts[i], pbar[i] = c, mean_p.detach()
        balance = balance + (c.double() * E / (k * n) * mean_p).sum()
        zsum = zsum + (lse ** 2).sum()
        tokens, live = tokens + n, live + 1
    b, z = BALANCE_COEF * balance / max(live, 1), Z_COEF * zsum / max(tokens, 1)
    if live == 0:
        zero = torch.zeros(3, dtype=torch.float64, device="cuda")
        return {"loss": zero, "counts": counts.to(torch.int32), "pbar": pbar,
                "dlogits": torch.zeros_like(l).detach()}
    dl, = torch.autograd.grad(b + z, l)
    return {"loss": torch.stack([b + z, b, z]).detach(), "counts": counts.to(torch.int32),
            "pbar": pbar, "dlogits": dl}


def _exact_grid(x):
    """Nearest values of the 4-bit grid at each block's scale 2^(floor(log2 max) - 2), ties to
    the even code, magnitudes above the grid's largest at that largest."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    _, ex = torch.frexp(top)                       # top = m 2^ex with m in [1/2, 1)
    scale = torch.exp2(torch.clamp(ex.double() - 3, min=-127.0))
    a = torch.clamp(b.abs() / scale, max=6.0)
    # spacing of the grid at each magnitude: 1/2 below 2, 1 below 4, then 2
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.round(a / step) * step               # round() takes ties to even
    q = torch.where(top > 0, q * torch.sign(b) * scale, torch.zeros_like(b))
    return q.reshape(x.shape)
