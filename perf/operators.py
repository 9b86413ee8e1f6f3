"""The operators around the fast-weight scans, as cases to be measured.

Three operators: the norm of queries and keys per head with the rotary positions in the same pass
(``rope`` and ``rope_bwd``), the gated linear recurrence on 64 x 64 per-head states (``scan``,
``scan_bwd`` and the one-token ``step``), and the gated feed-forward block that makes the In-Place
scan's keys (``ffn`` and ``ffn_bwd``). With ``own`` false ``run`` computes the plain form in
elementary torch operations; with ``own`` true it calls the package.
"""

import math

import torch

own = False

WIDTH = 64     # head width of the fast-weight states
BLOCK = 64     # tokens per block of the plain recurrence
NO_MEMORY = -1.0e4  # stands for a gate of minus infinity: exp of it is zero


def listed():
    return [
        # A training batch's queries and keys, straight from their projection (token-major), packed documents.
        {"name": "rope_train", "op": "rope", "batch": 8, "tokens": 2048, "hq": 12, "hk": 12, "width": 64, "rot": 64,
         "norm": "rms", "layout": "half", "scaling": "none", "start": 0, "documents": 5},
        # A long prompt with grouped heads, half of the head rotated, frequencies scaled for four times the length.
        {"name": "rope_long", "op": "rope", "batch": 1, "tokens": 32768, "hq": 32, "hk": 8, "width": 128, "rot": 64,
         "norm": "rms", "layout": "interleaved", "scaling": "yarn", "start": 98304, "documents": 1},
        # One token of every sequence in a serving batch: latency.
        {"name": "rope_token", "op": "rope", "batch": 32, "tokens": 1, "hq": 16, "hk": 16, "width": 64, "rot": 64,
         "norm": "l2", "layout": "half", "scaling": "linear", "start": 5000, "documents": 1},
        # Gradients of a training batch's queries and keys and of the norm's gains.
        {"name": "rope_back", "op": "rope_bwd", "batch": 4, "tokens": 8192, "hq": 16, "hk": 16, "width": 64, "rot": 32,
         "norm": "rms", "layout": "half", "scaling": "none", "start": 0, "documents": 3},
        # The gated scan over a training batch with documents that start afresh.
        {"name": "scan_train", "op": "scan", "batch": 8, "heads": 12, "tokens": 2048, "documents": 4, "initial": False},
        # One long sequence with few heads, of odd length, continued from a state.
        {"name": "scan_long", "op": "scan", "batch": 1, "heads": 4, "tokens": 65511, "documents": 1, "initial": True},
        # Gradients of a long training batch.
        {"name": "scan_back", "op": "scan_bwd", "batch": 4, "heads": 16, "tokens": 8192, "documents": 3, "initial": True},
        # One token of every sequence in a serving batch: the states are read and written.
        {"name": "scan_token", "op": "step", "batch": 64, "heads": 16},
        # The In-Place layer's feed-forward block over a long stretch of tokens.
        {"name": "ffn_long", "op": "ffn", "tokens": 8192, "d": 2560, "f": 9728, "activation": "silu", "save": False},
        # The same block for one token: the weights are read once.
        {"name": "ffn_token", "op": "ffn", "tokens": 1, "d": 2560, "f": 9728, "activation": "silu", "save": False},
        # An odd number of tokens through a smaller block, keeping what its backward pass needs.
        {"name": "ffn_odd", "op": "ffn", "tokens": 777, "d": 1000, "f": 2744, "activation": "gelu", "save": True},
        # Gradients of the block's input and weights.
        {"name": "ffn_back", "op": "ffn_bwd", "tokens": 4096, "d": 2560, "f": 9728, "activation": "silu"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "scan", "scan_bwd", "step", "ffn", "ffn", "ffn_bwd"])
    if op in ("rope", "rope_bwd"):
        width = rng.choice([64, 64, 96, 128, 256])
        hk = rng.randint(1, 16)
        hq = hk * rng.choice([1, 1, 2, 4])
        row = (hq + hk) * width
        tokens = _log(rng, 1, max(1, min(40000, 1 << 26) // max(1, row // 2048)))
        batch = rng.randint(1, max(1, min(64, (1 << 27) // (row * tokens))))
        return {"op": op, "batch": batch, "tokens": tokens, "hq": hq, "hk": hk, "width": width,
                "rot": rng.choice([16, 32, 48, 64, width]), "norm": rng.choice(["rms", "rms", "l2", "none"]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]), "start": _log(rng, 1, 500000) - 1,
                "documents": rng.randint(1, min(6, tokens))}
    if op in ("scan", "scan_bwd"):
        tokens = _log(rng, 1, 40000)
        pairs = _log(rng, 1, max(1, min(512, 400000 // tokens)))
        heads = rng.randint(1, pairs)
        return {"op": op, "batch": max(1, pairs // heads), "heads": heads, "tokens": tokens,
                "documents": rng.randint(1, min(5, tokens)), "initial": rng.random() < 0.5}
    if op == "step":
        return {"op": op, "batch": _log(rng, 1, 256), "heads": rng.randint(1, 40)}
    d, f = 8 * _log(rng, 8, 400), 8 * _log(rng, 8, 1300)
    top = max(1, min(8192, int(4.0e11 / (4.0 * d * f)))) if op == "ffn" else max(1, min(4096, int(6.0e11 / (8.0 * d * f))))
    case = {"op": op, "tokens": _log(rng, 1, top), "d": d, "f": f, "activation": rng.choice(["silu", "gelu"])}
    if op == "ffn":
        case["save"] = rng.random() < 0.5
    return case


def work(case):
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        n = case["batch"] * case["tokens"] * (case["hq"] + case["hk"]) * case["width"]
        pos = 8.0 * case["batch"] * case["tokens"]
        gains = 8.0 * case["width"] if case["norm"] == "rms" else 0.0
        if op == "rope":
            return {"bytes": 4.0 * n + pos + gains, "flops": 7.0 * n}
        # Without a norm the inputs themselves are not needed: the gradient is the rotation turned back.
        return {"bytes": (4.0 if case["norm"] == "none" else 6.0) * n + pos + 2.0 * gains, "flops": 14.0 * n}
    if op in ("scan", "scan_bwd"):
        pairs = case["batch"] * case["heads"]
        n = float(pairs * case["tokens"])
        state = 4.0 * WIDTH * WIDTH * pairs
        if op == "scan":
            # Per token: the state's decay and rank-one update and the output row.
            return {"bytes": n * (8.0 * WIDTH + 4.0) + state * (2 if case["initial"] else 1), "flops": 5.0 * n * WIDTH * WIDTH}
        return {"bytes": n * (14.0 * WIDTH + 8.0) + state * (3 if case["initial"] else 1), "flops": 14.0 * n * WIDTH * WIDTH}
    if op == "step":
        pairs = case["batch"] * case["heads"]
        return {"bytes": pairs * (8.0 * WIDTH * WIDTH + 8.0 * WIDTH + 4.0), "flops": 5.0 * pairs * WIDTH * WIDTH}
    T, d, f = case["tokens"], case["d"], case["f"]
    if op == "ffn":
        return {"bytes": 2.0 * (T * d + 2 * f * d + T * f * (3 if case["save"] else 1)), "flops": 4.0 * T * d * f}
    return {"bytes": 2.0 * (2 * T * d + 4 * f * d + 3 * T * f), "flops": 8.0 * T * d * f}


# ---- inputs -----------------------------------------------------------------------------


def _device():
    return torch.device("cuda", torch.cuda.current_device())


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=_device()) * std).to(dtype)


def _starts(case, gen, batch, tokens):
    """First tokens of each sequence's documents, as a truth value for each token."""
    first = torch.zeros(batch, tokens, dtype=torch.bool, device=_device())
    if case["documents"] > 1:
        at = torch.randint(1, max(2, tokens), (batch, case["documents"] - 1), generator=gen, device=_device())
        first.scatter_(1, at.clamp(max=tokens - 1), True)
    first[:, 0] = True
    return first


def _frequencies(case):
    """Radians per position of each rotated pair, and the rotation's magnitude (base 10000; a trained length of 32768)."""
    rot = min(case["rot"], case["width"])
    i = torch.arange(rot // 2, dtype=torch.float64, device=_device())
    base, factor, trained = 10000.0, 4.0, 32768.0
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    freq = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        return freq / factor, 1.0
    if case["scaling"] == "yarn":
        pair = lambda turns: rot * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return freq / factor * ramp + freq * (1.0 - ramp), 0.1 * math.log(factor) + 1.0
    return freq, 1.0


def prepare(case, seed):
    gen = torch.Generator(device=_device()).manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("rope", "rope_bwd"):
        B, T, D = case["batch"], case["tokens"], case["width"]
        # One projection's output holds each token's queries and keys: views of it, heads before tokens.
        x = _normal(gen, B, T, case["hq"] + case["hk"], D)
        s["q"], s["k"] = x[:, :, :case["hq"]].transpose(1, 2), x[:, :, case["hq"]:].transpose(1, 2)
        first = _starts(case, gen, B, T)
        t = torch.arange(T, device=_device()).expand(B, T)
        s["positions"] = t - torch.where(first, t, torch.zeros_like(t)).cummax(1).values + case["start"]
        s["freqs"], s["magnitude"] = _frequencies(case)
        s["wq"] = s["wk"] = None
        if case["norm"] == "rms":
            s["wq"], s["wk"] = (1.0 + _normal(gen, D, std=0.1, dtype=torch.float32) for _ in range(2))
        if op == "rope_bwd":
            s["dq"], s["dk"] = _normal(gen, B, case["hq"], T, D), _normal(gen, B, case["hk"], T, D)
        return s
    if op in ("scan", "scan_bwd"):
        B, H, T = case["batch"], case["heads"], case["tokens"]
        for name in ("q", "k", "v") + (("do",) if op == "scan_bwd" else ()):
            s[name] = _normal(gen, B, H, T, WIDTH)
        # Each head forgets at a rate of its own, from some tens of tokens to some thousands.
        rate = 2.0 + 6.0 * torch.rand(H, 1, generator=gen, device=_device())
        s["g"] = torch.nn.functional.logsigmoid(rate + _normal(gen, B, H, T, dtype=torch.float32))
        first = _starts(case, gen, B, T)
        first[:, 0] = False  # the call's first token goes on from the state before it
        s["g"] = s["g"].masked_fill(first[:, None, :], -math.inf)
        s["scale"] = WIDTH ** -0.5
        s["initial"] = _normal(gen, B, H, WIDTH, WIDTH, dtype=torch.float32) if case["initial"] else None
        if op == "scan_bwd":
            s["dfinal"] = _normal(gen, B, H, WIDTH, WIDTH, dtype=torch.float32) if case["initial"] else None
        return s
    if op == "step":
        B, H = case["batch"], case["heads"]
        for name in ("q", "k", "v"):
            s[name] = _normal(gen, B, H, WIDTH)
        s["g"] = torch.nn.functional.logsigmoid(4.0 + _normal(gen, B, H, dtype=torch.float32))
        s["scale"] = WIDTH ** -0.5
        s["state"] = _normal(gen, B, H, WIDTH, WIDTH, dtype=torch.float32)
        return s
    T, d, f = case["tokens"], case["d"], case["f"]
    s["x"] = _normal(gen, T, d)
    s["wg"], s["wu"] = _normal(gen, f, d, std=d ** -0.5), _normal(gen, f, d, std=d ** -0.5)
    if op == "ffn_bwd":
        s["dz"] = _normal(gen, T, f)
        # What the forward pass kept.
        s["g"], s["u"] = s["x"] @ s["wg"].t(), s["x"] @ s["wu"].t()
    return s


# ---- plain forms ------------------------------------------------------------------------


def _turn(x, cos, sin, layout, rot):
    """Rotates the first `rot` values of each row, pair by pair."""
    a = x[..., :rot]
    if layout == "half":
        p, r = a[..., :rot // 2], a[..., rot // 2:]
        y = torch.cat([p * cos - r * sin, r * cos + p * sin], -1)
    else:
        p, r = a[..., 0::2], a[..., 1::2]
        y = torch.stack([p * cos - r * sin, r * cos + p * sin], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _angles(s):
    a = s["positions"].double()[:, None, :, None] * s["freqs"]
    a = torch.remainder(a, 2.0 * math.pi).float()
    return torch.cos(a) * s["magnitude"], torch.sin(a) * s["magnitude"]


EPS = 1.0e-6


def _unit(x, norm):
    """x / its norm, and the reciprocal norm."""
    if norm == "none":
        return x, torch.ones_like(x[..., :1])
    m = (x * x).sum(-1, keepdim=True)
    r = torch.rsqrt((m / x.shape[-1] if norm == "rms" else m) + EPS)
    return x * r, r


def _plain_rope(s):
    c, out = s["case"], []
    cos, sin = _angles(s)
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = _unit(x.float(), c["norm"])[0]
        y = y * w if w is not None else y
        out.append(_turn(y, cos, sin, c["layout"], min(c["rot"], c["width"])).bfloat16())
    return out


def _plain_rope_bwd(s):
    c, out, gains = s["case"], [], []
    cos, sin = _angles(s)
    for x, w, dy in ((s["q"], s["wq"], s["dq"]), (s["k"], s["wk"], s["dk"])):
        n, r = _unit(x.float(), c["norm"])
        dy = _turn(dy.float(), cos, -sin, c["layout"], min(c["rot"], c["width"]))
        if w is not None:
            gains.append((dy * n).sum((0, 1, 2), dtype=torch.float64).float())
            dy = dy * w
        if c["norm"] != "none":
            dot = (dy * n).sum(-1, keepdim=True) / (c["width"] if c["norm"] == "rms" else 1.0)
            dy = r * (dy - n * dot)
        out.append(dy.bfloat16())
    return out + gains


def _blocks(x, fill=0.0):
    """[B, H, T, ...] in blocks of tokens, [B, H, n, BLOCK, ...], in 32 bits."""
    T = x.shape[2]
    n = -(-T // BLOCK)
    x = x.float() if x.dtype != torch.float64 else x
    if n * BLOCK != T:
        x = torch.cat([x, x.new_full(x.shape[:2] + (n * BLOCK - T,) + x.shape[3:], fill)], 2)
    return x.reshape(x.shape[:2] + (n, BLOCK) + x.shape[3:])


def _decays(g):
    """Within each block the decay from token j to token i and from and to its ends; and the
    sums of the gates to the start of each block (64 bits: they are long)."""
    b = _blocks(g.double().clamp(min=NO_MEMORY)).cumsum(-1)
    within = torch.exp((b[..., :, None] - b[..., None, :]).tril()).tril().float()
    total = b[..., -1].cumsum(-1)
    start = torch.cat([torch.zeros_like(total[..., :1]), total], -1)
    return b, within, start


def _states(local, start, first):
    """The state at the start of each block, from what each block adds."""
    n = local.shape[2]
    to = torch.exp((start[..., :n, None] - start[..., None, 1:]).tril(-1)).tril(-1).float()
    S = (to @ local.flatten(-2)).reshape(local.shape)
    if first is not None:
        S = S + torch.exp(start[..., :n]).float()[..., None, None] * first[:, :, None]
    return S


def _states_after(local, start, last):
    """The gradient of the state at the end of each block, from what each block adds."""
    n = local.shape[2]
    to = torch.exp((start[..., None, :n] - start[..., 1:, None]).triu(1)).triu(1).float()
    S = (to @ local.flatten(-2)).reshape(local.shape)
    if last is not None:
        S = S + torch.exp(start[..., -1:] - start[..., 1:]).float()[..., None, None] * last[:, :, None]
    return S


def _plain_scan(s):
    T = s["q"].shape[2]
    b, within, start = _decays(s["g"])
    q, k, v = (_blocks(s[n]) for n in ("q", "k", "v"))
    kw = k * torch.exp(b[..., -1:] - b).float()[..., None]
    local = kw.transpose(-1, -2) @ v
    S = _states(local, start, s["initial"])
    o = (q @ k.transpose(-1, -2) * within) @ v + torch.exp(b).float()[..., None] * (q @ S)
    final = torch.exp(b[..., -1, -1]).float()[..., None, None] * S[:, :, -1] + local[:, :, -1]
    return [(o * s["scale"]).flatten(2, 3)[:, :, :T].bfloat16(), final]


def _plain_scan_bwd(s):
    T, scale = s["q"].shape[2], s["scale"]
    b, within, start = _decays(s["g"])
    q, k, v, do = (_blocks(s[n]) for n in ("q", "k", "v", "do"))
    do = do * scale
    at, to = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None]
    S = _states((k * to).transpose(-1, -2) @ v, start, s["initial"])
    R = (q * at).transpose(-1, -2) @ do
    dS = _states_after(R, start, s["dfinal"])
    p, dp = q @ k.transpose(-1, -2), do @ v.transpose(-1, -2)
    dq_far, dk_far = at * (do @ S.transpose(-1, -2)), to * (v @ dS.transpose(-1, -2))
    dq, dk = (dp * within) @ k + dq_far, (dp * within).transpose(-1, -2) @ q + dk_far
    dv = (p * within).transpose(-1, -2) @ do + to * (k @ dS)
    # The gate of token t scales every pair with the key before t and the query at t or after.
    m = (p * dp * within).double().tril(-1)
    r, c = (q * dq_far).sum(-1).double(), (k * dk_far).sum(-1).double()
    after = lambda x: x.flip(-1).cumsum(-1).flip(-1)  # noqa: E731
    dg = after(m.sum(-1)) - after(m.sum(-2)) + after(r) + (c.cumsum(-1) - c)
    dg = dg + torch.exp(b[..., -1:]) * (S * dS).sum((-1, -2), dtype=torch.float64)[..., None]
    dg = dg.flatten(2, 3)[:, :, :T].masked_fill(s["g"] <= NO_MEMORY, 0.0)
    out = [x.flatten(2, 3)[:, :, :T].bfloat16() for x in (dq, dk, dv)] + [dg.float()]
    if s["initial"] is not None:
        out.append(torch.exp(b[:, :, 0, -1]).float()[..., None, None] * dS[:, :, 0] + R[:, :, 0])
    return out


def _plain_step(s):
    S = s["state"]
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    S.mul_(torch.exp(s["g"])[..., None, None]).add_(k[..., :, None] * v[..., None, :])
    return [(s["scale"] * (q[..., None, :] @ S).squeeze(-2)).bfloat16(), S]


def _act(x, kind):
    """The activation and its derivative."""
    if kind == "silu":
        y = torch.sigmoid(x)
        return x * y, y * (1.0 + x * (1.0 - y))
    phi = 0.5 * (1.0 + torch.erf(x * 0.5 ** 0.5))
    return x * phi, phi + x * torch.exp(-0.5 * x * x) * (2.0 * math.pi) ** -0.5


def _plain_ffn(s):
    x = s["x"].float()
    g, u = x @ s["wg"].float().t(), x @ s["wu"].float().t()
    z = (_act(g, s["case"]["activation"])[0] * u).bfloat16()
    return [z, g.bfloat16(), u.bfloat16()] if s["case"]["save"] else [z]


def _plain_ffn_bwd(s):
    x, g, u, dz = (s[n].float() for n in ("x", "g", "u", "dz"))
    a, da = _act(g, s["case"]["activation"])
    dg, du = dz * u * da, dz * a
    return [(dg @ s["wg"].float() + du @ s["wu"].float()).bfloat16(), (dg.t() @ x).bfloat16(), (du.t() @ x).bfloat16()]


_PLAIN = {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "scan": _plain_scan, "scan_bwd": _plain_scan_bwd,
          "step": _plain_step, "ffn": _plain_ffn, "ffn_bwd": _plain_ffn_bwd}


# ---- the package's calls ------------------------------------------------------------------


def _own(s):
    import chunked_weight_layers_b200 as cwl
    c, op = s["case"], s["op"]
    if op in ("rope", "rope_bwd"):
        how = dict(positions=s["positions"], freqs=s["freqs"], magnitude=s["magnitude"], norm=c["norm"], eps=EPS,
                   layout=c["layout"], q_weight=s["wq"], k_weight=s["wk"])
        if op == "rope":
            return list(cwl.qk_norm_rope(s["q"], s["k"], **how))
        return [x for x in cwl.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], **how) if x is not None]
    if op == "scan":
        return list(cwl.gated_scan(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], initial=s["initial"]))
    if op == "scan_bwd":
        return [x for x in cwl.gated_scan_backward(s["do"], s["q"], s["k"], s["v"], s["g"], scale=s["scale"],
                                                   initial=s["initial"], dfinal=s["dfinal"]) if x is not None]
    if op == "step":
        return [cwl.gated_scan_step(s["state"], s["q"], s["k"], s["v"], s["g"], scale=s["scale"]), s["state"]]
    if op == "ffn":
        z = cwl.gated_ffn(s["x"], s["wg"], s["wu"], activation=c["activation"], save=c["save"])
        return list(z) if c["save"] else [z]
    return list(cwl.gated_ffn_backward(s["dz"], s["x"], s["wg"], s["wu"], s["g"], s["u"], activation=c["activation"]))


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---- the definitions in 64 bits -------------------------------------------------------------


def _exact_rope(s, backward):
    c = s["case"]
    rot = min(c["rot"], c["width"])
    i = torch.arange(rot // 2, device=_device())
    lo, hi = (i, i + rot // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    turn = torch.polar(torch.full((1,), float(s["magnitude"]), dtype=torch.float64, device=_device()),
                       s["positions"].double()[:, None, :, None] * s["freqs"].double())
    out, gains = [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x = x.double()
        size = torch.ones_like(x[..., :1])
        if c["norm"] == "rms":
            size = (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        elif c["norm"] == "l2":
            size = (x.square().sum(-1, keepdim=True) + EPS).sqrt()
        gain = w.double() if w is not None else torch.ones(c["width"], dtype=torch.float64, device=_device())
        if not backward:
            y = x / size * gain
            z = torch.complex(y[..., lo], y[..., hi]) * turn
            y[..., lo], y[..., hi] = z.real, z.imag
            out.append(y)
            continue
        dy = dy.double().clone()
        z = torch.complex(dy[..., lo], dy[..., hi]) * turn.conj()
        dy[..., lo], dy[..., hi] = z.real, z.imag
        if w is not None:
            gains.append((dy * x / size).sum((0, 1, 2)))
        dn = dy * gain
        if c["norm"] == "none":
            out.append(dn)
        else:
            along = (dn * x).sum(-1, keepdim=True) / (c["width"] if c["norm"] == "rms" else 1)
            out.append(dn / size - x * along / size ** 3)
    return out + gains


def _exact_scan_pair(q, k, v, B, scale, S0, do, dST):
    """One (sequence, head): every query against every key before it, some rows at a time."""
    T = q.shape[0]
    rows = max(1, (1 << 25) // T)
    keys = torch.arange(T, device=q.device)
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=q.device)  # noqa: E731
    o, dq, dk, dv, by_row, by_col = new(T, WIDTH), new(T, WIDTH), new(T, WIDTH), new(T, WIDTH), new(T), new(T)
    for t in range(0, T, rows):
        e = min(T, t + rows)
        near = slice(0, e)
        w = scale * torch.exp((B[t:e, None] - B[None, near]).masked_fill(keys[None, near] > keys[t:e, None], -math.inf))
        p = w * (q[t:e] @ k[near].T)
        if do is None:
            o[t:e] = p @ v[near]
            continue
        dp = do[t:e] @ v[near].T
        dv[near] += p.T @ do[t:e]
        m = (p * dp).masked_fill_(keys[None, near] == keys[t:e, None], 0.0)
        by_row[t:e], by_col[near] = m.sum(1), by_col[near] + m.sum(0)
        dp *= w
        dq[t:e] = dp @ k[near]
        dk[near] += dp.T @ q[t:e]
    here, left = torch.exp(B)[:, None], torch.exp(B[-1] - B)[:, None]
    end = torch.exp(B[-1])
    if do is None:
        final = (left * k).T @ v
        if S0 is not None:
            o, final = o + scale * here * (q @ S0), final + end * S0
        return o, final
    dg = by_row.flip(0).cumsum(0).flip(0) - by_col.flip(0).cumsum(0).flip(0)
    dS0 = scale * (here * q).T @ do
    if S0 is not None:
        far = scale * here * (do @ S0.T)
        dq = dq + far
        dg = dg + (q * far).sum(1).flip(0).cumsum(0).flip(0)
    if dST is not None:
        far = left * (v @ dST.T)
        dk, dv, dS0 = dk + far, dv + left * (k @ dST), dS0 + end * dST
        past = (k * far).sum(1)
        dg = dg + past.cumsum(0) - past
    if S0 is not None and dST is not None:
        dg = dg + end * (S0 * dST).sum()
    return dq, dk, dv, dg, dS0


def _exact_scan(s, backward):
    B = s["g"].double().clamp(min=NO_MEMORY).cumsum(-1)
    T = B.shape[-1]
    if float(B.shape[0] * B.shape[1]) * T * T > 2.0e10:
        return None  # some tens of seconds
    dbl = lambda n, i, h: s[n][i, h].double() if s.get(n) is not None else None  # noqa: E731
    pairs = [[_exact_scan_pair(dbl("q", i, h), dbl("k", i, h), dbl("v", i, h), B[i, h], s["scale"], dbl("initial", i, h),
                               dbl("do", i, h), dbl("dfinal", i, h)) for h in range(B.shape[1])] for i in range(B.shape[0])]
    out = [torch.stack([torch.stack([p[n] for p in row]) for row in pairs]) for n in range(len(pairs[0][0]))]
    if backward:
        out[3] = out[3].masked_fill(s["g"] <= NO_MEMORY, 0.0)
        if s["initial"] is None:
            out = out[:4]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("rope", "rope_bwd"):
        return _exact_rope(s, op == "rope_bwd")
    if op in ("scan", "scan_bwd"):
        return _exact_scan(s, op == "scan_bwd")
    if op == "step":
        S = torch.einsum("bh,bhij->bhij", s["g"].double().exp(), s["state"].double())
        S = S + torch.einsum("bhi,bhj->bhij", s["k"].double(), s["v"].double())
        return [s["scale"] * torch.einsum("bhi,bhij->bhj", s["q"].double(), S), S]
    if op == "ffn":
        x = s["x"].double()
        g, u = torch.einsum("td,fd->tf", x, s["wg"].double()), torch.einsum("td,fd->tf", x, s["wu"].double())
        a = g / (1.0 + torch.exp(-g)) if case["activation"] == "silu" else 0.5 * g * torch.erfc(-g / math.sqrt(2.0))
        return [a * u, g, u] if case["save"] else [a * u]
    g = s["g"].double()
    if case["activation"] == "silu":
        e = torch.exp(-g)
        a, slope = g / (1.0 + e), 1.0 / (1.0 + e) + g * e / (1.0 + e) ** 2
    else:
        half = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        a, slope = g * half, half + g * torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
    dz, x = s["dz"].double(), s["x"].double()
    dg, du = dz * slope * s["u"].double(), dz * a
    dx = torch.einsum("tf,fd->td", dg, s["wg"].double()) + torch.einsum("tf,fd->td", du, s["wu"].double())
    return [dx, torch.einsum("tf,td->fd", dg, x), torch.einsum("tf,td->fd", du, x)]
