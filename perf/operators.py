"""Workloads of the operators between the adapted linears of a decoder layer.

Each case is one call that a serving program makes next to the fused merge and
the segmented apply: a projection with the merged weights, the gated pair of
projections of the feed-forward block, the epilogue of outputs that exist
already, and the rotation of queries and keys by position, with or without
norms of each head.  `run` computes a case in plain torch operations, or, with
`own` set, through the library.
"""
import math

import torch

own = False

BF16 = torch.bfloat16


def listed():
    return [
        # One token of one request through the 7B attention output: 4096 x 4096, the residual stream added.
        {"name": "project_decode_1", "op": "project", "T": 1, "K": 4096, "N": 4096, "act": "none", "bias": False,
         "residual": True, "out": "bf16"},
        # A rank's share (1 of 8) of the 7B down projection for an odd batch: 1376 input columns, fp32 partial sums.
        {"name": "project_partial_130", "op": "project", "T": 130, "K": 1376, "N": 4096, "act": "none", "bias": False,
         "residual": False, "out": "fp32"},
        # A long prompt through the 7B down projection, the residual stream added.
        {"name": "project_prompt_4096", "op": "project", "T": 4096, "K": 11008, "N": 4096, "act": "none",
         "bias": False, "residual": True, "out": "bf16"},
        # One token through the 7B feed-forward's gate and up projections.
        {"name": "gated_decode_1", "op": "gated", "T": 1, "K": 4096, "N": 11008, "act": "silu", "bias": False},
        # A decode batch of 64 sequences through the 13B gate and up projections.
        {"name": "gated_batch_64", "op": "gated", "T": 64, "K": 5120, "N": 13824, "act": "silu", "bias": False},
        # A prompt of odd length through the 7B gate and up projections, tanh-gelu and biases.
        {"name": "gated_prompt_2001", "op": "gated", "T": 2001, "K": 4096, "N": 11008, "act": "gelu_tanh",
         "bias": True},
        # The unmerged apply's gate and up outputs of a mixed decode batch of 64: silu(g) * u.
        {"name": "epilogue_gate_64", "op": "epilogue", "T": 64, "N": 11008, "act": "silu", "bias": False, "up": True,
         "residual": False, "in": "bf16", "out": "bf16"},
        # The all-reduced fp32 sums of a 13B row-parallel layer for a prompt: bias and residual, rounded once.
        {"name": "epilogue_partial_2047", "op": "epilogue", "T": 2047, "N": 5120, "act": "none", "bias": True,
         "up": False, "residual": True, "in": "fp32", "out": "bf16"},
        # A decode batch of 64 sequences at far positions, 7B heads.
        {"name": "rotary_decode_64", "op": "rotary", "T": 64, "Hq": 32, "Hk": 32, "D": 128, "rot": 128,
         "layout": "half", "scaled": False, "norm": False, "far": True},
        # A prompt of odd length, 13B heads, half of each head rotated in neighbouring pairs, frequencies stretched.
        {"name": "rotary_prompt_4097", "op": "rotary", "T": 4097, "Hq": 40, "Hk": 40, "D": 128, "rot": 64,
         "layout": "interleaved", "scaled": True, "norm": False, "far": False},
        # One token with 32 query and 8 key heads, each normalised.
        {"name": "norm_rotary_decode_1", "op": "rotary", "T": 1, "Hq": 32, "Hk": 8, "D": 128, "rot": 128,
         "layout": "half", "scaled": False, "norm": True, "far": True},
        # A long prompt with 32 query and 8 key heads, each normalised.
        {"name": "norm_rotary_prompt_8192", "op": "rotary", "T": 8192, "Hq": 32, "Hk": 8, "D": 128, "rot": 128,
         "layout": "half", "scaled": True, "norm": True, "far": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: tokens from one to a long prompt, widths of every multiple
    of eight (heads: even sizes) up to the 13B model's, every activation and form."""
    op = rng.choice(["project", "gated", "epilogue", "rotary"])
    acts = ["none", "relu", "silu", "gelu", "gelu_tanh"]
    if op in ("project", "gated"):
        K, N = 8 * _log(rng, 16, 1728), 8 * _log(rng, 16, 1728)
        most = 4096 * 11008 * 4096 // (K * N * (2 if op == "gated" else 1))
        T = _log(rng, 1, max(1, min(4096, most)))
        if op == "gated":
            return {"op": op, "T": T, "K": K, "N": N, "act": rng.choice(acts[1:]), "bias": rng.random() < 0.3}
        return {"op": op, "T": T, "K": K, "N": N, "act": rng.choice(acts), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5, "out": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "epilogue":
        return {"op": op, "T": _log(rng, 1, 4096), "N": 8 * _log(rng, 16, 1728), "act": rng.choice(acts),
                "bias": rng.random() < 0.5, "up": rng.random() < 0.5, "residual": rng.random() < 0.5,
                "in": rng.choice(["bf16", "fp32"]), "out": rng.choice(["bf16", "bf16", "fp32"])}
    D = rng.choice([64, 80, 96, 112, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 5, 8, 32])
    return {"op": op, "T": _log(rng, 1, 8192 * 128 * 8 // (D * Hk)) if Hk == 32 else _log(rng, 1, 8192),
            "Hq": Hk if Hk == 32 else Hk * rng.choice([1, 2, 4]), "Hk": Hk, "D": D,
            "rot": rng.choice([D, D, D // 2]), "layout": rng.choice(["half", "interleaved"]),
            "scaled": rng.random() < 0.5, "norm": rng.random() < 0.5, "far": rng.random() < 0.5}


def _frequencies(rot, scaled):
    """Radians per position of each rotated pair, in 64 bits, and the factor of the rotated values.
    Stretched 8 times by wavelength: pairs that turn more than 32 times within 4096 positions keep
    their frequency, those that turn less than once are slowed 8 times, a ramp between."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if not scaled:
        return f, 1.0
    pair = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot // 2 - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / 8 * ramp + f * (1 - ramp), 0.1 * math.log(8.0) + 1


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=BF16):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    c, s = case, {"case": case}
    if c["op"] in ("project", "gated"):
        s["x"] = normal(c["T"], c["K"])
        s["W"] = normal(c["N"], c["K"], std=0.02)
        s["bias"] = normal(c["N"], std=0.5) if c["bias"] else None
        if c["op"] == "gated":
            s["W_up"] = normal(c["N"], c["K"], std=0.02)
            s["bias_up"] = normal(c["N"], std=0.5) if c["bias"] else None
        else:
            s["residual"] = normal(c["T"], c["N"]) if c["residual"] else None
    elif c["op"] == "epilogue":
        kind = BF16 if c["in"] == "bf16" else torch.float32
        s["y"] = normal(c["T"], c["N"], dtype=kind)
        s["bias"] = normal(c["N"], std=0.5) if c["bias"] else None
        s["up"] = normal(c["T"], c["N"], dtype=kind) if c["up"] else None
        s["residual"] = normal(c["T"], c["N"]) if c["residual"] else None
    else:
        T, Hq, Hk, D = c["T"], c["Hq"], c["Hk"], c["D"]
        # the rows of one projection that holds q, k and v of a token side by side
        qkv = normal(T, (Hq + 2 * Hk) * D)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        if c["far"]:    # a decode batch: every sequence at a position of its own
            s["positions"] = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
        else:           # consecutive tokens of one prompt
            s["positions"] = torch.arange(T, device="cuda") + int(seed) % 1000
        f, s["factor"] = _frequencies(c["rot"], c["scaled"])
        s["freq"] = f.cuda()
        s["q_weight"] = 1 + normal(D, std=0.1) if c["norm"] else None
        s["k_weight"] = 1 + normal(D, std=0.1) if c["norm"] else None
    return s


def _act(v, name):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plus(v, *terms):
    for t in terms:
        if t is not None:
            v = v + t.float()
    return v


def _rotate(x, weight, cos, sin, layout):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    n = cos.shape[-1]
    y = x.clone()
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y.to(BF16)


def _plain(s):
    c = s["case"]
    if c["op"] == "project":
        y = _act(_plus(s["x"].float() @ s["W"].float().t(), s["bias"]), c["act"])
        y = _plus(y, s["residual"])
        return y if c["out"] == "fp32" else y.to(BF16)
    if c["op"] == "gated":
        x = s["x"].float()
        a = _act(_plus(x @ s["W"].float().t(), s["bias"]), c["act"])
        return (a * _plus(x @ s["W_up"].float().t(), s["bias_up"])).to(BF16)
    if c["op"] == "epilogue":
        y = _act(_plus(s["y"].float(), s["bias"]), c["act"])
        y = _plus(y if s["up"] is None else y * s["up"].float(), s["residual"])
        return y if c["out"] == "fp32" else y.to(BF16)
    angle = (s["positions"].double()[:, None] * s["freq"])[:, None, :]
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    return [_rotate(s["q"], s["q_weight"], cos, sin, c["layout"]),
            _rotate(s["k"], s["k_weight"], cos, sin, c["layout"])]


def _library(s):
    import adapter_merge_b200 as am
    c = s["case"]
    if c["op"] == "project":
        return am.project(s["x"], s["W"], bias=s["bias"], activation=c["act"], residual=s["residual"],
                          out_dtype=torch.float32 if c["out"] == "fp32" else BF16)
    if c["op"] == "gated":
        return am.gated_project(s["x"], s["W"], s["W_up"], bias_gate=s["bias"], bias_up=s["bias_up"],
                                activation=c["act"])
    if c["op"] == "epilogue":
        return am.epilogue(s["y"], bias=s["bias"], activation=c["act"], up=s["up"], residual=s["residual"],
                           out_dtype=torch.float32 if c["out"] == "fp32" else BF16)
    return list(am.rotary(s["q"], s["k"], s["positions"], s["freq"], layout=c["layout"], factor=s["factor"],
                          q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6))


def run(state):
    if own:
        return _library(state)
    return _plain(state)


def work(case):
    c, T = case, case["T"]
    size = {"bf16": 2, "fp32": 4}
    if c["op"] == "project":
        K, N = c["K"], c["N"]
        b = 2 * (T * K + N * K + (N if c["bias"] else 0) + (T * N if c["residual"] else 0)) + size[c["out"]] * T * N
        return {"bytes": b, "flops": 2 * T * N * K}
    if c["op"] == "gated":
        K, N = c["K"], c["N"]
        return {"bytes": 2 * (T * K + 2 * N * K + T * N + (2 * N if c["bias"] else 0)), "flops": 4 * T * N * K}
    if c["op"] == "epilogue":
        each = size[c["in"]] * (2 if c["up"] else 1) + (2 if c["residual"] else 0) + size[c["out"]]
        return {"bytes": T * c["N"] * each + (2 * c["N"] if c["bias"] else 0), "flops": 8 * T * c["N"]}
    values = T * (c["Hq"] + c["Hk"]) * c["D"]
    return {"bytes": 4 * values + 8 * T + 4 * c["rot"] + (4 * c["D"] if c["norm"] else 0),
            "flops": 3 * T * (c["Hq"] + c["Hk"]) * c["rot"] + (4 * values if c["norm"] else 0)}


def exact(case, seed):
    """The definitions in 64 bits, unrounded."""
    s, c = prepare(case, seed), case
    d = lambda t: t.to(torch.float64)  # noqa: E731

    def act(v):
        if c["act"] == "relu":
            return torch.where(v > 0, v, torch.zeros_like(v))
        if c["act"] == "silu":
            return v * torch.special.expit(v)
        if c["act"] == "gelu":
            return v * torch.special.ndtr(v)
        if c["act"] == "gelu_tanh":     # (1 + tanh u) / 2 = expit(2u)
            return v * torch.special.expit(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))
        return v

    if c["op"] in ("project", "gated"):
        v = torch.einsum("tk,nk->tn", d(s["x"]), d(s["W"]))
        v = act(v if s["bias"] is None else v + d(s["bias"]))
        if c["op"] == "gated":
            u = torch.einsum("tk,nk->tn", d(s["x"]), d(s["W_up"]))
            return v * (u if s["bias_up"] is None else u + d(s["bias_up"]))
        return v if s["residual"] is None else v + d(s["residual"])
    if c["op"] == "epilogue":
        v = act(d(s["y"]) if s["bias"] is None else d(s["y"]) + d(s["bias"]))
        v = v if s["up"] is None else v * d(s["up"])
        return v if s["residual"] is None else v + d(s["residual"])
    # one complex number per rotated pair, times e^(i position frequency)
    turn = s["factor"] * torch.exp(1j * torch.outer(d(s["positions"]), s["freq"]))[:, None, :]
    done = []
    for x, w in ((d(s["q"]), s["q_weight"]), (d(s["k"]), s["k_weight"])):
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6) * d(w)
        pairs, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["layout"] == "half":
            z = torch.complex(pairs[..., :c["rot"] // 2], pairs[..., c["rot"] // 2:]) * turn
            done.append(torch.cat([z.real, z.imag, rest], -1))
        else:
            z = torch.view_as_complex(pairs.reshape(*pairs.shape[:-1], -1, 2).contiguous()) * turn
            done.append(torch.cat([torch.view_as_real(z).flatten(-2), rest], -1))
    return done
