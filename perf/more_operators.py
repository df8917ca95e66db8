"""Cases for what stands between the 16-bit products of a layer: the forward product
with bias, activation, gate, dropout and residual in its epilogue, the gradient of
that epilogue, dropout by itself, rotary positions, and the norm of queries and keys
with the rotation, forward and backward.

Each case is one call.  `run` computes it either in plain torch operations in 32
bits (angles in 64), or, where `own` is true, with the library's entry points.
"""
import math

import torch

own = False

EPS = 1e-5
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]   # forge.ACT_NONE, ... in this order
NONE = dict(bias="", act="none", mul=False, residual=False, z=False, p=0.0, out="bf16")


def listed():
    return [
        # one new token through a SwiGLU gate: the weight's bytes are all that counts
        dict(name="linear_1_token", op="linear", bt=1, d_in=4096, d_out=14336,
             **{**NONE, "act": "silu", "mul": True}),
        # a small model's projection in training, odd sizes: everything the epilogue has
        dict(name="linear_333_all", op="linear", bt=333, d_in=1032, d_out=520,
             **{**NONE, "bias": "fp32", "act": "gelu", "residual": True, "z": True, "p": 0.1}),
        # the down projection onto the residual stream at a ragged token count
        dict(name="linear_2000_down", op="linear", bt=2000, d_in=14336, d_out=4096,
             **{**NONE, "residual": True}),
        # the gate projection of a long batch, in training
        dict(name="linear_8192_gate", op="linear", bt=8192, d_in=4096, d_out=14336,
             **{**NONE, "act": "silu", "mul": True, "z": True}),
        # the epilogue's gradient in a small model with biases and dropout
        dict(name="epilogue_bwd_333x520", op="epilogue_bwd", rows=333, cols=520, act="gelu",
             mul=False, bias=True, p=0.1),
        # the gradient of a long batch's SwiGLU product
        dict(name="epilogue_bwd_8192_gate", op="epilogue_bwd", rows=8192, cols=14336, act="silu",
             mul=True, bias=False, p=0.0),
        # dropout's gradient in a small model
        dict(name="dropout_64x520", op="dropout", rows=64, cols=520, residual=False, p=0.1),
        # dropout onto the residual stream of a long batch
        dict(name="dropout_8191", op="dropout", rows=8191, cols=4096, residual=True, p=0.1),
        # one new token's queries and keys, far into a long context
        dict(name="rope_1_token", op="rope", tokens=1, hq=32, hk=8, dim=128, rot=128, layout="half",
             scaling="llama3", fused=True, far=True, inverse=False),
        # the gradients of a long batch's rotated queries and keys
        dict(name="rope_bwd_8192", op="rope", tokens=8192, hq=32, hk=8, dim=128, rot=128,
             layout="half", scaling="llama3", fused=True, far=False, inverse=True),
        # a ragged batch, pairs side by side, part of each head rotated
        dict(name="qk_norm_rope_1999", op="qk", tokens=1999, hq=32, hk=8, dim=128, rot=64,
             layout="interleaved", scaling="yarn", fused=True, far=False, gain="bf16"),
        # the gradients of a long batch through rotation and norm
        dict(name="qk_norm_rope_bwd_8192", op="qk_bwd", tokens=8192, hq=32, hk=8, dim=128, rot=128,
             layout="half", scaling="none", fused=True, far=False, gain="fp32"),
    ]


def _log(rng, low, high, multiple=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / multiple)) * multiple))


def draw(rng):
    op = rng.choice(["linear", "linear", "epilogue_bwd", "dropout", "rope", "qk", "qk_bwd"])
    p = rng.choice([0.0, 0.05, 0.1, 0.5])
    if op == "linear":
        return dict(op=op, bt=_log(rng, 1, 8192), d_in=_log(rng, 64, 4096, 8),
                    d_out=_log(rng, 64, 14336, 8), bias=rng.choice(["", "bf16", "fp32"]),
                    act=rng.choice(ACTS), mul=rng.random() < 0.3, residual=rng.random() < 0.4,
                    z=rng.random() < 0.4, p=p, out=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "epilogue_bwd":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 14336, 8),
                    act=rng.choice(ACTS), mul=rng.random() < 0.5, bias=rng.random() < 0.5, p=p)
    if op == "dropout":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 4096, 8),
                    residual=rng.random() < 0.5, p=rng.choice([0.05, 0.1, 0.5]))
    dim = rng.choice([64, 80, 96, 128, 256])
    hk = _log(rng, 1, 8)
    case = dict(op=op, tokens=_log(rng, 1, 8192), hq=min(hk * rng.choice([1, 2, 4, 8]), 4096 // dim),
                hk=min(hk, 1024 // dim), dim=dim, rot=rng.choice([dim, dim // 2, 32, 24]),
                layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["none", "linear", "llama3", "yarn"]), fused=rng.random() < 0.6,
                far=rng.random() < 0.5)
    if op == "rope":
        return dict(case, inverse=rng.random() < 0.5)
    return dict(case, gain=rng.choice(["bf16", "fp32"]))


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _activations(g, rows, cols):
    """bf16 activations with a few columns far larger than the rest, as trained models have."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    heavy = torch.rand((cols,), generator=g, device="cuda") < 0.005
    return (x * torch.where(heavy, 20.0, 1.0)).to(torch.bfloat16)


def _frequencies(rot, scaling):
    """The angle of each pair per position, in 64 bits, and the rotated values' factor."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if scaling == "llama3":      # theta 500000, eight times a context of 8192
        f = 500000.0 ** (-i / rot)
        turns = 8192 * f / (2 * math.pi)
        mix = ((turns - 1) / (4 - 1)).clamp(0, 1)
        return (1 - mix) * f / 8 + mix * f, 1.0
    f = 10000.0 ** (-i / rot)
    if scaling == "linear":
        return f / 4, 1.0
    if scaling == "yarn":        # sixteen times a context of 4096
        at = [rot * math.log(4096 / (b * 2 * math.pi)) / (2 * math.log(10000.0)) for b in (32, 1)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i / 2 - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / 16 * ramp + f * (1 - ramp), 0.1 * math.log(16) + 1
    return f, 1.0


def _heads(g, case):
    """Queries and keys [tokens, heads, dim]: views of the projections' fused output, or apart."""
    t, hq, hk, dim = (case[k] for k in ("tokens", "hq", "hk", "dim"))
    if not case["fused"]:
        return _normal(g, (t, hq, dim), 1.0), _normal(g, (t, hk, dim), 2.0)
    qkv = _activations(g, t, (hq + 2 * hk) * dim).view(t, hq + 2 * hk, dim)
    return qkv[:, :hq], qkv[:, hq:hq + hk]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": case, "seed": int(seed) * 0x9E3779B97F4A7C15 % 2 ** 64, "offset": 7}
    new = lambda shape, dt=torch.bfloat16: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    if op == "linear":
        bt, d_in, d_out = case["bt"], case["d_in"], case["d_out"]
        s["X"] = _activations(g, bt, d_in)
        s["W"] = _normal(g, (d_out, d_in), d_in ** -0.5)
        s["bias"] = _normal(g, (d_out,), 0.5, _dt(case["bias"])) if case["bias"] else None
        s["mul"] = _normal(g, (bt, d_out), 1.0) if case["mul"] else None
        s["residual"] = _normal(g, (bt, d_out), 3.0) if case["residual"] else None
        s["Z"] = new((bt, d_out)) if case["z"] else None
        s["Y"] = new((bt, d_out), _dt(case["out"]))
    elif op == "epilogue_bwd":
        shape = (case["rows"], case["cols"])
        s["dY"], s["Z"] = _normal(g, shape, 1e-3), _normal(g, shape, 1.5)
        s["mul"] = _normal(g, shape, 1.0) if case["mul"] else None
        s["dZ"], s["dmul"] = new(shape), new(shape) if case["mul"] else None
        s["dbias"] = new((case["cols"],), torch.float32) if case["bias"] else None
        # scratch the program keeps for every layer of the model
        s["workspace"] = new((32 << 20,), torch.uint8)
    elif op == "dropout":
        shape = (case["rows"], case["cols"])
        s["x"], s["y"] = _normal(g, shape, 1.0), new(shape)
        s["residual"] = _normal(g, shape, 3.0) if case["residual"] else None
    else:
        t, dim = case["tokens"], case["dim"]
        s["q"], s["k"] = _heads(g, case)
        s["q_out"], s["k_out"] = new((t, case["hq"], dim)), new((t, case["hk"], dim))
        # a batch of sequences at positions of their own, or one prompt from some position on
        start = torch.randint(0, 100000, (t if case["far"] else 1,), generator=g, device="cuda")
        s["positions"] = start if case["far"] else start // 50 + torch.arange(t, device="cuda")
        f, s["magnitude"] = _frequencies(case["rot"], case["scaling"])
        s["angles"] = f.to("cuda")
        # what the library takes: turns per position as fractions of 2^64
        s["freqs"] = torch.round(f / (2 * math.pi) * 2.0 ** 64).to(torch.int64).to("cuda")
        if op != "rope":
            for n in ("q_gain", "k_gain"):
                s[n] = (1 + 0.2 * torch.randn((dim,), generator=g, device="cuda")).to(_dt(case["gain"]))
        if op == "qk_bwd":
            s["dq"] = _normal(g, (t, case["hq"], dim), 1e-3)
            s["dk"] = _normal(g, (t, case["hk"], dim), 1e-3)
            s["dq_gain"], s["dk_gain"] = new((dim,), torch.float32), new((dim,), torch.float32)
            s["workspace"] = new((8 << 20,), torch.uint8)
    return s


def _keep(rows, cols, s):
    """Which elements dropout keeps: Philox4x32-10 (Salmon et al. 2011), 16 bits an element."""
    low = 0xFFFFFFFF
    c0 = torch.arange(rows * cols // 8, device="cuda")
    c1, c2, c3 = c0 >> 32, torch.full_like(c0, s["offset"] & low), torch.full_like(c0, s["offset"] >> 32)
    c0, k0, k1 = c0 & low, s["seed"] & low, s["seed"] >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57       # modulo 2^64
        c0, c1, c2, c3 = (b >> 32) & low ^ c1 ^ k0, b & low, (a >> 32) & low ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2)
    return bits.view(rows, cols) >= round(s["case"]["p"] * 65536)


def _dropped(x, s):
    if s["case"]["p"] == 0:
        return x
    scale = 65536 / (65536 - round(s["case"]["p"] * 65536))
    return torch.where(_keep(*x.shape, s), x * scale, torch.zeros_like(x))


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        u = 1 / (1 + torch.exp(-z))
        return u * (1 + z * (1 - u))
    return torch.ones_like(z)


def _plain_linear(s):
    z = torch.matmul(s["X"].float(), s["W"].float().t())
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, s["case"]["act"])
    if s["mul"] is not None:
        y = y * s["mul"].float()
    y = _dropped(y, s)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = [y.to(s["Y"].dtype)]
    return out + [z.to(torch.bfloat16)] if s["Z"] is not None else out


def _plain_epilogue_bwd(s):
    act, z = s["case"]["act"], s["Z"].float()
    da, out = _dropped(s["dY"].float(), s), []
    if s["mul"] is not None:
        out.append((da * _act(z, act)).to(torch.bfloat16))
        da = da * s["mul"].float()
    dz = da * _act_slope(z, act)
    if s["dbias"] is not None:
        out.append(dz.sum(0))
    return [dz.to(torch.bfloat16)] + out


def _plain_dropout(s):
    y = _dropped(s["x"].float(), s)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(torch.bfloat16)]


def _rotate(x, s, sign):
    """x [tokens, heads, dim] in 32 bits, the first `rot` of each head rotated."""
    rot, half = s["case"]["rot"], s["case"]["rot"] // 2
    angle = s["positions"][:, None].double() * s["angles"]
    c = (angle.cos() * s["magnitude"]).float()[:, None]
    d = (angle.sin() * s["magnitude"] * sign).float()[:, None]
    r, rest = x[..., :rot], x[..., rot:]
    if s["case"]["layout"] == "half":
        a, b = r[..., :half], r[..., half:]
        return torch.cat([a * c - b * d, b * c + a * d, rest], 2)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * c - b * d, b * c + a * d], 3).flatten(2), rest], 2)


def _plain_rope(s):
    sign = -1.0 if s["case"]["inverse"] else 1.0
    return [_rotate(s[n].float(), s, sign).to(torch.bfloat16) for n in ("q", "k")]


def _rstd(x):
    return torch.rsqrt((x * x).mean(2, keepdim=True) + EPS)


def _plain_qk(s):
    q, k = s["q"].float(), s["k"].float()
    return [_rotate(x * _rstd(x) * s[n].float(), s, 1.0).to(torch.bfloat16)
            for x, n in ((q, "q_gain"), (k, "k_gain"))]


def _norm_bwd(dy, x, gain, s):
    dn, rstd = _rotate(dy.float(), s, -1.0), _rstd(x)
    xh, u = x * rstd, dn * gain.float()
    dx = rstd * (u - xh * (u * xh).mean(2, keepdim=True))
    return dx.to(torch.bfloat16), (dn * xh).sum((0, 1))


def _plain_qk_bwd(s):
    dq, dgq = _norm_bwd(s["dq"], s["q"].float(), s["q_gain"], s)
    dk, dgk = _norm_bwd(s["dk"], s["k"].float(), s["k_gain"], s)
    return [dq, dk, dgq, dgk]


def _own(s):
    from weight_gradient_gemm_gb300 import forge
    case = s["case"]
    op = case["op"]
    drop = dict(p=case.get("p", 0.0), seed=s["seed"], offset=s["offset"])
    if op == "linear":
        forge.linear_bf16(s["X"], s["W"], s["Y"], bias=s["bias"], act=ACTS.index(case["act"]),
                          mul=s["mul"], residual=s["residual"], Z=s["Z"], **drop)
        return [t for t in (s["Y"], s["Z"]) if t is not None]
    if op == "epilogue_bwd":
        forge.epilogue_backward(s["dY"], s["dZ"], Z=s["Z"], act=ACTS.index(case["act"]),
                                mul=s["mul"], dmul=s["dmul"], dbias=s["dbias"],
                                workspace=s["workspace"], **drop)
        return [t for t in (s["dZ"], s["dmul"], s["dbias"]) if t is not None]
    if op == "dropout":
        forge.dropout(s["x"], s["y"], residual=s["residual"], **drop)
        return [s["y"]]
    how = dict(positions=s["positions"], magnitude=s["magnitude"],
               layout=forge.ROPE_HALF if case["layout"] == "half" else forge.ROPE_INTERLEAVED)
    if op == "rope":
        forge.rope(s["q"], s["k"], s["freqs"], q_out=s["q_out"], k_out=s["k_out"],
                   inverse=case["inverse"], **how)
        return [s["q_out"], s["k_out"]]
    if op == "qk":
        forge.qk_norm_rope(s["q"], s["k"], s["q_gain"], s["k_gain"], s["freqs"], eps=EPS,
                           q_out=s["q_out"], k_out=s["k_out"], **how)
        return [s["q_out"], s["k_out"]]
    forge.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["q_gain"], s["k_gain"],
                                s["freqs"], eps=EPS, dq_out=s["q_out"], dk_out=s["k_out"],
                                dq_gain=s["dq_gain"], dk_gain=s["dk_gain"],
                                workspace=s["workspace"], **how)
    return [s["q_out"], s["k_out"], s["dq_gain"], s["dk_gain"]]


def run(state):
    if own:
        return _own(state)
    plain = {"linear": _plain_linear, "epilogue_bwd": _plain_epilogue_bwd,
             "dropout": _plain_dropout, "rope": _plain_rope, "qk": _plain_qk,
             "qk_bwd": _plain_qk_bwd}
    return plain[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "linear":
        bt, d_in, d_out = case["bt"], case["d_in"], case["d_out"]
        by = 2 * (bt * d_in + d_in * d_out) + bt * d_out * (4 if case["out"] == "fp32" else 2)
        by += 2 * bt * d_out * (case["mul"] + case["residual"] + case["z"])
        by += {"": 0, "bf16": 2, "fp32": 4}[case["bias"]] * d_out
        return {"bytes": by, "flops": 2 * bt * d_in * d_out}
    if op == "epilogue_bwd":
        n = case["rows"] * case["cols"]
        streams = 2 + (case["act"] != "none" or case["mul"]) + 2 * case["mul"]
        return {"bytes": 2 * n * streams + 4 * case["cols"] * case["bias"], "flops": 12 * n}
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * (3 if case["residual"] else 2), "flops": 2 * n}
    n = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
    small = 8 * case["tokens"] + 4 * case["rot"]
    if op == "rope":
        return {"bytes": 4 * n + small, "flops": 3 * n}
    small += 2 * case["dim"] * (2 if case["gain"] == "bf16" else 4)
    if op == "qk":
        return {"bytes": 4 * n + small, "flops": 7 * n}
    return {"bytes": 6 * n + small + 8 * case["dim"], "flops": 14 * n}


def _exact_keep(shape, s):
    """The kept elements as 0 or the scale: 32-bit products by 16-bit halves."""
    def mul32(a, m):     # high and low 32 bits of a * m
        lo, hi = (a & 65535) * m, (a >> 16) * m
        lo_hi = (lo >> 16) + (hi & 65535)
        return (hi >> 16) + (lo_hi >> 16), ((lo_hi & 65535) << 16) | (lo & 65535)

    n = shape[0] * shape[1] // 8
    block = torch.arange(n, device="cuda", dtype=torch.int64)
    x = [block % 2 ** 32, block // 2 ** 32, torch.zeros_like(block) + s["offset"] % 2 ** 32,
         torch.zeros_like(block) + s["offset"] // 2 ** 32]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
    for r in range(10):
        h0, l0 = mul32(x[0], 0xD2511F53)
        h1, l1 = mul32(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ ((key[0] + r * 0x9E3779B9) % 2 ** 32), l1,
             h0 ^ x[3] ^ ((key[1] + r * 0xBB67AE85) % 2 ** 32), l0]
    limit = round(s["case"]["p"] * 65536)
    out = torch.empty((n, 8), dtype=torch.float64, device="cuda")
    for j in range(8):
        out[:, j] = (x[j // 2] // 2 ** (16 * (j % 2)) % 65536 >= limit).double()
    return (out * (65536.0 / (65536 - limit))).reshape(shape)


def _exact_act(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.relu(z), torch.sign(torch.relu(z))
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / 2 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z ** 2 / 2) / (2 * math.pi) ** 0.5
    # the other two are z sigmoid(w)
    c = (8 / math.pi) ** 0.5
    w = z if act == "silu" else c * (z + 0.044715 * z ** 3)
    dw = torch.ones_like(z) if act == "silu" else c * (1 + 0.134145 * z ** 2)
    up, down = torch.sigmoid(w), torch.sigmoid(-w)
    return z * up, up + z * up * down * dw


def _exact_turn(x, s, sign):
    """x times the rotation of its token, pair by pair, as complex numbers."""
    rot, out = s["case"]["rot"], x.clone()
    pairs = (x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
             if s["case"]["layout"] == "half" else x[..., :rot].unflatten(-1, (rot // 2, 2)))
    by = torch.polar(torch.full_like(s["angles"], s["magnitude"]).expand(x.shape[0], -1),
                     sign * torch.outer(s["positions"].double(), s["angles"]))
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by.unsqueeze(1))
    out[..., :rot] = (turned.transpose(-1, -2) if s["case"]["layout"] == "half" else turned).flatten(-2)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = lambda t: t.to(torch.float64)  # noqa: E731
    if op == "linear":
        z = d(s["X"]) @ d(s["W"]).T
        z = z if s["bias"] is None else z + d(s["bias"])
        y = _exact_act(z, case["act"])[0]
        y = y if s["mul"] is None else y * d(s["mul"])
        y = y * _exact_keep(y.shape, s) if case["p"] else y
        y = y if s["residual"] is None else y + d(s["residual"])
        return [y, z] if case["z"] else [y]
    if op == "epilogue_bwd":
        a, slope = _exact_act(d(s["Z"]), case["act"])
        da = d(s["dY"]) * (_exact_keep(a.shape, s) if case["p"] else 1)
        dz = da * slope * (1 if s["mul"] is None else d(s["mul"]))
        out = [dz] if s["mul"] is None else [dz, da * a]
        return out + [torch.sum(dz, 0)] if case["bias"] else out
    if op == "dropout":
        y = d(s["x"]) * _exact_keep(s["x"].shape, s)
        return [y if s["residual"] is None else y + d(s["residual"])]
    if op == "rope":
        return [_exact_turn(d(s[n]), s, -1 if case["inverse"] else 1) for n in ("q", "k")]
    out, gains = [], []
    for n in ("q", "k"):
        x, gain = d(s[n]), d(s[n + "_gain"])
        r = 1 / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / case["dim"] + EPS)
        if op == "qk":
            out.append(_exact_turn(x * r * gain, s, 1))
            continue
        dn = _exact_turn(d(s["d" + n]), s, -1)
        dot = torch.sum(dn * gain * x, -1, keepdim=True)
        out.append(r * gain * dn - x * r ** 3 * dot / case["dim"])
        gains.append(torch.sum(dn * x * r, (0, 1)))
    return out + gains
