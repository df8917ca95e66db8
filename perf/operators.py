"""Cases for the operators around a linear layer's weight gradient: the RMS norm
in front of it (with the residual's addition and an 8-bit output) and its backward
pass, the 128-block quantiser, the 8-bit matrix products of the layer's forward
and input-gradient passes, and gradient clipping by the global norm.

Each case is one call (for clipping: the calls of one optimizer step).  `run`
computes it either in plain torch operations in 32 bits, or, where `own` is true,
with the library's entry points.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
BLOCK = 128          # columns (and for weights rows) that share one scale
F8_MAX = 448.0       # largest finite e4m3 value
TINY = 2.0 ** -126   # smallest scale of a block that is not all zero
EPS = 1e-5
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=10)

# The seven projections of a Llama-3.1-8B layer: (d_out, d_in).
LAYER = "4096x4096,1024x4096,1024x4096,4096x4096,14336x4096,14336x4096,4096x14336"


def listed():
    return [
        # one new token of a serving step: only latency counts
        dict(name="norm_1_token", op="norm", rows=1, cols=4096, residual=True, y=False, fp8=True,
             gain="bf16"),
        # a small training micro-batch: everything the backward pass and both products need
        dict(name="norm_512_all_outputs", op="norm", rows=512, cols=4096, residual=True, y=True,
             fp8=True, gain="fp32"),
        # the norm of a long batch without 8-bit output, at a ragged row count
        dict(name="norm_8191_bf16", op="norm", rows=8191, cols=4096, residual=True, y=True,
             fp8=False, gain="bf16"),
        # odd sizes: a small model's norm, columns that do not fill their last block
        dict(name="norm_bwd_333x1032", op="norm_bwd", rows=333, cols=1032, dsum=False,
             gain="bf16"),
        # the norm's backward pass on a long batch, with the residual stream's gradient
        dict(name="norm_bwd_8192", op="norm_bwd", rows=8192, cols=4096, dsum=True, gain="fp32"),
        # the output gradient of the gate projection, before the 8-bit input gradient
        dict(name="quantize_rows_8192", op="quant", rows=8192, cols=14336, block_rows=1),
        # a weight after its optimizer step, 128 x 128 blocks, the last ones ragged
        dict(name="quantize_weight_1000x4112", op="quant", rows=1000, cols=4112, block_rows=128),
        # one token through the gate projection: the weight's bytes are all that counts
        dict(name="linear_1_token", op="linear", bt=1, d_in=4096, d_out=14336),
        # the gate projection's forward pass on a long batch
        dict(name="linear_8192", op="linear", bt=8192, d_in=4096, d_out=14336),
        # the input gradient of the gate projection at a ragged token count
        dict(name="dgrad_2000", op="dgrad", bt=2000, d_in=4096, d_out=14336),
        # clipping and AdamW on a small model's matrices and gains: many launches, little work
        dict(name="clip_small", op="clip", shapes="264x520,520x264,1000x136", gains="520,1001,3",
             grad="bf16", moments="bf16", max_norm=1.0),
        # one layer's exact-accumulation buffers, clipped by their global norm and stepped
        dict(name="clip_layer", op="clip", shapes=LAYER, gains="4096,4096", grad="fp32",
             moments="fp32", max_norm=1.0),
    ]


def _log(rng, low, high, multiple=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / multiple)) * multiple))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quant", "linear", "dgrad", "clip"])
    gain = rng.choice(["bf16", "fp32"])
    if op == "norm":
        fp8 = rng.random() < 0.6
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192, 8),
                    residual=rng.random() < 0.7, y=not fp8 or rng.random() < 0.5, fp8=fp8,
                    gain=gain)
    if op == "norm_bwd":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192, 8),
                    dsum=rng.random() < 0.5, gain=gain)
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 14336, 8),
                    block_rows=rng.choice([1, 128]))
    if op in ("linear", "dgrad"):
        return dict(op=op, bt=_log(rng, 1, 8192), d_in=_log(rng, 256, 4096, 16),
                    d_out=_log(rng, 256, 14336, 16))
    n = rng.randint(1, 6)
    shapes = ",".join("%dx%d" % (_log(rng, 64, 4096, 8), _log(rng, 64, 4096, 8)) for _ in range(n))
    gains = ",".join(str(_log(rng, 1, 8192)) for _ in range(rng.randint(1, 4)))
    return dict(op=op, shapes=shapes, gains=gains, grad=rng.choice(["bf16", "fp32"]),
                moments=rng.choice(["bf16", "fp32"]), max_norm=rng.choice([0.25, 1.0, 1e6]))


def _pairs(text):
    return [tuple(int(v) for v in s.split("x")) for s in text.split(",")]


def _ceil(a, b):
    return -(-a // b)


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _activations(g, rows, cols, std=1.0):
    """bf16 activations with a few columns far larger than the rest, as trained models have."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    heavy = torch.rand((cols,), generator=g, device="cuda") < 0.005
    return (x * torch.where(heavy, 20.0 * std, std)).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    if op in ("norm", "norm_bwd"):
        rows, cols = case["rows"], case["cols"]
        s["gain"] = (1 + 0.2 * torch.randn((cols,), generator=g, device="cuda")).to(_dt(case["gain"]))
        s["x"] = _activations(g, rows, cols)
        if op == "norm":
            s["rstd"] = new((rows,), torch.float32)
            s["residual"] = _normal(g, (rows, cols), 3.0) if case["residual"] else None
            s["sum"] = new((rows, cols), torch.bfloat16) if case["residual"] else None
            s["y"] = new((rows, cols), torch.bfloat16) if case["y"] else None
            s["codes"] = new((rows, cols), F8) if case["fp8"] else None
            s["scales"] = new((rows, _ceil(cols, BLOCK)), torch.float32) if case["fp8"] else None
        else:
            # what the forward pass left: its input and its reciprocal norms
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dy"] = _normal(g, (rows, cols), 1e-3)
            s["dsum"] = _normal(g, (rows, cols), 1e-3) if case["dsum"] else None
            s["dx"] = new((rows, cols), torch.bfloat16)
            s["dgain"] = new((cols,), torch.float32)
            # scratch the program keeps for every norm of the model
            s["workspace"] = new((32 << 20,), torch.uint8)
    elif op == "quant":
        rows, cols, br = case["rows"], case["cols"], case["block_rows"]
        s["x"] = _normal(g, (rows, cols), 0.02) if br == BLOCK else _activations(g, rows, cols, 1e-3)
        s["codes"] = new((rows, cols), F8)
        s["scales"] = new((_ceil(rows, br), _ceil(cols, BLOCK)), torch.float32)
    elif op in ("linear", "dgrad"):
        bt, d_in, d_out = case["bt"], case["d_in"], case["d_out"]
        k = d_in if op == "linear" else d_out
        n = d_out if op == "linear" else d_in
        a = _activations(g, bt, k, 1.0 if op == "linear" else 1e-3)
        s["a"], s["sa"] = _plain_quantize(a, 1)
        s["w"], s["sw"] = _plain_quantize(_normal(g, (d_out, d_in), 0.02), BLOCK)
        s["out"] = new((bt, n), torch.bfloat16)
    else:
        shapes, gains = _pairs(case["shapes"]), _pairs(case["gains"])
        s["grads"] = [_normal(g, p, 2e-4, _dt(case["grad"])) for p in shapes]
        s["more"] = [_normal(g, p, 1e-3, torch.float32) for p in gains]
        s["w"] = [_normal(g, p, 0.02) for p in shapes]
        s["m"] = [_normal(g, p, 1e-4, _dt(case["moments"])) for p in shapes]
        s["v"] = [_normal(g, p, 1e-4, torch.float32).square().to(_dt(case["moments"])) for p in shapes]
        s["out"] = new((2,), torch.float32)   # the norm and the coefficient
        s["workspace"] = new((1 << 20,), torch.uint8)
    return s


def _plain_quantize(x, block_rows):
    """e4m3 codes of x and the scale of each block of block_rows x 128."""
    x = x.float()
    rows, cols = x.shape
    nr, nc = _ceil(rows, block_rows), _ceil(cols, BLOCK)
    pad = x.new_zeros((nr * block_rows, nc * BLOCK))
    pad[:rows, :cols] = x
    blocks = pad.view(nr, block_rows, nc, BLOCK)
    amax = blocks.abs().amax(dim=(1, 3))
    scales = torch.where(amax > 0, (amax / F8_MAX).clamp(min=TINY), torch.zeros_like(amax))
    by = torch.where(amax > 0, scales, torch.ones_like(amax))
    codes = (blocks / by[:, None, :, None]).clamp(-F8_MAX, F8_MAX).view(pad.shape)[:rows, :cols]
    return codes.to(F8), scales


def _spread(scales, block_rows, rows, cols):
    return scales.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def _plain_norm(s):
    x, r = s["x"].float(), s["residual"]
    h = x if r is None else x + r.float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * rstd * s["gain"].float()
    out = [rstd[:, 0]]
    if r is not None:
        out.append(h.to(torch.bfloat16))
    if s["y"] is not None:
        out.append(y.to(torch.bfloat16))
    if s["codes"] is not None:
        out.extend(_plain_quantize(y, 1))
    return out


def _plain_norm_bwd(s):
    xh = s["x"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    u = dy * s["gain"].float()
    dx = s["rstd"][:, None] * (u - xh * (u * xh).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return [dx.to(torch.bfloat16), (dy * xh).sum(0)]


def _plain_product(s):
    a, w = s["a"], s["w"]
    a = a.float() * _spread(s["sa"], 1, *a.shape)
    w = w.float() * _spread(s["sw"], BLOCK, *w.shape)
    y = torch.matmul(a, w.t() if s["case"]["op"] == "linear" else w)
    return [y.to(torch.bfloat16)]


def _plain_adamw(w, m, v, grad, coef):
    h = HYPER
    g = grad.float() * coef
    m1 = h["beta1"] * m.float() + (1 - h["beta1"]) * g
    v1 = h["beta2"] * v.float() + (1 - h["beta2"]) * g * g
    c1, c2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    step = (m1 / c1) / (torch.sqrt(v1 / c2) + h["eps"])
    w.copy_(w.float() * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * step)
    m.copy_(m1)
    v.copy_(v1)


def _plain_clip(s):
    squares = torch.stack([g.float().square().sum() for g in s["grads"] + s["more"]])
    norm = squares.sum().sqrt()
    coef = (s["case"]["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    [_plain_adamw(*t, coef) for t in zip(s["w"], s["m"], s["v"], s["grads"])]
    return [torch.stack([norm, coef]), s["w"], s["m"], s["v"]]


def _own(s):
    from weight_gradient_gemm_gb300 import forge
    op = s["case"]["op"]
    if op == "norm":
        forge.rmsnorm(s["x"], s["gain"], eps=EPS, residual=s["residual"], sum_out=s["sum"],
                      y=s["y"], codes=s["codes"], scales=s["scales"], rstd=s["rstd"])
        outs = (s["rstd"], s["sum"], s["y"], s["codes"], s["scales"])
        return [t for t in outs if t is not None]
    if op == "norm_bwd":
        forge.rmsnorm_backward(s["dy"], s["x"], s["gain"], s["rstd"], s["dx"], s["dgain"],
                               dsum=s["dsum"], workspace=s["workspace"])
        return [s["dx"], s["dgain"]]
    if op == "quant":
        forge.quantize_b128(s["x"], s["codes"], s["scales"], block_rows=s["case"]["block_rows"])
        return [s["codes"], s["scales"]]
    if op == "linear":
        forge.linear_fp8(s["a"], s["sa"], s["w"], s["sw"], s["out"])
        return [s["out"]]
    if op == "dgrad":
        forge.dgrad_fp8(s["a"], s["sa"], s["w"], s["sw"], s["out"])
        return [s["out"]]
    forge.grad_norm(s["grads"] + s["more"], s["case"]["max_norm"], s["out"],
                    workspace=s["workspace"])
    [forge.adamw_clip(g, w, m, v, s["out"], **HYPER)
     for g, w, m, v in zip(s["grads"], s["w"], s["m"], s["v"])]
    return [s["out"], s["w"], s["m"], s["v"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_bwd":
        return _plain_norm_bwd(state)
    if op == "quant":
        return list(_plain_quantize(state["x"], state["case"]["block_rows"]))
    if op in ("linear", "dgrad"):
        return _plain_product(state)
    return _plain_clip(state)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols = case["rows"], case["cols"]
        n, gain = rows * cols, cols * (2 if case["gain"] == "bf16" else 4)
        if op == "norm":
            by = 2 * n + gain + 4 * rows + (4 * n if case["residual"] else 0)
            by += (2 * n if case["y"] else 0)
            by += (n + 4 * rows * _ceil(cols, BLOCK) if case["fp8"] else 0)
            return {"bytes": by, "flops": 6 * n}
        by = 6 * n + gain + 4 * rows + 4 * cols + (2 * n if case["dsum"] else 0)
        return {"bytes": by, "flops": 9 * n}
    if op == "quant":
        n = case["rows"] * case["cols"]
        scales = _ceil(case["rows"], case["block_rows"]) * _ceil(case["cols"], BLOCK)
        return {"bytes": 3 * n + 4 * scales, "flops": 3 * n}
    if op in ("linear", "dgrad"):
        bt, d_in, d_out = case["bt"], case["d_in"], case["d_out"]
        k, n = (d_in, d_out) if op == "linear" else (d_out, d_in)
        scales = bt * _ceil(k, BLOCK) + _ceil(d_in, BLOCK) * _ceil(d_out, BLOCK)
        return {"bytes": bt * k + d_in * d_out + 2 * bt * n + 4 * scales,
                "flops": 2 * bt * d_in * d_out}
    params = sum(a * b for a, b in _pairs(case["shapes"]))
    more = sum(a for (a,) in _pairs(case["gains"]))
    grad, mom = (2 if case[k] == "bf16" else 4 for k in ("grad", "moments"))
    # the step needs the norm of every gradient first, so a gradient is read twice
    return {"bytes": params * (2 * grad + 4 + 4 * mom) + 4 * more + 8, "flops": 18 * params}


def _exact_quantize(y, block_rows):
    """The codes' values (rounded to e4m3, ties to even) and the scales, in 64 bits."""
    rows, cols = y.shape
    nr, nc = _ceil(rows, block_rows), _ceil(cols, BLOCK)
    big = torch.zeros((nr * block_rows, nc * BLOCK), dtype=torch.float64, device=y.device)
    big[:rows, :cols] = y
    amax = big.reshape(nr, block_rows, nc, BLOCK).abs().amax(dim=3).amax(dim=1)
    scales = torch.where(amax > 0, torch.clamp(amax / 448, min=TINY), amax)
    full = scales.repeat_interleave(block_rows, 0).repeat_interleave(BLOCK, 1)[:rows, :cols]
    q = torch.where(full > 0, y / full, torch.zeros_like(y)).clamp(-448, 448)
    # spacing of e4m3 around q: 2^(e-3), with e no lower than the smallest normal exponent
    step = torch.exp2(torch.clamp(torch.frexp(q)[1] - 1, min=-6).double() - 3)
    return torch.round(q / step) * step, scales


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = lambda t: t.to(torch.float64)  # noqa: E731
    if op == "norm":
        h = d(s["x"]) + (0 if s["residual"] is None else d(s["residual"]))
        rstd = 1 / torch.sqrt(torch.sum(h ** 2, 1) / case["cols"] + EPS)
        y = h * rstd.unsqueeze(1) * d(s["gain"])
        out = [rstd] + ([h] if case["residual"] else []) + ([y] if case["y"] else [])
        return out + (list(_exact_quantize(y, 1)) if case["fp8"] else [])
    if op == "norm_bwd":
        h, r, dy, gain = d(s["x"]), d(s["rstd"]).unsqueeze(1), d(s["dy"]), d(s["gain"])
        dot = torch.sum(dy * gain * h, 1, keepdim=True)
        dx = r * gain * dy - h * r ** 3 * dot / case["cols"]
        if case["dsum"]:
            dx += d(s["dsum"])
        return [dx, torch.sum(dy * (h * r), 0)]
    if op == "quant":
        return list(_exact_quantize(d(s["x"]), case["block_rows"]))
    if op in ("linear", "dgrad"):
        a = d(s["a"]) * d(s["sa"]).repeat_interleave(BLOCK, 1)[:, :s["a"].shape[1]]
        sw = d(s["sw"]).repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        w = d(s["w"]) * sw[:case["d_out"], :case["d_in"]]
        return [a @ (w.T if op == "linear" else w)]
    norm = math.sqrt(sum(float((d(g) ** 2).sum()) for g in s["grads"] + s["more"]))
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    ws, ms, vs = [], [], []
    for g, w, m, v in zip(s["grads"], s["w"], s["m"], s["v"]):
        g = d(g) * coef
        m = HYPER["beta1"] * d(m) + (1 - HYPER["beta1"]) * g
        v = HYPER["beta2"] * d(v) + (1 - HYPER["beta2"]) * g ** 2
        mh, vh = m / (1 - HYPER["beta1"] ** HYPER["step"]), v / (1 - HYPER["beta2"] ** HYPER["step"])
        w = d(w) * (1 - HYPER["lr"] * HYPER["weight_decay"])
        ws.append(w - HYPER["lr"] * mh / (torch.sqrt(vh) + HYPER["eps"]))
        ms.append(m)
        vs.append(v)
    return [torch.tensor([norm, coef], dtype=torch.float64), ws, ms, vs]
