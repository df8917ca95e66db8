"""The operators between a layer's 16-bit products in company: through the extension
and without it, on other streams, captured and replayed, from several threads, beside
memory that is not theirs, with waits that run out, and together as a block's forward
and backward pass."""
import threading

import numpy as np
import pytest
import torch

from oracle import layer as R
from tests.gpu_util import DEV, F, require_gpu
from tests.test_gpu_layer import EPILOGUES, call_linear, check_linear, f64, linear_case, ok, rand

pytestmark = pytest.mark.gpu
TIMEOUT = 9


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def every_call(bt=5, d_in=264, d_out=136, seed=1):
    """One call of each operator: a function of a stream, and its outputs."""
    b16 = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    X, W = rand(seed, (bt, d_in)), rand(seed + 1, (d_out, d_in), d_in ** -0.5)
    bias, mul, res = rand(seed + 2, (d_out,)), rand(seed + 3, (bt, d_out)), rand(seed + 4, (bt, d_out))
    Y, Z, dZ, dm, dr = (b16(bt, d_out) for _ in range(5))
    db, counter = torch.zeros(d_out, device=DEV), torch.tensor([3], device=DEV)
    qkv = rand(seed + 5, (bt, 8, 64))
    q, k = qkv[:, :4], qkv[:, 4:6]
    freqs, mag = F.rope_frequencies(64, 10000.0)
    pos = torch.arange(bt, device=DEV) * 7
    qo, ko, qn, kn, dq, dk = b16(bt, 4, 64), b16(bt, 2, 64), b16(bt, 4, 64), b16(bt, 2, 64), \
        b16(bt, 4, 64), b16(bt, 2, 64)
    gq, gk = (rand(seed + 6 + i, (64,), 1.0, torch.float32) for i in range(2))
    dgq, dgk = torch.zeros(64, device=DEV), torch.zeros(64, device=DEV)
    ws = torch.zeros(max(F.epilogue_backward_workspace_bytes(bt, d_out),
                         F.qk_norm_rope_backward_workspace_bytes(64)), dtype=torch.uint8, device=DEV)
    drop = dict(p=0.2, seed=11, offset=4, counter=counter)

    def run(stream=None):
        F.linear_bf16(X, W, Y, bias=bias, act=F.ACT_GELU_TANH, mul=mul, residual=res, Z=Z,
                      stream=stream, **drop)
        F.epilogue_backward(Y, dZ, Z=Z, act=F.ACT_GELU_TANH, mul=mul, dmul=dm, dbias=db,
                            workspace=ws, stream=stream, **drop)
        F.dropout(dZ, dr, residual=Y, stream=stream, **drop)
        F.rope(q, k, freqs, q_out=qo, k_out=ko, positions=pos, magnitude=mag, stream=stream)
        F.qk_norm_rope(q, k, gq, gk, freqs, eps=1e-5, q_out=qn, k_out=kn, positions=pos,
                       layout=F.ROPE_INTERLEAVED, stream=stream)
        F.qk_norm_rope_backward(qo, ko, q, k, gq, gk, freqs, eps=1e-5, dq_out=dq, dk_out=dk,
                                dq_gain=dgq, dk_gain=dgk, positions=pos,
                                layout=F.ROPE_INTERLEAVED, workspace=ws, stream=stream)

    outs = [Y, Z, dZ, dm, dr, db, qo, ko, qn, kn, dq, dk, dgq, dgk]
    return run, outs, dict(X=X, qkv=qkv, counter=counter)


NAMES = {"linear_bf16": 13, "epilogue_backward": 13, "dropout": 8, "rope": 10, "qk_norm_rope": 12,
         "qk_norm_rope_backward": 17}


def test_extension_and_ctypes_give_the_same(monkeypatch):
    run, outs, _ = every_call()
    taken, real = [], F._loaded()

    class Watch:
        def __getattr__(self, name):
            def fn(*a):
                st = getattr(real, name)(*a)
                taken.append((name, st, len(a)))
                return st
            return fn

    class Leave:
        def __getattr__(self, name):
            return lambda *a: -1

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    monkeypatch.setattr(F, "_call", Watch())
    for stream in (None, side, side.cuda_stream):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        run(stream)
        torch.cuda.synchronize()
        got.append([o.clone() for o in outs])
    assert {n: c for n, _, c in taken} == NAMES and all(st == 0 for _, st, _ in taken)
    monkeypatch.setattr(F, "_call", Leave())
    for o in outs:
        o.zero_()
    run()
    ok()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, outs))


def test_captured_and_replayed():
    for bt in (3, 300):
        run, outs, ins = every_call(bt=bt, seed=20)
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        for k in range(2):
            ins["X"].copy_(rand(30 + k, ins["X"].shape))
            ins["qkv"].copy_(rand(40 + k, ins["qkv"].shape))
            ins["counter"].add_(1)
            run()
            torch.cuda.synchronize()
            want = [o.clone() for o in outs]
            for o in outs:
                o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, outs))
    ok()


def test_several_threads_and_streams():
    """Eight threads, each with its own stream and buffers, at once."""
    cases = []
    for i, (bt, d_in, d_out) in enumerate([(1, 512, 264), (300, 2056, 520), (40, 1032, 136),
                                           (700, 264, 1032)] * 2):
        run, outs, _ = every_call(bt, d_in, d_out, seed=50 + i)
        run()
        torch.cuda.synchronize()
        cases.append((run, outs, [o.clone() for o in outs], torch.cuda.Stream()))
    bad = []

    def work(run, outs, want, stream):
        try:
            torch.cuda.set_device(DEV)
            for _ in range(20):
                run(stream)
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(outs, want)):
                bad.append("differs")
        except Exception as e:      # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=c) for c in cases]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not bad, bad
    ok()


def fenced(rows, cols, dtype=torch.bfloat16):
    """A matrix between two rows of sevens, and those rows."""
    pad = -(-cols // 64) * 64
    buf = torch.full((rows * cols + 2 * pad,), 7.0, device=DEV).to(dtype)
    return buf[pad:pad + rows * cols].view(rows, cols), (buf[:pad], buf[pad + rows * cols:])


def untouched(*edges):
    assert all(bool((e.float() == 7).all()) for pair in edges for e in pair)


@pytest.mark.parametrize("bt,d_in,d_out", [(1, 72, 8), (5, 136, 264), (33, 72, 72), (127, 264, 136),
                                           (129, 72, 136), (257, 136, 8), (300, 2056, 264),
                                           (513, 72, 520), (2001, 72, 1096)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_linear_leaves_the_rest_alone(bt, d_in, d_out, out):
    Y, ye = fenced(bt, d_out, out)
    Z, ze = fenced(bt, d_out)
    c = linear_case(bt, d_in, d_out, bias=torch.float32, act=R.SILU, residual=True, p=0.1)
    c["Y"], c["Z"] = Y, Z
    call_linear(c)
    check_linear(c)
    untouched(ye, ze)


def test_elementwise_leaves_the_rest_alone():
    for rows, cols in ((1, 8), (3, 264), (700, 136)):
        x, Z = rand(1, (rows, cols)), rand(2, (rows, cols))
        y, ye = fenced(rows, cols)
        dz, de = fenced(rows, cols)
        dm, me = fenced(rows, cols)
        db, be = fenced(1, cols, torch.float32)
        ws, wse = fenced(1, max(F.epilogue_backward_workspace_bytes(rows, cols) // 4, 64), torch.float32)
        F.dropout(x, y, p=0.1, seed=1)
        F.epilogue_backward(x, dz, Z=Z, act=F.ACT_SILU, mul=x, dmul=dm, dbias=db[0], workspace=ws)
        ok()
        untouched(ye, de, me, be, wse)


@pytest.mark.parametrize("dim,rot", [(64, 64), (80, 24), (8, 8), (256, 128)])
def test_heads_leave_the_rest_alone(dim, rot):
    """Queries and keys inside a wider buffer: what lies between, before and behind stays."""
    tokens, row = 37, 7 * dim + 64
    buf = torch.full((tokens + 2, row), 7.0, dtype=torch.bfloat16, device=DEV)
    q = buf[1:-1, :3 * dim].unflatten(1, (3, dim))
    k = buf[1:-1, 4 * dim:6 * dim].unflatten(1, (2, dim))
    freqs, _ = F.rope_frequencies(rot, 10000.0)
    g = torch.ones(dim, device=DEV)
    ws, wse = fenced(1, F.qk_norm_rope_backward_workspace_bytes(dim) // 4, torch.float32)
    dg = [fenced(1, dim, torch.float32) for _ in range(2)]
    x, y = rand(3, (tokens, 3, dim)), rand(4, (tokens, 2, dim))
    for layout in (F.ROPE_HALF, F.ROPE_INTERLEAVED):
        for call in (lambda: F.rope(q, k, freqs, layout=layout),
                     lambda: F.qk_norm_rope(q, k, g, g, freqs, eps=1e-5, layout=layout),
                     lambda: F.qk_norm_rope_backward(q, k, x, y, g, g, freqs, eps=1e-5,
                                                     dq_gain=dg[0][0][0], dk_gain=dg[1][0][0],
                                                     layout=layout, workspace=ws)):
            q.copy_(x)
            k.copy_(y)
            call()
            ok()
            assert not torch.equal(q, x) and bool(torch.isfinite(q).all() and torch.isfinite(k).all())
            rest = buf.clone()
            rest[1:-1, :3 * dim] = 7.0
            rest[1:-1, 4 * dim:6 * dim] = 7.0
            assert bool((rest == 7).all())
            untouched(wse, dg[0][1], dg[1][1])


@pytest.mark.parametrize("bt,d_in,d_out", [(65, 136, 19600), (100, 8, 20000), (128, 72, 40008)])
def test_linear_up_to_128_tokens_and_many_outputs(bt, d_in, d_out):
    """More tiles of 128 outputs than SMs: pairs with half of their rows empty."""
    c = linear_case(bt, d_in, d_out, **EPILOGUES["all"])
    call_linear(c)
    check_linear(c)


@pytest.mark.parametrize("bt,d_out,how", [
    (1, 264, {}), (40, 20000, {}), (128, 264, dict(splits=1)), (300, 520, dict(cg=1, splits=2)),
    (300, 520, dict(cg=2)), (300, 520, dict(cg=2, bn=256)), (1000, 2056, dict(cg=2, bn=128)),
    (2000, 2600, {})])
def test_fp32_outputs_of_long_reductions(bt, d_out, how, tune):
    """The tensor core cuts sums off: an instruction (16 products) loses less than 2^-23 of the
    sum so far.  Over 512 elements, whose j-th of 32 partial sums is about sqrt(j / 32) of the
    512's, that is less than 2^-23 (2 / 3) 32 of it.  What the 32 sums of 512 lose is
    independent (it has the sign of each, and they are random), so in the 2-norm it is that
    share of the whole; adding them in fp32 costs 2^-24 each.  (Cut off throughout, 16384
    elements lose 1.2 10^-9 each, 1.9 10^-5 in all.)"""
    tune(**how)
    c = linear_case(bt, 16384, d_out, residual=False, out=torch.float32)
    call_linear(c)
    want = c["X"].double() @ c["W"].double().t()
    off = float((c["Y"].double() - want).norm() / want.norm())
    assert off <= 2.0 ** -23 * 2 / 3 * 32 + 32 * 2.0 ** -24


@pytest.mark.parametrize("bt,d_out,how", [
    (1, 264, {}), (40, 20000, {}), (128, 264, dict(splits=1)), (300, 520, dict(cg=1, splits=2)),
    (300, 520, dict(cg=2)), (1000, 2056, dict(cg=2, bn=128))])
@pytest.mark.parametrize("d_in", [512, 16384])
def test_fp32_outputs_of_operands_of_one_sign(bt, d_out, how, d_in, tune):
    """Products of one sign: what is cut off adds up instead of averaging out.  An instruction
    loses between nothing and one unit in the last place of the sum so far, on average half of
    at most 2^-23 of it; the i-th of 32 partial sums is i / 32 of the 512's, so that 512
    elements lose 2^-24 (1 + ... + 32) / 32 = 16.5 2^-24 of their sum.  Adding the 32 sums of
    512 in fp32 rounds the i-th time by at most 2^-24 i / 32, either way: the root of the
    squares is 3.4 2^-24.  (1024 elements in one sum would lose twice 16.5 2^-24 less the
    seventh part by which half a unit is below 2^-24 on average: 28.)"""
    tune(**how)
    g = torch.Generator().manual_seed(7)
    X, W = (torch.randn(s, generator=g).abs().bfloat16().to(DEV) for s in ((bt, d_in), (d_out, d_in)))
    Y = torch.empty((bt, d_out), device=DEV)
    F.linear_bf16(X, W, Y)
    ok()
    want = X.double() @ W.double().t()
    assert float((Y.double() - want).norm() / want.norm()) <= (16.5 + 3.4) * 2.0 ** -24


@pytest.mark.parametrize("group_m", [-3, 1, 2, 64, 1000])
def test_linear_tile_order(group_m, tune):
    """Groups of tile rows of any size (what lies outside 1..64: automatic)."""
    tune(cg=2, group_m=group_m)
    c = linear_case(1100, 136, 2056, **EPILOGUES["all"])
    call_linear(c)
    check_linear(c)


@pytest.mark.parametrize("heads", [(0, 2), (2, 0), (0, 0)])
def test_kinds_without_heads(heads):
    """A kind without heads: the other is as alone, its gain's gradient is zero."""
    dim, tokens = 64, 9
    freqs, _ = F.rope_frequencies(dim, 10000.0)
    x = [rand(1 + i, (tokens, h, dim)) for i, h in enumerate(heads)]
    dy = [rand(3 + i, (tokens, h, dim)) for i, h in enumerate(heads)]
    g = [rand(5 + i, (dim,), 1.0, torch.float32) for i in range(2)]
    ws = torch.empty(F.qk_norm_rope_backward_workspace_bytes(dim), dtype=torch.uint8, device=DEV)
    dg = [torch.full((dim,), 7.0, device=DEV) for _ in range(2)]
    out = [torch.empty_like(t) for t in x]
    F.qk_norm_rope_backward(*dy, *x, *g, freqs, eps=1e-5, dq_out=out[0], dk_out=out[1],
                            dq_gain=dg[0], dk_gain=dg[1], workspace=ws)
    for i, h in enumerate(heads):
        if h == 0:
            ok()
            assert bool((dg[i] == 0).all())
            continue
        one, dg1 = torch.empty_like(x[i]), torch.empty(dim, device=DEV)
        F.qk_norm_rope_backward(dy[i], None, x[i], None, g[i], None, freqs, eps=1e-5, dq_out=one,
                                dq_gain=dg1, workspace=ws)
        ok()
        assert torch.equal(out[i], one) and torch.equal(dg[i], dg1)   # the same blocks
    for fn in (lambda o: F.rope(*x, freqs, q_out=o[0], k_out=o[1]),
               lambda o: F.qk_norm_rope(*x, *g, freqs, eps=1e-5, q_out=o[0], k_out=o[1])):
        fn(out)
        ok()


@pytest.mark.parametrize("bt,d_in,d_out,how", [
    (3, 4104, 264, {}), (100, 1032, 520, {}), (3, 264, 40000, {}),            # few tokens
    (300, 4104, 520, dict(cg=1, splits=4)), (700, 264, 2056, dict(cg=1, splits=1)),
    (700, 520, 2056, dict(cg=2)), (3000, 264, 2600, dict(cg=2))])             # pairs
def test_linear_waits_run_out(bt, d_in, d_out, how, tune):
    """The first copy waits for bytes that never come: the kernel records the timeout and
    returns, the context stays usable, and what lies beside the outputs is not touched."""
    tune(**how)
    Y, ye = fenced(bt, d_out)
    Z, ze = fenced(bt, d_out)
    c = linear_case(bt, d_in, d_out, **EPILOGUES["all"])
    c["Y"], c["Z"] = Y, Z
    call_linear(c)
    want = [Y.clone(), Z.clone()]
    F.set_wait_limit_ns(20_000_000)
    try:
        F.debug_drop_first_arrival(True)
        F.linear_bf16(c["X"], c["W"], Y, bias=c["bias"], act=c["act"], mul=c["mul"],
                      residual=c["residual"], Z=Z, p=c["p"], seed=1)
        assert F.device_error() == TIMEOUT
        assert F.device_error() == 0      # cleared
    finally:
        F.debug_drop_first_arrival(False)
        F.set_wait_limit_ns(2_000_000_000)
    untouched(ye, ze)
    call_linear(c)
    assert torch.equal(Y, want[0]) and torch.equal(Z, want[1])


@pytest.mark.parametrize("bt,d_in,d_out,how", [
    (3, 4104, 264, {}), (100, 1032, 520, dict(splits=1)), (300, 4104, 520, dict(cg=1, splits=2)),
    (700, 1032, 2056, dict(cg=2)), (40, 1032, 20000, {})])
def test_linear_waits_run_out_with_fp32_outputs(bt, d_in, d_out, how, tune):
    tune(**how)
    Y, ye = fenced(bt, d_out, torch.float32)
    c = linear_case(bt, d_in, d_out, act=R.SILU, residual=True, out=torch.float32)
    c["Y"] = Y
    call_linear(c)
    want = Y.clone()
    F.set_wait_limit_ns(20_000_000)
    try:
        F.debug_drop_first_arrival(True)
        F.linear_bf16(c["X"], c["W"], Y, act=c["act"], residual=c["residual"])
        assert F.device_error() == TIMEOUT
        assert F.device_error() == 0      # cleared
    finally:
        F.debug_drop_first_arrival(False)
        F.set_wait_limit_ns(2_000_000_000)
    untouched(ye)
    call_linear(c)
    assert torch.equal(Y, want)


def test_python_refusals():
    x, w, y = rand(1, (4, 256)), rand(2, (8, 256)), torch.empty((4, 8), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        F.linear_bf16(x, w[:, :128], y)
    with pytest.raises(ValueError):
        F.linear_bf16(x[:, ::2], w[:, ::2], y)
    with pytest.raises(TypeError):
        F.linear_bf16(x.half(), w, y)
    with pytest.raises(ValueError):
        F.linear_bf16(x, w, y, residual=x)
    with pytest.raises(ValueError):
        F.linear_bf16(x, w, y, bias=torch.zeros(4, device=DEV))
    for kw in (dict(act=9), dict(p=1.0), dict(Z=y)):
        with pytest.raises(F.ForgeError):
            F.linear_bf16(x, w, y, **kw)
    with pytest.raises((ValueError, TypeError)):
        F.dropout(x, x, p=0.5, seed=1, counter=torch.zeros(1, device=DEV))
    q, f = rand(3, (4, 2, 64)), torch.zeros(32, dtype=torch.int64, device=DEV)
    g = torch.ones(64, device=DEV)
    for call in (lambda: F.rope(q.transpose(1, 2), None, f), lambda: F.rope(q[0], None, f),
                 lambda: F.rope(q, q[:3], f), lambda: F.rope(q, None, f.float()),
                 lambda: F.rope(q, None, f, positions=torch.arange(3, device=DEV)),
                 lambda: F.qk_norm_rope(q, None, g[:8], None, f, eps=1e-5),
                 lambda: F.qk_norm_rope(q, q.clone(), g, None, f, eps=1e-5),
                 lambda: F.qk_norm_rope_backward(q, None, q[:, :1], None, g, None, f, eps=1e-5)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(F.ForgeError):
        F.rope(q[:, :, :60], None, f[:8])                       # dim not a multiple of 8
    with pytest.raises(F.ForgeError):
        F.rope(q, None, torch.zeros(40, dtype=torch.int64, device=DEV))      # wider than a head
    with pytest.raises(F.ForgeError):
        F.rope(q, q, f)                                          # the same heads twice
    with pytest.raises(F.ForgeError):
        F.qk_norm_rope_backward(q, None, q.clone(), None, g, None, f, eps=1e-5,
                                dq_gain=torch.zeros(64, device=DEV))          # no workspace
    ok()


# ---------------------------------------------------------------- together
class Block:
    """The linear layers, norms and rotations of a block, without attention itself (the
    rotated queries, keys and the values go straight into the output projection), forward
    and backward, with everything the backward pass needs kept from the forward one."""

    def __init__(self, bt=37, d=128, hq=2, hk=1, dim=32, ff=264, p=0.1):
        self.bt, self.d, self.hq, self.hk, self.dim, self.p = bt, d, hq, hk, dim, p
        n = (hq + 2 * hk) * dim
        self.par = dict(g1=1 + rand(1, (d,), 0.2, torch.float32), Wqkv=rand(2, (n, d), d ** -0.5),
                        bqkv=rand(3, (n,), 0.3, torch.float32),
                        gq=1 + rand(4, (dim,), 0.2, torch.float32),
                        gk=1 + rand(5, (dim,), 0.2, torch.float32), Wo=rand(6, (d, n), n ** -0.5),
                        bo=rand(7, (d,), 0.3, torch.float32), g2=1 + rand(8, (d,), 0.2, torch.float32),
                        Wg=rand(9, (ff, d), d ** -0.5), Wu=rand(10, (ff, d), d ** -0.5),
                        Wd=rand(11, (d, ff), ff ** -0.5))
        self.x, self.dout = rand(12, (bt, d)), rand(13, (bt, d))
        self.freqs, self.mag = F.rope_frequencies(dim, 10000.0)
        self.pos = torch.arange(bt, device=DEV) + 100

    def b16(self, *s):
        return torch.empty(s, dtype=torch.bfloat16, device=DEV)

    def heads(self, t):
        v = t.view(self.bt, self.hq + 2 * self.hk, self.dim)
        return v[:, :self.hq], v[:, self.hq:self.hq + self.hk]

    def run(self):
        P, bt, d = self.par, self.bt, self.d
        n, ff = P["Wqkv"].shape[0], P["Wg"].shape[0]
        f32 = dict(device=DEV)
        how = dict(positions=self.pos, magnitude=self.mag)
        # forward
        n1, r1 = self.b16(bt, d), torch.empty(bt, **f32)
        F.rmsnorm(self.x, P["g1"], eps=1e-5, y=n1, rstd=r1)
        qkv = self.b16(bt, n)
        F.linear_bf16(n1, P["Wqkv"], qkv, bias=P["bqkv"])
        rot = qkv.clone()
        F.qk_norm_rope(*self.heads(rot), P["gq"], P["gk"], self.freqs, eps=1e-5, **how)
        h = self.b16(bt, d)
        drop = dict(p=self.p, seed=5, offset=1)
        F.linear_bf16(rot, P["Wo"], h, bias=P["bo"], residual=self.x, **drop)
        n2, r2 = self.b16(bt, d), torch.empty(bt, **f32)
        F.rmsnorm(h, P["g2"], eps=1e-5, y=n2, rstd=r2)
        up, Z, a, out = self.b16(bt, ff), self.b16(bt, ff), self.b16(bt, ff), self.b16(bt, d)
        F.linear_bf16(n2, P["Wu"], up)
        F.linear_bf16(n2, P["Wg"], a, act=F.ACT_SILU, mul=up, Z=Z)
        F.linear_bf16(a, P["Wd"], out, residual=h)
        # backward
        G = {k: torch.empty(v.shape, **f32) for k, v in P.items()}
        ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
        da = self.b16(bt, ff)
        F.dgrad(self.dout, P["Wd"], da)
        F.wgrad(a, self.dout, G["Wd"])
        dz, dup = self.b16(bt, ff), self.b16(bt, ff)
        F.epilogue_backward(da, dz, Z=Z, act=F.ACT_SILU, mul=up, dmul=dup)
        dn, dn_u = self.b16(bt, d), self.b16(bt, d)
        F.dgrad(dz, P["Wg"], dn)
        F.dgrad(dup, P["Wu"], dn_u)
        F.wgrad(n2, dz, G["Wg"])
        F.wgrad(n2, dup, G["Wu"])
        dn += dn_u
        dh = self.b16(bt, d)
        F.rmsnorm_backward(dn, h, P["g2"], r2, dh, G["g2"], dsum=self.dout, workspace=ws)
        do = self.b16(bt, d)
        F.epilogue_backward(dh, do, dbias=G["bo"], workspace=ws, **drop)
        drot = self.b16(bt, n)
        F.dgrad(do, P["Wo"], drot)
        F.wgrad(rot, do, G["Wo"])
        q, k = self.heads(qkv)
        F.qk_norm_rope_backward(*self.heads(drot), q, k, P["gq"], P["gk"], self.freqs, eps=1e-5,
                                dq_gain=G["gq"], dk_gain=G["gk"], workspace=ws, **how)
        F.epilogue_backward(drot, dbias=G["bqkv"], workspace=ws)
        dn1, dx = self.b16(bt, d), self.b16(bt, d)
        F.dgrad(drot, P["Wqkv"], dn1)
        F.wgrad(n1, drot, G["Wqkv"])
        F.rmsnorm_backward(dn1, self.x, P["g1"], r1, dx, G["g1"], dsum=dh, workspace=ws)
        return out, dx, G

    def exact(self):
        """The same in fp64 by autograd."""
        P = {k: torch.from_numpy(f64(v)).requires_grad_() for k, v in self.par.items()}
        x = torch.from_numpy(f64(self.x)).requires_grad_()
        norm = lambda t, g: t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-5) * g  # noqa: E731
        qkv = norm(x, P["g1"]) @ P["Wqkv"].T + P["bqkv"]
        v = qkv.view(self.bt, -1, self.dim)
        rad = torch.from_numpy(R.frequencies(self.dim, 10000.0)[0])
        w = torch.outer(self.pos.cpu().double(), rad)[:, None]

        def turn(t):
            a, b = t.chunk(2, -1)
            return torch.cat([a * w.cos() - b * w.sin(), b * w.cos() + a * w.sin()], -1)

        q = turn(norm(v[:, :self.hq], P["gq"]))
        k = turn(norm(v[:, self.hq:self.hq + self.hk], P["gk"]))
        rot = torch.cat([q, k, v[:, self.hq + self.hk:]], 1).reshape(self.bt, -1)
        keep = torch.from_numpy(R.keep(self.bt, self.d, self.p, 5, 1))
        h = x + keep * (rot @ P["Wo"].T + P["bo"])
        n2 = norm(h, P["g2"])
        out = h + (torch.nn.functional.silu(n2 @ P["Wg"].T) * (n2 @ P["Wu"].T)) @ P["Wd"].T
        out.backward(torch.from_numpy(f64(self.dout)))
        return out, x.grad, {k: v.grad for k, v in P.items()}


@pytest.mark.parametrize("bt", [1, 37, 300])
def test_a_block_together(bt):
    """Forward and backward of a block against autograd in fp64.  On the longest path 16
    tensors are rounded to bf16, each by at most 2^-8 of its values; the layers between
    are near-isometries (weights of variance 1 / d_in, norms, a residual stream), so a
    result is off by at most about 16 2^-8 of its own norm."""
    block = Block(bt=bt)
    out, dx, G = block.run()
    ok()
    want, dx64, G64 = block.exact()
    off = lambda a, b: np.linalg.norm(f64(a) - b.detach().numpy()) / np.linalg.norm(b.detach().numpy())  # noqa: E731
    assert off(out, want) <= 16 * 2.0 ** -8
    assert off(dx, dx64) <= 16 * 2.0 ** -8
    for name in G:
        assert off(G[name], G64[name]) <= 16 * 2.0 ** -8, name
    out2, dx2, G2 = block.run()
    assert torch.equal(out, out2) and torch.equal(dx, dx2)
    assert all(torch.equal(G[k], G2[k]) for k in G)
