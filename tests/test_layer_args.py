"""Refusals of the operators between a layer's 16-bit products (host checks: no GPU is
touched), and pins of their fp64 definitions."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import layer as R
from weight_gradient_gemm_gb300 import _build
from weight_gradient_gemm_gb300 import forge as F

# fake, aligned, far apart addresses: never dereferenced
A, B, C, D, E, G, H, J = (1 << k for k in (20, 30, 34, 36, 38, 40, 42, 44))
OK, NULL, ALIGN, SHAPE, FORMAT, HYPER, ALIAS, ARCH = range(8)
F32, BF16 = F.DT_FP32, F.DT_BF16
# what a call that passes every check answers with here: there is no GB300, or the driver
# cannot be asked for one
REACHED = (ARCH, 8, 10)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return F.lib()


@pytest.fixture(autouse=True)
def _no_gpu_touched():
    if torch.cuda.is_available():
        pytest.skip("the addresses are not the GPU's")


def test_header_declares_the_operators():
    names = F.header_functions()
    for n in ("forge_linear_bf16", "forge_epilogue_backward",
              "forge_epilogue_backward_workspace_bytes", "forge_dropout", "forge_rope",
              "forge_qk_norm_rope", "forge_qk_norm_rope_backward",
              "forge_qk_norm_rope_backward_workspace_bytes", "forge_rope_frequencies"):
        assert n in names


def drop(p=0.0, seed=0, offset=0, counter=None):
    return F.ForgeDrop(p, seed, offset, counter)


def lin(L, X=A, W=B, Y=C, dt=BF16, bt=4, d_in=256, d_out=512, bias=None, bdt=F32, act=0, mul=None,
        res=None, z=None, d=None):
    e = F.ForgeEpilogue(bias, bdt, act, mul, res, z, d or drop())
    return L.forge_linear_bf16(X, W, Y, dt, ctypes.byref(e), bt, d_in, d_out, None)


def test_linear_refusals(L):
    assert lin(L, bt=0) == OK
    assert L.forge_linear_bf16(A, B, C, BF16, None, 0, 256, 512, None) == OK
    for kw in (dict(bt=-1), dict(d_in=0), dict(d_out=0), dict(d_in=4), dict(d_out=12),
               dict(bt=1 << 31), dict(d_in=1 << 31), dict(d_out=1 << 31)):
        assert lin(L, **kw) == SHAPE, kw
    for kw in (dict(dt=2), dict(bias=D, bdt=7), dict(act=-1), dict(act=5)):
        assert lin(L, **kw) == FORMAT, kw
    for p in (-0.1, 1.0, float("nan"), float("inf")):
        assert lin(L, d=drop(p)) == HYPER, p
    assert lin(L, d=drop(0.5, counter=D + 4)) == ALIGN
    for kw in (dict(X=None), dict(W=None), dict(Y=None)):
        assert lin(L, **kw) == NULL, kw
    for kw in (dict(X=A + 8), dict(W=B + 2), dict(Y=C + 8), dict(bias=D + 8), dict(mul=D + 2),
               dict(res=D + 4), dict(z=D + 8)):
        assert lin(L, **kw) == ALIGN, kw
    for kw in (dict(Y=A), dict(Y=B + 4096), dict(bias=C), dict(z=C), dict(z=A), dict(z=D, mul=D),
               dict(z=D, res=D), dict(res=C + 16), dict(mul=C + 1024), dict(res=C, dt=F32),
               dict(mul=C, dt=F32), dict(d=drop(0.5, counter=C + 8)), dict(z=D, bias=D)):
        assert lin(L, **kw) == ALIAS, kw
    for kw in (dict(), dict(res=C), dict(mul=C), dict(res=D, mul=E, z=G, bias=H), dict(bt=1 << 20),
               dict(d=drop(0.9999999))):
        assert lin(L, **kw) in REACHED, kw


def bwd(L, dy=A, z=B, mul=None, act=4, d=None, dz=C, dm=None, db=None, rows=4, cols=256, ws=None,
        wb=0):
    return L.forge_epilogue_backward(dy, z, mul, act, None if d is None else ctypes.byref(d), dz,
                                     dm, db, rows, cols, ws, wb, None)


def test_epilogue_backward_refusals(L):
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=20), dict(rows=1 << 31),
               dict(rows=1 << 30, cols=1 << 16)):
        assert bwd(L, **kw) == SHAPE, kw
    assert bwd(L, act=5) == FORMAT and bwd(L, d=drop(1.0)) == HYPER
    for kw in (dict(dz=None), dict(dy=None), dict(z=None), dict(dm=D), dict(z=None, act=0, mul=E,
                                                                          dm=D)):
        assert bwd(L, **kw) == NULL, kw
    for kw in (dict(dy=A + 8), dict(z=B + 2), dict(mul=D + 8), dict(dz=C + 8), dict(mul=E, dm=D + 8),
               dict(db=D + 4), dict(db=D, ws=E + 8, wb=64)):
        assert bwd(L, **kw) == ALIGN, kw
    for kw in (dict(dz=A + 16), dict(dz=B + 512), dict(mul=E, dm=C), dict(db=A), dict(db=C),
               dict(db=D, ws=D, wb=4096), dict(db=D, ws=A, wb=4096), dict(db=D, ws=C, wb=4096),
               dict(mul=E, dm=E + 16), dict(d=drop(0.5, counter=C))):
        assert bwd(L, **kw) == ALIAS, kw
    for kw in (dict(dz=A), dict(dz=B), dict(mul=E, dz=E, dm=B), dict(mul=E, dm=E),
               dict(z=None, act=0), dict(z=None, act=0, mul=E), dict(rows=0)):
        assert bwd(L, **kw) in REACHED, kw


def test_dropout_refusals(L):
    def d(x=A, r=None, y=B, dr=drop(0.1), rows=4, cols=256):
        return L.forge_dropout(x, r, y, None if dr is None else ctypes.byref(dr), rows, cols, None)
    assert d(rows=0) == OK
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=4), dict(rows=1 << 30, cols=1 << 20)):
        assert d(**kw) == SHAPE, kw
    assert d(dr=None) == NULL and d(x=None) == NULL and d(y=None) == NULL
    assert d(dr=drop(1.5)) == HYPER and d(dr=drop(0.1, counter=C + 1)) == ALIGN
    assert d(x=A + 8) == ALIGN and d(y=B + 2) == ALIGN and d(r=C + 8) == ALIGN
    assert d(y=A + 16) == ALIAS and d(r=C, y=C + 32) == ALIAS and d(dr=drop(0.1, counter=B + 8)) == ALIAS
    for kw in (dict(y=A), dict(r=C, y=C), dict(dr=drop(0.1, counter=C))):
        assert d(**kw) in REACHED, kw


def heads(x=A, y=A, tokens=4, h=3, dim=64, xs=None, ys=None, gain=None, dy=None, dys=None, dg=None):
    xs = xs or (h * dim, dim)
    ys, dys = ys or xs, dys or xs
    return F.ForgeHeads(x, y, xs[0], xs[1], ys[0], ys[1], h, gain, dy, dys[0], dys[1], dg)


def rope(L, sets=None, n=None, freqs=G, pos=None, mag=1.0, dim=64, layout=0, tokens=4, head_dim=64,
         inverse=0):
    sets = [heads()] if sets is None else sets
    arr = (F.ForgeHeads * 2)(*sets)
    rot = F.ForgeRotation(freqs, pos, mag, dim, layout)
    return L.forge_rope(arr, len(sets) if n is None else n, ctypes.byref(rot), inverse, tokens,
                        head_dim, None)


def test_rope_refusals(L):
    assert L.forge_rope(None, 1, None, 0, 4, 64, None) == NULL
    for kw in (dict(n=0), dict(n=3), dict(tokens=-1), dict(tokens=1 << 31), dict(head_dim=0),
               dict(head_dim=60), dict(head_dim=264), dict(dim=0), dict(dim=72), dict(dim=12)):
        assert rope(L, **kw) == SHAPE, kw
    assert rope(L, layout=2) == FORMAT
    assert rope(L, mag=float("nan")) == HYPER and rope(L, mag=float("inf")) == HYPER
    assert rope(L, freqs=None) == NULL and rope(L, freqs=G + 4) == ALIGN
    assert rope(L, pos=H + 4) == ALIGN
    for kw, want in ((dict(x=None), NULL), (dict(y=None), NULL), (dict(x=A + 8), ALIGN),
                     (dict(y=B + 2), ALIGN), (dict(h=-1), SHAPE), (dict(h=1025), SHAPE),
                     (dict(xs=(196, 64)), SHAPE), (dict(xs=(192, -64)), SHAPE),
                     (dict(xs=(1 << 41, 64)), SHAPE),
                     (dict(y=B, ys=(192, 0)), ALIAS), (dict(y=B, ys=(0, 64)), ALIAS),
                     (dict(y=B, ys=(128, 64)), ALIAS), (dict(y=B, ys=(64, 128)), ALIAS),
                     (dict(y=A + 16), ALIAS), (dict(ys=(256, 64)), ALIAS), (dict(y=G), ALIAS)):
        assert rope(L, [heads(**kw)]) == want, kw
    # two kinds of heads
    row = (5 * 64, 64)
    q = dict(xs=row, h=3)
    assert rope(L, [heads(**q), heads(A + 2 * 3 * 64, A + 2 * 3 * 64, h=2, xs=row)]) in REACHED
    assert rope(L, [heads(**q), heads(A + 2 * 2 * 64, A + 2 * 2 * 64, h=2, xs=row)]) == ALIAS
    assert rope(L, [heads(**q), heads(B, A + 2 * 3 * 64, h=2, xs=row)]) in REACHED
    assert rope(L, [heads(**q), heads(B, A + 2 * 64, h=2, xs=row)]) == ALIAS
    assert rope(L, [heads(y=B), heads(C, B, h=2)]) == ALIAS
    # [heads][tokens][dim] and padded rows
    assert rope(L, [heads(y=B, ys=(64, 4 * 64))]) in REACHED
    assert rope(L, [heads(y=B, ys=(512, 64))]) in REACHED
    assert rope(L, [heads(xs=(0, 0), y=B, ys=(192, 64))]) in REACHED      # read again and again
    # one token or head: its stride is not used
    assert rope(L, [heads(xs=(3, 64))], tokens=1) in REACHED
    assert rope(L, [heads(h=1, xs=(64, 7))]) in REACHED
    # nothing to do
    assert rope(L, [heads(None, None, h=0)]) in (OK,) + REACHED
    assert rope(L, [heads(None, None)], tokens=0, freqs=None) in (OK,) + REACHED


def qk(L, sets=None, gdt=F32, eps=1e-5, tokens=4, pos=None):
    sets = [heads(y=B, gain=C)] if sets is None else sets
    arr = (F.ForgeHeads * 2)(*sets)
    rot = F.ForgeRotation(G, pos, 1.0, 64, 0)
    return L.forge_qk_norm_rope(arr, len(sets), gdt, eps, ctypes.byref(rot), tokens, 64, None)


def test_qk_norm_rope_refusals(L):
    assert qk(L) in REACHED
    assert qk(L, gdt=2) == FORMAT
    for eps in (-1.0, float("nan"), float("inf")):
        assert qk(L, eps=eps) == HYPER
    assert qk(L, [heads(y=B)]) == NULL
    assert qk(L, [heads(y=B, gain=C + 8)]) == ALIGN
    assert qk(L, [heads(y=B, gain=B + 64)]) == ALIAS
    assert qk(L, [heads(y=B, gain=C), heads(D, E, gain=B)]) == ALIAS


def qkb(L, sets=None, ws=H, wb=1 << 24, tokens=4):
    sets = [heads(y=B, gain=C, dy=D, dg=E)] if sets is None else sets
    arr = (F.ForgeHeads * 2)(*sets)
    rot = F.ForgeRotation(G, None, 1.0, 64, 0)
    return L.forge_qk_norm_rope_backward(arr, len(sets), F32, 1e-5, ctypes.byref(rot), tokens, 64, ws,
                                         wb, None)


def test_qk_norm_rope_backward_refusals(L):
    assert qkb(L) in REACHED
    assert qkb(L, [heads(y=B, gain=C, dg=E)]) == NULL
    assert qkb(L, [heads(y=B, gain=C, dy=D + 8, dg=E)]) == ALIGN
    assert qkb(L, [heads(y=B, gain=C, dy=D, dg=E + 4)]) == ALIGN
    for kw in (dict(y=D + 16), dict(dg=B), dict(dg=A), dict(dg=D + 64), dict(dg=C), dict(dg=G)):
        base = dict(y=B, gain=C, dy=D, dg=E)
        base.update(kw)
        assert qkb(L, [heads(**base)]) == ALIAS, kw
    assert qkb(L, [heads(y=B, gain=C, dy=D, dg=E), heads(J, J + (1 << 20), gain=C, dy=J + (1 << 21),
                                                         dg=E + 128)]) == ALIAS
    for kw in (dict(y=D), dict(y=A), dict(y=B, dg=None)):      # in place of dy or x; no dgain
        base = dict(y=B, gain=C, dy=D, dg=E)
        base.update(kw)
        assert qkb(L, [heads(**base)]) in REACHED, kw


def test_heads_side_by_side_within_a_projection(L):
    # [tokens, heads, 3, dim]: queries, keys and values of a head next to each other
    row, size = (3 * 3 * 64, 3 * 64), 2 * 64
    q, k, v = (heads(A + i * size, A + i * size, xs=row) for i in range(3))
    assert rope(L, [q, k]) in REACHED and rope(L, [k, v]) in REACHED and rope(L, [v, q]) in REACHED
    assert rope(L, [heads(A, A + size, xs=row), heads(A + 2 * size, B, xs=row, ys=(192, 64))]) in REACHED
    # [tokens, heads, keys and values, dim] beside queries of another buffer
    assert rope(L, [heads(B, B), heads(A, A, xs=(2 * 3 * 64, 2 * 64))]) in REACHED
    # one that reaches into its neighbour, and two in one place
    assert rope(L, [q, heads(A + size // 2, A + size // 2, xs=row)]) == ALIAS
    assert rope(L, [q, heads(B, A, xs=row)]) == ALIAS
    assert rope(L, [q, heads(A + 2 * size + 64, A + 2 * size + 64, xs=row)]) == ALIAS
    qs = [heads(A + i * size, A + i * size, xs=row, gain=C) for i in range(2)]
    assert qk(L, qs) in REACHED
    grads = [heads(A + i * size, D + i * size, xs=row, gain=C, dy=D + i * size, dg=E + 1024 * i)
             for i in range(2)]
    assert qkb(L, grads) in REACHED


def test_frequencies_refusals(L):
    table, mag = (ctypes.c_uint64 * 128)(), ctypes.c_float()

    def f(dim=64, theta=1e4, kind=0, factor=2.0, context=4096.0, low=1.0, high=4.0, out=True):
        s = F.ForgeRopeScaling(kind, factor, context, low, high)
        return L.forge_rope_frequencies(dim, theta, ctypes.byref(s),
                                        ctypes.addressof(table) if out else None,
                                        ctypes.addressof(mag))
    assert f() == OK and L.forge_rope_frequencies(64, 1e4, None, ctypes.addressof(table),
                                                  ctypes.addressof(mag)) == OK
    for kw in (dict(dim=0), dict(dim=12), dict(dim=264), dict(dim=-8)):
        assert f(**kw) == SHAPE, kw
    assert f(out=False) == NULL and f(kind=5) == FORMAT and f(kind=-1) == FORMAT
    for kw in (dict(theta=1.0), dict(theta=float("nan")), dict(theta=float("inf")),
               dict(kind=1, factor=0.5), dict(kind=2, factor=float("inf")),
               dict(kind=3, context=0.0), dict(kind=3, low=0.0), dict(kind=4, low=4.0),
               dict(kind=4, high=float("inf"))):
        assert f(**kw) == HYPER, kw


@pytest.mark.parametrize("scale", ["none", "linear", "ntk", "llama3", "yarn"])
@pytest.mark.parametrize("dim", [8, 24, 64, 128, 256])
def test_frequencies_against_the_definition(scale, dim):
    kw = {"none": {}, "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
          "llama3": dict(factor=8.0, context=8192.0, low=1.0, high=4.0),
          "yarn": dict(factor=16.0, context=4096.0, low=1.0, high=32.0)}[scale]
    ids = {"none": F.ROPE_SCALE_NONE, "linear": F.ROPE_SCALE_LINEAR, "ntk": F.ROPE_SCALE_NTK,
           "llama3": F.ROPE_SCALE_LLAMA3, "yarn": F.ROPE_SCALE_YARN}
    for theta in (10000.0, 500000.0):
        table, mag = F.rope_frequencies(dim, theta, scaling=ids[scale], device="cpu", **kw)
        rad, mag64 = R.frequencies(dim, theta, scale, **kw)
        turns = table.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
        # doubles on both sides: a few 2^-53 of at most 1 / (2 pi) turns
        assert np.abs(turns - rad / (2 * np.pi)).max() <= 2.0 ** -52
        assert abs(mag - mag64) <= 2.0 ** -24 * mag64


@pytest.mark.parametrize("kind,name,high", [(F.ROPE_SCALE_LLAMA3, "llama3", 4.0),
                                            (F.ROPE_SCALE_YARN, "yarn", 32.0)])
def test_frequencies_are_mixed_up_to_the_usual_turns(kind, name, high):
    kw = dict(factor=16.0, context=4096.0)
    table, mag = F.rope_frequencies(128, 10000.0, scaling=kind, device="cpu", **kw)
    given, mag2 = F.rope_frequencies(128, 10000.0, scaling=kind, high=high, device="cpu", **kw)
    assert torch.equal(table, given) and mag == mag2
    rad, mag64 = R.frequencies(128, 10000.0, name, low=1.0, high=high, **kw)
    turns = table.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    # doubles on both sides, as above
    assert np.abs(turns - rad / (2 * np.pi)).max() <= 2.0 ** -52
    assert abs(mag - mag64) <= 2.0 ** -24 * mag64
    other, _ = F.rope_frequencies(128, 10000.0, scaling=kind, high=36.0 - high, device="cpu", **kw)
    assert not torch.equal(table, other)


def test_python_checks_without_a_gpu():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    w = torch.zeros((8, 256), dtype=torch.bfloat16)
    y = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        F.linear_bf16(x, w, y)
    with pytest.raises(ValueError, match="2-D"):
        F.linear_bf16(x[0], w, y)
    with pytest.raises(ValueError, match="CUDA"):
        F.epilogue_backward(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        F.dropout(x, x, p=0.1, seed=1)
    q, f = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        F.rope(q, None, f)
    with pytest.raises(ValueError, match="CUDA"):
        F.qk_norm_rope(q, q, torch.ones(64), torch.ones(64), f, eps=1e-5)
    with pytest.raises(F.ForgeError):
        F.rope_frequencies(12, 10000.0, device="cpu")


# ---------------------------------------------------------------- definitions
def test_philox_against_known_answers():
    # Random123's published vectors
    full = (1 << 32) - 1
    assert R.philox4x32_10((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert R.philox4x32_10((full,) * 4, (full,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6,
                                                         0x6D5451FD]
    assert R.philox4x32_10((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
                           (0xA4093822, 0x299F31D0)) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420,
                                                         0x24126EA1]


def test_keep_is_the_generators_words():
    seed, offset, p = 0x123456789ABCDEF0, (7 << 32) + 5, 0.3
    got = R.keep(3, 16, p, seed, offset)
    t = R.threshold(p)
    for b in range(6):
        w = R.philox4x32_10((b, 0, 5, 7), (0x9ABCDEF0, 0x12345678))
        u = [(w[j // 2] >> (16 * (j % 2))) & 0xFFFF for j in range(8)]
        assert got.reshape(-1, 8)[b].tolist() == [65536 / (65536 - t) if x >= t else 0.0 for x in u]
    assert R.threshold(0.9999999) == 65535 and R.threshold(0.0) == 0


@pytest.mark.parametrize("kind", [R.RELU, R.GELU, R.GELU_TANH, R.SILU])
def test_activation_slopes_by_differences(kind):
    z, t = np.linspace(-6, 6, 121) + 0.013, 1e-6
    num = (R.act(z + t, kind) - R.act(z - t, kind)) / (2 * t)
    assert np.abs(num - R.act_slope(z, kind)).max() < 1e-8
    pairs = {R.GELU: "none", R.GELU_TANH: "tanh"}
    if kind in pairs:
        want = torch.nn.functional.gelu(torch.from_numpy(z), approximate=pairs[kind]).numpy()
    else:
        want = (torch.relu if kind == R.RELU else torch.nn.functional.silu)(torch.from_numpy(z)).numpy()
    assert np.abs(R.act(z, kind) - want).max() < 1e-14


def test_linear_gradients_by_autograd():
    g = torch.Generator().manual_seed(0)
    X, W, b = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((3, 8), (16, 8), (16,)))
    m, r, dY = (torch.randn((3, 16), generator=g, dtype=torch.float64) for _ in range(3))
    f = torch.from_numpy(R.keep(3, 16, 0.4, 1, 2))
    for t in (b, m, r):
        t.requires_grad_()
    Z = X @ W.T + b
    Z.retain_grad()
    Y = r + torch.nn.functional.silu(Z) * m * f
    Y.backward(dY)
    n = lambda t: t.detach().numpy()  # noqa: E731
    z, y = R.linear(n(X), n(W), n(b), R.SILU, n(m), n(r), n(f))
    assert np.abs(y - n(Y)).max() < 1e-12
    dz, dm, db = R.epilogue_backward(n(dY), z, R.SILU, n(m), n(f))
    for got, want in ((dz, Z.grad), (dm, m.grad), (db, b.grad), (n(dY), r.grad)):
        assert np.abs(got - n(want)).max() < 1e-12


@pytest.mark.parametrize("layout", [R.HALF, R.INTERLEAVED])
def test_rotation_is_a_rotation(layout):
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (5, 2, 24))
    rad, _ = R.frequencies(16, 100.0)
    pos = rng.integers(-1000, 1000, 5)
    y = R.rotate(x, pos, rad, 1.0, layout)
    assert np.abs((y ** 2).sum(2) - (x ** 2).sum(2)).max() < 1e-12
    assert np.abs(R.rotate(y, pos, rad, 1.0, layout, True) - x).max() < 1e-12
    assert np.array_equal(y[..., 16:], x[..., 16:])
    # a query and a key meet by the distance of their positions alone
    a, b = x[:1], x[1:2]
    dot = lambda p, q: (R.rotate(a, [p], rad, 1.0, layout) * R.rotate(b, [q], rad, 1.0, layout)).sum(2)  # noqa: E731
    assert np.abs(dot(17, 5) - dot(112, 100)).max() < 1e-12


def test_head_norm_gradients_by_differences():
    rng = np.random.default_rng(4)
    x, dn, g, t = rng.normal(0, 1, (2, 3, 8)), rng.normal(0, 1, (2, 3, 8)), rng.normal(1, 0.2, 8), 1e-6
    dx, dg = R.head_norm_backward(dn, x, g, 1e-3)
    loss = lambda xx, gg: (dn * R.head_norm(xx, gg, 1e-3)).sum()  # noqa: E731
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = t
        assert abs((loss(x + e, g) - loss(x - e, g)) / (2 * t) - dx[at]) < 1e-7
    for j in range(8):
        e = np.zeros_like(g)
        e[j] = t
        assert abs((loss(x, g + e) - loss(x, g - e)) / (2 * t) - dg[j]) < 1e-7
