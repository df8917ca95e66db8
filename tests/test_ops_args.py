"""Refusals of the operators around the weight gradient (host checks: no GPU is
touched), and pins of their fp64 definitions."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import ops as R
from weight_gradient_gemm_gb300 import _build
from weight_gradient_gemm_gb300 import forge as F

# fake, aligned, far apart addresses: never dereferenced
A, B, C, D, E, G, H = (1 << k for k in (20, 30, 34, 36, 38, 40, 42))
OK, NULL, ALIGN, SHAPE, FORMAT, HYPER, ALIAS = range(7)
F32, BF16 = F.DT_FP32, F.DT_BF16


@pytest.fixture(scope="module")
def L():
    _build.build()
    return F.lib()


def test_header_declares_the_operators():
    names = F.header_functions()
    for n in ("forge_rmsnorm", "forge_rmsnorm_backward", "forge_rmsnorm_backward_workspace_bytes",
              "forge_quantize_b128", "forge_linear_fp8", "forge_dgrad_fp8", "forge_grad_norm",
              "forge_grad_norm_workspace_bytes", "forge_adamw_clip"):
        assert n in names


def norm(L, x=A, r=None, g=B, gt=F32, s=None, y=C, c=None, sc=None, rstd=None, rows=4, cols=256,
         eps=1e-5):
    return L.forge_rmsnorm(x, r, g, gt, s, y, c, sc, rstd, rows, cols, eps, None)


def test_rmsnorm_refusals(L):
    assert norm(L, rows=0) == OK
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=12), dict(cols=32776), dict(rows=1 << 31)):
        assert norm(L, **kw) == SHAPE, kw
    assert norm(L, gt=2) == FORMAT
    for eps in (-1.0, float("nan"), float("inf")):
        assert norm(L, eps=eps) == HYPER
    for kw in (dict(x=None), dict(g=None), dict(y=None), dict(c=D), dict(sc=E)):
        assert norm(L, **kw) == NULL, kw
    for kw in (dict(x=A + 2), dict(r=A + 8), dict(g=B + 4), dict(s=D + 2), dict(y=C + 8),
               dict(c=D + 8, sc=E), dict(c=D, sc=E + 4), dict(rstd=D + 4)):
        assert norm(L, **kw) == ALIGN, kw
    for kw in (dict(y=A), dict(y=A + 16), dict(c=A, sc=E), dict(c=D, sc=B), dict(rstd=C),
               dict(r=D, y=D), dict(s=C), dict(s=A + 16), dict(r=D, s=D + 16), dict(s=B)):
        assert norm(L, **kw) == ALIAS, kw


def bwd(L, dy=A, h=B, g=C, gt=BF16, rstd=D, ds=None, dx=E, dg=None, rows=4, cols=256, ws=None,
        wb=0):
    return L.forge_rmsnorm_backward(dy, h, g, gt, rstd, ds, dx, dg, rows, cols, ws, wb, None)


def test_rmsnorm_backward_refusals(L):
    for kw in (dict(rows=-1), dict(cols=4), dict(cols=40000)):
        assert bwd(L, **kw) == SHAPE, kw
    assert bwd(L, gt=7) == FORMAT
    for kw in (dict(dy=None), dict(h=None), dict(g=None), dict(rstd=None), dict(dx=None)):
        assert bwd(L, **kw) == NULL, kw
    for kw in (dict(dy=A + 2), dict(dx=E + 8), dict(rstd=D + 4), dict(ds=G + 8), dict(dg=G + 4)):
        assert bwd(L, **kw) == ALIGN, kw
    for kw in (dict(dx=A), dict(dx=B), dict(ds=G, dx=G + 16), dict(dg=E), dict(dg=C),
               dict(dg=G, ws=G, wb=4096), dict(dg=G, ws=A, wb=4096)):
        assert bwd(L, **kw) == ALIAS, kw


def test_quantize_refusals(L):
    def q(x=A, c=B, s=C, rows=4, cols=256, br=1):
        return L.forge_quantize_b128(x, c, s, rows, cols, br, None)
    assert q(rows=0) == OK
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=20), dict(rows=(1 << 31) - 1, br=128,
                                                               cols=(1 << 31) - 8)):
        assert q(**kw) == SHAPE, kw
    assert q(br=64) == FORMAT
    for k in "xcs":
        assert q(**{k: None}) == NULL
    assert q(x=A + 8) == ALIGN and q(c=B + 8) == ALIGN and q(s=C + 4) == ALIGN
    assert q(c=A) == ALIAS and q(s=B) == ALIAS and q(s=A + 1024) == ALIAS


@pytest.mark.parametrize("name", ["forge_linear_fp8", "forge_dgrad_fp8"])
def test_product_refusals(L, name):
    def p(a=A, sa=B, w=C, sw=D, o=E, dt=BF16, bt=4, d_in=256, d_out=512):
        return getattr(L, name)(a, sa, w, sw, o, dt, bt, d_in, d_out, None)
    assert p(bt=0) == OK
    for kw in (dict(bt=-1), dict(d_in=0), dict(d_out=0), dict(d_in=24), dict(d_out=8),
               dict(bt=1 << 31), dict(d_in=1 << 31)):
        assert p(**kw) == SHAPE, kw
    assert p(dt=5) == FORMAT
    for k in ("a", "sa", "w", "sw", "o"):
        assert p(**{k: None}) == NULL
    for kw in (dict(a=A + 8), dict(sa=B + 4), dict(w=C + 1), dict(sw=D + 8), dict(o=E + 2)):
        assert p(**kw) == ALIGN, kw
    for kw in (dict(o=A), dict(o=B), dict(o=C + 4096), dict(o=D)):
        assert p(**kw) == ALIAS, kw


def test_grad_norm_refusals(L):
    def n(items=((A, 100, F32),), count=None, mx=1.0, out=B, ws=C, wb=1 << 20):
        arr = (F.ForgeGrad * len(items))(*[F.ForgeGrad(*i) for i in items])
        return L.forge_grad_norm(ctypes.addressof(arr) if items else None,
                                 len(items) if count is None else count, mx, out, ws, wb, None)
    assert n(count=-1) == SHAPE
    assert n(items=(), count=1) == NULL and n(out=None) == NULL
    assert n(items=((None, 5, F32),)) == NULL
    assert n(out=B + 2) == ALIGN and n(ws=C + 8) == ALIGN and n(items=((A + 4, 5, F32),)) == ALIGN
    for mx in (0.0, -1.0, float("nan")):
        assert n(mx=mx) == HYPER
    assert n(items=((A, 5, 3),)) == FORMAT
    assert n(items=((A, -1, F32),)) == SHAPE
    assert n(out=A) == ALIAS and n(out=C) == ALIAS and n(ws=A + 16) == ALIAS


def test_adamw_clip_refusals(L):
    def a(dw=A, coef=B, w=C, m=D, v=E, dt=F32, fmt=F.MOM_FP32, step=1):
        return L.forge_adamw_clip(dw, dt, coef, w, F.ForgeMoment(m, None), F.ForgeMoment(v, None),
                                  64, 64, 1e-3, 0.9, 0.999, 1e-8, 0.0, step, fmt, None)
    assert a(dw=None) == NULL and a(coef=None) == NULL
    assert a(coef=B + 2) == ALIGN
    assert a(coef=C) == ALIAS and a(coef=D + 64) == ALIAS
    assert a(step=0) == HYPER and a(fmt=9) == FORMAT


def test_python_checks_without_a_gpu():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        F.quantize_b128(x, *F.alloc_b128(4, 256, device="cpu"))
    with pytest.raises(ValueError, match="block_rows"):
        F.quantize_b128(x, *F.alloc_b128(4, 256, device="cpu"), block_rows=3)
    with pytest.raises(ValueError, match="block_rows"):
        F.alloc_b128(4, 256, 2, device="cpu")
    with pytest.raises(ValueError, match="2-D"):
        F.rmsnorm(x[0], x[0], eps=0.0)
    with pytest.raises(ValueError, match="CUDA"):
        F.grad_norm([x], 1.0, torch.zeros(2), workspace=torch.zeros(16))


# ---------------------------------------------------------------- definitions
def test_e4m3_rounding_against_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, 1, 4000), rng.normal(0, 100, 4000), rng.normal(0, 1e-2, 4000),
                        np.linspace(-448, 448, 8001), [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = x.astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(R.e4m3_round(x), want)
    assert R.e4m3_round(np.array([1e4, -1e4])).tolist() == [448.0, -448.0]


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_definition(block_rows):
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, (200, 300))
    x[:128, :128] = 0
    codes, scales = R.quantize(x, block_rows)
    assert scales.shape == (200 if block_rows == 1 else 2, 3)
    back = R.dequantize(codes, scales, block_rows)
    full = R.spread(scales, block_rows, x.shape)
    assert (np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, full * 2.0 ** -10) * (1 + 1e-12)).all()
    assert (back[:128, :128] == 0).all() and (scales[:1, 0] == 0).all()
    assert R.block_amax(codes, block_rows)[-1].tolist() == [448.0] * 3
    # rounding is to the nearest code: no neighbouring code is closer
    assert np.array_equal(R.e4m3_round(codes), codes)


def test_norm_gradients_by_differences():
    rng = np.random.default_rng(2)
    x, r, dy, ds = (rng.normal(0, 1, (3, 16)) for _ in range(4))
    g = rng.normal(1, 0.2, 16)

    def loss(xx, rr, gg):
        h, _, y = R.rmsnorm(xx, rr, gg, 1e-3)
        return (y * dy).sum() + (h * ds).sum()

    h, rstd, _ = R.rmsnorm(x, r, g, 1e-3)
    dx, dg = R.rmsnorm_backward(dy, h, g, rstd, ds)
    t = 1e-6
    for i in range(3):
        for j in range(16):
            e = np.zeros_like(x)
            e[i, j] = t
            for num in (loss(x + e, r, g) - loss(x - e, r, g), loss(x, r + e, g) - loss(x, r - e, g)):
                assert abs(num / (2 * t) - dx[i, j]) < 1e-7
    for j in range(16):
        e = np.zeros_like(g)
        e[j] = t
        assert abs((loss(x, r, g + e) - loss(x, r, g - e)) / (2 * t) - dg[j]) < 1e-7


def test_grad_norm_definition():
    grads = [np.array([3.0, 0.0]), np.array([[4.0]])]
    assert R.grad_norm(grads, 10.0) == (5.0, 1.0)
    norm, coef = R.grad_norm(grads, 1.0)
    assert norm == 5.0 and abs(coef - 0.2) < 1e-6
