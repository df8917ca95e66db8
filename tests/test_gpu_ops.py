"""The operators around the weight gradient against their fp64 definitions
(oracle/ops.py): the RMS norm and its gradients, the 128-block quantiser, the
8-bit products and clipping by the global gradient norm.

Tolerances.  u = 2^-24 is fp32's unit roundoff, 2^-8 bf16's.  A value computed in
fp32 by a chain of k roundings and rounded once to bf16 is held to
(2^-8 + k u) of itself plus what the roundings of larger terms leave.
"""
import numpy as np
import pytest
import torch

from oracle import ops as R
from tests.gpu_util import DEV, F, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rand(seed, shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ok():
    st = F.device_error()
    assert st == 0, F.status_string(st)


def within(got, ref, bound):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref)[bad].max()))


def check_codes(codes, scales, x64, block_rows, rel, absolute):
    """Codes and scales of x64, known to within rel of itself plus absolute
    (an array): each scale within rel of its block's, and each decoded value no
    further than half a code step from x (a step is at most 2^-3 of the value,
    2^-9 scales below the normal codes)."""
    ref_scales = R.quantize(x64, block_rows)[1]
    s = f64(scales)
    err = R.block_amax(absolute, block_rows)
    within(s, ref_scales, (rel + 2 * U) * ref_scales + (err / 448) + 2.0 ** -149)
    back = R.dequantize(f64(codes), s, block_rows)
    full = R.spread(np.maximum(s, ref_scales), block_rows, x64.shape)
    half = np.maximum(np.abs(x64) * 2.0 ** -4, full * 2.0 ** -10)
    within(back, x64, half * (1 + 4 * U) + (rel + 4 * U) * np.abs(x64) + absolute)


# ---------------------------------------------------------------- the norm
NORM_SHAPES = [(1, 8), (1, 4096), (2, 136), (3, 1032), (7, 128), (65, 264), (5, 8200),
               (3, 16392), (2, 32768), (333, 520), (1300, 64), (5000, 128), (1251, 1544),
               (640, 4096), (613, 4104), (610, 8192)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("gain_dtype", [torch.float32, torch.bfloat16])
def test_rmsnorm(rows, cols, res, gain_dtype):
    x = rand(1, (rows, cols))
    r = rand(2, (rows, cols), 3.0) if res else None
    gain = (1 + rand(3, (cols,), 0.2, torch.float32)).to(gain_dtype)
    y = torch.empty_like(x)
    s = torch.empty_like(x) if res else None
    rstd = torch.empty(rows, device=DEV)
    codes, scales = F.alloc_b128(rows, cols)
    F.rmsnorm(x, gain, eps=1e-5, residual=r, sum_out=s, y=y, codes=codes, scales=scales, rstd=rstd)
    ok()
    h64, rstd64, y64 = R.rmsnorm(f64(x), f64(r) if res else None, f64(gain), 1e-5)
    # the sum of `cols` squares is a tree over runs of at most 32 products: at
    # most 32 + 16 roundings of a sum of positive terms, half of that in rstd,
    # and rsqrt's 2 ulp; h itself is rounded once (its error is h's own)
    rel = (24 + 1 + 4) * U
    within(f64(rstd), rstd64, rel * rstd64)
    if res:
        within(f64(s), h64, (BF + 2 * U) * np.abs(h64))
    yrel = rel + 4 * U
    within(f64(y), y64, (BF + yrel) * np.abs(y64))
    check_codes(codes, scales, y64, 1, yrel, np.zeros_like(y64))


@pytest.mark.parametrize("rows,cols", [(400, 4096), (310, 4104), (1200, 1032), (200, 8200),
                                       (2500, 1024), (2000, 1024), (2600, 520), (1217, 768)])
@pytest.mark.parametrize("res", [False, True])
def test_rmsnorm_more_rows_than_one_wave(rows, cols, res):
    test_rmsnorm(rows, cols, res, torch.bfloat16)


def test_rmsnorm_each_output_alone():
    x, r, gain = rand(1, (5, 392)), rand(2, (5, 392)), rand(3, (392,), 1.0, torch.float32)
    y, s, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(5, device=DEV)
    codes, scales = F.alloc_b128(5, 392)
    F.rmsnorm(x, gain, eps=1e-6, residual=r, sum_out=s, y=y, codes=codes, scales=scales, rstd=rstd)
    y2 = torch.empty_like(x)
    F.rmsnorm(x, gain, eps=1e-6, residual=r, y=y2)
    c2, s2 = F.alloc_b128(5, 392)
    F.rmsnorm(x, gain, eps=1e-6, residual=r, codes=c2, scales=s2)
    assert torch.equal(y, y2) and torch.equal(codes.view(torch.uint8), c2.view(torch.uint8))
    assert torch.equal(scales, s2)
    # the sum in place of either input
    for take in (0, 1):
        xi, ri = x.clone(), r.clone()
        F.rmsnorm(xi, gain, eps=1e-6, residual=ri, sum_out=(xi, ri)[take], y=y2)
        assert torch.equal((xi, ri)[take], s) and torch.equal(y, y2)
        assert torch.equal((ri, xi)[take], (r, x)[take])
    ok()


def test_rmsnorm_zero_rows_and_extremes():
    cols = 256
    gain = torch.ones(cols, device=DEV)
    x = torch.zeros((4, cols), dtype=torch.bfloat16, device=DEV)
    x[1, 5] = 1e-30                     # squares underflow: eps alone is left
    x[2] = 2.0 ** 40                    # squares far from overflow
    x[3, 130] = float("nan")
    y, rstd = torch.empty_like(x), torch.empty(4, device=DEV)
    codes, scales = F.alloc_b128(4, cols)
    F.rmsnorm(x, gain, eps=1e-6, y=y, codes=codes, scales=scales, rstd=rstd)
    ok()
    assert torch.equal(y[0], x[0]) and f64(codes)[0].max() == 0 and f64(scales)[0].max() == 0
    assert abs(float(rstd[0]) - 1e3) < 1e-3 and abs(float(rstd[1]) - 1e3) < 1e-3
    assert (f64(y)[2] == 1).all() and (f64(codes)[2] == 448).all()
    assert torch.isnan(y[3]).all() and torch.isnan(scales[3]).all()
    assert torch.isnan(codes[3].float()).all()
    none = torch.empty((0, cols), dtype=torch.bfloat16, device=DEV)
    F.rmsnorm(none, gain, eps=1e-6, y=torch.empty_like(none))
    ok()


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("with_dsum", [False, True])
@pytest.mark.parametrize("gain_dtype", [torch.float32, torch.bfloat16])
def test_rmsnorm_backward(rows, cols, with_dsum, gain_dtype):
    h = rand(4, (rows, cols), 2.0)
    dy = rand(5, (rows, cols), 1e-2)
    dsum = rand(6, (rows, cols), 1e-2) if with_dsum else None
    gain = (1 + rand(3, (cols,), 0.2, torch.float32)).to(gain_dtype)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-5)).float()
    dx, dgain = torch.empty_like(h), torch.empty(cols, device=DEV)
    ws = torch.empty(F.rmsnorm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    F.rmsnorm_backward(dy, h, gain, rstd, dx, dgain, dsum=dsum, workspace=ws)
    ok()
    d64, h64, g64, r64 = f64(dy), f64(h), f64(gain), f64(rstd)
    dx64, dg64 = R.rmsnorm_backward(d64, h64, g64, r64, f64(dsum) if with_dsum else None)
    xh = np.abs(h64 * r64[:, None])
    u = np.abs(d64 * g64)
    # each term carries at most 6 roundings; the row's dot product at most 64
    # more of its terms' magnitude
    mean_abs = (u * xh).mean(1, keepdims=True)
    noise = r64[:, None] * (6 * U * u + 80 * U * xh * mean_abs)
    if with_dsum:
        noise += U * np.abs(f64(dsum))
    within(f64(dx), dx64, (BF + 2 * U) * np.abs(dx64) + noise)
    # a column's sum: at most rows additions, each within u of the partial sum
    within(f64(dgain), dg64, (min(rows, 60) + 30) * U * (np.abs(d64) * xh).sum(0) + 1e-30)
    again = torch.empty_like(dgain)
    dx2 = dsum.clone() if with_dsum else torch.empty_like(dx)     # dX in place of dsum
    F.rmsnorm_backward(dy, h, gain, rstd, dx2, again, dsum=dx2 if with_dsum else None, workspace=ws)
    assert torch.equal(again, dgain) and torch.equal(dx, dx2)
    dx3 = torch.empty_like(dx)
    F.rmsnorm_backward(dy, h, gain, rstd, dx3, dsum=dsum)
    assert torch.equal(dx, dx3)
    ok()


@pytest.mark.parametrize("rows,cols", [(1500, 1032), (800, 520), (2100, 512), (1024, 4096),
                                       (2000, 2048), (400, 8192), (320, 16384), (305, 14336),
                                       (2000, 1024), (1281, 1032), (769, 520), (2049, 256)])
@pytest.mark.parametrize("with_dsum", [False, True])
def test_rmsnorm_backward_between_one_wave_and_many(rows, cols, with_dsum):
    test_rmsnorm_backward(rows, cols, with_dsum, torch.float32)


def test_rmsnorm_backward_many_wide_rows():
    # rows too wide for the stream and too many for one launch; dX on a few rows
    rows, cols = 4200, 16392
    h, dy = rand(4, (rows, cols), 2.0), rand(5, (rows, cols), 1e-2)
    gain = 1 + rand(3, (cols,), 0.2, torch.float32)
    rstd = (1 / torch.sqrt(h.float().square().mean(1) + 1e-5))
    dx, dgain = torch.empty_like(h), torch.empty(cols, device=DEV)
    ws = torch.empty(F.rmsnorm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    F.rmsnorm_backward(dy, h, gain, rstd, dx, dgain, workspace=ws)
    ok()
    dg64, mag = torch.zeros(cols, dtype=torch.float64, device=DEV), 0.0
    for r in range(0, rows, 600):
        t = dy[r:r + 600].double() * (h[r:r + 600].double() * rstd[r:r + 600, None].double())
        dg64 += t.sum(0)
        mag = mag + t.abs().sum(0)
    within(f64(dgain), f64(dg64), 90 * U * f64(mag) + 1e-30)
    pick = torch.tensor([0, 1, 303, 304, 2111, 4199], device=DEV)
    d64, h64, g64, r64 = f64(dy[pick]), f64(h[pick]), f64(gain), f64(rstd[pick])
    dx64, _ = R.rmsnorm_backward(d64, h64, g64, r64, None)
    xh, u = np.abs(h64 * r64[:, None]), np.abs(d64 * g64)
    noise = r64[:, None] * (6 * U * u + 80 * U * xh * (u * xh).mean(1, keepdims=True))
    within(f64(dx[pick]), dx64, (BF + 2 * U) * np.abs(dx64) + noise)


def test_rmsnorm_backward_against_differences():
    # L = sum(dy * y): its central differences in h and in the gain, in fp64
    rows, cols, eps = 3, 40, 1e-5
    h, dy = rand(7, (rows, cols)), rand(8, (rows, cols))
    gain = rand(9, (cols,), 1.0, torch.float32)
    h64, d64, g64 = f64(h), f64(dy), f64(gain)
    rstd = torch.from_numpy(R.rmsnorm(h64, None, g64, eps)[1]).float().to(DEV)
    dx, dgain = torch.empty_like(h), torch.empty(cols, device=DEV)
    ws = torch.empty(F.rmsnorm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    F.rmsnorm_backward(dy, h, gain, rstd, dx, dgain, workspace=ws)
    ok()
    t = 1e-5

    def loss(hh, gg):
        return (d64 * R.rmsnorm(hh, None, gg, eps)[2]).sum()

    for i in range(rows):
        for j in range(cols):
            e = np.zeros_like(h64)
            e[i, j] = t
            num = (loss(h64 + e, g64) - loss(h64 - e, g64)) / (2 * t)
            assert abs(num - float(dx[i, j])) <= BF * abs(num) + 1e-5
    for j in range(cols):
        e = np.zeros_like(g64)
        e[j] = t
        num = (loss(h64, g64 + e) - loss(h64, g64 - e)) / (2 * t)
        assert abs(num - float(dgain[j])) <= 1e-5


def test_rmsnorm_backward_no_rows():
    none = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    dgain = torch.full((64,), 7.0, device=DEV)
    F.rmsnorm_backward(none, none, torch.ones(64, device=DEV), torch.empty(0, device=DEV), none,
                       dgain)
    ok()
    assert float(dgain.abs().max()) == 0.0


# ---------------------------------------------------------------- quantiser
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 4096), (3, 136), (129, 264), (128, 128),
                                       (300, 1032), (777, 640), (5, 14336)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(rows, cols, block_rows):
    x = rand(11, (rows, cols)) * (10.0 ** torch.linspace(-6, 3, cols, device=DEV))
    x = x.to(torch.bfloat16)
    codes, scales = F.alloc_b128(rows, cols, block_rows)
    F.quantize_b128(x, codes, scales, block_rows=block_rows)
    ok()
    x64 = f64(x)
    check_codes(codes, scales, x64, block_rows, 0.0, np.zeros_like(x64))


@pytest.mark.parametrize("rows,cols", [(5000, 2056), (40, 80000), (80000, 40)])
def test_quantize_more_blocks_than_resident(rows, cols):
    test_quantize(rows, cols, 128)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_blocks(block_rows):
    x = torch.zeros((130, 640), dtype=torch.bfloat16, device=DEV)
    x[0, 128:256] = 1e-38          # scale held at 2^-126
    x[0, 256] = float("nan")
    x[0, 384] = float("inf")
    x[0, 512:640] = torch.linspace(-448, 448, 128, device=DEV).to(torch.bfloat16)
    codes, scales = F.alloc_b128(130, 640, block_rows)
    F.quantize_b128(x, codes, scales, block_rows=block_rows)
    ok()
    back = R.dequantize(f64(codes), f64(scales), block_rows)
    assert (back[0, :128] == 0).all() and float(scales[0, 0]) == 0.0
    assert float(scales[0, 1]) == 2.0 ** -126
    within(back[0, 128:256], f64(x)[0, 128:256], 2.0 ** -4 * 1e-38)
    assert np.isnan(back[0, 256:512]).all()
    assert float(scales[0, 4]) == 1.0
    within(f64(codes)[0, 512:], R.e4m3_round(f64(x)[0, 512:]), 0.0)
    F.quantize_b128(x[:0], codes[:0], scales[:0], block_rows=block_rows)
    ok()


# ---------------------------------------------------------------- products
def random_codes(seed, rows, cols, block_rows):
    """Codes over the whole e4m3 range and scales of every size."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (rows, cols), generator=g, dtype=torch.uint8)
    c[(c & 0x7F) == 0x7F] = 0x30           # no NaN
    sr = rows if block_rows == 1 else -(-rows // 128)
    s = torch.exp2(torch.randn((sr, -(-cols // 128)), generator=g) * 2 - 6)
    return c.view(torch.float8_e4m3fn).to(DEV), s.float().to(DEV)


def check_product(out, a64, w64, k, dtype):
    ref, mag = a64 @ w64, np.abs(a64) @ np.abs(w64)
    # inside a block the tensor core adds 128 exact products in groups; each
    # addition is within 2^-23 of the partial sums' magnitude (truncation
    # included), of which there are at most 4 per block plus the group's own
    # alignment; outside, one product and one addition per block
    tol = (16 + -(-k // 128) + 2) * 2.0 ** -23 * mag
    within(f64(out), ref, tol + ((BF + U) * np.abs(ref) if dtype == torch.bfloat16 else 0))


PRODUCTS = [(1, 16, 16), (1, 4096, 1024), (2, 128, 128), (5, 144, 272), (16, 512, 640),
            (17, 1040, 48), (33, 272, 1296), (64, 2064, 528), (65, 640, 272), (128, 256, 256),
            (129, 400, 400), (257, 1040, 656), (300, 128, 1040), (512, 1024, 2048),
            (700, 2320, 144), (1, 14336, 256)]


@pytest.mark.parametrize("bt,d_in,d_out", PRODUCTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_fp8(bt, d_in, d_out, dtype):
    X, xs = random_codes(21, bt, d_in, 1)
    W, ws = random_codes(22, d_out, d_in, 128)
    Y = torch.empty((bt, d_out), dtype=dtype, device=DEV)
    F.linear_fp8(X, xs, W, ws, Y)
    ok()
    check_product(Y, R.dequantize(f64(X), f64(xs), 1), R.dequantize(f64(W), f64(ws), 128).T, d_in,
                  dtype)
    again = torch.empty_like(Y)
    F.linear_fp8(X, xs, W, ws, again)
    assert torch.equal(Y, again)


@pytest.mark.parametrize("bt,d_in,d_out", PRODUCTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dgrad_fp8(bt, d_in, d_out, dtype):
    dY, ds = random_codes(23, bt, d_out, 1)
    W, ws = random_codes(24, d_out, d_in, 128)
    dX = torch.empty((bt, d_in), dtype=dtype, device=DEV)
    F.dgrad_fp8(dY, ds, W, ws, dX)
    ok()
    check_product(dX, R.dequantize(f64(dY), f64(ds), 1), R.dequantize(f64(W), f64(ws), 128), d_out,
                  dtype)


@pytest.mark.parametrize("bt", [3, 200])
def test_products_keep_out_of_bounds_untouched(bt):
    # outputs inside a larger buffer: what surrounds them does not change
    X, xs = random_codes(25, bt, 272, 1)
    W, ws = random_codes(26, 144, 272, 128)
    buf = torch.full(((bt + 2) * 144,), 5.0, dtype=torch.bfloat16, device=DEV)
    F.linear_fp8(X, xs, W, ws, buf[144:-144].view(bt, 144))
    ok()
    assert (buf[:144] == 5).all() and (buf[-144:] == 5).all()


@pytest.mark.parametrize("bt", [4, 300])
def test_products_pass_nan_on(bt):
    # a token whose block holds a NaN has a NaN row, the other rows do not
    x = rand(27, (bt, 256))
    x[2, 200] = float("nan")
    X, xs = F.alloc_b128(bt, 256)
    F.quantize_b128(x, X, xs)
    W, ws = random_codes(28, 160, 256, 128)
    Y = torch.empty((bt, 160), dtype=torch.bfloat16, device=DEV)
    F.linear_fp8(X, xs, W, ws, Y)
    ok()
    bad = torch.isnan(Y)
    assert bad[2].all() and not bad[:2].any() and not bad[3:].any()


def test_products_no_tokens():
    W, ws = random_codes(29, 64, 64, 128)
    X, xs = random_codes(29, 0, 64, 1)
    F.linear_fp8(X, xs, W, ws, torch.empty((0, 64), dtype=torch.bfloat16, device=DEV))
    F.dgrad_fp8(X, xs, W, ws, torch.empty((0, 64), dtype=torch.bfloat16, device=DEV))
    ok()


# ---------------------------------------------------------------- clipping
def run_norm(grads, max_norm):
    out = torch.empty(2, device=DEV)
    ws = torch.empty(F.grad_norm_workspace_bytes(max(1, len(grads))), dtype=torch.uint8, device=DEV)
    F.grad_norm(grads, max_norm, out, workspace=ws)
    ok()
    return out


@pytest.mark.parametrize("sizes", [[1], [7], [8, 0, 9], [16384, 16385, 3], [1000003], [5] * 600,
                                   [70000] * 40])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grad_norm(sizes, dtype):
    grads = [rand(30 + i, (n,), 10.0 ** (i % 5 - 4), dtype) for i, n in enumerate(sizes)]
    if len(grads) > 1:
        grads[1] = grads[1].float()      # both types in one call
    norm, coef = R.grad_norm([f64(g) for g in grads], 0.5)
    got = run_norm(grads, 0.5)
    # 32 fp32 additions at most before fp64 takes over
    within(f64(got)[:1], np.array([norm]), 40 * U * norm)
    within(f64(got)[1:], np.array([coef]), 40 * U * coef)
    assert torch.equal(got, run_norm(grads, 0.5))


def test_grad_norm_extremes():
    big = torch.full((3000,), 1e30, device=DEV)
    tiny = torch.full((3000,), 1e-30, device=DEV)
    zero = torch.zeros(40000, device=DEV)
    for g, each in ((big, 1e30), (tiny, 1e-30)):
        norm = f64(g)[0] * np.sqrt(3000.0)
        got = run_norm([zero, g], 1.0)
        assert abs(float(got[0]) - norm) <= 4 * U * norm
        assert abs(float(got[1]) - min(1.0, 1 / (norm + 1e-6))) <= 1e-6 * float(got[1])
    assert f64(run_norm([zero], 1.0)).tolist() == [0.0, 1.0]
    assert f64(run_norm([], 1.0)).tolist() == [0.0, 1.0]
    zero[39999] = float("inf")
    assert f64(run_norm([zero], 1.0)).tolist() == [np.inf, 0.0]
    zero[0] = float("nan")
    assert torch.isnan(run_norm([zero], 1.0)).all()


@pytest.mark.parametrize("fmt", [torch.float32, torch.bfloat16, torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_adamw_clip(fmt, dtype):
    # the step equals forge_adamw's on a gradient scaled beforehand, bit for bit
    d_out, d_in = 40, 256
    hyper = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=3)
    g = rand(40, (d_out, d_in), 1e-2, dtype)
    w0 = rand(41, (d_out, d_in), 0.02)
    kind = {torch.float32: F.MOM_FP32, torch.bfloat16: F.MOM_BF16, torch.int8: F.MOM_INT8_B128,
            torch.float8_e4m3fn: F.MOM_FP8_E4M3}[fmt]

    def step(call):
        m, v, ms, vs = F.alloc_moments(d_out, d_in, kind, DEV)
        if kind == F.MOM_FP8_E4M3:
            ms[:2] = 1e-5
            vs[:2] = 1e-5
        W = w0.clone()
        call(W, m, v, dict(hyper, m_scale=ms, v_scale=vs))
        ok()
        return [t.view(torch.uint8) for t in (W, m, v)]

    for coef in (1.0, 0.25):
        clip = torch.tensor([9.0, coef], device=DEV)
        pre = (g.float() * coef) if coef != 1.0 else g
        a = step(lambda W, m, v, kw: F.adamw_clip(g, W, m, v, clip, **kw))
        b = step(lambda W, m, v, kw: F.adamw(pre, W, m, v, **kw))
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---------------------------------------------------------------- streams
def test_operators_on_another_stream():
    # inputs written late on a side stream, operators enqueued behind them there
    rows, cols = 256, 1024
    side = torch.cuda.Stream()
    gain = torch.ones(cols, device=DEV)
    ref_x = rand(50, (rows, cols))
    W, ws = random_codes(51, 512, cols, 128)
    g = rand(52, (rows, cols), 1.0, torch.float32)
    torch.cuda.synchronize()

    def work(x, grad, stream):
        codes, scales = F.alloc_b128(rows, cols)
        Y = torch.empty((rows, 512), dtype=torch.bfloat16, device=DEV)
        out = torch.empty(2, device=DEV)
        wsp = torch.empty(F.grad_norm_workspace_bytes(1), dtype=torch.uint8, device=DEV)
        F.rmsnorm(x, gain, eps=1e-5, codes=codes, scales=scales, stream=stream)
        F.linear_fp8(codes, scales, W, ws, Y, stream=stream)
        F.grad_norm([grad], 1.0, out, workspace=wsp, stream=stream)
        return Y, out

    want = work(ref_x, g, None)
    torch.cuda.synchronize()
    x = torch.zeros_like(ref_x)
    grad = torch.zeros_like(g)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x.copy_(ref_x)
        grad.copy_(g)
        got = work(x, grad, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_operators_in_a_graph():
    rows, cols = 64, 512
    x, gain = rand(60, (rows, cols)), torch.ones(cols, device=DEV)
    W, ws = random_codes(61, 256, cols, 128)
    codes, scales = F.alloc_b128(rows, cols)
    Y = torch.empty((rows, 256), dtype=torch.bfloat16, device=DEV)

    def step():
        F.rmsnorm(x, gain, eps=1e-5, codes=codes, scales=scales)
        F.linear_fp8(codes, scales, W, ws, Y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (62, 63):
        x.copy_(rand(seed, (rows, cols)))
        step()
        want = Y.clone()
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def test_repeated_launches_agree():
    # many launches back to back with cold and warm operands: every tile form
    # of the products gives the same bits each time
    for bt, d_in, d_out in ((1, 4096, 2048), (20, 2048, 4096), (100, 4096, 1024), (300, 4096, 1024),
                            (1500, 2048, 2048)):
        X, xs = random_codes(70, bt, d_in, 1)
        W, ws = random_codes(71, d_out, d_in, 128)
        Y = [torch.empty((bt, d_out), dtype=torch.bfloat16, device=DEV) for _ in range(40)]
        flush = torch.empty(64 << 20, dtype=torch.float32, device=DEV)
        for i, y in enumerate(Y):
            if i % 8 == 0:
                flush.fill_(float(i))
            F.linear_fp8(X, xs, W, ws, y)
        ok()
        assert all(torch.equal(Y[0], y) for y in Y[1:]), (bt, d_in, d_out)


def test_offsets_past_32_bits():
    # more than 2^31 elements: the last rows are where a narrow offset would show
    rows, cols = 540000, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    tail = rand(80, (200, cols))
    x[-200:] = tail
    codes, scales = F.alloc_b128(rows, cols)
    F.quantize_b128(x, codes, scales)
    ok()
    c2, s2 = F.alloc_b128(200, cols)
    F.quantize_b128(tail, c2, s2)
    assert torch.equal(codes[-200:].view(torch.uint8), c2.view(torch.uint8))
    assert torch.equal(scales[-200:], s2) and float(scales[0].max()) == 0.0
    gain = torch.ones(cols, device=DEV)
    y, y2 = torch.empty_like(x), torch.empty_like(tail)
    F.rmsnorm(x, gain, eps=1e-5, y=y)
    F.rmsnorm(tail, gain, eps=1e-5, y=y2)
    ok()
    assert torch.equal(y[-200:], y2)
    del x
    # the product's output offsets, and the gradient norm's
    W, ws = random_codes(81, cols, 128, 128)
    X, xs = random_codes(82, rows, 128, 1)
    F.linear_fp8(X, xs, W, ws, y)
    F.linear_fp8(X[-200:].clone(), xs[-200:].clone(), W, ws, y2)
    ok()
    assert torch.equal(y[-200:], y2)
    y.zero_()
    y[-1, -1] = 3.0
    assert f64(run_norm([y], 6.0)).tolist() == [3.0, 1.0]


def test_example_trains():
    from examples import fp8_layer
    losses, norms = fp8_layer.train(steps=30, bt=256, d_in=384, d_out=640)
    assert losses[-1] < 0.2 * losses[0], losses
    assert all(np.isfinite(norms))
