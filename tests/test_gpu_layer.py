"""The operators between a layer's 16-bit products against their fp64 definitions
(oracle/layer.py): the forward product with its epilogue, the epilogue's gradient,
dropout, rotary positions, and the norm of queries and keys with the rotation.

Tolerances.  U = 2^-24 is fp32's unit roundoff, BF = 2^-8 bf16's.  Each bound counts
the fp32 roundings on the way, by the magnitude of the terms they act on, and one
rounding to the output's type.
"""
import numpy as np
import pytest
import torch

from oracle import layer as R
from tests.gpu_util import DEV, F, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8
KINDS = [R.NONE, R.RELU, R.GELU, R.GELU_TANH, R.SILU]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rand(seed, shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def ok():
    st = F.device_error()
    assert st == 0, F.status_string(st)


def within(got, ref, bound):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.nanmax(np.abs(got - ref)[bad])))


def out_round(dtype):
    return BF if dtype == torch.bfloat16 else U


def act_error(z, kind):
    """What computing act(z) in fp32 from an exact z may be off by.  ReLU is exact.  The
    argument of the exponential (w; for GELU z^2 / 2 inside erfc) carries four roundings,
    which e^-w turns into a relative |w| times that; the hardware's exponential has
    2 + 1.2 |w| ulp, quotient and products a few more.  Below 2^-120 results may be lost."""
    if kind in (R.NONE, R.RELU):
        return 0.0
    w = {R.GELU: z * z, R.GELU_TANH: np.abs(R._tanh_arg(z)[0]), R.SILU: np.abs(z)}[kind]
    return (16 + 8 * w) * U * np.abs(R.act(z, kind)) + 2.0 ** -120


def slope_error(z, kind):
    """The same for act'(z): s and z s (1 - s) w' carry act's relative error, and 1 - s is
    off by a few roundings of 1 itself.  An exponential below the smallest normal number,
    2^-126, comes out as zero.  z w' e^-w is largest where e^-w passes 2^-126, w = 87.3:
    z w' is 87.3 there for SILU and, z being 10.6, 10.6 (1 + 0.134 10.6^2) 1.6 < 2^9 for
    GELU_TANH; so less than 2^-117 is lost."""
    if kind in (R.NONE, R.RELU):
        return 0.0
    lost = 2.0 ** -112
    if kind == R.GELU:
        dw, w = 1.0, z * z
        terms = 0.5 + np.abs(z)
        return (16 + 8 * w) * U * np.abs(R.act_slope(z, kind)) + 16 * U * terms + lost
    w, dw = R._tanh_arg(z) if kind == R.GELU_TANH else (z, 1.0)
    s, t = R._sigmoid(w), R._sigmoid(-w)
    return ((16 + 8 * np.abs(w)) * U * (s + np.abs(z) * s * t * dw)
            + 8 * U * s * (1 + np.abs(z) * dw) + lost)


# ---------------------------------------------------------------- the product
EPILOGUES = {
    "plain": {},
    "fp32": dict(out=torch.float32),
    "all": dict(bias=torch.float32, act=R.GELU, mul=True, residual=True, z=True, p=0.1),
    "gate": dict(act=R.SILU, mul=True, z=True),
    "dropped": dict(bias=torch.bfloat16, act=R.RELU, p=0.5),
    "residual": dict(residual=True),
    "all_fp32": dict(bias=torch.bfloat16, act=R.GELU_TANH, mul=True, residual=True, z=True, p=0.25,
                     out=torch.float32),
    "residual_fp32": dict(residual=True, act=R.RELU, out=torch.float32),
    "z_fp32": dict(bias=torch.float32, z=True, out=torch.float32),
}
SHAPES = [(1, 8, 8), (1, 4096, 1024), (2, 128, 128), (5, 144, 272), (16, 512, 640), (17, 1040, 48),
          (33, 272, 1296), (64, 2064, 528), (65, 640, 272), (128, 256, 256), (129, 400, 400),
          (257, 1040, 656), (300, 136, 1040), (333, 1032, 520), (512, 1024, 2048), (700, 2320, 144),
          (1, 14336, 256), (100, 72, 24)]
SEED, OFFSET = 0x123456789ABCDEF0, 5


def linear_case(bt, d_in, d_out, bias=None, act=R.NONE, mul=False, residual=False, z=False, p=0.0,
                out=torch.bfloat16):
    shape = (bt, d_out)
    return dict(X=rand(1, (bt, d_in)), W=rand(2, (d_out, d_in), d_in ** -0.5), act=act, p=p,
                bias=rand(3, (d_out,), 0.5, bias) if bias is not None else None,
                mul=rand(4, shape) if mul else None,
                residual=rand(5, shape, 3.0) if residual else None,
                Z=torch.full(shape, 7.0, dtype=torch.bfloat16, device=DEV) if z else None,
                Y=torch.full(shape, 7.0, dtype=out, device=DEV))


def call_linear(c, **more):
    F.linear_bf16(c["X"], c["W"], c["Y"], bias=c["bias"], act=c["act"], mul=c["mul"],
                  residual=c["residual"], Z=c["Z"], p=c["p"], seed=SEED, offset=OFFSET, **more)
    ok()


def check_linear(c, Y=None, residual=None, mul=None):
    """Against fp64.  Inside the product, each instruction adds 16 exact products to the
    accumulator with a truncation of at most 2^-22 of the partial sums' magnitude."""
    X, W, bias = f64(c["X"]), f64(c["W"]), f64(c["bias"])
    mul = f64(c["mul"]) if mul is None else mul
    residual = f64(c["residual"]) if residual is None else residual
    k = X.shape[1]
    factor = R.keep(X.shape[0], W.shape[0], c["p"], SEED, OFFSET) if c["p"] else None
    Z, want = R.linear(X, W, bias, c["act"], mul, residual, factor)
    mag = np.abs(X) @ np.abs(W).T + (0 if bias is None else np.abs(bias))
    zerr = (-(-k // 16) + 4) * 2.0 ** -22 * mag
    if c["Z"] is not None:
        within(f64(c["Z"]), Z, BF * np.abs(Z) + zerr)
    a = R.act(Z, c["act"])
    err = 1.2 * zerr + act_error(Z, c["act"]) + 4 * U * np.abs(a)   # |act'| is below 1.13
    scale = (1.0 if mul is None else np.abs(mul)) * (1.0 if factor is None else factor)
    err = err * scale + 2 * U * np.abs(want)
    Y = c["Y"] if Y is None else Y
    rd = out_round(Y.dtype)
    within(f64(Y), want, rd * np.abs(want) + (1 + rd) * err)


@pytest.mark.parametrize("bt,d_in,d_out", SHAPES)
@pytest.mark.parametrize("name", sorted(EPILOGUES))
def test_linear(bt, d_in, d_out, name):
    c = linear_case(bt, d_in, d_out, **EPILOGUES[name])
    call_linear(c)
    check_linear(c)
    first = [t.clone() for t in (c["Y"], c["Z"]) if t is not None]
    call_linear(c)
    assert all(torch.equal(a, b) for a, b in zip(first, [t for t in (c["Y"], c["Z"]) if t is not None]))


@pytest.mark.parametrize("bt,d_in,d_out", [(1, 64, 8), (40, 200, 328), (300, 136, 1040),
                                           (700, 1024, 1160), (2100, 72, 2600), (1, 8, 40000)])
@pytest.mark.parametrize("cg,bn,splits", [(1, 0, 1), (1, 0, 2), (1, 0, 8), (2, 0, 0), (2, 128, 0),
                                          (2, 256, 0)])
@pytest.mark.parametrize("name", ["plain", "all", "all_fp32"])
def test_linear_by_tile(bt, d_in, d_out, cg, bn, splits, name, tune):
    """Both forms, also where the other would be taken, by tile and split, also of
    reductions with fewer steps than CTAs, with several tiles a pair."""
    tune(cg=cg, bn=bn, splits=splits)
    c = linear_case(bt, d_in, d_out, **EPILOGUES[name])
    call_linear(c)
    check_linear(c)


@pytest.mark.parametrize("bt", [1, 16, 31, 64, 128])
@pytest.mark.parametrize("splits", [1, 2, 4, 8])
def test_linear_by_splits(bt, splits, tune):
    """Few tokens: every split, also of reductions with fewer steps than CTAs."""
    tune(splits=splits)
    for d_in, d_out in ((64, 136), (264, 640), (2056, 264)):
        c = linear_case(bt, d_in, d_out, **EPILOGUES["all"])
        call_linear(c)
        check_linear(c)


@pytest.mark.parametrize("bt,d_out", [(2000, 4096), (1000, 4800), (2000, 3400), (1500, 5000),
                                      (520, 88), (2300, 2200)])
@pytest.mark.parametrize("name", ["all", "fp32", "gate"])
def test_linear_by_tile_width(bt, d_out, name):
    """Sizes that take tiles of other widths (the rule counts waves)."""
    c = linear_case(bt, 136, d_out, **EPILOGUES[name])
    call_linear(c)
    check_linear(c)


def test_linear_few_tokens_more_tiles_than_sms():
    for bt in (1, 20, 50, 100):
        c = linear_case(bt, 200, 128 * 320 + 8, **EPILOGUES["gate"])
        call_linear(c)
        check_linear(c)


@pytest.mark.parametrize("bt", [3, 100, 300])
def test_linear_in_place(bt):
    c = linear_case(bt, 264, 520, **EPILOGUES["all"])
    call_linear(c)
    want = c["Y"].clone()
    for name in ("residual", "mul"):
        d = dict(c, **{name: c[name].clone()})
        d["Y"] = d[name]
        call_linear(d)
        assert torch.equal(d["Y"], want)


@pytest.mark.parametrize("bt", [4, 300])
def test_linear_special_values(bt):
    """NaN and infinities stay in their rows and columns; a dropped element is zero
    whatever it was."""
    d_in, d_out = 136, 264
    c = linear_case(bt, d_in, d_out, p=0.5, act=R.SILU)
    c["X"][1, 3] = float("nan")
    c["W"][5, 7] = float("inf")
    call_linear(c)
    keep = R.keep(bt, d_out, 0.5, SEED, OFFSET) > 0
    Y = f64(c["Y"])
    assert (Y[~keep] == 0).all()
    assert np.isnan(Y[1][keep[1]]).all()
    rest = np.ones_like(keep)
    rest[1] = False
    rest[:, 5] = False
    assert np.isfinite(Y[rest]).all()
    # +inf through the activation stays, -inf gives zero
    x = f64(c["X"])[:, 7]
    for r in range(bt):
        if r != 1 and keep[r, 5]:
            assert Y[r, 5] == (np.inf if x[r] > 0 else 0.0)


@pytest.mark.parametrize("bt,d_out", [(3, 256), (300, 256), (300, 264), (1100, 1040)])
@pytest.mark.parametrize("name", ["all", "all_fp32"])
def test_linear_at_16_byte_alignment(bt, d_out, name):
    """Matrices that start 16 bytes behind a 32-byte boundary, rows of 32 bytes or not."""
    c = linear_case(bt, 136, d_out, **EPILOGUES[name])
    call_linear(c)
    want = [c["Y"].clone(), c["Z"].clone()]

    def shifted(t):
        n = 16 // t.element_size()
        buf = torch.empty(t.numel() + 2 * n, dtype=t.dtype, device=DEV)
        out = buf[n:n + t.numel()].view(t.shape)
        assert out.data_ptr() % 32 == 16
        out.copy_(t)
        return out

    for k in ("X", "W", "bias", "mul", "residual", "Z", "Y"):
        d = dict(c, Z=torch.zeros_like(c["Z"]), Y=torch.zeros_like(c["Y"]))
        for name_ in (k,) if k != "Y" else ("X", "W", "bias", "mul", "residual", "Z", "Y"):
            d[name_] = shifted(d[name_])
        call_linear(d)
        assert torch.equal(d["Y"], want[0]) and torch.equal(d["Z"], want[1]), k


def test_more_than_2_to_the_31_elements():
    """Outputs and dropout blocks whose indexes pass 32 bits: the last rows."""
    bt, d_in, d_out, last = 140000, 8, 16384, 3
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    X, W = rand(1, (bt, d_in)), rand(2, (d_out, d_in))
    Y = torch.empty((bt, d_out), dtype=torch.bfloat16, device=DEV)
    F.linear_bf16(X, W, Y, p=0.5, seed=SEED, offset=OFFSET)
    ok()
    blocks = np.arange((bt - last) * d_out // 8, bt * d_out // 8)
    pick = [0, 1, len(blocks) // 2, len(blocks) - 1]
    want = np.array([[(w >> s) & 0xFFFF for w in R.philox4x32_10(
        (int(blocks[i]) & 0xFFFFFFFF, int(blocks[i]) >> 32, OFFSET, 0),
        (SEED & 0xFFFFFFFF, SEED >> 32)) for s in (0, 16)] for i in pick]) >= 32768
    Z, _ = R.linear(f64(X[-last:]), f64(W))
    kept = f64(Y[-last:]).reshape(-1, 8)
    assert np.array_equal(kept[pick] != 0, want)
    ref = np.where(kept != 0, 2 * Z.reshape(-1, 8), 0.0)
    within(kept, ref, BF * np.abs(ref) + 1e-5)
    y2 = torch.empty_like(Y)
    F.dropout(Y, y2, p=0.5, seed=SEED, offset=OFFSET)
    F.epilogue_backward(Y, Y, p=0.5, seed=SEED, offset=OFFSET)      # in place, the same mask
    ok()
    within(f64(y2[-last:]), 2 * kept.reshape(last, -1), BF * np.abs(2 * kept.reshape(last, -1)))
    assert torch.equal(Y, y2)


def test_linear_no_tokens():
    none = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    F.linear_bf16(none, rand(2, (24, 64)), torch.empty((0, 24), dtype=torch.bfloat16, device=DEV))
    ok()


def test_activations_and_their_slopes_over_the_range():
    """act(z) by a product with the identity, act'(z) by the gradient of ones."""
    n = 64
    z = torch.cat([torch.linspace(-20, 20, 40 * n), torch.tensor([1e30, -1e30, 200.0, -200.0, 0.0,
                   -0.0, 1e-30, -1e-30] * (n // 8))]).to(torch.bfloat16).view(-1, n).to(DEV)
    one = torch.eye(n, dtype=torch.bfloat16, device=DEV)
    for kind in KINDS:
        Y = torch.empty(z.shape, device=DEV)
        F.linear_bf16(z, one, Y, act=kind)
        z64 = f64(z)
        with np.errstate(over="ignore", invalid="ignore"):
            big = np.abs(z64) > 100
            ref = np.where(big, np.where(z64 > 0, z64, z64 if kind == R.NONE else 0.0),
                           R.act(np.where(big, 0.0, z64), kind))
            err = np.where(big, 0.0, act_error(np.where(big, 0.0, z64), kind))
        within(f64(Y), ref, 2 * U * np.abs(ref) + err + 1e-37)
        dz = torch.empty_like(z)
        F.epilogue_backward(torch.ones_like(z), dz, Z=z, act=kind)
        ok()
        zs = np.where(big, 0.0, z64)
        ref = np.where(big, (z64 > 0) | (kind == R.NONE), R.act_slope(zs, kind))
        within(f64(dz), ref, BF * np.abs(ref) + np.where(big, 0.0, slope_error(zs, kind)))


# ---------------------------------------------------------------- its gradient
BWD_SHAPES = [(1, 8), (1, 4096), (2, 136), (7, 128), (33, 264), (65, 1032), (333, 520), (1300, 64),
              (5000, 40), (700, 2056), (40, 14336)]


@pytest.mark.parametrize("rows,cols", BWD_SHAPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mul", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_epilogue_backward(rows, cols, kind, mul, p):
    dY, Z = rand(11, (rows, cols), 1e-2), rand(12, (rows, cols), 1.5)
    m = rand(13, (rows, cols)) if mul else None
    dZ, dm = torch.empty_like(Z), torch.empty_like(Z) if mul else None
    db = torch.empty(cols, device=DEV)
    how = dict(Z=Z, act=kind, mul=m, p=p, seed=SEED, offset=OFFSET)
    ws = torch.empty(max(F.epilogue_backward_workspace_bytes(rows, cols), 16), dtype=torch.uint8,
                     device=DEV)
    F.epilogue_backward(dY, dZ, dmul=dm, dbias=db, workspace=ws, **how)
    ok()
    factor = R.keep(rows, cols, p, SEED, OFFSET) if p else np.ones((rows, cols))
    m64 = f64(m) if mul else np.ones((rows, cols))
    z64, d64 = f64(Z), f64(dY)
    dz64, dm64, db64 = R.epilogue_backward(d64, z64, kind, m64, factor)
    da = np.abs(d64) * factor
    zerr = da * np.abs(m64) * slope_error(z64, kind) + 4 * U * np.abs(dz64)
    within(f64(dZ), dz64, BF * np.abs(dz64) + 1.01 * zerr)
    if mul:
        within(f64(dm), dm64, BF * np.abs(dm64) + 1.01 * da * act_error(z64, kind)
               + 4 * U * np.abs(dm64))
    # a column's sum: rows / 16 additions in a thread, 16 joined, then the partial rows'
    adds = rows / 16 + 16 + 100
    within(f64(db), db64, zerr.sum(0) + adds * U * np.abs(dz64).sum(0) + 1e-30)
    # the same without dbias, each output alone, and in place of each input
    dz2, dm2 = torch.empty_like(Z), torch.empty_like(Z) if mul else None
    F.epilogue_backward(dY, dz2, dmul=dm2, **how)
    assert torch.equal(dz2, dZ) and (not mul or torch.equal(dm2, dm))
    db2 = torch.empty_like(db)
    F.epilogue_backward(dY, dbias=db2, workspace=ws, **how)
    assert torch.equal(db2, db)
    for dst in ("dY", "Z") + (("mul",) if mul else ()):
        t = dict(dY=dY.clone(), Z=Z.clone(), mul=m.clone() if mul else None)
        F.epilogue_backward(t["dY"], t[dst], Z=t["Z"], act=kind, mul=t["mul"], p=p, seed=SEED,
                            offset=OFFSET, dmul=t["mul"] if mul and dst != "mul" else None,
                            dbias=db2, workspace=ws)
        assert torch.equal(t[dst], dZ) and torch.equal(db2, db)
        if mul and dst != "mul":
            assert torch.equal(t["mul"], dm)
    ok()


def test_epilogue_backward_of_dropped_elements_is_zero():
    """Whatever Z, mul and dY hold there."""
    rows, cols = 40, 264
    keep = R.keep(rows, cols, 0.5, SEED, OFFSET) > 0
    gone = torch.from_numpy(~keep).to(DEV)
    for bad in (float("nan"), float("inf"), -float("inf")):
        dY, Z, m = rand(1, (rows, cols)), rand(2, (rows, cols)), rand(3, (rows, cols))
        for t in (dY, Z, m):
            t[gone] = bad
        for kind in KINDS:
            dZ, dm, db = torch.empty_like(Z), torch.empty_like(Z), torch.empty(cols, device=DEV)
            F.epilogue_backward(dY, dZ, Z=Z, act=kind, mul=m, dmul=dm, dbias=db, p=0.5, seed=SEED,
                                offset=OFFSET,
                                workspace=torch.empty(1 << 20, dtype=torch.uint8, device=DEV))
            ok()
            for t in (dZ, dm):
                assert bool((t[gone] == 0).all()) and bool(torch.isfinite(t).all())
            assert bool(torch.isfinite(db).all())


def test_epilogue_backward_without_z():
    dY, m = rand(11, (20, 264)), rand(13, (20, 264))
    dZ, db = torch.empty_like(dY), torch.empty(264, device=DEV)
    F.epilogue_backward(dY, dbias=db, workspace=torch.empty(1 << 20, dtype=torch.uint8, device=DEV))
    within(f64(db), f64(dY).sum(0), 40 * U * np.abs(f64(dY)).sum(0))
    F.epilogue_backward(dY, dZ, mul=m)
    ok()
    ref = f64(dY) * f64(m)
    within(f64(dZ), ref, BF * np.abs(ref) + U * np.abs(ref))


def test_epilogue_backward_no_rows():
    none = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    db = torch.full((64,), 7.0, device=DEV)
    F.epilogue_backward(none, none, dbias=db)
    ok()
    assert float(db.abs().max()) == 0.0


@pytest.mark.parametrize("kind", KINDS[1:])
def test_epilogue_backward_against_differences(kind):
    """L = sum(dY * Y) as fp64 computes it: its central differences in Z, mul and bias."""
    rows, cols, t = 3, 16, 1e-5
    Z, m, dY = rand(21, (rows, cols), 1.5), rand(22, (rows, cols)), rand(23, (rows, cols))
    Z[0, 0] = 0.5       # away from ReLU's corner
    dZ, dm, db = torch.empty_like(Z), torch.empty_like(Z), torch.empty(cols, device=DEV)
    F.epilogue_backward(dY, dZ, Z=Z, act=kind, mul=m, dmul=dm, dbias=db, p=0.25, seed=9, offset=2)
    ok()
    factor = R.keep(rows, cols, 0.25, 9, 2)
    z64, m64, d64 = f64(Z), f64(m), f64(dY)

    def loss(z, mm):
        return (d64 * R.act(z, kind) * mm * factor).sum()

    for i in range(rows):
        for j in range(cols):
            e = np.zeros_like(z64)
            e[i, j] = t
            for got, num in ((dZ, loss(z64 + e, m64) - loss(z64 - e, m64)),
                             (dm, loss(z64, m64 + e) - loss(z64, m64 - e))):
                num /= 2 * t
                assert abs(num - float(got[i, j])) <= BF * abs(num) + 1e-6
    for j in range(cols):
        e = np.zeros_like(z64)
        e[:, j] = t
        num = (loss(z64 + e, m64) - loss(z64 - e, m64)) / (2 * t)
        assert abs(num - float(db[j])) <= 1e-5 * (1 + abs(num))


# ---------------------------------------------------------------- dropout
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 40), (64, 520), (1000, 1032), (2049, 512)])
@pytest.mark.parametrize("p", [0.1, 0.5, 0.999, 1e-6, 0.0])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(rows, cols, p, residual):
    x, r = rand(31, (rows, cols)), rand(32, (rows, cols), 3.0) if residual else None
    x[x == 0] = 1.0
    y = torch.empty_like(x)
    seed, offset = (1 << 63) + 12345, (1 << 40) + 3
    F.dropout(x, y, p=p, seed=seed, offset=offset, residual=r)
    ok()
    factor = R.keep(rows, cols, p, seed, offset)
    ref = f64(x) * factor + (f64(r) if residual else 0)
    within(f64(y), ref, BF * np.abs(ref) + 2 * U * np.abs(f64(x) * factor))
    if not residual:
        assert np.array_equal(f64(y) == 0, factor == 0)
    else:
        assert torch.equal(y[torch.from_numpy(factor == 0).to(DEV)],
                           r[torch.from_numpy(factor == 0).to(DEV)])
    for place in ("x", "r")[:1 + residual]:
        t = dict(x=x.clone(), r=r.clone() if residual else None)
        F.dropout(t["x"], t[place], p=p, seed=seed, offset=offset, residual=t["r"])
        assert torch.equal(t[place], y)


def test_dropout_share_and_independence():
    x = torch.ones((512, 4096), dtype=torch.bfloat16, device=DEV)
    kept = []
    for seed, offset in ((1, 0), (2, 0), (1, 1)):
        y = torch.empty_like(x)
        F.dropout(x, y, p=0.25, seed=seed, offset=offset)
        kept.append((y != 0).double())
        # 2^21 draws: five standard deviations of the share are 0.0015
        assert abs(float(kept[-1].mean()) - 0.75) < 0.0015
    for a, b in ((0, 1), (0, 2), (1, 2)):
        c = ((kept[a] - 0.75) * (kept[b] - 0.75)).mean() / (0.75 * 0.25)
        assert abs(float(c)) < 0.004
    ok()


def test_dropout_counter_in_a_replayed_graph():
    x = rand(33, (40, 264))
    y, c = torch.empty_like(x), torch.zeros(1, dtype=torch.int64, device=DEV)
    F.dropout(x, y, p=0.5, seed=3, offset=10, counter=c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        F.dropout(x, y, p=0.5, seed=3, offset=10, counter=c)
        c += 1
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(f64(y) != 0, (R.keep(40, 264, 0.5, 3, 10 + i) > 0) & (f64(x) != 0))
    c.fill_(-11)     # modulo 2^64
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(f64(y) != 0, (R.keep(40, 264, 0.5, 3, -1) > 0) & (f64(x) != 0))
    ok()


# ---------------------------------------------------------------- rotary positions
HEADS = [(1, 1, 1, 64, 64, "dense"), (1, 32, 8, 128, 128, "fused"), (5, 3, 1, 80, 32, "fused"),
         (33, 8, 2, 96, 24, "dense"), (7, 4, 4, 256, 256, "heads"), (200, 6, 3, 128, 64, "heads"),
         (300, 16, 2, 64, 48, "fused"), (3000, 5, 1, 128, 128, "fused"), (9, 2, 0, 8, 8, "dense"),
         (64, 9, 7, 40, 16, "fused"), (11, 33, 5, 248, 136, "heads")]
SCALES = {"none": dict(), "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
          "llama3": dict(factor=8.0, context=8192.0, low=1.0, high=4.0),
          "yarn": dict(factor=16.0, context=4096.0, low=1.0, high=32.0)}
SCALE_ID = {"none": F.ROPE_SCALE_NONE, "linear": F.ROPE_SCALE_LINEAR, "ntk": F.ROPE_SCALE_NTK,
            "llama3": F.ROPE_SCALE_LLAMA3, "yarn": F.ROPE_SCALE_YARN}


def heads(seed, tokens, hq, hk, dim, how, std=1.0):
    """Queries and keys as dense tensors, views of one fused buffer, or [heads, tokens, dim]."""
    if how == "fused":
        qkv = rand(seed, (tokens, hq + 2 * hk, dim), std)
        return qkv[:, :hq], qkv[:, hq:hq + hk] if hk else None
    if how == "heads":
        return (rand(seed, (hq, tokens, dim), std).transpose(0, 1),
                rand(seed + 1, (hk, tokens, dim), std).transpose(0, 1))
    return rand(seed, (tokens, hq, dim), std), rand(seed + 1, (tokens, hk, dim), std) if hk else None


def positions_of(tokens, how):
    g = torch.Generator().manual_seed(8)
    if how == "far":
        return torch.randint(0, 1 << 31, (tokens,), generator=g).to(DEV)
    return torch.randint(-100, 4096, (tokens,), generator=g).to(DEV) if how == "any" else None


def pair_sum(x, half, layout):
    """|a| + |b| of each rotated element's pair; |x| of the others."""
    out = np.abs(x)
    ia, ib = ((np.arange(half), np.arange(half) + half) if layout == R.HALF
              else (2 * np.arange(half), 2 * np.arange(half) + 1))
    s = out[..., ia] + out[..., ib]
    out[..., ia], out[..., ib] = s, s
    return out


def turn_error(pos, rad):
    """How far a computed cosine or sine may be off: the phase's rounding to fp32 (2^-24 of
    half a turn), sincospi's 2 ulp, the magnitude's and the product's roundings; and the
    fp64 definition's own angle, 2^-52 of it."""
    return 16 * U + 2.0 ** -51 * np.max(np.abs(np.asarray(pos, np.float64))) * np.max(rad)


@pytest.mark.parametrize("tokens,hq,hk,dim,rot,how", HEADS)
@pytest.mark.parametrize("layout", [R.HALF, R.INTERLEAVED])
@pytest.mark.parametrize("scale", ["none", "llama3", "yarn"])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(tokens, hq, hk, dim, rot, how, layout, scale, inverse):
    q, k = heads(41, tokens, hq, hk, dim, how)
    freqs, mag = F.rope_frequencies(rot, 500000.0, scaling=SCALE_ID[scale], **SCALES[scale])
    rad, mag64 = R.frequencies(rot, 500000.0, scale, **SCALES[scale])
    assert abs(mag - mag64) <= U * mag64
    pos = positions_of(tokens, "far" if scale == "llama3" else ("any" if scale == "yarn" else None))
    pos64 = np.arange(tokens) if pos is None else pos.cpu().numpy()
    qo = torch.empty((tokens, hq, dim), dtype=torch.bfloat16, device=DEV)
    ko = torch.empty((tokens, hk, dim), dtype=torch.bfloat16, device=DEV) if hk else None
    F.rope(q, k, freqs, q_out=qo, k_out=ko, positions=pos, magnitude=mag, layout=layout,
           inverse=inverse)
    ok()
    for x, y in ((q, qo), (k, ko)):
        if x is None:
            continue
        ref = R.rotate(f64(x), pos64, rad, mag, layout, inverse)
        within(f64(y), ref, BF * np.abs(ref)
               + turn_error(pos64, rad) * mag * pair_sum(f64(x), rot // 2, layout))
        assert torch.equal(y[..., rot:], x[..., rot:])      # what does not turn is copied
    # in place, on the views themselves; what lies between them stays
    if how == "fused" and hk:
        buf = q._base
        rest = buf[:, hq + hk:].clone()
        F.rope(q, k, freqs, positions=pos, magnitude=mag, layout=layout, inverse=inverse)
        ok()
        assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(buf[:, hq + hk:], rest)


def test_rope_inverse_is_the_gradient():
    """sum(dy * R x) = sum(R' dy * x) up to the outputs' roundings."""
    q, _ = heads(43, 20, 4, 0, 64, "dense")
    dy, _ = heads(45, 20, 4, 0, 64, "dense")
    freqs, mag = F.rope_frequencies(48, 10000.0, scaling=F.ROPE_SCALE_YARN, **SCALES["yarn"])
    y, dx = torch.empty_like(q), torch.empty_like(q)
    for layout in (F.ROPE_HALF, F.ROPE_INTERLEAVED):
        F.rope(q, None, freqs, q_out=y, magnitude=mag, layout=layout)
        F.rope(dy, None, freqs, q_out=dx, magnitude=mag, layout=layout, inverse=True)
        a, b = f64(dy) * f64(y), f64(dx) * f64(q)
        assert abs(a.sum() - b.sum()) <= BF * (np.abs(a).sum() + np.abs(b).sum())
        t, rad = 1e-5, R.frequencies(48, 10000.0, "yarn", **SCALES["yarn"])[0]
        x64, d64 = f64(q), f64(dy)
        for i in (0, 5, 23, 24, 40, 47, 48, 63):
            e = np.zeros_like(x64)
            e[7, 2, i] = t
            num = ((d64 * (R.rotate(x64 + e, np.arange(20), rad, mag, layout)
                           - R.rotate(x64 - e, np.arange(20), rad, mag, layout))).sum()) / (2 * t)
            assert abs(num - float(dx[7, 2, i])) <= BF * abs(num) + 1e-5
    ok()


def test_rope_no_tokens_or_heads():
    freqs, _ = F.rope_frequencies(32, 10000.0)
    for shape in ((0, 4, 64), (5, 0, 64)):
        q = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        F.rope(q, q.clone(), freqs)
    q, k = rand(1, (5, 4, 64)), torch.empty((5, 0, 64), dtype=torch.bfloat16, device=DEV)
    want = q.clone()
    F.rope(want, None, freqs)
    F.rope(q, k, freqs)
    assert torch.equal(q, want)
    ok()


def test_rope_offsets_beyond_32_bits():
    """A key cache of more than 2^32 elements, rotated in its last rows."""
    tokens, stride = 3, (1 << 31) + 64
    if torch.cuda.mem_get_info()[0] < 3 * (2 * stride * 2):
        pytest.skip("needs 26 GB")
    buf = torch.empty(2 * stride + 256, dtype=torch.bfloat16, device=DEV)
    q = buf.as_strided((tokens, 2, 64), (stride, 64, 1))
    q.copy_(rand(47, (tokens, 2, 64)))
    freqs, _ = F.rope_frequencies(64, 10000.0)
    want = q.contiguous()
    F.rope(want, None, freqs)
    F.rope(q, None, freqs)
    ok()
    assert torch.equal(q.contiguous(), want)


def test_rope_frequencies_against_the_definition():
    for rot in (8, 24, 64, 128, 256):
        for scale, kw in SCALES.items():
            table, mag = F.rope_frequencies(rot, 10000.0, scaling=SCALE_ID[scale], device="cpu", **kw)
            rad, mag64 = R.frequencies(rot, 10000.0, scale, **kw)
            got = (table.numpy().astype(np.uint64).astype(np.float64)) / 2.0 ** 64 * 2 * np.pi
            assert np.abs(got - rad).max() <= 1e-14 and abs(mag - mag64) <= U * mag64


# ---------------------------------------------------------------- the norm of heads
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,how", HEADS)
@pytest.mark.parametrize("layout", [R.HALF, R.INTERLEAVED])
@pytest.mark.parametrize("gain_dtype", [torch.float32, torch.bfloat16])
def test_qk_norm_rope(tokens, hq, hk, dim, rot, how, layout, gain_dtype):
    q, k = heads(51, tokens, hq, hk, dim, how, 2.0)
    gains = [(1 + rand(53 + i, (dim,), 0.2, torch.float32)).to(gain_dtype) for i in range(2)]
    freqs, mag = F.rope_frequencies(rot, 10000.0)
    rad, _ = R.frequencies(rot, 10000.0)
    pos = positions_of(tokens, "any")
    pos64 = pos.cpu().numpy()
    eps = 1e-5
    qo = torch.empty((tokens, hq, dim), dtype=torch.bfloat16, device=DEV)
    ko = torch.empty((tokens, hk, dim), dtype=torch.bfloat16, device=DEV) if hk else None
    how_ = dict(eps=eps, positions=pos, layout=layout)
    kg = gains[1] if hk else None
    F.qk_norm_rope(q, k, gains[0], kg, freqs, q_out=qo, k_out=ko, **how_)
    ok()
    # the mean of squares: at most 16 + 5 roundings of positive terms, half of it in the
    # root, two products and the root's 2 ulp
    rel = 24 * U
    for x, y, g in ((q, qo, gains[0]), (k, ko, gains[1])):
        if x is None:
            continue
        n = R.head_norm(f64(x), f64(g), eps)
        ref = R.rotate(n, pos64, rad, 1.0, layout)
        within(f64(y), ref, BF * np.abs(ref)
               + (turn_error(pos64, rad) + rel) * pair_sum(n, rot // 2, layout))
    # gradients, with and without those of the gains, in place of dq and dk and of q and k
    dq, dk = heads(57, tokens, hq, hk, dim, "dense", 1e-2)
    dqo, dko = torch.empty_like(dq), torch.empty_like(dk) if hk else None
    dg = [torch.empty(dim, device=DEV), torch.empty(dim, device=DEV) if hk else None]
    ws = torch.empty(F.qk_norm_rope_backward_workspace_bytes(dim), dtype=torch.uint8, device=DEV)
    F.qk_norm_rope_backward(dq, dk, q, k, gains[0], kg, freqs, dq_out=dqo, dk_out=dko,
                            dq_gain=dg[0], dk_gain=dg[1], workspace=ws, **how_)
    ok()
    for x, dy, dx, g, dgain in ((q, dq, dqo, gains[0], dg[0]), (k, dk, dko, gains[1], dg[1])):
        if x is None:
            continue
        x64, g64 = f64(x), f64(g)
        dn = R.rotate(f64(dy), pos64, rad, 1.0, layout, True)
        dx64, dg64 = R.head_norm_backward(dn, x64, g64, eps)
        r = 1 / np.sqrt((x64 * x64).mean(2, keepdims=True) + eps)
        xh = np.abs(x64 * r)
        d = pair_sum(f64(dy), rot // 2, layout)
        terr = turn_error(pos64, rad)
        u, uerr = np.abs(g64) * d, (terr + 4 * U) * np.abs(g64) * d
        noise = r * (uerr + rel * u + xh * ((uerr + (rel + 40 * U) * u) * xh).mean(2, keepdims=True)
                     + 3 * rel * xh * (u * xh).mean(2, keepdims=True))
        within(f64(dx), dx64, BF * np.abs(dx64) + 1.01 * noise)
        # dgain: a lane's heads one after the other, then warps and blocks
        adds = min(tokens * x.shape[1], 200) + 100
        within(f64(dgain), dg64, ((terr + rel + adds * U) * d * xh).sum((0, 1)) + 1e-30)
    da, db = dq.clone(), dk.clone() if hk else None
    F.qk_norm_rope_backward(da, db, q, k, gains[0], kg, freqs, **how_)
    assert torch.equal(da, dqo) and (not hk or torch.equal(db, dko))
    again = torch.empty(dim, device=DEV)
    qc, kc = q.clone(), k.clone() if hk else None
    F.qk_norm_rope_backward(dq, dk, qc, kc, gains[0], kg, freqs, dq_out=qc, dk_out=kc,
                            dq_gain=again, workspace=ws, **how_)
    assert torch.equal(qc, dqo) and (not hk or torch.equal(kc, dko)) and torch.equal(again, dg[0])
    F.qk_norm_rope(q, k, gains[0], kg, freqs, **how_)      # the forward pass in place
    assert torch.equal(q, qo) and (not hk or torch.equal(k, ko))
    ok()


def test_qk_norm_rope_backward_against_differences():
    tokens, h, dim, rot, eps, t = 2, 3, 16, 8, 1e-3, 1e-5
    q, dy = rand(61, (tokens, h, dim)), rand(62, (tokens, h, dim))
    g = rand(63, (dim,), 1.0, torch.float32)
    freqs, _ = F.rope_frequencies(rot, 100.0)
    rad = R.frequencies(rot, 100.0)[0]
    for layout in (R.HALF, R.INTERLEAVED):
        dx, dg = torch.empty_like(q), torch.empty(dim, device=DEV)
        ws = torch.empty(F.qk_norm_rope_backward_workspace_bytes(dim), dtype=torch.uint8, device=DEV)
        F.qk_norm_rope_backward(dy, None, q, None, g, None, freqs, eps=eps, dq_out=dx, dq_gain=dg,
                                workspace=ws, layout=layout)
        ok()
        x64, g64, d64 = f64(q), f64(g), f64(dy)

        def loss(x, gg):
            return (d64 * R.rotate(R.head_norm(x, gg, eps), np.arange(tokens), rad, 1.0, layout)).sum()

        for at in np.ndindex(x64.shape):
            e = np.zeros_like(x64)
            e[at] = t
            num = (loss(x64 + e, g64) - loss(x64 - e, g64)) / (2 * t)
            assert abs(num - float(dx[at])) <= BF * abs(num) + 1e-5
        for j in range(dim):
            e = np.zeros_like(g64)
            e[j] = t
            num = (loss(x64, g64 + e) - loss(x64, g64 - e)) / (2 * t)
            assert abs(num - float(dg[j])) <= 1e-5 * (1 + abs(num))


def test_qk_norm_rope_zero_heads_and_no_tokens():
    dim = 64
    freqs, _ = F.rope_frequencies(dim, 10000.0)
    g = torch.ones(dim, device=DEV)
    q = torch.zeros((3, 2, dim), dtype=torch.bfloat16, device=DEV)
    q[1, 0, 5] = float("nan")
    F.qk_norm_rope(q, None, g, None, freqs, eps=1e-6)
    ok()
    assert torch.isnan(q[1, 0]).all() and float(q[0].abs().max()) == 0 and float(q[1, 1].abs().max()) == 0
    none = torch.empty((0, 2, dim), dtype=torch.bfloat16, device=DEV)
    dg = [torch.full((dim,), 7.0, device=DEV) for _ in range(2)]
    ws = torch.empty(F.qk_norm_rope_backward_workspace_bytes(dim), dtype=torch.uint8, device=DEV)
    F.qk_norm_rope_backward(none, none, none, none, g, g, freqs, eps=1e-6, dq_gain=dg[0],
                            dk_gain=dg[1], workspace=ws)
    ok()
    assert float(dg[0].abs().max()) == 0 and float(dg[1].abs().max()) == 0
