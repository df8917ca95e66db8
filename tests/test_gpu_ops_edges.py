"""The operators around the weight gradient where they can go wrong: ties between
two codes and scales far apart, against their fp64 definitions (oracle/ops.py)."""
import numpy as np
import pytest
import torch

from oracle import ops as R
from tests.gpu_util import DEV, F, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ok():
    st = F.device_error()
    assert st == 0, F.status_string(st)


# ---------------------------------------------------------------- quantiser
def every_quotient(block_rows):
    """bf16 rows in which each of the 128 significands an amax can have meets each
    that another entry can have, 0 to 19 powers of two below it: 2560 rows of two
    blocks with one amax, 1 + m / 128 (or, for block_rows 128, 128 x 128 blocks
    with one amax)."""
    sig = np.arange(128, 256) / 128.0
    amax = sig[:, None, None]
    x = np.broadcast_to(sig * 2.0 ** -np.arange(20.0)[:, None], (128, 20, 128))
    x = np.where(x <= amax, x, -x / 2)               # both signs, none above amax
    if block_rows == 1:
        rows = np.concatenate([x, -x], 2)            # [128, 20, 256]
        rows[:, :, 0] = rows[:, :, 255] = amax[:, :, 0]   # the other block has what this hides
        return rows.reshape(2560, 256)
    rows = np.zeros((128, 128, 128))
    rows[:, :20] = x
    rows[:, 20:40] = -x
    rows[:, 127, 127] = amax[:, 0, 0]
    return rows.reshape(128 * 128, 128)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("power", [0, -100, 127])
def test_quantize_rounds_every_quotient_to_the_nearest_code(block_rows, power):
    # 448 x is exact in fp64 and the division correctly rounded, so a tie is a tie
    # and nothing else comes near one: the codes have to be equal
    x64 = every_quotient(block_rows) * 2.0 ** power
    # whole blocks, and rows whose last block is partial (another kernel)
    for cols in (x64.shape[1], x64.shape[1] - 8):
        part = np.ascontiguousarray(x64[:, :cols])
        a = R.spread(R.block_amax(part, block_rows), block_rows, part.shape)
        x = torch.from_numpy(part).to(torch.bfloat16).to(DEV)
        assert np.array_equal(f64(x), part)
        codes, scales = F.alloc_b128(*x.shape, block_rows)
        F.quantize_b128(x, codes, scales, block_rows=block_rows)
        ok()
        held = a < 448 * 2.0 ** -126                 # the scale is 2^-126
        bad = f64(codes) != R.e4m3_round(np.where(held, part * 2.0 ** 126, part * 448 / a))
        assert not bad.any(), int(bad.sum())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_keeps_the_sign_of_zero(block_rows):
    x = torch.zeros((3, 136), device=DEV)
    x[:, 1::2] = -0.0
    x[0, 2], x[1, 4] = 1.53125, -3.25      # 448 / amax rounded up and down
    codes, scales = F.alloc_b128(3, 136, block_rows)
    F.quantize_b128(x.bfloat16(), codes, scales, block_rows=block_rows)
    ok()
    assert torch.equal(torch.signbit(codes.float()), torch.signbit(x))


# ---------------------------------------------------------------- the norm's codes
@pytest.mark.parametrize("rows,cols", [(4096, 4096), (600, 4096), (9000, 512), (3000, 1032),
                                       (500, 8328), (60, 32768), (20000, 136)])
@pytest.mark.parametrize("gain", ["fp32", "bf16", "one"])
@pytest.mark.parametrize("res", [False, True])
def test_rmsnorm_codes(rows, cols, gain, res):
    # rstd is common to a row: the codes are those of h gain, in fp64 exact here.  The
    # kernel's quotients carry at most six roundings (h rstd gain, its amax, their
    # reciprocal, the product): within 6 x 2^-24 of halfway either code may be taken
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x = torch.randn((rows, cols), generator=g, device=DEV).bfloat16()
    r = torch.randn((rows, cols), generator=g, device=DEV).bfloat16() if res else None
    w = torch.ones(cols, device=DEV) if gain == "one" else \
        1 + 0.2 * torch.randn(cols, generator=g, device=DEV)
    w = w.to(torch.bfloat16 if gain == "bf16" else torch.float32)
    codes, scales = F.alloc_b128(rows, cols)
    F.rmsnorm(x, w, eps=1e-5, residual=r, codes=codes, scales=scales)
    ok()
    h = x.float() + r.float() if res else x.float()
    y = torch.zeros((rows, -(-cols // 128) * 128), dtype=torch.float64, device=DEV)
    y[:, :cols] = h.double() * w.double()
    a = y.view(rows, -1, 128).abs().amax(2).repeat_interleave(128, 1)[:, :cols]
    q = y[:, :cols] * 448 / a
    step = torch.exp2(torch.clamp(torch.frexp(q)[1] - 1, min=-6).double() - 3)
    got = codes.double()
    bad = (got - q).abs() > step / 2 + q.abs() * 6 * 2.0 ** -24
    assert not bad.any(), int(bad.sum())


# ---------------------------------------------------------------- products
def product_case(seed, op, bt, d_in, d_out, codes=256):
    """Random operands of one product: code bytes below `codes` (with both signs) and
    scales around one; the call, and its reference from the codes and scales given."""
    g = torch.Generator().manual_seed(seed)
    k, n = (d_in, d_out) if op == "linear" else (d_out, d_in)

    def matrix(rows, cols, block_rows):
        c = torch.randint(0, min(codes, 128), (rows, cols), generator=g, dtype=torch.uint8)
        c |= torch.randint(0, 2, (rows, cols), generator=g, dtype=torch.uint8) << 7
        c[(c & 0x7F) == 0x7F] = 0x30           # no NaN
        sr = rows if block_rows == 1 else -(-rows // 128)
        s = torch.exp2(torch.randn((sr, -(-cols // 128)), generator=g))
        return c.view(torch.float8_e4m3fn), s.float()

    return matrix(bt, k, 1), matrix(d_out, d_in, 128), k, n


def check(op, a, sa, w, sw, k, n, dtype=torch.float32):
    out = torch.empty((a.shape[0], n), dtype=dtype, device=DEV)
    call = F.linear_fp8 if op == "linear" else F.dgrad_fp8
    call(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), out)
    ok()
    a64, w64 = R.dequantize(f64(a), f64(sa), 1), R.dequantize(f64(w), f64(sw), 128)
    if op == "linear":
        w64 = w64.T
    a64, w64 = (torch.from_numpy(np.ascontiguousarray(t)).to(DEV) for t in (a64, w64))
    ref, mag = a64 @ w64, a64.abs() @ w64.abs()
    # inside a block the tensor core adds 128 exact products in groups, at most 4
    # alignments of 2^-23 of the partial sums' magnitude and the groups' own;
    # outside, one product and one addition per block; below 2^-126 a step is 2^-149
    nb = -(-k // 128)
    tol = (18 + nb) * 2.0 ** -23 * mag + (nb + 1) * 2.0 ** -149
    if dtype == torch.bfloat16:
        tol = tol + (2.0 ** -8 + 2.0 ** -24) * ref.abs()
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((out.double() - ref).abs()[bad].max()))
    return out


# the forms of the products: up to 16, 32, 64 and 128 tokens, with the reduction on
# one CTA and on several, tiles of one CTA and of a pair
FORMS = [(3, {}), (3, dict(splits=1)), (30, {}), (50, {}), (100, dict(splits=2)), (200, {}),
         (300, dict(cg=2))]


@pytest.mark.parametrize("op", ["linear", "dgrad"])
@pytest.mark.parametrize("bt,how", FORMS)
@pytest.mark.parametrize("case", ["tiny", "huge", "rising", "rising_to_huge"])
def test_products_of_scales_outside_fp32(tune, op, bt, how, case):
    # each scale is one the format allows, and so is the result; their product is not
    tune(**how)
    d_in, d_out = 2576, 2320
    small = case in ("huge", "rising_to_huge")       # sums of 2^-10: codes below 2^-6
    (a, sa), (w, sw), k, n = product_case(90, op, bt, d_in, d_out, 8 if small else 256)
    if case == "tiny":          # sums up to 2^20 times 2^-140
        sa, sw = sa * 2.0 ** -110, sw * 2.0 ** -30
    elif case == "huge":        # times 2^127
        sa, sw = sa * 2.0 ** 85, sw * 2.0 ** 42
    elif case == "rising":      # empty blocks, then products on both sides of 2^-120
        a.view(torch.uint8)[:, :3 * 128] = 0
        sa[:, :3] = 0
        sa[:, 3:9] *= 2.0 ** -100
        sa[:, 9:] *= 2.0 ** -97
        sw *= 2.0 ** -22
    else:                       # products on both sides of 2^100
        sa[:, :9] *= 2.0 ** 60
        sa[:, 9:] *= 2.0 ** 63
        sw *= 2.0 ** 39
    out = check(op, a, sa, w, sw, k, n)
    assert torch.isfinite(out).all() and float(out.abs().max()) > 0


@pytest.mark.parametrize("op", ["linear", "dgrad"])
@pytest.mark.parametrize("bt,how", FORMS)
@pytest.mark.parametrize("zero", ["weight", "tokens", "blocks"])
def test_products_of_zeros(tune, op, bt, how, zero):
    # zero scales: a weight that has not left its initial zeros, masked tokens, and
    # blocks of both that never meet another
    tune(**how)
    (a, sa), (w, sw), k, n = product_case(91, op, bt, 2576, 2320)
    if zero == "weight":
        w.view(torch.uint8).zero_()
        sw.zero_()
    elif zero == "tokens":
        a.view(torch.uint8)[::2] = 0
        sa[::2] = 0
    else:
        nb = sa.shape[1]
        for b in range(nb):
            part = a.view(torch.uint8)[:, b * 128:(b + 1) * 128]
            if b % 2:
                part.zero_()
                sa[:, b] = 0
            elif op == "linear":
                w.view(torch.uint8)[:, b * 128:(b + 1) * 128] = 0
                sw[:, b] = 0
            else:
                w.view(torch.uint8)[b * 128:(b + 1) * 128] = 0
                sw[b] = 0
    out = check(op, a, sa, w, sw, k, n)
    assert bool((out[::2] == 0).all()) and (zero == "tokens" or not out.any())
