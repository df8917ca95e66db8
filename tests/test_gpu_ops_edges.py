"""The operators around the weight gradient where they can go wrong: ties between
two codes, against their fp64 definitions (oracle/ops.py)."""
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
