"""Every form of the operators' kernels against the fp64 definitions: tiles of one
CTA and of a pair with several tiles each, few tokens with the reduction split
unevenly or with more tiles than SMs, the norm's streams of wide rows, and sums
written in place.  tests/test_host_code.py pins that these shapes take the forms
they are here for."""
import pytest
import torch

from tests import test_gpu_ops as ops
from tests.gpu_util import DEV, F, require_gpu
from tests.test_gpu_ops_edges import check, product_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def product(op, bt, d_in, d_out, dtype=torch.float32, seed=95):
    (a, sa), (w, sw), k, n = product_case(seed, op, bt, d_in, d_out)
    return check(op, a, sa, w, sw, k, n, dtype)


# ---------------------------------------------------------------- products
# (bt, k, n): two tiles and more for every CTA or pair, reductions of 3 to 17
# blocks that end inside a block and inside a batch of scales
LONG = [(1500, 2064, 4112), (2000, 1040, 4112), (2311, 272, 5200)]


@pytest.mark.parametrize("op", ["linear", "dgrad"])
@pytest.mark.parametrize("bt,k,n", LONG)
@pytest.mark.parametrize("cg", [0, 1, 2])
def test_products_of_several_tiles(tune, op, bt, k, n, cg):
    tune(cg=cg)
    d_in, d_out = (k, n) if op == "linear" else (n, k)
    product(op, bt, d_in, d_out)


@pytest.mark.parametrize("op", ["linear", "dgrad"])
@pytest.mark.parametrize("cg", [1, 2])
@pytest.mark.parametrize("bt,d_in,d_out", [(1, 16, 16), (3, 272, 144), (128, 1040, 400),
                                           (130, 400, 16), (257, 144, 272), (700, 2320, 1040)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_products_with_the_tile_given(tune, op, cg, bt, d_in, d_out, dtype):
    tune(cg=cg)
    product(op, bt, d_in, d_out, dtype)


@pytest.mark.parametrize("op", ["linear", "dgrad"])
@pytest.mark.parametrize("splits", [1, 2, 4, 8])
@pytest.mark.parametrize("bt,k,n", [(1, 1152, 272), (16, 2176, 144), (17, 4352, 272),
                                    (60, 656, 400), (100, 2320, 144), (5, 128, 272)])
def test_products_with_the_split_given(tune, op, splits, bt, k, n):
    # 9, 17, 34, 6, 19 blocks and a single one on 1 to 8 CTAs
    tune(splits=splits)
    d_in, d_out = (k, n) if op == "linear" else (n, k)
    product(op, bt, d_in, d_out)


FEW = [(bt, n) for bt in (1, 16, 20, 50, 100) for n in (19600, 39184)]


@pytest.mark.parametrize("op", ["linear", "dgrad"])
@pytest.mark.parametrize("bt,n", FEW)
def test_few_tokens_with_more_tiles_than_sms(op, bt, n):
    k = 1040
    d_in, d_out = (k, n) if op == "linear" else (n, k)
    product(op, bt, d_in, d_out, torch.bfloat16)


# ---------------------------------------------------------------- the norm
STREAMS = [(400, 8200), (330, 16384), (1217, 9224)]
BACKWARD_STREAMS = [(1100, 8200), (600, 16384), (2100, 4104)]


@pytest.mark.parametrize("rows,cols", STREAMS)
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("gain_dtype", [torch.float32, torch.bfloat16])
def test_rmsnorm_streams_of_two_vectors_a_thread(rows, cols, res, gain_dtype):
    ops.test_rmsnorm(rows, cols, res, gain_dtype)


@pytest.mark.parametrize("rows,cols", BACKWARD_STREAMS)
@pytest.mark.parametrize("with_dsum", [False, True])
@pytest.mark.parametrize("gain_dtype", [torch.float32, torch.bfloat16])
def test_rmsnorm_backward_streams_of_wide_rows(rows, cols, with_dsum, gain_dtype):
    ops.test_rmsnorm_backward(rows, cols, with_dsum, gain_dtype)


# a warp per row; a block per row with one, two and four vectors a thread; streams
# with one and two
IN_PLACE = [(1300, 392), (300, 4096), (320, 4096), (40, 4104), (40, 8200), (7, 16392),
            (640, 4096), (400, 8200), (5000, 1032)]


@pytest.mark.parametrize("rows,cols", IN_PLACE)
@pytest.mark.parametrize("take", [0, 1])
def test_rmsnorm_sum_in_place(rows, cols, take):
    # the sum in place of x or of the residual: the same bits as beside them
    x, r = ops.rand(1, (rows, cols)), ops.rand(2, (rows, cols), 3.0)
    gain = ops.rand(3, (cols,), 1.0, torch.float32)

    def run(xi, ri, s):
        y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
        codes, scales = F.alloc_b128(rows, cols)
        F.rmsnorm(xi, gain, eps=1e-6, residual=ri, sum_out=s, y=y, codes=codes, scales=scales,
                  rstd=rstd)
        ops.ok()
        return [s, y, rstd, codes.view(torch.uint8), scales]

    want = run(x, r, torch.empty_like(x))
    assert torch.equal(want[0], (x.float() + r.float()).bfloat16())
    both = [x.clone(), r.clone()]
    got = run(*both, both[take])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(both[1 - take], (x, r)[1 - take])
