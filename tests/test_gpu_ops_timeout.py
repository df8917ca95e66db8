"""Bounded waits of the norm's, the quantiser's and the 8-bit products' kernels that
run out: the testing aid lets the first copy wait for bytes that never come.  The
kernel records FORGE_ERR_DEVICE_TIMEOUT and returns, the context stays usable, and
what lies beside the outputs is not touched."""
import pytest
import torch

from tests.gpu_util import DEV, F, require_gpu
from tests.test_gpu_ops import rand
from tests.test_gpu_ops_edges import product_case

pytestmark = pytest.mark.gpu
TIMEOUT = 9


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def runs_out(call, outputs):
    """The call with the first arrival dropped, then as usual, against itself before."""
    call()
    assert F.device_error() == 0
    want = [t.clone() for t in outputs]
    F.set_wait_limit_ns(20_000_000)
    try:
        F.debug_drop_first_arrival(True)
        call()
        assert F.device_error() == TIMEOUT
        assert F.device_error() == 0      # cleared
    finally:
        F.debug_drop_first_arrival(False)
        F.set_wait_limit_ns(2_000_000_000)
    call()
    assert F.device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(outputs, want))


def fenced(rows, cols, dtype):
    """A matrix between two rows of sevens, and those rows."""
    buf = torch.full(((rows + 2) * cols,), 7.0, device=DEV).to(dtype)
    return buf[cols:-cols].view(rows, cols), (buf[:cols], buf[-cols:])


def untouched(*edges):
    assert all(bool((e.float() == 7).all()) for pair in edges for e in pair)


@pytest.mark.parametrize("rows,cols", [(640, 4096), (400, 8200), (5000, 1032)])
@pytest.mark.parametrize("res", [False, True])
def test_rmsnorm(rows, cols, res):
    x, r = rand(1, (rows, cols)), rand(2, (rows, cols)) if res else None
    gain = torch.ones(cols, device=DEV)
    y, ye = fenced(rows, cols, torch.bfloat16)
    s, se = fenced(rows, cols, torch.bfloat16)
    codes, scales = F.alloc_b128(rows, cols)
    rstd = torch.empty(rows, device=DEV)
    runs_out(lambda: F.rmsnorm(x, gain, eps=1e-5, residual=r, sum_out=s, y=y, codes=codes,
                               scales=scales, rstd=rstd),
             [y, s, codes.view(torch.uint8), scales, rstd])
    untouched(ye, se)


@pytest.mark.parametrize("rows,cols", [(2100, 4104), (600, 16384), (2000, 1032)])
@pytest.mark.parametrize("with_dsum", [False, True])
def test_rmsnorm_backward(rows, cols, with_dsum):
    h, dy = rand(1, (rows, cols)), rand(2, (rows, cols), 1e-2)
    dsum = rand(3, (rows, cols), 1e-2) if with_dsum else None
    gain, rstd = torch.ones(cols, device=DEV), torch.ones(rows, device=DEV)
    dx, edge = fenced(rows, cols, torch.bfloat16)
    dgain = torch.empty(cols, device=DEV)
    ws = torch.empty(F.rmsnorm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    runs_out(lambda: F.rmsnorm_backward(dy, h, gain, rstd, dx, dgain, dsum=dsum, workspace=ws),
             [dx, dgain])
    untouched(edge)


@pytest.mark.parametrize("rows,cols", [(8, 16), (300, 1040), (5000, 4112)])
def test_quantize(rows, cols):
    x = rand(1, (rows, cols))
    codes, edge = fenced(rows, cols, torch.float8_e4m3fn)
    scales = F.alloc_b128(rows, cols, 128)[1]
    runs_out(lambda: F.quantize_b128(x, codes, scales, block_rows=128),
             [codes.view(torch.uint8), scales])
    untouched(edge)


@pytest.mark.parametrize("op", ["linear", "dgrad"])
@pytest.mark.parametrize("bt,how", [(3, {}), (3, dict(splits=1)), (3, dict(splits=8)), (30, {}),
                                    (50, dict(splits=4)), (100, {}), (200, dict(cg=1)),
                                    (300, dict(cg=2)), (1500, dict(cg=1)), (2000, dict(cg=2))])
def test_products(tune, op, bt, how):
    # the last two with several tiles a CTA or pair
    tune(**how)
    k, n = 2064, 4112
    d_in, d_out = (k, n) if op == "linear" else (n, k)
    (a, sa), (w, sw), _, _ = product_case(7, op, bt, d_in, d_out)
    args = [t.to(DEV) for t in (a, sa, w, sw)]
    out, edge = fenced(bt, n, torch.bfloat16)
    runs_out(lambda: (F.linear_fp8 if op == "linear" else F.dgrad_fp8)(*args, out), [out])
    untouched(edge)
