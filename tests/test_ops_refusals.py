"""What the operators around the weight gradient refuse, they refuse before
anything is enqueued (host checks: no GPU is touched)."""
import ctypes

import pytest

from weight_gradient_gemm_gb300 import _build
from weight_gradient_gemm_gb300 import forge as F

SHAPE = 3


@pytest.fixture(scope="module")
def L():
    _build.build()
    return F.lib()


@pytest.mark.parametrize("sizes", [[1 << 44], [1 << 43, 1 << 43], [64] * 128 + [1 << 44],
                                   [64] * 200 + [1 << 43, 3 << 42, 1 << 43, 8]])
def test_grad_norm_refuses_too_many_values_first(L, sizes):
    # more work units than one launch counts: in the first launch's tensors, or in
    # those of a second one.  (The addresses are never dereferenced; a device is
    # asked for only after the refusal.)
    at, items = 1 << 50, []
    for n in sizes:
        items.append(F.ForgeGrad(at, n, F.DT_BF16))
        at += 2 * n + (-2 * n) % 16
    arr = (F.ForgeGrad * len(items))(*items)
    st = L.forge_grad_norm(ctypes.addressof(arr), len(items), 1.0, 1 << 20, 1 << 21, 1 << 20, None)
    assert st == SHAPE
