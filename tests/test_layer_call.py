"""The extension's calls of the operators between a layer's 16-bit products leave,
undone, what they do not take."""
import pytest
import torch

from weight_gradient_gemm_gb300 import _build
from weight_gradient_gemm_gb300 import forge as F

NAMES = {"linear_bf16": 13, "epilogue_backward": 13, "dropout": 8, "rope": 10, "qk_norm_rope": 12,
         "qk_norm_rope_backward": 17}


@pytest.fixture(scope="module")
def call():
    _build.build()
    return F._loaded()


@pytest.mark.parametrize("name", sorted(NAMES))
def test_leaves_what_it_does_not_take(call, name):
    fn, n = getattr(call, name), NAMES[name]
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    h = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for args in ((), (None,) * (n - 1), (None,) * (n + 1), (None,) * n, ("a",) * n, (1,) * n,
                 (x,) * n, (h,) * n, (x,) * (n - 1) + (None,), ([x],) + (None,) * (n - 1)):
        assert fn(*args) == -1
