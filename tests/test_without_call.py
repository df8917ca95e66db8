"""Without the CPython extension of the operators' calls the library is whole: it
loads, and every call goes through forge.py's own checks."""
import os

import pytest
import torch

from weight_gradient_gemm_gb300 import _build
from weight_gradient_gemm_gb300 import forge as F


@pytest.fixture
def unloaded(monkeypatch):
    """forge.py as before its library was loaded."""
    _build.build()
    monkeypatch.setattr(F, "_lib", None)
    monkeypatch.setattr(F, "_call", None)


def check_ctypes_path():
    with pytest.warns(UserWarning):
        lib = F.lib()
    assert F.header_functions() and lib.forge_status_string(0)
    assert F._loaded().rmsnorm(*[None] * 10) == -1
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        F.rmsnorm(x, x[0], eps=1e-5, y=x)
    with pytest.raises(ValueError, match="CUDA"):
        F.grad_norm([x], 1.0, torch.zeros(2), workspace=torch.zeros(16))


def test_loads_without_the_extension(unloaded, monkeypatch, tmp_path):
    monkeypatch.setattr(F, "CALL_PATH", os.path.join(tmp_path, "absent.so"))
    check_ctypes_path()


def test_loads_beside_a_file_that_is_no_extension(unloaded, monkeypatch, tmp_path):
    path = os.path.join(tmp_path, "_forge_call.so")
    with open(path, "w") as f:
        f.write("not a library")
    monkeypatch.setattr(F, "CALL_PATH", path)
    check_ctypes_path()


def test_leaves_an_extension_of_another_torch_alone(unloaded, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.1.0+other")
    check_ctypes_path()


def test_takes_the_extension_that_was_built(unloaded):
    F.lib()
    assert F._call.torch_version == torch.__version__.split("+")[0]


@pytest.mark.parametrize("compiler", ["/nonexistent/g++", "false"])
def test_builds_without_the_extension(monkeypatch, tmp_path, compiler):
    stale = os.path.join(tmp_path, "_forge_call.so")
    with open(stale, "w") as f:
        f.write("from an older source")
    os.utime(stale, (1, 1))
    monkeypatch.setattr(_build, "CALL", stale)
    monkeypatch.setattr(_build, "CXX", compiler)
    with pytest.warns(UserWarning, match="ctypes"):
        assert _build.build() == _build.LIB
    assert not os.path.exists(stale)


@pytest.mark.gpu
def test_operators_run_without_the_extension(unloaded, monkeypatch, tmp_path):
    monkeypatch.setattr(F, "CALL_PATH", os.path.join(tmp_path, "absent.so"))
    x = torch.randn(5, 256, device="cuda").bfloat16()
    gain, y, want = torch.ones(256, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    with pytest.warns(UserWarning):
        F.rmsnorm(x, gain, eps=1e-5, y=y)
    monkeypatch.undo()
    F.rmsnorm(x, gain, eps=1e-5, y=want)
    assert F.device_error() == 0 and torch.equal(y, want)
