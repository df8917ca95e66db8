"""The CPython extension that carries the calls of the operators around the
weight gradient: it takes what is valid and leaves the rest, undone, to the
checks of forge.py."""
import pytest
import torch

from weight_gradient_gemm_gb300 import _build
from weight_gradient_gemm_gb300 import forge as F


@pytest.fixture(scope="module")
def call():
    _build.build()
    return F._loaded()


NAMES = {"rmsnorm": 10, "rmsnorm_backward": 9, "quantize": 5, "linear": 6, "dgrad": 6,
         "grad_norm": 5, "adamw_clip": 12}


@pytest.mark.parametrize("name", sorted(NAMES))
def test_leaves_what_it_does_not_take(call, name):
    fn, n = getattr(call, name), NAMES[name]
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    for args in ((), (None,) * (n - 1), (None,) * (n + 1),      # another number of arguments
                 (None,) * n, ("a",) * n, (1,) * n,             # no tensors
                 (x,) * n, (x,) * (n - 1) + (None,),            # not on a GPU
                 ([x],) + (None,) * (n - 1)):
        assert fn(*args) == -1


def test_bind_refuses_what_is_no_address(call):
    with pytest.raises(TypeError):
        call.bind()
    with pytest.raises(TypeError):
        call.bind(*["a"] * 7)
    assert call.rmsnorm(*[None] * 10) == -1


def layer(dev="cuda"):
    bt, d_in, d_out = 3, 256, 144
    t = dict(x=torch.randn(bt, d_in), g=torch.ones(d_in), dy=torch.randn(bt, d_in))
    t = {k: v.to(dev, torch.bfloat16) for k, v in t.items()}
    t["rstd"] = torch.empty(bt, device=dev)
    t["codes"], t["scales"] = F.alloc_b128(bt, d_in, device=dev)
    t["W"], t["ws"] = F.alloc_b128(d_out, d_in, 128, device=dev)
    w = torch.randn(d_out, d_in).to(dev, torch.bfloat16)
    return bt, d_in, d_out, t, w


@pytest.mark.gpu
def test_takes_valid_calls_with_the_same_results(monkeypatch):
    """Every operator's plain call is taken (status 0), and gives bit for bit
    what the call through ctypes gives."""
    torch.manual_seed(5)
    bt, d_in, d_out, t, w = layer()
    dy_c, dy_s = F.alloc_b128(bt, d_out)
    F.quantize_b128(torch.randn(bt, d_out).cuda().bfloat16(), dy_c, dy_s)
    g32 = torch.randn(d_out, d_in).cuda()
    ws = torch.empty(max(F.rmsnorm_backward_workspace_bytes(bt, d_in),
                         F.grad_norm_workspace_bytes(2)), dtype=torch.uint8, device="cuda")

    def run(side):
        o = [torch.zeros(bt, d_in, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
        dg, clip = torch.zeros(d_in, device="cuda"), torch.zeros(2, device="cuda")
        Y = torch.zeros(bt, d_out, device="cuda")
        W, m, v = w.clone(), torch.zeros_like(g32), torch.zeros_like(g32)
        torch.cuda.synchronize()      # the fills above are on the current stream
        F.rmsnorm(t["x"], t["g"], eps=1e-5, y=o[0], codes=t["codes"], scales=t["scales"],
                  rstd=t["rstd"], stream=side)
        F.rmsnorm_backward(t["dy"], t["x"], t["g"], t["rstd"], o[1], dg, workspace=ws, stream=side)
        F.quantize_b128(w, t["W"], t["ws"], block_rows=128, stream=side)
        F.linear_fp8(t["codes"], t["scales"], t["W"], t["ws"], Y, stream=side)
        F.dgrad_fp8(dy_c, dy_s, t["W"], t["ws"], o[2], stream=side)
        F.grad_norm([g32, o[1]], 0.5, clip, workspace=ws, stream=side)
        F.adamw_clip(g32, W, m, v, clip, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8,
                     weight_decay=0.1, step=7, stream=side)
        torch.cuda.synchronize()
        return [a.float() for a in (*o, dg, clip, Y, W, m, v, t["codes"].float(), t["scales"])]

    taken = []
    real = F._loaded()

    class Watch:
        def __getattr__(self, name):
            def fn(*a):
                st = getattr(real, name)(*a)
                taken.append((name, st))
                return st
            return fn

    class Leave:
        def __getattr__(self, name):
            return lambda *a: -1

    side = torch.cuda.Stream()
    monkeypatch.setattr(F, "_call", Watch())
    got = [run(None), run(side), run(side.cuda_stream)]
    assert sorted({n for n, _ in taken}) == sorted(NAMES)
    assert all(st == 0 for _, st in taken) and len(taken) == 21
    monkeypatch.setattr(F, "_call", Leave())
    want = run(None)
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_reports_the_librarys_refusals(monkeypatch):
    """A status of the library itself comes back as ForgeError."""
    _, _, _, t, _ = layer()
    with pytest.raises(F.ForgeError):
        F.rmsnorm(t["x"], t["g"], eps=-1.0, rstd=t["rstd"])
    with pytest.raises(F.ForgeError):
        F.rmsnorm(t["x"], t["g"], eps=1e-5, y=t["x"])
    with pytest.raises((ValueError, TypeError)):
        F.rmsnorm(t["x"], t["g"][:8], eps=1e-5, rstd=t["rstd"])
    with pytest.raises((ValueError, TypeError)):
        F.quantize_b128(t["x"].t(), t["codes"], t["scales"])
