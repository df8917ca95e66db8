"""Heads where the other tests do not go, against the fp64 definitions: eps = 0 with head counts
that leave lanes without a head, and queries, keys and values side by side within a head."""
import numpy as np
import pytest
import torch

from oracle import layer as R
from tests.gpu_util import DEV, F, require_gpu
from tests.test_gpu_layer import BF, U, f64, heads, ok, pair_sum, rand, turn_error, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("tokens,hq,hk,dim,rot", [
    (1, 1, 2, 64, 64), (9, 3, 1, 128, 128), (9, 5, 2, 256, 64), (40, 12, 1, 128, 64),
    (40, 12, 5, 64, 64), (300, 5, 3, 128, 128), (17, 33, 3, 80, 32), (17, 7, 1, 40, 24),
    (3000, 12, 1, 256, 256)])
@pytest.mark.parametrize("layout", [R.HALF, R.INTERLEAVED])
def test_without_eps(tokens, hq, hk, dim, rot, layout):
    q, k = heads(71, tokens, hq, hk, dim, "fused", 2.0)
    dq, dk = heads(73, tokens, hq, hk, dim, "dense", 1e-2)
    gains = [1 + rand(75 + i, (dim,), 0.2, torch.float32) for i in range(2)]
    freqs, _ = F.rope_frequencies(rot, 10000.0)
    rad, _ = R.frequencies(rot, 10000.0)
    pos64 = np.arange(tokens)
    ws = torch.empty(F.qk_norm_rope_backward_workspace_bytes(dim), dtype=torch.uint8, device=DEV)
    y = [torch.empty_like(t) for t in (dq, dk)]
    dx = [torch.empty_like(t) for t in (dq, dk)]
    dg = [torch.full((dim,), 7.0, device=DEV) for _ in range(2)]
    F.qk_norm_rope(q, k, *gains, freqs, eps=0.0, q_out=y[0], k_out=y[1], layout=layout)
    F.qk_norm_rope_backward(dq, dk, q, k, *gains, freqs, eps=0.0, dq_out=dx[0], dk_out=dx[1],
                            dq_gain=dg[0], dk_gain=dg[1], workspace=ws, layout=layout)
    ok()
    # bounds: as with eps (test_gpu_layer.py, test_qk_norm_rope), every head's mean square is
    # far from zero
    rel, terr = 24 * U, turn_error(pos64, rad)
    for x, dy, g, got, gotx, gotg in zip((q, k), (dq, dk), gains, y, dx, dg):
        x64, g64 = f64(x), f64(g)
        n = R.head_norm(x64, g64, 0.0)
        ref = R.rotate(n, pos64, rad, 1.0, layout)
        within(f64(got), ref, BF * np.abs(ref) + (terr + rel) * pair_sum(n, rot // 2, layout))
        dx64, dg64 = R.head_norm_backward(R.rotate(f64(dy), pos64, rad, 1.0, layout, True), x64, g64,
                                          0.0)
        r = 1 / np.sqrt((x64 * x64).mean(2, keepdims=True))
        xh, d = np.abs(x64 * r), pair_sum(f64(dy), rot // 2, layout)
        u, uerr = np.abs(g64) * d, (terr + 4 * U) * np.abs(g64) * d
        noise = r * (uerr + rel * u + xh * ((uerr + (rel + 40 * U) * u) * xh).mean(2, keepdims=True)
                     + 3 * rel * xh * (u * xh).mean(2, keepdims=True))
        within(f64(gotx), dx64, BF * np.abs(dx64) + 1.01 * noise)
        adds = min(tokens * x.shape[1], 200) + 100
        within(f64(gotg), dg64, ((terr + rel + adds * U) * d * xh).sum((0, 1)) + 1e-30)


@pytest.mark.parametrize("tokens", [1, 37])
def test_queries_keys_and_values_of_a_head_side_by_side(tokens):
    """[tokens, heads, 3, dim]: in place on the views is as apart; the values stay."""
    h, dim = 5, 64
    qkv, grad = rand(81, (tokens, h, 3, dim)), rand(82, (tokens, h, 3, dim))
    freqs, _ = F.rope_frequencies(dim, 10000.0)
    gains = [1 + rand(83 + i, (dim,), 0.2, torch.float32) for i in range(2)]
    ws = torch.empty(F.qk_norm_rope_backward_workspace_bytes(dim), dtype=torch.uint8, device=DEV)
    dg = torch.empty(4, dim, device=DEV)
    calls = [lambda x, d, g: F.rope(*x, freqs),
             lambda x, d, g: F.qk_norm_rope(*x, *gains, freqs, eps=1e-5),
             lambda x, d, g: F.qk_norm_rope_backward(*d, *x, *gains, freqs, eps=1e-5, dq_gain=g[0],
                                                     dk_gain=g[1], workspace=ws)]
    for call in calls:
        views = qkv.clone(), grad.clone()
        call(*[(t[:, :, 0], t[:, :, 1]) for t in views], dg[:2])
        apart = [[t[:, :, i].contiguous() for i in range(2)] for t in (qkv, grad)]
        call(*apart, dg[2:])
        ok()
        for got, want, start in zip(views, apart, (qkv, grad)):
            assert torch.equal(got[:, :, 0], want[0]) and torch.equal(got[:, :, 1], want[1])
            assert torch.equal(got[:, :, 2], start[:, :, 2])
    assert torch.equal(dg[:2], dg[2:])
