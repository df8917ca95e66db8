"""The norm of queries and keys with eps = 0, against the fp64 definitions: a head count that
leaves lanes without a head must not reach the gains' gradients."""
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
