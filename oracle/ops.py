"""fp64 definitions of the operators around the weight gradient (test
infrastructure): the RMS norm and its gradients, the 128-block e4m3 format, the
products of quantised matrices and the clipped gradient norm.  Plain numpy."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
BLOCK = 128


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to even), saturating at +-448."""
    x = np.clip(np.asarray(x, np.float64), -E4M3_MAX, E4M3_MAX)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.round(x / step) * step


def block_amax(x: np.ndarray, block_rows: int) -> np.ndarray:
    rows, cols = x.shape
    out = np.empty((-(-rows // block_rows), -(-cols // BLOCK)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = np.abs(x[i * block_rows:(i + 1) * block_rows,
                                 j * BLOCK:(j + 1) * BLOCK]).max()
    return out


def spread(scales: np.ndarray, block_rows: int, shape) -> np.ndarray:
    full = np.repeat(np.repeat(scales, block_rows, 0), BLOCK, 1)
    return full[:shape[0], :shape[1]]


def quantize(x: np.ndarray, block_rows: int):
    """Code values and scales of x in the 128-block format."""
    x = np.asarray(x, np.float64)
    a = block_amax(x, block_rows)
    scales = np.where(a > 0, np.maximum(a / E4M3_MAX, 2.0 ** -126), 0.0)
    s = spread(scales, block_rows, x.shape)
    return e4m3_round(np.divide(x, s, out=np.zeros_like(x), where=s > 0)), scales


def dequantize(codes: np.ndarray, scales: np.ndarray, block_rows: int) -> np.ndarray:
    return codes.astype(np.float64) * spread(scales.astype(np.float64), block_rows, codes.shape)


def rmsnorm(x, residual, gain, eps):
    """h, rstd, y."""
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * gain


def rmsnorm_backward(dy, h, gain, rstd, dsum):
    """dX and dgain from the given rstd."""
    xh = h * rstd[:, None]
    u = dy * gain
    dx = rstd[:, None] * (u - xh * (u * xh).mean(1, keepdims=True))
    return (dx if dsum is None else dx + dsum), (dy * xh).sum(0)


def grad_norm(grads, max_norm):
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))
