"""fp64 definitions of the operators between a layer's 16-bit products (test
infrastructure): activations and their derivatives, the dropout generator, the
product's epilogue and its gradient, rotary positions, and the norm of queries and
keys.  Plain numpy."""
from __future__ import annotations

import math

import numpy as np

NONE, RELU, GELU, GELU_TANH, SILU = range(5)
HALF, INTERLEAVED = 0, 1
_erf = np.vectorize(math.erf, otypes=[float])
_erfc = np.vectorize(math.erfc, otypes=[float])


def _sigmoid(w):
    with np.errstate(over="ignore"):
        return np.where(w >= 0, 1 / (1 + np.exp(-np.abs(w))), np.exp(-np.abs(w)) / (1 + np.exp(-np.abs(w))))


def _tanh_arg(z):
    c = 2 * math.sqrt(2 / math.pi)
    return c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z ** 2)


def act(z, kind):
    if kind == RELU:
        return np.maximum(z, 0.0)
    if kind == GELU:
        return z * 0.5 * _erfc(-z / math.sqrt(2))
    if kind == GELU_TANH:
        return z * _sigmoid(_tanh_arg(z)[0])
    if kind == SILU:
        return z * _sigmoid(z)
    return z


def act_slope(z, kind):
    if kind == RELU:
        return (z > 0).astype(float)
    if kind == GELU:
        return 0.5 * _erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == GELU_TANH:
        w, dw = _tanh_arg(z)
        return _sigmoid(w) + z * _sigmoid(w) * _sigmoid(-w) * dw
    if kind == SILU:
        return _sigmoid(z) + z * _sigmoid(z) * _sigmoid(-z)
    return np.ones_like(z)


def philox4x32_10(counter, key):
    """One block of Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw 2011), in
    Python integers."""
    mask = (1 << 32) - 1
    c, k = list(counter), list(key)
    for r in range(10):
        if r:
            k = [(k[0] + 0x9E3779B9) & mask, (k[1] + 0xBB67AE85) & mask]
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & mask, (p >> 32) ^ c[3] ^ k[1], p & mask]
    return c


def threshold(p: float) -> int:
    return min(int(np.rint(float(np.float32(p)) * 65536.0)), 65535)


def keep(rows: int, cols: int, p: float, seed: int, offset: int) -> np.ndarray:
    """The factor of each element: 0 where dropped, else 65536 / (65536 - T)."""
    t = threshold(p)
    block = np.arange(rows * cols // 8, dtype=np.uint64)
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    full = lambda v: np.full(block.shape, v, np.uint64)  # noqa: E731
    offset %= 1 << 64
    c = [block & low, block >> sh, full(offset & 0xFFFFFFFF), full(offset >> 32)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for r in range(10):
        if r:
            k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> sh) ^ c[1] ^ np.uint64(k[0]), p1 & low, (p0 >> sh) ^ c[3] ^ np.uint64(k[1]),
             p0 & low]
    u = np.stack([(c[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF) for j in range(8)], 1)
    return (u.reshape(rows, cols) >= t) * (65536.0 / (65536 - t))


def linear(X, W, bias=None, kind=NONE, mul=None, residual=None, factor=None):
    """Z and Y."""
    Z = X @ W.T + (0.0 if bias is None else bias)
    Y = act(Z, kind) * (1.0 if mul is None else mul) * (1.0 if factor is None else factor)
    return Z, Y + (0.0 if residual is None else residual)


def epilogue_backward(dY, Z, kind=NONE, mul=None, factor=None):
    """dZ, dmul and dbias."""
    dA = dY * (1.0 if factor is None else factor)
    dZ = dA * (1.0 if mul is None else mul) * act_slope(Z, kind)
    return dZ, dA * act(Z, kind), dZ.sum(0)


def frequencies(dim, theta, kind="none", factor=1.0, context=0.0, low=1.0, high=4.0):
    """Radians per position of each pair, and the magnitude."""
    i = np.arange(dim // 2, dtype=np.float64)
    if kind == "ntk":
        theta = theta * factor ** (dim / (dim - 2))
    f = theta ** (-2 * i / dim)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "llama3":
        wave = 2 * math.pi / f
        mixed = (context / wave - low) / (high - low)
        out = np.where(wave > context / low, f / factor,
                       np.where(wave < context / high, f, (1 - mixed) * f / factor + mixed * f))
        return out, 1.0
    if kind == "yarn":
        at = lambda turns: dim * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), dim - 1)
        ramp = np.clip((i - a) / max(b - a, 0.001), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    return f, 1.0


def rotate(x, positions, radians, magnitude=1.0, layout=HALF, inverse=False):
    """x [tokens, heads, dim]; the first 2 len(radians) elements of each head turn."""
    half = len(radians)
    w = np.outer(np.asarray(positions, np.float64), radians)[:, None] * (-1 if inverse else 1)
    c, s = magnitude * np.cos(w), magnitude * np.sin(w)
    out = np.array(x, np.float64)
    ia, ib = ((np.arange(half), np.arange(half) + half) if layout == HALF
              else (2 * np.arange(half), 2 * np.arange(half) + 1))
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    return out


def head_norm(x, gain, eps):
    return x * gain / np.sqrt((x * x).mean(2, keepdims=True) + eps)


def head_norm_backward(dn, x, gain, eps):
    """dx and dgain."""
    r = 1 / np.sqrt((x * x).mean(2, keepdims=True) + eps)
    xh, u = x * r, dn * gain
    return r * (u - xh * (u * xh).mean(2, keepdims=True)), (dn * xh).sum((0, 1))
