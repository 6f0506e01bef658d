"""CPU oracle of the 8-bit blocks, the RMS norm and the products by expert.  TEST INFRASTRUCTURE ONLY; float64 numpy, the
definitions as include/moe_blocks8.h, moe_rmsnorm.h and moe_linear.h write them.  It shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def scale_of(amax):
    """The smallest 2^e, e >= -127, with amax <= 448 x 2^e; 1 where amax is 0."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, -127, dtype=np.int64)
    for k in range(-127, 121):
        e = np.where(amax > 448 * 2.0 ** k, k + 1, e)
    return np.where(amax == 0, 1.0, 2.0 ** e.astype(np.float64))


def e4m3(v):
    """To the nearest e4m3 value, ties to even; NaN stays NaN.  |v| <= 448."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    with np.errstate(invalid="ignore", divide="ignore"):
        exp = np.floor(np.log2(np.where(a > 0, a, 1.0)))
        exp = np.where(2.0 ** exp > a, exp - 1, exp)            # where the logarithm was rounded
        exp = np.where(2.0 ** (exp + 1) <= a, exp + 1, exp)
        step = 2.0 ** (np.maximum(exp, -6) - 3)
        return np.rint(v / step) * step


def _codes(v, scale):
    with np.errstate(invalid="ignore"):
        q = e4m3(np.where(np.isfinite(v), np.clip(v / scale, -448, 448), np.nan))
        return np.where((scale >= 2.0 ** 120) & (np.abs(q) > 240), np.sign(q) * 240, q)


def _finite_max(v, axis):
    return np.where(np.isfinite(v), np.abs(v), 0.0).max(axis=axis)


def pack(x):
    """(codes [n, h] as values, scales [n, ceil(h / 128)])."""
    x = np.asarray(x, dtype=np.float64)
    n, h = x.shape
    codes, scales = np.zeros((n, h)), np.ones((n, -(-h // BLOCK)))
    for b in range(scales.shape[1]):
        at = slice(b * BLOCK, min(h, (b + 1) * BLOCK))
        if n:
            scales[:, b] = scale_of(_finite_max(x[:, at], 1))
        codes[:, at] = _codes(x[:, at], scales[:, b:b + 1])
    return codes, scales


def unpack(codes, scales):
    return codes * np.repeat(scales, BLOCK, axis=1)[:, :codes.shape[1]]


def pack_weight(w):
    """(codes [E, O, K] as values, scales [E, ceil(O / 128), ceil(K / 128)])."""
    w = np.asarray(w, dtype=np.float64)
    E, O, K = w.shape
    codes, scales = np.zeros(w.shape), np.ones((E, -(-O // BLOCK), -(-K // BLOCK)))
    for i in range(scales.shape[1]):
        for j in range(scales.shape[2]):
            at = (slice(None), slice(i * BLOCK, min(O, (i + 1) * BLOCK)), slice(j * BLOCK, min(K, (j + 1) * BLOCK)))
            scales[:, i, j] = scale_of(_finite_max(w[at], (1, 2)))
            codes[at] = _codes(w[at], scales[:, i, j][:, None, None])
    return codes, scales


def unpack_weight(codes, scales):
    _, O, K = codes.shape
    return codes * np.repeat(np.repeat(scales, BLOCK, axis=1)[:, :O], BLOCK, axis=2)[:, :, :K]


def rms_forward(h, weight, eps):
    """(y, rstd) of the rows as they are kept."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * (1 if weight is None else np.asarray(weight, dtype=np.float64)), rstd


def rms_backward(h, weight, dy, dh, eps):
    xh, rstd = rms_forward(h, None, eps)
    dy = np.asarray(dy, dtype=np.float64)
    t = dy * (1 if weight is None else np.asarray(weight, dtype=np.float64))
    dx = rstd[:, None] * (t - xh * (t * xh).mean(axis=1, keepdims=True))
    return dx if dh is None else dx + np.asarray(dh, dtype=np.float64), (dy * xh).sum(axis=0)


def linear(x, w, offsets):
    """y [n, O], and the sum of the terms' magnitudes [n, O]."""
    y = np.zeros((x.shape[0], w.shape[1]))
    size = np.zeros_like(y)
    for e in range(w.shape[0]):
        at = slice(offsets[e], offsets[e + 1])
        y[at] = x[at] @ w[e].T
        size[at] = np.abs(x[at]) @ np.abs(w[e]).T
    return y, size


def linear_dx(dy, w, offsets):
    return linear(dy, np.swapaxes(w, 1, 2), offsets)


def linear_dw(dy, x, offsets, E):
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    size = np.zeros_like(dw)
    for e in range(E):
        at = slice(offsets[e], offsets[e + 1])
        dw[e] = dy[at].T @ x[at]
        size[e] = np.abs(dy[at]).T @ np.abs(x[at])
    return dw, size
