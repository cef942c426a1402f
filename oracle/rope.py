"""Plain definition of the rotation by positions and its gradient (float64
numpy), one pair of values at a time.

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import _f64


def frequencies(rotary: int, base: float = 10000.0, factor: float = 1.0, original_len: int = 0, low: float = 1.0,
                high: float = 32.0) -> np.ndarray:
    """Angles per position, in radians."""
    out = []
    for i in range(rotary // 2):
        theta = 1.0 / base ** (2 * i / rotary)
        if original_len:
            wavelength = 2 * math.pi / theta
            g = (original_len / wavelength - low) / (high - low)
            g = 0.0 if g < 0 else 1.0 if g > 1 else g
            theta = (1 - g) * (theta / factor) + g * theta
        else:
            theta /= factor
        out.append(theta)
    return np.array(out)


def _indices(rotary: int, half: bool):
    i = np.arange(rotary // 2)
    return (i, i + rotary // 2) if half else (2 * i, 2 * i + 1)


def rotate(x, positions, theta, half: bool, mscale: float = 1.0, back: bool = False):
    """x [T, heads, d] turned by the positions' angles (back: the transpose)."""
    x = _f64(x)
    a, b = _indices(2 * len(theta), half)
    # the position in 64 bits, the angle modulo a turn
    t = np.asarray(positions, dtype=np.float64)[:, None, None] * theta
    c, s = mscale * np.cos(t), mscale * np.sin(t)
    if back:
        s = -s
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def spread(x, theta, half: bool, mscale: float = 1.0):
    """|x_a| + |x_b| in both places of every pair, |x| elsewhere: what the error
    of a rotated value is in proportion to."""
    x = np.abs(_f64(x))
    a, b = _indices(2 * len(theta), half)
    y = x.copy()
    y[..., a] = y[..., b] = abs(mscale) * (x[..., a] + x[..., b])
    return y


def norm(x, weight, eps: float):
    x = _f64(x)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * _f64(weight)


def forward(x, positions, theta, half: bool, mscale: float = 1.0, weight=None, eps: float = 1e-6):
    return rotate(x if weight is None else norm(x, weight, eps), positions, theta, half, mscale)


def backward(dy, x, positions, theta, half: bool, mscale: float = 1.0, weight=None, eps: float = 1e-6):
    """(dx, dweight): the chain rule through the pairs, then through x / r with
    r = sqrt(mean(x^2) + eps), whose own gradient is x / (d r)."""
    g = rotate(dy, positions, theta, half, mscale, back=True)
    if weight is None:
        return g, None
    x, w = _f64(x), _f64(weight)
    r = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x / r).sum((0, 1))
    dr = -(g * w * x).sum(-1, keepdims=True) / r ** 2
    return g * w / r + dr * x / (x.shape[-1] * r), dw
