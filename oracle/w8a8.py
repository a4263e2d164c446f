"""The 8-bit linear path and rotary positions, written plainly in float64.

ORACLE -- test infrastructure only; the product package never imports it.

    quantize_rows    t = max(max |y|, 2^-100), scale = t / 448, codes = e4m3(y * (448 / t))
    rmsnorm          h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight
    linear, gated    z = (a w^T) sa sw + bias; act(z) + residual, or act(gate) * up
    rope             pair (a, b) -> (a c - b s, b c + a s), angle = position * freq
"""

from __future__ import annotations

import numpy as np

from .formats import E4M3_MAX, rn32, ue4m3_decode, ue4m3_encode

FLOOR = 2.0 ** -100


def e4m3(v: np.ndarray) -> np.ndarray:
    """The E4M3 value nearest to v (ties to the even code, saturating)."""
    return np.copysign(ue4m3_decode(ue4m3_encode(np.abs(v))), v)


def quantize_rows(y: np.ndarray):
    """(E4M3 values, float32 scales) of the rows of y, each float32 step rounded as stated:
    RN32(448 / t), RN32(t / 448), RN32(y * RN32(448 / t))."""
    t = np.maximum(np.abs(y).max(1), FLOOR)
    return e4m3(rn32(y * rn32(E4M3_MAX / t)[:, None])), rn32(t / E4M3_MAX)


def rmsnorm(x, weight=None, residual=None, eps=1e-6):
    """(h, y), nothing rounded."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else residual)
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h, y if weight is None else y * weight


def act(z, kind):
    with np.errstate(over="ignore"):
        if kind == "silu":
            return z / (1.0 + np.exp(-z))
        if kind == "gelu":
            return 0.5 * z * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (z + 0.044715 * z ** 3)))
    return z


def product(a, sa, w, sw, bias=None):
    """(z, the sum of its terms' magnitudes)."""
    s = np.outer(sa, sw)
    b = 0.0 if bias is None else bias
    return (a @ w.T) * s + b, (np.abs(a) @ np.abs(w).T) * np.abs(s) + np.abs(b)


def cos_sin(positions, freq, axis=None, scale=1.0):
    """[M, P] tables; positions [M, A] whole numbers."""
    axis = np.zeros(len(freq), np.int64) if axis is None else axis
    angle = positions[:, axis].astype(np.float64) * freq
    return scale * np.cos(angle), scale * np.sin(angle)


def rope(x, cos, sin, interleaved):
    """x [M, heads, D] turned by cos, sin [M, P]; columns from 2P on unchanged."""
    y = np.array(x, np.float64)
    P = cos.shape[1]
    first, second = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    a, b = x[..., first], x[..., second]
    c, s = cos[:, None], sin[:, None]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y
