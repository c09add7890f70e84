"""fp64 definition of the per-head norm and position rotation of queries and keys
(the serving and training paths' ``stt_rope``), and its gradient."""

import numpy as np


def _pairs(R, interleaved):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate(x, positions, freq, interleaved, amplitude=1.0, sign=1.0):
    """x [tokens, heads, D] rotated by sign * positions [tokens] * freq [R/2]."""
    y = x.astype(np.float64).copy()
    if freq is None or len(freq) == 0:
        return y
    a, b = _pairs(2 * len(freq), interleaved)
    t = positions.astype(np.float64)[:, None] * np.asarray(freq, np.float64)[None]
    c, s = amplitude * np.cos(t)[:, None], sign * amplitude * np.sin(t)[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, w, eps, positions, freq, interleaved, amplitude=1.0):
    """y [tokens, heads, D] of x: RMS norm with weight w (None: none), rotation."""
    n = x
    if w is not None:
        n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w
    return rotate(n, positions, freq, interleaved, amplitude)


def norm_rope_grad(dy, x, w, eps, positions, freq, interleaved, amplitude=1.0):
    """(dx, dw) for dy; also the sums of absolute terms that bound their rounding:
    (|terms| of dx, |terms| of dw).  dw is None without a weight."""
    u = rotate(dy, positions, freq, interleaved, amplitude, -1.0)
    if w is None:
        return u, None, np.abs(u), None
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh, uw = x * r, u * w
    dw = (u * xh).sum((0, 1))
    dx = r * (uw - xh * np.mean(uw * xh, -1, keepdims=True))
    terms = r * (np.abs(uw) + np.abs(xh) * np.mean(np.abs(uw * xh), -1, keepdims=True))
    return dx, dw, terms, np.abs(u * xh).sum((0, 1))
