"""CPU oracle of the norm and rotation of queries and keys, forward and backward, in float64.

TEST INFRASTRUCTURE, as the other oracles.  The plain definition; nothing is taken from the library.
"""
from __future__ import annotations

import numpy as np

__all__ = ["qk_norm_rope", "qk_norm_rope_backward"]


def _turn(n, positions, inv_freq, neighbours, axes, sign):
    """n [T, heads, d] with its pairs as complex numbers, each times e^{i sign angle}."""
    P = inv_freq.shape[0]
    pos = np.atleast_2d(np.asarray(positions, np.float64))
    angle = pos[list(axes) if axes is not None else [0] * P].T * inv_freq.astype(np.float64)  # [T, P]
    i = np.arange(P)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + P)
    y = n.copy()
    z = (n[..., a] + 1j * n[..., b]) * np.exp(1j * sign * angle)[:, None]
    y[..., a], y[..., b] = z.real, z.imag
    return y


def qk_norm_rope(x, w, positions, inv_freq, eps=1e-6, neighbours=False, axes=None):
    """One of the two tensors, x [T, heads, d]."""
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _turn(x * r * w, positions, inv_freq, neighbours, axes, 1)


def qk_norm_rope_backward(dy, x, w, positions, inv_freq, eps=1e-6, neighbours=False, axes=None):
    """dx and dw."""
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dn = _turn(dy, positions, inv_freq, neighbours, axes, -1)
    xh = x * r
    dh = dn * w
    return r * (dh - xh * (dh * xh).mean(-1, keepdims=True)), (dn * xh).sum((0, 1))
