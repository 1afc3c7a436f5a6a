"""CPU oracle of the layer and RMS norm of a row's slices, forward and backward, in float64.

TEST INFRASTRUCTURE, as the other oracles.  The plain definition; nothing is taken from the library.
"""
from __future__ import annotations

import numpy as np

__all__ = ["layer_norm", "layer_norm_backward"]


def _silu(z):
    s = 1 / (1 + np.exp(-z))
    return z * s, s * (1 + z * (1 - s))


def _parts(x, w, b, z, groups, rms, gate_after, eps):
    rows, width = x.shape
    gate, slope = _silu(z) if z is not None else (1.0, 0.0)
    u = (x * gate if z is not None and not gate_after else x).reshape(rows, groups, width // groups)
    mean = u.mean(-1) * (0.0 if rms else 1.0)
    rstd = 1 / np.sqrt(((u - mean[..., None]) ** 2).mean(-1) + eps)
    h = (u - mean[..., None]) * rstd[..., None]
    v = h.reshape(rows, width) * w + (0.0 if b is None else b)
    return gate, slope, mean, rstd, h, v


def layer_norm(x, w, b=None, z=None, groups=1, rms=False, gate_after=False, eps=1e-5):
    """y, mean and rstd [rows, groups]; arguments float64."""
    gate, _, mean, rstd, _, v = _parts(x, w, b, z, groups, rms, gate_after, eps)
    return (v * gate if z is not None and gate_after else v), mean, rstd


def layer_norm_backward(dy, x, w, b=None, z=None, groups=1, rms=False, gate_after=False, eps=1e-5):
    """dx, dw, db, dz (dz None without a gate)."""
    gate, slope, _, rstd, h, v = _parts(x, w, b, z, groups, rms, gate_after, eps)
    dv = dy * gate if z is not None and gate_after else dy
    dz = dy * v * slope if z is not None and gate_after else None
    hf = h.reshape(x.shape)
    e = (dv * w).reshape(h.shape)
    du = e - h * (e * h).mean(-1, keepdims=True)
    if not rms:
        du = du - e.mean(-1, keepdims=True)
    du = (du * rstd[..., None]).reshape(x.shape)
    if z is not None and not gate_after:
        dz = du * x * slope
        du = du * gate
    return du, (dv * hf).sum(0), dv.sum(0), dz
