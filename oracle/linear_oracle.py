"""CPU oracle of linear attention with a fixed decay a head, forward and backward, in float64, token by token.

TEST INFRASTRUCTURE, as the other oracles.  The plain recurrences; nothing is taken from the library.
"""
from __future__ import annotations

import numpy as np

__all__ = ["linear_scan", "linear_scan_backward", "linear_step"]


def _heads(x, H):
    """[T, heads, d] with every head repeated for the states that share it."""
    return np.repeat(x, H // x.shape[1], axis=1)


def _shared(dx, heads):
    T, H, d = dx.shape
    return dx.reshape(T, heads, H // heads, d).sum(2)


def _start(init, slot_map, s, shape):
    """The state that sequence s starts from, or None for a padded one."""
    if init is None:
        return np.zeros(shape)
    if not 0 <= slot_map[s] < init.shape[0]:
        return None
    return init[slot_map[s]].copy()


def linear_scan(q, k, v, log_decay, cu, init=None, slot_map=None, scale=None, sizes=False):
    """o [T, H, dv] and the final states [N, H, dk, dv]; arguments float64, init [slots, H, dk, dv].  sizes: the same
    sums of absolute values, which errors are measured by."""
    H, (T, _, dk), dv = log_decay.shape[0], q.shape, v.shape[2]
    scale = dk ** -0.5 if scale is None else scale
    if sizes:
        q, k, v = np.abs(q), np.abs(k), np.abs(v)
        init = np.abs(init) if init is not None else None
    q, k, v, lam = _heads(q, H), _heads(k, H), _heads(v, H), np.exp(log_decay)[:, None, None]
    o, ends = np.zeros((T, H, dv)), np.zeros((len(cu) - 1, H, dk, dv))
    for s in range(len(cu) - 1):
        S = _start(init, slot_map, s, (H, dk, dv))
        if S is None:
            continue
        for t in range(cu[s], cu[s + 1]):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
        ends[s] = S
    return o, ends


def linear_scan_backward(do, q, k, v, log_decay, cu, init=None, slot_map=None, dfinal=None, scale=None, sizes=False):
    """dq, dk, dv shaped as q, k, v, and dinit [N, H, dk, dv]."""
    H, (T, _, dk_), dv_ = log_decay.shape[0], q.shape, v.shape[2]
    scale = dk_ ** -0.5 if scale is None else scale
    heads = [x.shape[1] for x in (q, k, v)]
    if sizes:
        do, q, k, v = np.abs(do), np.abs(q), np.abs(k), np.abs(v)
        init = np.abs(init) if init is not None else None
        dfinal = np.abs(dfinal) if dfinal is not None else None
    q, k, v, lam = _heads(q, H), _heads(k, H), _heads(v, H), np.exp(log_decay)[:, None, None]
    N = len(cu) - 1
    dq, dk, dv, dinit = np.zeros((T, H, dk_)), np.zeros((T, H, dk_)), np.zeros((T, H, dv_)), np.zeros((N, H, dk_, dv_))
    for s in range(N):
        S = _start(init, slot_map, s, (H, dk_, dv_))
        if S is None:
            continue
        for t in range(cu[s], cu[s + 1]):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.einsum("hv,hkv->hk", do[t], S)
        dS = dfinal[s].copy() if dfinal is not None else np.zeros((H, dk_, dv_))
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            dS = dS + scale * q[t][:, :, None] * do[t][:, None, :]
            dk[t] = np.einsum("hv,hkv->hk", v[t], dS)
            dv[t] = np.einsum("hk,hkv->hv", k[t], dS)
            dS = lam * dS
        dinit[s] = dS
    return _shared(dq, heads[0]), _shared(dk, heads[1]), _shared(dv, heads[2]), dinit


def linear_step(q, k, v, log_decay, states, scale=None):
    """One token for each row of states [B, H, dk, dv]: o [B, H, dv] and the states after it."""
    H = log_decay.shape[0]
    scale = q.shape[2] ** -0.5 if scale is None else scale
    q, k, v = _heads(q, H), _heads(k, H), _heads(v, H)
    S = np.exp(log_decay)[:, None, None] * states + k[..., :, None] * v[..., None, :]
    return scale * np.einsum("bhk,bhkv->bhv", q, S), S
