"""CPU oracle of the Mamba2 recurrence over packed sequences, forward and backward, in float64.

TEST INFRASTRUCTURE, as the other oracles.  Token by token: the forward pass is the token update of
``mamba2_oracle`` (all heads of a token at once), the backward pass walks the same tokens in reverse
with every state kept.
"""
from __future__ import annotations

import numpy as np

from .gdn_oracle import _slot_ok
from .mamba2_oracle import m2_gates

__all__ = ["mamba2_scan", "mamba2_scan_backward"]


def _heads(v, H):
    return np.repeat(v, H // v.shape[0], axis=0)


def mamba2_scan(x, Bm, Cm, dt, A_log, dt_bias, Dskip, cu, init=None, slot_map=None, sizes=False):
    """x [T, H, d], Bm, Cm [T, G, n], dt [T, H] in float64; init [slots, H, d, n] with slot_map, or None for zero states.
    Returns y [T, H, d] and the final states [N, H, d, n] before rounding (a padded sequence's are zero).
    sizes: the sums of the terms' absolute values in place of the sums."""
    T, H, d = x.shape
    N, n = len(cu) - 1, Bm.shape[2]
    g, dtp = m2_gates(dt, A_log, dt_bias)
    size = np.abs if sizes else (lambda v: v)
    y, final = np.zeros((T, H, d)), np.zeros((N, H, d, n))
    for s in range(N):
        if init is not None and not _slot_ok(int(slot_map[s]), init.shape[0]):
            continue
        S = size(np.array(init[int(slot_map[s])])) if init is not None else np.zeros((H, d, n))
        for t in range(cu[s], cu[s + 1]):
            S = np.exp(g[t])[:, None, None] * S + (dtp[t][:, None] * size(x[t]))[:, :, None] * size(_heads(Bm[t], H))[:, None]
            y[t] = np.einsum("hpn,hn->hp", S, size(_heads(Cm[t], H))) + size(Dskip[:, None] * x[t])
        final[s] = S
    return y, final


def mamba2_scan_backward(dy, x, Bm, Cm, dt, A_log, dt_bias, Dskip, cu, init=None, slot_map=None, dfinal=None, sizes=False):
    """dx, dBm, dCm, ddt, dA_log, ddt_bias, dD, dinit [N, H, d, n]; sizes as above."""
    T, H, d = x.shape
    N, G, n = len(cu) - 1, Bm.shape[1], Bm.shape[2]
    g, dtp = m2_gates(dt, A_log, dt_bias)
    slope = 1 / (1 + np.exp(-(dt + dt_bias)))
    A = np.exp(A_log)
    size, sign = (np.abs, 1.0) if sizes else ((lambda v: v), -1.0)
    dx, dB, dC, ddt = np.zeros_like(x), np.zeros_like(Bm), np.zeros_like(Cm), np.zeros_like(dt)
    dA, dD, dinit = np.zeros(H), np.zeros(H), np.zeros((N, H, d, n))
    for s in range(N):
        if init is not None and not _slot_ok(int(slot_map[s]), init.shape[0]):
            continue
        S = size(np.array(init[int(slot_map[s])])) if init is not None else np.zeros((H, d, n))
        states = [S]
        for t in range(cu[s], cu[s + 1]):
            S = np.exp(g[t])[:, None, None] * S + (dtp[t][:, None] * size(x[t]))[:, :, None] * size(_heads(Bm[t], H))[:, None]
            states.append(S)
        dS = size(np.array(dfinal[s])) if dfinal is not None else np.zeros((H, d, n))
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            S, before = states[t - cu[s] + 1], states[t - cu[s]]
            o, xt, Bt, Ct = size(dy[t]), size(x[t]), size(_heads(Bm[t], H)), size(_heads(Cm[t], H))
            dS = dS + o[:, :, None] * Ct[:, None]
            dC[t] = np.einsum("hpn,hp->hn", S, o).reshape(G, H // G, n).sum(1)
            X = np.einsum("hpn,hn->hp", dS, Bt)
            dx[t] = dtp[t][:, None] * X + size(Dskip[:, None]) * o
            dB[t] = (dtp[t][:, None] * np.einsum("hpn,hp->hn", dS, xt)).reshape(G, H // G, n).sum(1)
            dg = np.exp(g[t]) * (dS * before).sum((1, 2))
            ddt[t] = ((xt * X).sum(1) + sign * A * dg) * slope[t]
            dA += sign * A * dtp[t] * dg
            dD += (o * xt).sum(1)
            dS = np.exp(g[t])[:, None, None] * dS
        dinit[s] = dS
    return dx, dB, dC, ddt, dA, ddt.sum(0), dD, dinit
