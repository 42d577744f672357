"""The gated linear recurrence, its gradient and the 8-bit checkpoint's values in float64, position by position.

For one sequence in scan order (k = 0 first), per channel:

    log a_k = -8 softplus(lam) sigmoid(r_k)
    h_k     = a_k h_{k-1} + sqrt(1 - a_k^2) sigmoid(g_k) x_k

The gradient is the chain rule applied to these lines, last position first.
"""
from __future__ import annotations

import numpy as np

__all__ = ["gated_coefficients", "gated_scan_forward", "gated_scan_entering", "gated_scan_backward", "act8_values"]

RATE = 8.0
TILE = 64
GROUP = 64


def _sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def gated_coefficients(r, g, lam):
    """(a, beta, sigmoid(r), sigmoid(g), log a) of rows [n, E]."""
    sr, sg = _sigmoid(r), _sigmoid(g)
    la = -RATE * np.logaddexp(0.0, lam) * sr
    return np.exp(la), np.sqrt(-np.expm1(2.0 * la)), sr, sg, la


def gated_scan_forward(x, r, g, lam, h0):
    """States [n, E] after each position."""
    a, beta, _, sg, _ = gated_coefficients(r, g, lam)
    h = np.array(h0, np.float64)
    out = np.empty_like(x)
    for k in range(x.shape[0]):
        # a closed input gate times an infinite x is NaN here as in IEEE arithmetic
        h = a[k] * h + beta[k] * (sg[k] * x[k])
        out[k] = h
    return out


def gated_scan_entering(x, r, g, lam, h0, starts=None):
    """The state that enters each position, [n, E].  With `starts` (a row for every TILE-th position) each tile is
    run from its own start, as a gradient that recomputes tiles does."""
    a, beta, _, sg, _ = gated_coefficients(r, g, lam)
    h = np.array(h0, np.float64)
    out = np.empty_like(x)
    for k in range(x.shape[0]):
        if starts is not None and k % TILE == 0:
            h = starts[k // TILE]
        out[k] = h
        h = a[k] * h + beta[k] * (sg[k] * x[k])
    return out


def gated_scan_backward(x, r, g, lam, h0, dy, dh_last, starts=None):
    """(dx, dr, dg, dlam, dh0) for dy [n, E] and dh_last [E]."""
    a, beta, sr, sg, la = gated_coefficients(r, g, lam)
    enters = gated_scan_entering(x, r, g, lam, h0, starts)
    D = np.array(dh_last, np.float64)
    dx, dr, dg = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    dlam = np.zeros(x.shape[1])
    slope = -RATE * _sigmoid(lam)
    for k in range(x.shape[0] - 1, -1, -1):
        G = dy[k] + D
        dx[k] = G * beta[k] * sg[k]
        dg[k] = G * beta[k] * x[k] * sg[k] * (1.0 - sg[k])
        with np.errstate(divide="ignore", invalid="ignore"):
            dla = np.where(la[k] == 0.0, 0.0, G * (a[k] * enters[k] - sg[k] * x[k] * a[k] ** 2 / beta[k]))
        dr[k] = dla * la[k] * (1.0 - sr[k])
        dlam += dla * sr[k] * slope
        D = a[k] * G
    return dx, dr, dg, dlam, D


def act8_values(v):
    """What an 8-bit checkpoint of rows v [m, cols] stands for: e4m3 values times a power of two per 64 channels."""
    v = np.asarray(v, np.float64)
    out = np.empty_like(v)
    for c in range(0, v.shape[1], GROUP):
        p = v[:, c:c + GROUP]
        fine = np.isfinite(p)
        top = np.max(np.where(fine, np.abs(p), 0.0), axis=1, keepdims=True)
        _, e = np.frexp(top / 448.0)                       # top / 448 = m 2^e, 1/2 <= m < 1 (exact: only e is used)
        k = np.where(np.ldexp(448.0, e - 1) >= top, e - 1, e)
        k = np.maximum(np.where(top > 0, k, -126), -126)
        u = np.ldexp(np.where(fine, p, 0.0), -k)
        _, ue = np.frexp(u)
        grid = np.ldexp(1.0, np.maximum(ue - 1, -6) - 3)   # 3 fraction bits, and 2^-9 below the normal range
        q = np.ldexp(np.rint(u / grid) * grid, k)          # rint: ties to even
        q = np.clip(q, -np.ldexp(240.0, 120), np.ldexp(240.0, 120))   # 256 * 2^120 is no fp32 number
        out[:, c:c + GROUP] = np.where(fine, q, np.nan)
    return out
