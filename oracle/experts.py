"""Layers of experts in e4m3, in 64 bits from the definitions (loops over slots
and experts).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

A slot is one choice of a token (slot = token * topk + j); the slots of expert e
have the rows offsets[e] .. offsets[e + 1], in the order of their slots; ids outside
[0, experts) have no row.  e4m3 rows: bytes [rows][Kp], scales [Kp/128][rows];
weights: bytes [experts][N][Kp], scales [experts][Np/128][Kp/128].
"""
from __future__ import annotations

import numpy as np

from .codecs import e4m3_to_f64, e8m0_to_f64
from .mx import E4M3_MAGNITUDES, nearest_code, padded, quant_e4m3, scale_exponent


def sort(ids, experts: int):
    """(place [tokens][topk], order [slots], offsets [experts + 1])."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    place = np.full(flat.size, -1, np.int32)
    order = np.full(flat.size, -1, np.int32)
    offsets = np.zeros(experts + 1, np.int32)
    row = 0
    for e in range(experts):
        offsets[e] = row
        slots = np.flatnonzero(flat == e)
        place[slots] = row + np.arange(len(slots))
        order[row:row + len(slots)] = slots
        row += len(slots)
    offsets[experts] = row
    return place.reshape(ids.shape), order, offsets


def dequant_rows(q, scale):
    """Values [rows][Kp] of e4m3 rows."""
    rows = q.shape[0]
    with np.errstate(invalid="ignore"):
        return (e4m3_to_f64(q).reshape(rows, -1, 128) * e8m0_to_f64(scale).T[..., None]).reshape(rows, -1)


def quant_rows(x):
    """(bytes [rows][Kp], scales [Kp/128][rows])."""
    return quant_e4m3(np.asarray(x, np.float64))


def quant_weights(w):
    """(bytes [N][Kp], scales [Np/128][Kp/128]) of one matrix [N][K]."""
    w = np.asarray(w, np.float64)
    n, k = w.shape
    full = np.zeros((padded(n), padded(k)))
    full[:n, :k] = w
    b = full.reshape(padded(n) // 128, 128, padded(k) // 128, 128)
    bad = ~np.isfinite(b).all((1, 3))
    b = np.where(bad[:, None, :, None], 0.0, b)
    e = scale_exponent(np.abs(b).max((1, 3)), 448.0, 8, "ceil")
    idx = nearest_code(np.ldexp(b, -e[:, None, :, None]), E4M3_MAGNITUDES)
    code = (idx + 128 * np.signbit(b)).astype(np.uint8).reshape(padded(n), padded(k))[:n]
    return code, np.where(bad, 255, e + 127).astype(np.uint8)


def dequant_weights(q, scale):
    """Values [N][Kp] of one matrix."""
    n, k = q.shape
    s = np.repeat(e8m0_to_f64(scale), 128, 0)[:n]
    with np.errstate(invalid="ignore"):
        return (e4m3_to_f64(q).reshape(n, -1, 128) * s[..., None]).reshape(n, k)


def product(a, b, offsets):
    """(C, Abs) [rows][N] of values a [rows][K] and b [experts][N][K]; rows of no
    expert are zero."""
    c = np.zeros((a.shape[0], b.shape[1]))
    t = np.zeros_like(c)
    for e, (lo, hi) in enumerate(zip(offsets[:-1], offsets[1:])):
        c[lo:hi] = a[lo:hi] @ b[e].T
        t[lo:hi] = np.abs(a[lo:hi]) @ np.abs(b[e]).T
    return c, t


def wgrad(d, a, offsets):
    """(dB, Abs) [experts][N][K] of values d [rows][N] and a [rows][K]."""
    parts = list(zip(offsets[:-1], offsets[1:]))
    return (np.stack([d[lo:hi].T @ a[lo:hi] for lo, hi in parts]),
            np.stack([np.abs(d[lo:hi]).T @ np.abs(a[lo:hi]) for lo, hi in parts]))


def combine(x, place, weights=None, r=None):
    """(Y, Abs) [tokens][cols]: sums and sums of magnitudes."""
    tokens, topk = place.shape
    y = np.zeros((tokens, x.shape[1])) if r is None else np.array(r, np.float64)
    t = np.abs(y)
    for i in range(tokens):
        for j in range(topk):
            if 0 <= place[i, j] < x.shape[0]:
                v = x[place[i, j]] * (1.0 if weights is None else weights[i, j])
                y[i] += v
                t[i] += np.abs(v)
    return y, t


def combine_grad(dy, x, place, weights=None):
    """(dX [rows][cols], dW [tokens][topk], its Abs); rows without a slot are zero."""
    dx, dw, t = np.zeros(x.shape), np.zeros(place.shape), np.zeros(place.shape)
    for i in range(place.shape[0]):
        for j in range(place.shape[1]):
            r = place[i, j]
            if 0 <= r < x.shape[0]:
                dx[r] = dy[i] * (1.0 if weights is None else weights[i, j])
                dw[i, j] = dy[i] @ x[r]
                t[i, j] = np.abs(dy[i]) @ np.abs(x[r])
    return dx, dw, t


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(g, np.float64)))


def glu(x):
    """silu(g) * u of x = [g | u]."""
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    return g * sigmoid(g) * u


def glu_grad(dy, x):
    """(dX, terms) for x = [g | u]: the terms' magnitudes bound the fp32 errors, which
    are largest where s + g s (1 - s) cancels."""
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    dy, s = np.asarray(dy, np.float64), sigmoid(g)
    dx = np.concatenate([dy * u * (s + g * s * (1.0 - s)), dy * g * s], 1)
    return dx, np.concatenate([np.abs(dy * u) * (s + np.abs(g * s)), np.abs(dy * g * s)], 1)
