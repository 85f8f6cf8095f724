"""The gradients of the routing path and the 4-bit expert layer in binary64
(numpy), with bounds of the fp32 kernels' errors that follow from the
arithmetic; shared by the CPU tests (which check these formulas against
differences of the oracle's forward) and the GPU tests.

u = 2^-24 is half a step of fp32, relative to the value.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # rounding to the row dtype
TINY = {"bf16": 2.0 ** -133, "f32": 2.0 ** -149}    # smallest subnormal steps


def combine_backward(dy, E, w, inv, k):
    """(dE rows by sorted position, NaN where no slot names the row; dw; the
    sum of |dy * E| behind each dw)."""
    T, d = dy.shape
    dE = np.full(E.shape, np.nan)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        r = inv.reshape(T, k)[:, j]
        t = np.nonzero(r >= 0)[0]
        dE[r[t]] = w[t, j, None].astype(np.float64) * dy[t]
        p = dy[t] * E[r[t]]
        dw[t, j], mag[t, j] = p.sum(1), np.abs(p).sum(1)
    return dE, dw, mag


def gather_backward(dxs, inv, k, add=None):
    """(dx, the sum of the terms' magnitudes)."""
    T = len(inv) // k
    dx = np.zeros((T, dxs.shape[1]))
    mag = np.zeros_like(dx)
    for j in range(k):
        r = inv.reshape(T, k)[:, j]
        t = np.nonzero(r >= 0)[0]
        dx[t] += dxs[r[t]]
        mag[t] += np.abs(dxs[r[t]])
    if add is not None:
        dx += add
        mag += np.abs(add)
    return dx, mag


def dlogits(L, idx, g, scale, softmax=False, eps=1e-20):
    """(dL [T, N], bound of the fp32 kernel's error of each entry).

    sigmoid: expf is within 1 ulp (2 u), so s and 1 - s are within 6 u, their
    sum within 12 u, its reciprocal within 13 u; the mean of g within 26 u of M
    = sum |g| s / S, and the product of all factors within 64 u of
    scale / S * s (1 - s) * (|g| + M).
    softmax: the exponent's argument is off by u |L - max|, so p is off by at
    most P = (16 + 2 max|L - max| + N / 32) u relative, and dL by
    (2 P + 16 u) scale * p * (sum of the entry's |g| + M)."""
    L, g = np.asarray(L, np.float64), np.asarray(g, np.float64)
    T, N = L.shape
    k = idx.shape[1]
    ok = (idx >= 0) & (idx < N)
    e = np.where(ok, idx, 0)
    rows = np.arange(T)[:, None]
    g = np.where(ok, g, 0.0)
    dL, err = np.zeros((T, N)), np.zeros((T, N))
    if softmax:
        z = L - L.max(1, keepdims=True)
        p = np.exp(z)
        p /= p.sum(1, keepdims=True)
        ps = np.where(ok, p[rows, e], 0.0)
        mean = (g * ps).sum(1, keepdims=True)
        M = (np.abs(g) * ps).sum(1, keepdims=True)
        gs, ga = np.zeros((T, N)), np.zeros((T, N))
        for j in range(k):
            np.add.at(gs, (np.arange(T), e[:, j]), g[:, j])
            np.add.at(ga, (np.arange(T), e[:, j]), np.abs(g[:, j]))
        P = (16 + 2 * np.abs(z).max() + N / 32) * U
        return scale * p * (gs - mean), scale * p * (2 * P + 16 * U) * (ga + M)
    Lc = L[rows, e]
    s = np.where(ok, 1 / (1 + np.exp(-Lc)), 0.0)
    c = 1 / (1 + np.exp(Lc))
    S = s.sum(1, keepdims=True) + eps
    mean = (g * s).sum(1, keepdims=True) / S
    M = (np.abs(g) * s).sum(1, keepdims=True) / S
    dl = scale / S * (g - mean) * s * c
    b = 64 * U * scale / S * (np.abs(g) + M) * s * c
    for j in range(k):
        np.add.at(dL, (np.arange(T), e[:, j]), dl[:, j])
        np.add.at(err, (np.arange(T), e[:, j]), b[:, j] + U * np.abs(dl[:, j]))
    return dL, err


def products(dL, err, x, W, add=None, n_dx=None, n_dw=None):
    """dx = dL.W (+ add), dW = dL^T.x and their error bounds: the entries'
    errors carried through, plus one u per fp32 term of each sum (n_dx, n_dw:
    the most terms a sum has)."""
    dx = dL @ W
    mag = np.abs(dL) @ np.abs(W)
    if add is not None:
        dx = dx + add
        mag = mag + np.abs(add)
    n_dx = (n_dx or dL.shape[1]) + 2
    n_dw = (n_dw or dL.shape[0]) + 2
    return (dx, err @ np.abs(W) + n_dx * U * mag,
            dL.T @ x, err.T @ np.abs(x) + n_dw * U * (np.abs(dL).T @ np.abs(x)))


def check(got, want, bound, dtype="f32", name=""):
    """|got - want| <= bound plus half a step of the output's type."""
    got = np.asarray(got, np.float64)
    tol = bound + HALF_STEP[dtype] * (np.abs(want) + bound) + TINY[dtype]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (
        f"{name}: {bad.sum()} of {bad.size} beyond the bound, first at "
        f"{np.argwhere(bad)[0].tolist()}: got {got[bad][0]!r} want {np.asarray(want)[bad][0]!r} "
        f"tolerance {tol[bad][0]!r}")
    return float((np.abs(got - want) / tol).max()) if got.size else 0.0


def expert_w4(x, perm, offsets, q, scales, group, k):
    """(out by sorted row, sum of |scale * q * x| behind each, sum of |scale *
    x|) in binary64."""
    N, n_out, half = q.shape
    d = 2 * half
    rows = len(perm)
    out, mag, magx = (np.zeros((rows, n_out)) for _ in range(3))
    for e in range(N):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        v = np.empty((n_out, d))
        v[:, 0::2] = (q[e] & 15).astype(np.float64) - 8
        v[:, 1::2] = (q[e] >> 4).astype(np.float64) - 8
        sc = np.repeat(scales[e].astype(np.float64), group, axis=1)[:, :d]
        v *= sc
        xe = x[perm[a:b] // k]
        out[a:b] = xe @ v.T
        mag[a:b] = np.abs(xe) @ np.abs(v).T
        magx[a:b] = np.abs(xe) @ np.abs(sc).T
    return out, mag, magx
