"""The selective state space scan and the layer norm in fp64: the token loop h <- exp(dt A) h + dt u B,
y = (sum_n C h + skip u) silu(z) with dt = softplus(delta + dt_bias), A = -exp(A_log) (a row of the update-rule table's
gated-linear kind with a diagonal state for each channel), its adjoint walked backwards with the forward states kept, and
the layer norm behind a residual add with its gradients.  Channel d reads B and C of group d // (D // G).
"""
from __future__ import annotations

import numpy as np


def sequences(T, cu=None, B=1):
    """Token ranges of the sequences in the flattened token order."""
    if cu is None:
        return [(i * T, (i + 1) * T) for i in range(B)]
    return [(int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def _parts(u, delta, A_log, B, C, skip, dt_bias, z):
    nB, T, D = u.shape
    f = lambda x, *s: np.asarray(x, np.float64).reshape(nB * T, *s)   # noqa: E731
    G, N = B.shape[2:]
    x = f(delta, D) + (0 if dt_bias is None else np.asarray(dt_bias, np.float64))
    dt = np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))
    grow = lambda m: np.repeat(f(m, G, N), D // G, 1)   # noqa: E731
    return (f(u, D), x, dt, -np.exp(np.asarray(A_log, np.float64)), grow(B), grow(C),
            np.zeros(D) if skip is None else np.asarray(skip, np.float64), None if z is None else f(z, D))


def _states(u, dt, A, B, spans, h0):
    """Every token's state after it, and each sequence's last."""
    hs, finals = np.zeros((*u.shape, A.shape[1])), []
    for i, (t0, t1) in enumerate(spans):
        h = np.zeros_like(A) if h0 is None else np.array(h0[i], np.float64)
        for t in range(t0, t1):
            h = np.exp(dt[t][:, None] * A) * h + (dt[t] * u[t])[:, None] * B[t]
            hs[t] = h
        finals.append(h)
    return hs, np.stack(finals) if finals else np.zeros((0, *A.shape))


def forward(u, delta, A_log, B, C, h0=None, skip=None, dt_bias=None, z=None, cu=None):
    """u, delta, z [B, T, D], B, C [B, T, G, N] -> (y [B, T, D], h_final [nseq, D, N])."""
    U, _, dt, A, Bm, Cm, sk, Z = _parts(u, delta, A_log, B, C, skip, dt_bias, z)
    hs, finals = _states(U, dt, A, Bm, sequences(u.shape[1], cu, u.shape[0]), h0)
    y = (hs * Cm).sum(-1) + sk * U
    return (y if Z is None else y * Z * _sigmoid(Z)).reshape(u.shape), finals


def step(u, delta, A_log, B, C, h, skip=None, dt_bias=None, z=None, slots=None):
    """One token per row: (y [N, D], the pool of states after it); idle rows (slot outside the pool) give zeros."""
    h, y = np.array(h, np.float64), np.zeros(u.shape)
    for n in range(len(u)):
        at = n if slots is None else int(slots[n])
        if 0 <= at < len(h):
            row = lambda x: None if x is None else x[n][None, None]   # noqa: E731
            o, hn = forward(row(u), row(delta), A_log, row(B), row(C), h[at][None], skip, dt_bias, row(z))
            y[n], h[at] = o[0, 0], hn[0]
    return y, h


def backward(u, delta, A_log, B, C, dy, h0=None, dh_final=None, skip=None, dt_bias=None, z=None, cu=None):
    """(du, ddelta, dA_log, dB, dC, dskip, ddt_bias, dz or None, dh0) of a loss whose gradients at (y, h_final) are dy
    and dh_final."""
    U, x, dt, A, Bm, Cm, sk, Z = _parts(u, delta, A_log, B, C, skip, dt_bias, z)
    spans = sequences(u.shape[1], cu, u.shape[0])
    G, N = B.shape[2:]
    dY = np.asarray(dy, np.float64).reshape(U.shape)
    hs, _ = _states(U, dt, A, Bm, spans, h0)
    full = (hs * Cm).sum(-1) + sk * U
    p, dz = dY, None
    if Z is not None:
        s = _sigmoid(Z)
        p, dz = dY * Z * s, (dY * full * s * (1 + Z * (1 - s))).reshape(u.shape)
    dU, ddt = sk * p, np.zeros_like(U)
    dB, dC = np.zeros_like(Bm), hs * p[..., None]
    dA, dh0 = np.zeros_like(A), []
    for i, (t0, t1) in enumerate(spans):
        lam = np.zeros_like(A) if dh_final is None else np.array(dh_final[i], np.float64)
        for t in range(t1 - 1, t0 - 1, -1):
            prev = hs[t - 1] if t > t0 else (np.zeros_like(A) if h0 is None else np.asarray(h0[i], np.float64))
            lam = lam + Cm[t] * p[t][:, None]
            q = (lam * Bm[t]).sum(-1)
            dU[t] += dt[t] * q
            dB[t] = lam * (dt[t] * U[t])[:, None]
            lam = np.exp(dt[t][:, None] * A) * lam
            ddt[t] = U[t] * q + (A * lam * prev).sum(-1)
            dA += dt[t][:, None] * lam * prev
        dh0.append(lam)
    ddelta = ddt * _sigmoid(x)
    fold = lambda m: m.reshape(*u.shape[:2], G, u.shape[2] // G, N).sum(3)   # noqa: E731
    return (dU.reshape(u.shape), ddelta.reshape(u.shape), dA * A, fold(dB), fold(dC), (p * U).sum(0), ddelta.sum(0), dz,
            np.stack(dh0) if dh0 else np.zeros((0, *A.shape)))


def layer_norm(x, w, bias=None, residual=None, eps=1e-5):
    """(n, r): r = x + residual, n = (r - mean r) / sqrt(var r + eps) w + bias."""
    r = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    d = r - r.mean(-1, keepdims=True)
    n = d / np.sqrt((d * d).mean(-1, keepdims=True) + eps) * w
    return n if bias is None else n + bias, r


def layer_norm_backward(x, w, dn, residual=None, dr=None, eps=1e-5):
    """(dx, dw, dbias); dx is the gradient of residual too."""
    r = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    d = r - r.mean(-1, keepdims=True)
    inv = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    rh, h = d * inv, np.asarray(dn, np.float64) * w
    dx = inv * (h - h.mean(-1, keepdims=True) - rh * (h * rh).mean(-1, keepdims=True))
    rows = tuple(range(r.ndim - 1))
    return dx if dr is None else dx + dr, (dn * rh).sum(rows), np.asarray(dn, np.float64).sum(rows)
