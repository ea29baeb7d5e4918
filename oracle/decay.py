"""Linear attention with a decay for each value head, and the norms, gate and residual around a block, in
fp64: the token loop S <- a S + k v^T, o = scale S^T q with a = exp(log_decay[h]) (the update-rule table's
row below the delta rule on the learn-llm page "linear attention", the decay a constant of the head), its
adjoint walked backwards with the forward states kept, and RMSNorm / sigmoid gate / residual with their
gradients.  Value head h reads query/key head h // (Hv // Hqk).
"""
from __future__ import annotations

import numpy as np


def _a(log_decay):
    return np.exp(np.asarray(log_decay, np.float64))[:, None, None]


def sequences(T, cu=None, B=1):
    """Token ranges of the sequences in the flattened token order."""
    if cu is None:
        return [(i * T, (i + 1) * T) for i in range(B)]
    return [(int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def forward(q, k, v, log_decay, S0=None, scale=1.0, cu=None):
    """q, k [B, T, Hqk, dk], v [B, T, Hv, dv] -> (out [B, T, Hv, dv], S_final [nseq, Hv, dk, dv])."""
    B, T, Hqk, dk = q.shape
    Hv, dv = v.shape[2:]
    G = Hv // Hqk
    Q, K = (np.repeat(x.reshape(B * T, Hqk, dk).astype(np.float64), G, 1) for x in (q, k))
    V = v.reshape(B * T, Hv, dv).astype(np.float64)
    a = _a(log_decay)
    out, finals = np.zeros((B * T, Hv, dv)), []
    for i, (t0, t1) in enumerate(sequences(T, cu, B)):
        S = np.zeros((Hv, dk, dv)) if S0 is None else np.array(S0[i], np.float64)
        for t in range(t0, t1):
            S = a * S + K[t][:, :, None] * V[t][:, None, :]
            out[t] = scale * np.einsum("hk,hkv->hv", Q[t], S)
        finals.append(S)
    return out.reshape(B, T, Hv, dv), np.stack(finals) if finals else np.zeros((0, Hv, dk, dv))


def step(q, k, v, log_decay, S, slots=None, scale=1.0):
    """One token per row: (out [N, Hv, dv], the pool of states after it); idle rows (slot outside the pool)
    give zeros."""
    S = np.array(S, np.float64)
    N, Hv, dv = v.shape
    out = np.zeros((N, Hv, dv))
    for n in range(N):
        at = n if slots is None else int(slots[n])
        if 0 <= at < len(S):
            o, Sn = forward(q[n][None, None], k[n][None, None], v[n][None, None], log_decay, S[at][None], scale)
            out[n], S[at] = o[0, 0], Sn[0]
    return out, S


def backward(q, k, v, log_decay, dout, S0=None, dS_final=None, scale=1.0, cu=None):
    """(dq, dk, dv, dS0) of a loss whose gradients at (out, S_final) are dout and dS_final."""
    B, T, Hqk, dk = q.shape
    Hv, dv = v.shape[2:]
    G = Hv // Hqk
    Q, K = (np.repeat(x.reshape(B * T, Hqk, dk).astype(np.float64), G, 1) for x in (q, k))
    V, dO = (x.reshape(B * T, Hv, dv).astype(np.float64) for x in (v, dout))
    a = _a(log_decay)
    dQ, dK, dV, dS0 = np.zeros_like(Q), np.zeros_like(K), np.zeros_like(V), []
    for i, (t0, t1) in enumerate(sequences(T, cu, B)):
        S = np.zeros((Hv, dk, dv)) if S0 is None else np.array(S0[i], np.float64)
        for t in range(t0, t1):
            S = a * S + K[t][:, :, None] * V[t][:, None, :]
            dQ[t] = scale * np.einsum("hkv,hv->hk", S, dO[t])
        lam = np.zeros((Hv, dk, dv)) if dS_final is None else np.array(dS_final[i], np.float64)
        for t in range(t1 - 1, t0 - 1, -1):
            lam = lam + scale * Q[t][:, :, None] * dO[t][:, None, :]
            dK[t] = np.einsum("hkv,hv->hk", lam, V[t])
            dV[t] = np.einsum("hkv,hk->hv", lam, K[t])
            lam = a * lam
        dS0.append(lam)
    fold = lambda x: x.reshape(B, T, Hqk, G, dk).sum(3)   # noqa: E731
    return fold(dQ), fold(dK), dV.reshape(B, T, Hv, dv), np.stack(dS0) if dS0 else np.zeros((0, Hv, dk, dv))


def _parts(x, b, w_post, w_pre, gate, c, eps):
    x, b = np.asarray(x, np.float64), np.asarray(b, np.float64)
    s = 1.0 if gate is None else 1.0 / (1.0 + np.exp(-np.asarray(gate, np.float64)))
    c = 1.0 if c is None else np.asarray(c, np.float64)
    ib = 1.0 / np.sqrt((b * b).mean(-1, keepdims=True) + eps)
    y = b * ib * w_post
    r = x + c * s * y
    ir = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return b, s, c, ib, y, r, ir


def block_norm(x, b, w_post, w_pre, gate=None, res_scale=None, eps=1e-6):
    """(r, n): r = x + res_scale sigmoid(gate) RMSNorm(b) w_post, n = RMSNorm(r) w_pre."""
    *_, r, ir = _parts(x, b, w_post, w_pre, gate, res_scale, eps)
    return r, r * ir * w_pre


def block_norm_backward(x, b, w_post, w_pre, dr, dn, gate=None, res_scale=None, eps=1e-6):
    """(dx, db, dw_post, dw_pre, dgate or None, dres_scale or None)."""
    b, s, c, ib, y, r, ir = _parts(x, b, w_post, w_pre, gate, res_scale, eps)
    rows = tuple(range(r.ndim - 1))
    h = dn * w_pre
    dx = dr + ir * (h - r * ir * (h * r * ir).mean(-1, keepdims=True))
    e = dx * c * s * w_post
    db = ib * (e - b * ib * (e * b * ib).mean(-1, keepdims=True))
    dgate = dc = None
    if gate is not None:
        dgate = dx * c * y * s * (1 - s)
        if np.asarray(gate).shape[-1] == 1 and r.shape[-1] != 1:
            dgate = dgate.sum(-1, keepdims=True)
    if res_scale is not None:
        dc = (dx * s * y).sum(rows)
    return dx, db, (dx * c * s * b * ib).sum(rows), (dn * r * ir).sum(rows), dgate, dc
