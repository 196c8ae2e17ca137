"""fp64 oracles of the language-model operators: head norms with rotation, the gated delta rule.

Written from the definitions in include/litela.h (numpy, float64, one token after another, the
gradients by the chain rule of the recurrence) and independent of the CUDA code: it shares no
code, layout trick or chunking with it.
"""
from __future__ import annotations

import numpy as np


def _pairs(rot, interleaved):
    lo = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    return lo, lo + (1 if interleaved else rot // 2)


def qk_norm_rope(x, Hq, Hk, wq, wk, cos, sin, pos, eps, interleaved, dout=None):
    """x: [B, N, heads, d]; wq, wk [d] or None; cos, sin [P, rot/2] or None; pos [B, N].
    Returns out, or with dout (dx, dwq, dwk).  Rows at a negative position: zeros."""
    x = np.asarray(x, np.float64)
    d, h = x.shape[-1], Hq + Hk
    w = np.ones((h, d))
    if wq is not None:
        w[:Hq] = wq
    if wk is not None:
        w[Hq:] = wk
    rot = 0 if cos is None else 2 * cos.shape[1]
    lo, hi = _pairs(rot, interleaved)
    real = pos >= 0
    at = np.where(real, pos, 0)
    if rot:
        over = at >= cos.shape[0]
        c, s = (np.asarray(t, np.float64)[np.minimum(at, cos.shape[0] - 1)][:, :, None] for t in (cos, sin))
        c, s = np.where(over[:, :, None, None], np.nan, c), np.where(over[:, :, None, None], np.nan, s)
    a = x[:, :, :h]
    r = 1.0 / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
    keep = real[:, :, None, None]
    if dout is None:
        y = a * r * w
        if rot:
            u, v = y[..., lo].copy(), y[..., hi].copy()
            y[..., lo], y[..., hi] = u * c - v * s, v * c + u * s
        return np.where(keep, np.concatenate((y, x[:, :, h:]), 2), 0.0)
    dout = np.where(keep, np.asarray(dout, np.float64), 0.0)
    t = dout[:, :, :h].copy()
    if rot:
        u, v = t[..., lo].copy(), t[..., hi].copy()
        t[..., lo], t[..., hi] = u * c + v * s, v * c - u * s
    dw = (t * a * r).sum((0, 1))
    t = t * w
    dx = r * t - a * r ** 3 * (t * a).mean(-1, keepdims=True)
    return np.concatenate((dx, dout[:, :, h:]), 2), dw[:Hq].sum(0), dw[Hq:].sum(0)


def gated_delta(q, k, v, g, beta, scale, state=None, grads=None):
    """One sequence: q, k [N, Hk, d], v [N, Hv, d], g, beta [N, Hv], state [Hv, d, d] or None.
    Returns (out, state_out); with grads = (dout, dstate_out) also the gradients
    (dq, dk, dv, dg, dbeta, dstate_in)."""
    q, k, v, g, beta = (np.asarray(t, np.float64) for t in (q, k, v, g, beta))
    N, Hv, d = v.shape
    Hk = q.shape[1]
    group = Hv // Hk
    qh, kh = np.repeat(q, group, 1), np.repeat(k, group, 1)
    S = np.zeros((Hv, d, d)) if state is None else np.asarray(state, np.float64).copy()
    alpha = np.exp(g)
    out, states, err = np.zeros((N, Hv, d)), [S], np.zeros((N, Hv, d))
    for n in range(N):
        A = alpha[n][:, None, None] * S
        err[n] = v[n] - np.einsum("hij,hi->hj", A, kh[n])
        S = A + np.einsum("hi,hj->hij", kh[n], beta[n][:, None] * err[n])
        out[n] = scale * np.einsum("hij,hi->hj", S, qh[n])
        states.append(S)
    if grads is None:
        return out, S
    do, dS = (np.asarray(t, np.float64) for t in grads)
    G = dS.copy()
    dq, dk = np.zeros((N, Hv, d)), np.zeros((N, Hv, d))
    dv, dg, db = np.zeros((N, Hv, d)), np.zeros((N, Hv)), np.zeros((N, Hv))
    for n in reversed(range(N)):
        dq[n] = scale * np.einsum("hij,hj->hi", states[n + 1], do[n])
        G = G + scale * np.einsum("hi,hj->hij", qh[n], do[n])
        du = np.einsum("hij,hi->hj", G, kh[n])
        db[n] = (du * err[n]).sum(-1)
        dv[n] = beta[n][:, None] * du
        A = alpha[n][:, None, None] * states[n]
        dk[n] = np.einsum("hij,hj->hi", G, beta[n][:, None] * err[n]) - np.einsum("hij,hj->hi", A, dv[n])
        G = G - np.einsum("hi,hj->hij", kh[n], dv[n])
        dg[n] = (G * A).sum((-1, -2))
        G = alpha[n][:, None, None] * G
    share = lambda t: t.reshape(N, Hk, group, d).sum(2)  # noqa: E731
    return out, S, (share(dq), share(dk), dv, dg, db, G)
