"""Oracles of the layers beside the scan, in 64 bits on the CPU, one token after the other.

    qk_norm(x, w, inv_freq, positions, eps, mode, interleaved)              -> y
    qk_norm_backward(x, w, inv_freq, positions, eps, mode, interleaved, dy) -> dx, dw
    delta(q, k, v, g, beta, h0, scale, lengths)                             -> y, h_final
    delta_backward(q, k, v, g, beta, h0, scale, lengths, dy, dh_final)      -> dict of gradients

All arguments are numpy arrays (None where absent); layouts as in include/pdssm.h.
"""
from __future__ import annotations

import numpy as np


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(z, inv_freq, positions, interleaved, sign):
    if inv_freq is None:
        return z
    a, b = _pairs(2 * len(inv_freq), interleaved)
    t = positions.astype(np.float64)[:, :, None, None] * inv_freq.astype(np.float64)
    c, s = np.cos(t), sign * np.sin(t)
    out = z.copy()
    out[..., a] = z[..., a] * c - z[..., b] * s
    out[..., b] = z[..., b] * c + z[..., a] * s
    return out


def _places(x, positions):
    return np.broadcast_to(np.arange(x.shape[1]), x.shape[:2]) if positions is None else positions


def qk_norm(x, w, inv_freq, positions, eps, mode, interleaved):
    x = x.astype(np.float64)
    m = (x * x).sum(-1, keepdims=True)
    if mode == "rms":
        m = m / x.shape[-1]
    z = x / np.sqrt(m + eps)
    if w is not None:
        z = z * w.astype(np.float64)
    return _turn(z, inv_freq, _places(x, positions), interleaved, 1.0)


def qk_norm_backward(x, w, inv_freq, positions, eps, mode, interleaved, dy):
    x, n = x.astype(np.float64), x.shape[-1]
    d = _turn(dy.astype(np.float64), inv_freq, _places(x, positions), interleaved, -1.0)
    share = 1.0 / n if mode == "rms" else 1.0
    s = np.sqrt(share * (x * x).sum(-1, keepdims=True) + eps)
    dw = (d * x / s).sum((0, 1, 2))
    if w is not None:
        d = d * w.astype(np.float64)
    dx = d / s - x * share * (d * x).sum(-1, keepdims=True) / s ** 3
    return dx, dw


def _prepare(q, k, v, g, beta, h0, scale, lengths):
    q, k, v, g, beta = (np.asarray(x, np.float64) for x in (q, k, v, g, beta))
    Bt, L, H, P = v.shape
    r = H // q.shape[2]
    q, k = np.repeat(q, r, 2), np.repeat(k, r, 2)
    h = np.zeros((Bt, H, q.shape[-1], P)) if h0 is None else np.array(h0, np.float64)
    ends = np.full(Bt, L) if lengths is None else np.clip(lengths, 0, L)
    return q * scale, k, v, np.exp(g), beta, h, ends


def delta(q, k, v, g, beta, h0=None, scale=1.0, lengths=None):
    q, k, v, a, beta, h, ends = _prepare(q, k, v, g, beta, h0, scale, lengths)
    y = np.zeros_like(v)
    for b in range(v.shape[0]):
        for t in range(ends[b]):
            for i in range(v.shape[2]):
                f = a[b, t, i] * h[b, i]
                e = v[b, t, i] - f.T @ k[b, t, i]
                h[b, i] = f + beta[b, t, i] * np.outer(k[b, t, i], e)
                y[b, t, i] = h[b, i].T @ q[b, t, i]
    return y, h


def delta_backward(q, k, v, g, beta, h0, scale, lengths, dy, dh_final=None):
    qk_heads = q.shape[2]
    q, k, v, a, beta, h, ends = _prepare(q, k, v, g, beta, h0, scale, lengths)
    dy = np.asarray(dy, np.float64)
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, a, beta))
    dh0 = np.zeros_like(h)
    for b in range(v.shape[0]):
        for i in range(v.shape[2]):
            states = [h[b, i]]
            for t in range(ends[b]):
                f = a[b, t, i] * states[-1]
                states.append(f + beta[b, t, i] * np.outer(k[b, t, i], v[b, t, i] - f.T @ k[b, t, i]))
            x = np.zeros_like(h[b, i]) if dh_final is None else np.array(dh_final[b, i], np.float64)
            for t in range(ends[b] - 1, -1, -1):
                f = a[b, t, i] * states[t]
                e = v[b, t, i] - f.T @ k[b, t, i]
                x = x + np.outer(q[b, t, i], dy[b, t, i])
                dq[b, t, i] = scale * states[t + 1] @ dy[b, t, i]
                du = x.T @ k[b, t, i]
                dv[b, t, i] = beta[b, t, i] * du
                db[b, t, i] = du @ e
                dk[b, t, i] = x @ (beta[b, t, i] * e) - f @ dv[b, t, i]
                x = x - np.outer(k[b, t, i], dv[b, t, i])
                dg[b, t, i] = (x * f).sum()
                x = a[b, t, i] * x
            dh0[b, i] = x
    r = v.shape[2] // qk_heads

    def shared(d):
        return d.reshape(d.shape[0], d.shape[1], qk_heads, r, d.shape[3]).sum(3)

    return {"dq": shared(dq), "dk": shared(dk), "dv": dv, "dg": dg, "dbeta": db, "dh0": dh0}
