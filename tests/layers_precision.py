"""What the delta rule's fp32 results may be off by, in units of 2^-24 (the largest relative error of one rounding to fp32; of a norm over
many values a rounding makes about 1 / sqrt(3) of it), as norms over a (sequence, head)'s slice.

A chunk takes a state through three products, one after the other. Their sums of up to 3 N / 16, 24 and 12 accumulations, and some 8
products of single values, are (24 + 24 + 12 + 8) / 3 = 23 squared units for N = 128, the four factors exp(..), off by up to 4 units
each, another 4 x 4 / 3 x 4 = 21 at most: sqrt(44) = 6.6 units. A step takes beta (2 - beta), or three quarters, of the part along its
key out of what is remembered, so N / 0.38 steps are, five chunks for N = 128: 6.6 sqrt(5) = 14.8.

* h_final, dh0: 14.8; 18.
* dbeta = <du, e>: both factors are the chunk's own, 6.6 sqrt(2), through two states of 14.8 that they share half of: 18; 24.
* dg, a sum of terms <X, H'>, <dy, y> and -<dv, v> that may cancel: its size is the root of the sum of the terms' usual sizes
  squared, |x| |w| / sqrt(n) for a dot product of n values. One of factors that are off by 14.8 each is off by 14.8 sqrt(2) of that, and
  the terms' errors are independent: 21; 24.
"""
import numpy as np

from oracle import layers

UNIT = 2.0 ** -24
BOUNDS = {"h_final": 18, "dh0": 18, "dbeta": 24, "dg": 24}


def npy(t):
    return t.detach().double().cpu().numpy()


def backward_oracle(a, h0, dy, dh, lengths=None):
    x = [npy(a[n]) for n in ("q", "k", "v", "g", "beta")]
    scale = a["q"].shape[-1] ** -0.5
    y, h = layers.delta(*x, npy(h0), scale, lengths)
    return y, h, layers.delta_backward(*x, npy(h0), scale, lengths, npy(dy), npy(dh))


def ends(a, h0, dy, dh, chunk):
    """|X| |H'| of every chunk's end."""
    q, k, v, g, beta = (npy(a[n]) for n in ("q", "k", "v", "g", "beta"))
    r = v.shape[2] // q.shape[2]
    q, k, g = q.repeat(r, 2) * q.shape[-1] ** -0.5, k.repeat(r, 2), np.exp(g)
    L, at, h, x = v.shape[1], [], npy(h0), npy(dh)
    for t in range(L):
        h = g[:, t, :, None, None] * h
        h = h + k[:, t, :, :, None] * (beta[:, t, :, None] * (v[:, t] - (k[:, t, :, None] @ h)[..., 0, :]))[:, :, None]
        if (t + 1) % chunk == 0 or t + 1 == L:
            at.append(np.linalg.norm(h, axis=(2, 3)))
    for t in range(L - 1, -1, -1):
        if (t + 1) % chunk == 0 or t + 1 == L:
            at[t // chunk] = at[t // chunk] * np.linalg.norm(x, axis=(2, 3))
        x = x + q[:, t, :, :, None] * npy(dy)[:, t, :, None]
        x = g[:, t, :, None, None] * (x - k[:, t, :, :, None] * (beta[:, t, :, None] * (k[:, t, :, None] @ x)[..., 0, :])[:, :, None])
    return at


def gate_terms(a, h0, y, want, dy, dh, chunk):
    """The size of what dg_i is a sum of: <X, H'> and, over the chunk's j >= i, <dy_j, y_j> and <dv_j, v_j>."""
    L, P, N = y.shape[1], y.shape[3], a["q"].shape[3]
    size = lambda x, w: (x ** 2).sum(-1) * (w ** 2).sum(-1) / P  # noqa: E731
    local, M = size(npy(dy), y) + size(want["dv"], npy(a["v"])), np.zeros(y.shape[:3])
    for i, end in enumerate(ends(a, h0, dy, dh, chunk)):
        t = slice(i * chunk, min(L, (i + 1) * chunk))
        M[:, t] = end[:, None] ** 2 / (N * P) + local[:, t][:, ::-1].cumsum(1)[:, ::-1]
    return np.sqrt(M)


def slices_off(got, h, want, terms):
    """The largest slice's error of each fp32 result, in units."""
    out = {}
    for n, w, axes in (("h_final", h, (2, 3)), ("dh0", want["dh0"], (2, 3)), ("dbeta", want["dbeta"], (1,)), ("dg", want["dg"], (1,))):
        size = np.linalg.norm(terms if n == "dg" else w, axis=axes)
        out[n] = float((np.linalg.norm(got[n] - w, axis=axes) / size).max()) / UNIT
    return out
