"""CPU oracle of the operators around the layer -- TEST INFRASTRUCTURE ONLY.

Like the rest of ``oracle/``, only tests may import this module; it shares no
code with the CUDA library.  Double precision throughout, from the formulas:

* residual addition + RMS norm + 1x128 scaling:
    h = x + resid (rounded to the stream's type by the caller),
    rstd = (mean h^2 + eps)^-1/2,  y = h rstd w,
    S = amax / 448 (or the smallest power of two with amax <= 448 S) per 128
    channels;
* its backward, with n = h rstd and g = dy w:
    dx = dres + rstd (g - n mean(g n)),  dw = sum over rows of dy n;
* the sequence-wise balance loss of packed sequences ("DeepSeek-V3 Technischer
  Bericht" (xyznot.com/de), Methode section 2, in the technical report's form):
    f_i = N_r / (K_r L) picks_i,  loss = alpha sum_i f_i (1/L) sum_t s_ti / sum_j s_tj;
* the gradient of the router's logits z from the gates' gradient (picks held
  fixed, g_k = route_scale s_k / sum_sel s) and from the balance loss.
"""
from __future__ import annotations

import numpy as np


def rmsnorm(h, w, eps):
    """(y, rstd) of rows h."""
    h = np.asarray(h, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * (1.0 if w is None else np.asarray(w, np.float64)), rstd


def tile_amax(y):
    return np.abs(y).reshape(y.shape[0], -1, 128).max(axis=2)


def rmsnorm_backward(dy, h, rstd, w=None, dres=None):
    dy, h, rstd = (np.asarray(a, np.float64) for a in (dy, h, rstd))
    n = h * rstd[:, None]
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dx = rstd[:, None] * (g - n * (g * n).mean(axis=1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, (dy * n).sum(axis=0)


def sigmoid(z):
    """(s, 1 - s), neither by a difference."""
    z = np.asarray(z, np.float64)
    e = np.exp(-np.abs(z))
    big, small = 1.0 / (1.0 + e), e / (1.0 + e)
    return np.where(z >= 0, big, small), np.where(z >= 0, small, big)


def seq_counts(idx, off, Nr):
    """int64 [n_seq, Nr] picks per sequence; indices outside [0, Nr) do not count."""
    out = np.zeros((len(off) - 1, Nr), np.int64)
    for s, (a, b) in enumerate(zip(off[:-1], off[1:])):
        e = np.asarray(idx[a:b]).reshape(-1)
        e = e[(e >= 0) & (e < Nr)]
        np.add.at(out[s], e, 1)
    return out


def balance_loss(z, idx, off, alpha, Kr=None):
    """(loss [n_seq], counts)."""
    s, _ = sigmoid(z)
    Nr = s.shape[1]
    Kr = idx.shape[1] if Kr is None else Kr
    counts = seq_counts(idx, off, Nr)
    p = s / s.sum(axis=1, keepdims=True)
    loss = np.zeros(len(off) - 1)
    for i, (a, b) in enumerate(zip(off[:-1], off[1:])):
        L = b - a
        if L > 0:
            loss[i] = alpha * (counts[i] * Nr / (Kr * L) * p[a:b].sum(axis=0) / L).sum()
    return loss, counts


def router_dlogits(z, idx, Kr=None, dgate=None, route_scale=1.0, off=None, counts=None, dloss=None, alpha=0.0):
    """dz, and the sum of the magnitudes of the terms it is made of (for error bounds)."""
    s, om = sigmoid(z)
    T, Nr = s.shape
    Kr = idx.shape[1] if Kr is None else Kr
    dz, mag = np.zeros((T, Nr)), np.zeros((T, Nr))
    if off is not None:
        p = s / s.sum(axis=1, keepdims=True)
        for i, (a, b) in enumerate(zip(off[:-1], off[1:])):
            L = b - a
            if L <= 0:
                continue
            f = np.asarray(counts[i], np.float64) * Nr / (Kr * L)
            k = (1.0 if dloss is None else float(dloss[i])) * alpha / L
            fp = (f * p[a:b]).sum(axis=1, keepdims=True)
            dz[a:b] += k * p[a:b] * om[a:b] * (f - fp)
            mag[a:b] += abs(k) * p[a:b] * om[a:b] * (f + fp)
    if dgate is not None:
        sel = np.take_along_axis(s, idx, axis=1)
        gh = sel / sel.sum(axis=1, keepdims=True)
        r = route_scale * np.asarray(dgate, np.float64)
        tot = (r * gh).sum(axis=1, keepdims=True)
        mtot = (np.abs(r) * gh).sum(axis=1, keepdims=True)
        d = np.take_along_axis(om, idx, axis=1) * gh * (r - tot)
        m = np.take_along_axis(om, idx, axis=1) * gh * (np.abs(r) + mtot)
        for t in range(T):
            np.add.at(dz[t], idx[t], d[t])
            np.add.at(mag[t], idx[t], m[t])
    return dz, mag
