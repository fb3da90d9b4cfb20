"""Oracle of the dense half of a residual block -- dropout, the dense layer,
group norm over the rows of each graph -- in float64 (test infrastructure
only).

Definitions followed
--------------------
* Dropout (Srivastava et al., JMLR 2014, scaled at training time): with
  T = round(65536 p) an element is kept when its 16-bit draw is at least T and
  then scaled by 65536 / (65536 - T), held as fp32.  The draw of element j of
  the row with stream id `node`: number j % 8 of the Philox4x32-10 block at
  counter (j // 8, node, call, 1) under (seed low, seed high), two draws per
  word, low half first.
* Dense layer: Z = X W + b, Out = R + dropout(act(Z)); the gradients by the
  chain rule.
* Group norm (Wu and He, ECCV 2018) over each graph's rows and each group of
  adjacent channels, then an affine per channel and an activation.
"""
from __future__ import annotations

import math

import numpy as np

from .lowbit import philox4x32_10

ACTS = ("none", "relu", "leaky_relu", "gelu", "silu")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def drop_factor(rows, d, p, seed, call=0, nodes=None, row0=0):
    """float64 [rows, d]: 0 where dropped, else the scale (an fp32 value)."""
    T = int(math.floor(float(np.float32(p)) * 65536 + 0.5))
    if T == 0:
        return np.ones((rows, d))
    if T == 65536:
        return np.zeros((rows, d))
    ids = np.arange(rows, dtype=np.int64) + row0 if nodes is None else np.asarray(nodes, np.int64)
    out = np.zeros((rows, d))
    scale = float(np.float32(65536.0 / (65536 - T)))
    for j in range(d):
        if j % 8 == 0:
            ctr = np.zeros((rows, 4), np.uint64)
            ctr[:, 0] = j // 8
            ctr[:, 1] = ids.astype(np.uint64) & np.uint64(0xFFFFFFFF)
            ctr[:, 2] = call & 0xFFFFFFFF
            ctr[:, 3] = 1
            block = philox4x32_10(ctr, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)).astype(np.int64)
        word = block[:, (j % 8) // 2]
        u = word % 65536 if j % 2 == 0 else word // 65536
        out[:, j] = np.where(u >= T, scale, 0.0)
    return out


def drop(x, factor):
    """x with the factor applied; a dropped element is 0 whatever it held."""
    return np.where(factor == 0.0, 0.0, np.where(factor == 0.0, 0.0, x) * factor)


def act(z, kind, slope=0.01):
    if kind == "relu":
        return np.where(z < 0, 0.0, z)
    if kind == "leaky_relu":
        return np.where(z > 0, z, slope * z)
    if kind == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    return z


def act_grad(z, kind, slope=0.01):
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "leaky_relu":
        return np.where(z > 0, 1.0, slope)
    if kind == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def dense_forward(X, W, b, kind, slope, factor, R):
    """(Z, Out)."""
    Z = X @ W + (0.0 if b is None else b)
    Y = drop(act(Z, kind, slope), factor)
    return Z, Y + (0.0 if R is None else R)


def dense_backward(X, W, Z, kind, slope, factor, G):
    """(dZ, dW, db, dX)."""
    dZ = drop(G, factor)
    if kind != "none":
        dZ = dZ * act_grad(Z, kind, slope)
    return dZ, X.T @ dZ, dZ.sum(0), dZ @ W.T


def norm_stats(X, groups, seg, eps):
    """mean, rstd [graphs, groups] (mean 0 and var 0 for a graph without rows)."""
    n_seg, D = len(seg) - 1, X.shape[1] // groups
    mean, rstd = np.zeros((n_seg, groups)), np.full((n_seg, groups), 1.0 / math.sqrt(eps) if eps > 0 else np.inf)
    for i in range(n_seg):
        x = X[seg[i]:seg[i + 1]]
        if x.shape[0] == 0:
            continue
        x = x.reshape(x.shape[0], groups, D)
        mean[i] = x.mean((0, 2))
        rstd[i] = 1.0 / np.sqrt(((x - mean[i][None, :, None]) ** 2).mean((0, 2)) + eps)
    return mean, rstd


def norm_forward(X, groups, seg, w, b, kind, slope, mean, rstd, Out):
    """Out with the rows of every graph replaced (the others as given)."""
    Out = Out.copy()
    D = X.shape[1] // groups
    for i in range(len(seg) - 1):
        r = slice(seg[i], seg[i + 1])
        z = (X[r] - np.repeat(mean[i], D)) * np.repeat(rstd[i], D) * w + b
        Out[r] = act(z, kind, slope)
    return Out


def norm_backward(X, groups, seg, w, b, kind, slope, mean, rstd, G, dX):
    """(dw, db, dX), dX's rows of no graph as given."""
    dX = dX.copy()
    n, d = X.shape
    D = d // groups
    dw, db = np.zeros(d), np.zeros(d)
    for i in range(len(seg) - 1):
        r = slice(seg[i], seg[i + 1])
        if seg[i + 1] <= seg[i]:
            continue
        rs = np.repeat(rstd[i], D)
        xhat = (X[r] - np.repeat(mean[i], D)) * rs
        a = act_grad(xhat * w + b, kind, slope) * G[r]
        dw += (a * xhat).sum(0)
        db += a.sum(0)
        h = a * w
        m1 = np.repeat(h.reshape(-1, groups, D).mean((0, 2)), D)
        m2 = np.repeat((h * xhat).reshape(-1, groups, D).mean((0, 2)), D)
        dX[r] = rs * (h - m1 - xhat * m2)
    return dw, db, dX
