"""Plain float64 definitions of the steps around the experts' products -- TEST
INFRASTRUCTURE ONLY, as ``oracle.moe``: one row at a time, from the formulas.

Functions that sum also return the sum of the terms' magnitudes, which the
tests' error bounds are made of.
"""
from __future__ import annotations

import numpy as np

from .moe import e2m1_decode, e8m0_decode, unpack_codes

__all__ = ["invert_perm", "gather_rows", "combine_rows", "combine_rows_grad", "swiglu", "swiglu_grad", "packed_weights",
           "matmul_packed"]


def invert_perm(perm, size: int) -> np.ndarray:
    """positions[perm[p]] = p, the last p of an assignment named twice, -1 elsewhere; entries outside [0, size) count
    for nothing."""
    positions = np.full(size, -1, np.int32)
    for p, a in enumerate(perm):
        if 0 <= a < size:
            positions[a] = p
    return positions


def gather_rows(x, perm, top_k: int, x_order: str, weights=None) -> np.ndarray:
    """out[p] = (weights[perm[p]] *) x[perm[p] // top_k or perm[p]]; NaN rows where perm names no assignment."""
    x = np.asarray(x, np.float64)
    slots = x.shape[0] * (top_k if x_order == "token" else 1)
    out = np.full((len(perm), x.shape[1]), np.nan)
    for p, a in enumerate(perm):
        if 0 <= a < slots:
            out[p] = x[a // top_k if x_order == "token" else a]
            if weights is not None:
                out[p] *= float(weights.reshape(-1)[a])
    return out


def combine_rows(y, weights, positions, T: int, top_k: int, y_shared=None):
    """(out [T][d], sum of |terms|): out[t] = sum_j weights[t][j] y[positions[t top_k + j]] + y_shared[t]."""
    y = np.asarray(y, np.float64)
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for a in range(T * top_k):
        p = a if positions is None else positions[a]
        if 0 <= p < y.shape[0]:
            term = y[p] * (1.0 if weights is None else float(weights.reshape(-1)[a]))
            out[a // top_k] += term
            mag[a // top_k] += np.abs(term)
    if y_shared is not None:
        out, mag = out + y_shared, mag + np.abs(y_shared)
    return out, mag


def combine_rows_grad(dout, y, weights, positions):
    """(dy, dweights [T][top_k], sum of |terms| of dweights); NaN rows of dy that no position names."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    T, k = weights.shape
    dy, dw, mag = np.full(y.shape, np.nan), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = t * k + j if positions is None else positions[t * k + j]
            if 0 <= p < y.shape[0]:
                dy[p] = float(weights[t, j]) * dout[t]
                dw[t, j] = (dout[t] * y[p]).sum()
                mag[t, j] = np.abs(dout[t] * y[p]).sum()
    return dy, dw, mag


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


def swiglu(gu) -> np.ndarray:
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=1)
    return g * _sigmoid(g) * u


def swiglu_grad(gu, dh):
    """(dgu, a magnitude of its terms): d/dg of g s(g) u is u s (1 + g (1 - s)), 1 - s(g) = s(-g)."""
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=1)
    dh, s, t = np.asarray(dh, np.float64), _sigmoid(g), _sigmoid(-g)
    return (np.concatenate([dh * u * s * (1 + g * t), dh * g * s], axis=1),
            np.concatenate([np.abs(dh * u) * s * (1 + np.abs(g) * t), np.abs(dh * g * s)], axis=1))


def packed_weights(codes, scales, biases):
    """(W, magnitude of its two terms) float64 [..., N][K] of 4-bit codes uint32 [..., N][K / 8]; biases None: MXFP4."""
    K = codes.shape[-1] * 8
    q = unpack_codes(codes, 4, K)
    spread = lambda t: np.repeat(t, K // t.shape[-1], axis=-1)  # noqa: E731
    if biases is None:
        w = e2m1_decode(q) * spread(e8m0_decode(scales))
        return w, np.abs(w)
    s, b = spread(np.asarray(scales, np.float64)), spread(np.asarray(biases, np.float64))
    return s * q + b, np.abs(s) * q + np.abs(b)


def matmul_packed(x, codes, scales, biases):
    """(x W^T, sum of |terms|), the terms being x * code * scale and x * bias."""
    w, mag = packed_weights(codes, scales, biases)
    x = np.asarray(x, np.float64)
    return x @ w.T, np.abs(x) @ mag.T
