"""Plain float64 definitions of the block-scaled FP8 quantiser and the products
grouped by expert -- TEST INFRASTRUCTURE ONLY, as ``oracle.moe``.

The quantiser's definition names its fp32 roundings (scale, reciprocal,
product); each is made with one numpy float32 operation. Everything else is
float64, one row or one expert at a time.
"""
from __future__ import annotations

import numpy as np

from .moe import e4m3_decode, silu

__all__ = ["e4m3_encode", "quantize_block", "swiglu_quantize_block", "dequant_block", "source_rows",
           "grouped_matmul", "grouped_matmul_dw"]

_E4M3 = e4m3_decode(np.arange(127, dtype=np.uint8))  # the finite non-negative values, ascending by code


def e4m3_encode(v) -> np.ndarray:
    """Codes of the nearest E4M3 values (ties to the even code); |v| up to 448 and what rounds to it."""
    a = np.abs(np.asarray(v, np.float64))
    hi = np.clip(np.searchsorted(_E4M3, a), 1, 126)
    below, above = a - _E4M3[hi - 1], _E4M3[hi] - a
    code = np.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)
    return (code | (np.signbit(v) << 7)).astype(np.uint8)


def quantize_block(x, block_rows: int, pow2: bool):
    """x float32 [rows][cols] -> (codes uint8, scales float32): per block s = max(fl(amax / 448), 2^-126), the
    quotient raised to a power of two if pow2; code = e4m3(fl(x * fl(1 / s))); NaN scale and codes 0 for a block
    with a value that is not finite."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((-(-rows // block_rows), -(-cols // 128)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * block_rows:(i + 1) * block_rows, 128 * j:128 * (j + 1)]
            b = x[at]
            if not np.isfinite(b).all():
                scales[i, j] = np.nan
                continue
            amax = np.abs(b).max()
            s = amax / np.float32(448)
            if pow2 and s > 0:
                m, e = np.frexp(float(amax) / 448)
                s = np.float32(np.ldexp(1.0, int(e) - (m == 0.5)))
            s = max(np.float32(s), np.float32(2.0 ** -126))
            scales[i, j] = s
            codes[at] = e4m3_encode(b * (np.float32(1) / s))
    return codes, scales


def swiglu_quantize_block(gu, pow2: bool):
    """gu [rows][gate | up] -> quantize_block of silu(gate) * up rounded to float32, 1 x 128."""
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=1)
    return quantize_block((silu(g) * u).astype(np.float32), 1, pow2)


def dequant_block(codes, scales, block_rows: int) -> np.ndarray:
    """What the codes stand for, float64."""
    rows, cols = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), block_rows, axis=0)[:rows], 128, axis=1)[:, :cols]
    return e4m3_decode(codes) * s


def source_rows(m, order: str, perm, top_k: int) -> np.ndarray:
    """The rows of m in bucket order."""
    if order == "bucket":
        return m
    return m[perm // top_k if order == "token" else perm]


def grouped_matmul(x, w, offsets):
    """x [rows][Q] in bucket order, w [E][C][Q], float64 -> (y [rows][C], sum of |products|); rows of no bucket NaN."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    mag = np.full_like(y, np.nan)
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            y[lo:hi] = x[lo:hi] @ w[e].T
            mag[lo:hi] = np.abs(x[lo:hi]) @ np.abs(w[e]).T
    return y, mag


def grouped_matmul_dw(x, dy, offsets):
    """x [rows][K], dy [rows][N] in bucket order -> (dw [E][N][K], sum of |products|)."""
    E = len(offsets) - 1
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    mag = np.zeros_like(dw)
    for e in range(E):
        lo, hi = offsets[e], max(offsets[e + 1], offsets[e])
        dw[e] = dy[lo:hi].T @ x[lo:hi]
        mag[e] = np.abs(dy[lo:hi]).T @ np.abs(x[lo:hi])
    return dw, mag
