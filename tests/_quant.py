"""What a SwiGLU quantiser may answer, decided value by value in 64 bits."""
import numpy as np

import oracle


def check_swiglu(codes, scales, gu, pow2):
    """codes uint8 [rows][inner] and scales fp32 for gu (float64 of the inputs) as moe_swiglu_quantize_block defines
    them, up to the last bits of h = silu(gate) * up in fp32.

    h: 2 ulp for the exponential and half an ulp for each of the sum, the quotient and the product are less than
    2^-21 relative to it, with the oracle's own rounding of h. A scale has that error and two roundings; with pow2 it is
    the oracle's unless amax / 448 is that close to a power of two, where it may be the neighbour. A code is the
    oracle's (for the scale that was given), or its neighbour where h / scale is within 2^-19 of the value halfway
    between the two (the errors of h and of the scale, the reciprocal and the product). Signs agree but at zero."""
    gate, up = np.split(np.asarray(gu, np.float64), 2, axis=1)
    h = oracle.silu(gate) * up
    rows, inner = h.shape
    want_codes, want_scales = oracle.quantize_block(h.astype(np.float32), 1, pow2)
    assert codes.shape == want_codes.shape and scales.shape == want_scales.shape
    rel = np.abs(scales.astype(np.float64) / want_scales - 1)
    if pow2:
        amax = np.stack([np.abs(h[:, j:j + 128]).max(1) for j in range(0, inner, 128)], 1)
        m, _ = np.frexp(amax / 448)
        near = np.minimum(np.abs(m * 2 - 1), np.abs(1 - m)) <= 2.0 ** -20
        factor = scales.astype(np.float64) / want_scales
        assert np.all((factor == 1) | (near & ((factor == 2) | (factor == 0.5)))), "scales"
    else:
        assert np.all(rel <= 2.0 ** -21 + 2.0 ** -23), "scales"
    s = np.repeat(scales.astype(np.float64), 128, axis=1)[:, :inner]
    q = h / s
    # where a power of two moved, the codes belong to the scale that was given
    want = np.where(np.repeat(rel > 2.0 ** -20, 128, axis=1)[:, :inner], oracle.e4m3_encode(np.clip(q, -448, 448)),
                    want_codes).astype(int)
    got = codes.astype(int)
    g, w = got & 127, want & 127
    assert np.all((g == w) | (np.abs(g - w) == 1)) and g.max() <= 126, "codes"
    half = (oracle.e4m3_decode(g.astype(np.uint8)) + oracle.e4m3_decode(w.astype(np.uint8))) / 2
    assert np.all((g == w) | (np.abs(np.abs(q) - half) <= 2.0 ** -19 * half)), "codes away from a boundary"
    assert np.all((got >> 7 == want >> 7) | (g == 0) & (w <= 1)), "signs"
