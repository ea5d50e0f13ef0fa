"""Pins of the oracle's block-scaled FP8 quantiser and grouped products, on the CPU."""
import numpy as np
import pytest
import torch

import oracle
from tests._quant import check_swiglu


def test_e4m3_encode_inverts_decode_and_rounds_to_even():
    codes = np.concatenate([np.arange(127), 128 + np.arange(127)]).astype(np.uint8)
    assert np.array_equal(oracle.e4m3_encode(oracle.e4m3_decode(codes)), codes)
    v = oracle.e4m3_decode(np.arange(127, dtype=np.uint8))
    mid = (v[:-1] + v[1:]) / 2
    got = oracle.e4m3_encode(mid)
    assert np.array_equal(got, np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127)))
    assert np.array_equal(oracle.e4m3_encode(mid * (1 - 1e-9)), np.arange(126))
    assert np.array_equal(oracle.e4m3_encode(mid * (1 + 1e-9)), np.arange(1, 127))


def test_e4m3_encode_matches_torch():
    x = torch.randn(20000, generator=torch.Generator().manual_seed(3)) * 60
    x = x.clamp(-448, 448)
    assert np.array_equal(oracle.e4m3_encode(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_block_error_and_scales(block_rows, pow2):
    rng = np.random.default_rng(7)
    x = (rng.standard_normal((130, 272)) * np.exp(rng.standard_normal(272))).astype(np.float32)
    codes, scales = oracle.quantize_block(x, block_rows, pow2)
    d = oracle.dequant_block(codes, scales, block_rows)
    s = np.repeat(np.repeat(scales, block_rows, 0)[:130], 128, 1)[:, :272].astype(np.float64)
    # half a step of e4m3 relative to the value, or of its subnormals (2^-9) times the scale, and fp32 roundings
    assert np.all(np.abs(d - x) <= np.maximum(np.abs(x) * (2.0 ** -4 + 2.0 ** -22), s * 2.0 ** -10 * (1 + 2.0 ** -22)))
    if pow2:
        m, _ = np.frexp(scales)
        assert np.all(m == 0.5)
    b = np.abs(d[:block_rows, :128]).max()
    assert b <= np.abs(x[:block_rows, :128]).max() * (1 + 2.0 ** -4)


def test_quantize_block_special_blocks():
    x = np.zeros((4, 256), np.float32)
    x[1, 5] = np.inf
    x[2, 200] = np.nan
    x[3, :] = 448 * 2.0 ** -3
    codes, scales = oracle.quantize_block(x, 1, True)
    assert scales[0, 0] == np.float32(2.0 ** -126) and not codes[0].any()
    assert np.isnan(scales[1, 0]) and scales[1, 1] == np.float32(2.0 ** -126)
    assert np.isnan(scales[2, 1]) and not codes[2].any()
    assert np.all(scales[3] == 2.0 ** -3) and np.all(codes[3] == 126)


def test_grouped_products_against_loops_and_differences():
    rng = np.random.default_rng(9)
    off = np.array([0, 3, 3, 7])
    x, w, dy = rng.standard_normal((7, 4)), rng.standard_normal((3, 5, 4)), rng.standard_normal((7, 5))
    y, _ = oracle.grouped_matmul(x, w, off)
    expert = [0, 0, 0, 2, 2, 2, 2]
    for p in range(7):
        assert np.allclose(y[p], w[expert[p]] @ x[p])
    # the product is linear in x and in w, so a difference of any size gives the gradient
    dw, _ = oracle.grouped_matmul_dw(x, dy, off)
    dx, _ = oracle.grouped_matmul(dy, w.transpose(0, 2, 1), off)
    for _ in range(4):
        tw, tx = rng.standard_normal(w.shape), rng.standard_normal(x.shape)
        assert np.isclose(((oracle.grouped_matmul(x, w + tw, off)[0] - y) * dy).sum(), (dw * tw).sum())
        assert np.isclose(((oracle.grouped_matmul(x + tx, w, off)[0] - y) * dy).sum(), (dx * tx).sum())
    assert not dw[1].any()


def _swiglu_inputs(rows, inner, seed):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((rows, 2 * inner)) * np.exp(rng.standard_normal(2 * inner))).astype(np.float32)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,inner", [(1, 16), (6, 2048), (33, 272)])
def test_swiglu_check_accepts_the_oracle_and_refuses_mistakes(rows, inner, pow2):
    """The value-by-value check of the SwiGLU quantiser: scales off by a factor of two (with any codes), other codes,
    a few flipped signs or codes one step away are all refused."""
    gu = _swiglu_inputs(rows, inner, rows)
    codes, scales = oracle.swiglu_quantize_block(gu, pow2)
    check_swiglu(codes, scales, gu, pow2)
    rng = np.random.default_rng(1)
    big = np.argmax(np.abs(codes.astype(int) & 127))
    flipped, stepped = codes.copy(), codes.copy()
    flipped.flat[big] ^= 0x80
    stepped.flat[big] -= 1
    one_block = scales.copy()
    one_block[0, 0] *= 2
    wrong = [(np.zeros_like(codes), scales * 2), (codes, scales * 2), (codes, scales / 2), (codes, one_block),
             (rng.integers(0, 127, codes.shape).astype(np.uint8), scales / 2), (flipped, scales), (stepped, scales),
             (np.zeros_like(codes), scales), (codes, scales * np.float32(1 + 2.0 ** -18))]
    for c, s in wrong:
        with pytest.raises(AssertionError):
            check_swiglu(c, s, gu, pow2)


def test_swiglu_check_allows_a_power_of_two_only_where_it_is_near():
    """amax / 448 a power of two up to the last bits: either scale is right, with its own codes; a code on a boundary
    may be either neighbour."""
    gu = np.zeros((1, 32), np.float32)
    gu[0, :16], gu[0, 16:] = 60.0, np.arange(16) / 60         # silu(60) = 60 but for e^-60
    gu[0, 31] = np.float32(448) / np.float32(60)              # 448 up to a rounding
    codes, scales = oracle.swiglu_quantize_block(gu, True)
    check_swiglu(codes, scales, gu, True)
    h = (gu[0, :16] * gu[0, 16:]).astype(np.float64)
    for s in (1.0, 2.0):
        check_swiglu(oracle.e4m3_encode(np.clip(h / s, -448, 448))[None], np.full((1, 1), s, np.float32), gu, True)
    with pytest.raises(AssertionError):
        check_swiglu(oracle.e4m3_encode(h / 4)[None], np.full((1, 1), 4.0, np.float32), gu, True)
