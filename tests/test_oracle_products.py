"""Pins of the oracle's block-scaled FP8 quantiser and grouped products, on the CPU."""
import numpy as np
import pytest
import torch

import oracle


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
