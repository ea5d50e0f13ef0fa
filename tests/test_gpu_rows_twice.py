"""Rows of y that two assignments name: combine_rows counts them for each, and of
its gradient every element of dy's row is one of the two gradients' (which one is
not specified), while dw and the other rows are as ever."""
import numpy as np
import pytest
import torch

import quantized_sparse_moe_amd as qm
from tests._steps import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,d", [(40, 3, 65), (61, 4, 4100), (700, 2, 1003)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_named_twice(T, k, d, dtype):
    """Small integers, so that every sum and product is exact."""
    rng = np.random.default_rng(d)
    n = T * k
    positions = rng.permutation(n).astype(np.int32)
    twice = rng.choice(n, 10, replace=False).reshape(5, 2)
    positions[twice[:, 1]] = positions[twice[:, 0]]
    y, dout = rng.integers(-4, 5, (n, d)).astype(np.float32), rng.integers(-4, 5, (T, d)).astype(np.float32)
    w = rng.integers(-3, 4, (T, k)).astype(np.float32)
    args = dev(y, dtype), dev(w), dev(positions)
    want = (w[:, :, None] * y[positions].reshape(T, k, d)).sum(1)
    assert np.array_equal(qm.combine_rows(*args, out_dtype="f32").cpu().numpy(), want)
    dy, dw = qm.combine_rows_grad(dev(dout, dtype), *args, out=torch.full((n, d), 99.0, dtype=dtype, device="cuda"))
    assert np.array_equal(dw.cpu().numpy(), (dout[:, None] * y[positions].reshape(T, k, d)).sum(2))
    grads = w.reshape(-1)[:, None] * dout.repeat(k, 0)
    dy = dy.float().cpu().numpy()
    once = np.setdiff1d(np.arange(n), twice.reshape(-1))
    assert np.array_equal(dy[positions[once]], grads[once])
    for a, b in twice:
        row = dy[positions[a]]
        assert ((row == grads[a]) | (row == grads[b])).all()
    assert (dy[np.setdiff1d(np.arange(n), positions)] == 99).all()
