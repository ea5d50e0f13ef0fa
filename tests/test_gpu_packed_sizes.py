"""The 4-bit products at sizes that decide how a launch is laid out, against the
float64 oracle. Errors allowed as in test_gpu_packed.py: (K + 2 K / g + 8) *
2^-23 of the sum of |x s q| + |x b|, then one rounding to the type."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm
from tests._steps import DT, close, dev, routing
from tests.test_gpu_packed import FORMATS, on_device, sampled, tolerance, weights

pytestmark = pytest.mark.gpu


def some_columns(y, at):
    return y[:, torch.from_numpy(at).cuda()]


@pytest.mark.parametrize("fmt,group", [("affine", 64), ("mxfp4", 32)])
def test_short_contractions_of_more_results_than_a_grid_has_threads(fmt, group):
    """65600 x 66000 results of K = 64, 8.7 GB of bf16: a workgroup takes several rows of x."""
    M, N, K = 65600, 66000, 64
    rng = np.random.default_rng(group)
    x = torch.from_numpy(rng.standard_normal((M, K))).bfloat16()
    codes, s, b = weights(rng, (N,), K, fmt, group)
    y = qm.matmul_packed(x.cuda(), *on_device((codes, s, b)),
                         out=torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda"))
    assert all(torch.isfinite(part).all() for part in y.split(8192))
    at, rows = sampled(N), np.r_[np.arange(20), 65000:65080, M - 60:M]   # the second round of rows begins near 65000
    want, mag = oracle.matmul_packed(x[rows].double().numpy(), codes[at], s[at], None if b is None else b[at])
    close(some_columns(y[torch.from_numpy(rows).cuda()], at), want, tolerance(mag, K, group), "bf16")


@pytest.mark.parametrize("fmt,group", [("affine", 32), ("affine", 64), ("mxfp4", 32)])
def test_short_contractions_of_many_grouped_rows(fmt, group):
    """More rows than a grid has in y, a last workgroup of columns that ends inside a wave."""
    T, k, E, N, K = 17500, 4, 70, 300, 64
    rng, off, perm, _ = routing(group, T, k, E, 1.0)
    x = torch.from_numpy(rng.standard_normal((T, K))).to(torch.float16)
    codes, s, b = weights(rng, (E, N), K, fmt, group)
    y = qm.grouped_matmul_packed(x.cuda(), *on_device((codes, s, b)), dev(off), perm=dev(perm), top_k=k, x_order="token",
                                 out_dtype="f32", out=torch.full((T * k, N), float("nan"), device="cuda"))
    rows = oracle.source_rows(x.double().numpy(), "token", perm, k)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        want, mag = oracle.matmul_packed(rows[r], codes[e], s[e], None if b is None else b[e])
        close(y[r], want, tolerance(mag, K, group), "f32")
