"""The 4-bit products at sizes that decide how a launch is laid out, against the
float64 oracle. Errors allowed as in test_gpu_packed.py: (K + 2 K / g + 8) *
2^-23 of the sum of |x s q| + |x b|, then one rounding to the type."""
import os
import re

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


# The kernel that each size reaches goes by these: rows of x, tiles of 16 rows of the matrix, workgroups.
RULE = {"kFewRows": 20, "kSmallTiles": 512, "kEnoughGroups": 192}
TILES = [  # M, N, K: 21 to 32 rows and 192 tiles of 256 columns: 32 rows by 256 columns, no shared contraction
    (21, 50000, 256), (32, 49200, 672), (27, 48900, 1184),
]
STREAMS = [  # up to 20 rows and more than 512 tiles, x in several segments, rows of scales that end inside a block
    (7, 9001, 8160), (12, 9000, 7072), (15, 8300, 8160), (8, 8209, 4096),
]


def test_the_sizes_here_fit_the_rule():
    """A changed rule may lead these sizes to other kernels: choose sizes for the ones they are meant for again."""
    with open(os.path.join(os.path.dirname(qm.__file__), "csrc", "product_packed.hip")) as f:
        source = f.read()
    for name, value in RULE.items():
        assert re.search(rf"\b{name} = (\d+)", source).group(1) == str(value), name
    assert all(M > RULE["kFewRows"] and -(-N // 256) >= RULE["kEnoughGroups"] for M, N, _ in TILES)
    assert all(M <= RULE["kFewRows"] and -(-N // 16) > RULE["kSmallTiles"] for M, N, _ in STREAMS)


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("M,N,K", TILES + STREAMS)
def test_wide_matrices(fmt, group, dtype, out, M, N, K):
    K -= K % group
    rng = np.random.default_rng(M + N + K)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(DT[dtype])
    codes, s, b = weights(rng, (N,), K, fmt, group)
    y = qm.matmul_packed(x.cuda(), *on_device((codes, s, b)), out=torch.full((M, N), float("nan"), dtype=DT[out], device="cuda"))
    assert torch.isfinite(y).all()
    at = sampled(N)
    want, mag = oracle.matmul_packed(x.double().numpy(), codes[at], s[at], None if b is None else b[at])
    close(some_columns(y, at), want, tolerance(mag, K, group), out)


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("orders", [("token", "bucket"), ("bucket", "slot")], ids="-".join)
def test_many_buckets_of_two_tiles_of_rows(fmt, group, orders):
    """200 experts with 22 rows on average, up to several times that: tiles of 32 rows by 256 columns."""
    T, k, E, N, K = 1100, 4, 200, 300, 416
    K -= K % group
    rng, off, perm, _ = routing(group, T, k, E, 0.5)
    x = torch.from_numpy(rng.standard_normal((T if orders[0] == "token" else T * k, K))).to(torch.bfloat16)
    codes, s, b = weights(rng, (E, N), K, fmt, group)
    y = qm.grouped_matmul_packed(x.cuda(), *on_device((codes, s, b)), dev(off), perm=dev(perm), top_k=k, x_order=orders[0],
                                 out_order=orders[1], out=torch.full((T * k, N), float("nan"), device="cuda"))
    assert torch.isfinite(y).all()
    if orders[1] == "slot":
        y = y[dev(perm).long()]
    rows, at = oracle.source_rows(x.double().numpy(), orders[0], perm, k), sampled(N)
    for e in [*np.argsort(-np.diff(off))[:6], *rng.integers(0, E, 20), E - 1]:
        r = slice(off[e], off[e + 1])
        want, mag = oracle.matmul_packed(rows[r], codes[e][at], s[e][at], None if b is None else b[e][at])
        close(some_columns(y[r], at), want, tolerance(mag, K, group), "f32")
