"""The 4-bit products against the float64 oracle: every format, group, type,
order, row counts from one up, odd numbers of rows of the matrix, contractions
that end inside a chunk, empty and long buckets, masked neighbours with NaN.

Error allowed (computed in the test): out = sum over groups of s * (sum x q) + b *
(sum x), all in fp32 with rounding or truncation at each step, so (K + 2 K / g + 8)
* 2^-23 of the sum of |x s q| + |x b| (oracle.packed_weights' magnitude); then one
rounding to the type. Integers small enough to be exact are compared for equality."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm
from tests._steps import DT, close, dev, routing

pytestmark = pytest.mark.gpu

FORMATS = [("affine", 32), ("affine", 64), ("affine", 128), ("mxfp4", 32)]


def weights(rng, lead, K, fmt, group):
    """(codes uint32, scales, biases) of random codes."""
    codes = rng.integers(0, 1 << 32, (*lead, K // 8), dtype=np.uint64).astype(np.uint32)
    shape = (*lead, K // group)
    if fmt == "mxfp4":
        return codes, rng.integers(115, 125, shape).astype(np.uint8), None
    s = (np.exp(0.5 * rng.standard_normal(shape)) * 0.01).astype(np.float16)
    return codes, s, (-7.5 * s * (1 + 0.3 * rng.standard_normal(shape))).astype(np.float16)


def on_device(w):
    codes, s, b = w
    return dev(codes.view(np.int32)), dev(s), None if b is None else dev(b)


def tolerance(mag, K, group):
    return (K + 2 * K // group + 8) * 2.0 ** -23 * mag


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64, 65, 130])
def test_rows_of_x(fmt, group, M):
    rng = np.random.default_rng(M + group)
    for dtype, N, K in (("bf16", 37, 640), ("f16", 200, 384)):
        x = torch.from_numpy(rng.standard_normal((M, K))).to(DT[dtype])
        w = weights(rng, (N,), K, fmt, group)
        want, mag = oracle.matmul_packed(x.double().numpy(), *w)
        for out in (None, "f32"):
            y = qm.matmul_packed(x.cuda(), *on_device(w), out_dtype=out)
            assert y.shape == (M, N) and y.dtype == DT[out or dtype]
            close(y, want, tolerance(mag, K, group), out or dtype)


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("N", [1, 15, 16, 17, 128, 1000, 4099])
def test_rows_of_the_matrix(fmt, group, N):
    rng = np.random.default_rng(N + group)
    for M, K, out in ((1, 1024, "bf16"), (7, 256, "f16")):
        x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16)
        w = weights(rng, (N,), K, fmt, group)
        want, mag = oracle.matmul_packed(x.double().numpy(), *w)
        close(qm.matmul_packed(x.cuda(), *on_device(w), out_dtype=out), want, tolerance(mag, K, group), out)


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("groups", [1, 2, 3, 5, 7, 13, 31, 63, 101])
def test_contractions_that_end_anywhere(fmt, group, groups):
    rng = np.random.default_rng(groups)
    K = group * groups
    for M, N, dtype in ((1, 50, "f16"), (13, 33, "bf16"), (40, 20, "f16")):
        x = torch.from_numpy(rng.standard_normal((M, K))).to(DT[dtype])
        w = weights(rng, (N,), K, fmt, group)
        want, mag = oracle.matmul_packed(x.double().numpy(), *w)
        close(qm.matmul_packed(x.cuda(), *on_device(w), out_dtype="f32"), want, tolerance(mag, K, group), "f32")


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_code_at_every_place(fmt, group, dtype):
    """Unit rows of x pick single weights: each must be its value, exactly (affine with integer scale and bias)."""
    K, N = 128, 16
    codes = np.array([[(n + k) % 16 for k in range(K)] for n in range(N)])
    words = np.zeros((N, K // 8), np.uint32)
    for j in range(8):
        words |= codes[:, j::8].astype(np.uint32) << np.uint32(4 * j)
    rng = np.random.default_rng(0)
    if fmt == "mxfp4":
        w = (words, rng.integers(120, 134, (N, K // group)).astype(np.uint8), None)
    else:
        w = (words, rng.integers(1, 9, (N, K // group)).astype(np.float16), rng.integers(-60, 60, (N, K // group)).astype(np.float16))
    y = qm.matmul_packed(torch.eye(K, device="cuda", dtype=DT[dtype]), *on_device(w), out_dtype="f32")
    assert np.array_equal(y.cpu().numpy().T, oracle.packed_weights(*w)[0])


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_integers_are_exact(fmt, group):
    """Codes, scales, biases and x small integers: every sum is one below 2^24."""
    rng = np.random.default_rng(1)
    M, N, K = 21, 70, 1152
    x = rng.integers(-3, 4, (M, K)).astype(np.float32)
    codes = rng.integers(0, 1 << 32, (N, K // 8), dtype=np.uint64).astype(np.uint32)
    if fmt == "mxfp4":
        w = (codes, rng.integers(127, 131, (N, K // group)).astype(np.uint8), None)     # values to 48
    else:
        w = (codes, rng.integers(-3, 4, (N, K // group)).astype(np.float16), rng.integers(-40, 40, (N, K // group)).astype(np.float16))
    want, _ = oracle.matmul_packed(x, *w)
    y = qm.matmul_packed(dev(x, torch.bfloat16), *on_device(w), out_dtype="f32")
    assert np.array_equal(y.double().cpu().numpy(), want)


GROUPED = [  # T, k, E, N, K
    (1, 1, 1, 16, 128), (1, 6, 256, 136, 256), (1, 8, 9, 40, 1024), (5, 2, 7, 33, 384), (33, 4, 9, 64, 256),
    (97, 6, 64, 48, 128), (130, 3, 16, 100, 384), (300, 4, 5, 32, 256), (12, 6, 600, 20, 128),
]
ORDERS = [("bucket", "bucket"), ("token", "bucket"), ("bucket", "slot"), ("slot", "slot"), ("token", "slot")]


@pytest.mark.parametrize("shape", GROUPED, ids=str)
@pytest.mark.parametrize("orders", ORDERS, ids="-".join)
def test_grouped(shape, orders):
    T, k, E, N, K = shape
    rng, off, perm, _ = routing(sum(shape), T, k, E, 1.0)
    for fmt, group in FORMATS:
        dtype = ["bf16", "f16"][rng.integers(2)]
        out = ["f32", dtype][rng.integers(2)]
        x = torch.from_numpy(rng.standard_normal((T if orders[0] == "token" else T * k, K))).to(DT[dtype])
        w = weights(rng, (E, N), K, fmt, group)
        rows = oracle.source_rows(x.double().numpy(), orders[0], perm, k)
        want, mag = np.empty((T * k, N)), np.empty((T * k, N))
        for e in range(E):
            s = slice(off[e], off[e + 1])
            if off[e + 1] > off[e]:
                want[s], mag[s] = oracle.matmul_packed(rows[s], w[0][e], w[1][e], None if w[2] is None else w[2][e])
        if orders[1] == "slot":
            want, mag = want[np.argsort(perm)], mag[np.argsort(perm)]
        codes, s, b = on_device(w)
        y = qm.grouped_matmul_packed(x.cuda(), codes, s, b, dev(off), perm=dev(perm), top_k=k, x_order=orders[0],
                                     out_order=orders[1], out_dtype=out,
                                     out=torch.full((T * k, N), float("nan"), dtype=DT[out], device="cuda"))
        assert y.shape == (T * k, N)
        close(y, want, tolerance(mag, K, group), out)


def sampled(N):
    """Rows of a matrix of N: the first, the last and some between."""
    rng = np.random.default_rng(N)
    return np.unique(np.r_[np.arange(min(N, 20)), np.arange(max(N - 35, 0), N), rng.integers(0, N, 60)])


LARGE = [  # M, N, K (a multiple of every group, or of the smaller ones): more than 512 tiles of 16 rows
    (1, 8209, 4096), (1, 20000, 640), (1, 8209, 160), (2, 8300, 2208), (4, 8209, 1088), (5, 8209, 2976), (8, 9001, 8192),
    (9, 8209, 544), (16, 8209, 8192), (16, 8400, 3104), (13, 8209, 128), (17, 12500, 672), (20, 50000, 256), (33, 13000, 1184),
    (40, 3000, 2080), (64, 49200, 160), (65, 12400, 320), (150, 5000, 544),
]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_matrices(fmt, group, M, N, K):
    """Whole waves of tiles, contractions that end inside a step, a block of scales or a segment of x; sampled rows of
    the matrix against the oracle, and every result finite and written."""
    K -= K % group
    rng = np.random.default_rng(M + N + K)
    dtype, out = (("bf16", "f32"), ("f16", "f16"))[rng.integers(2)]
    x = torch.from_numpy(rng.standard_normal((M, K))).to(DT[dtype])
    codes, s, b = weights(rng, (N,), K, fmt, group)
    y = qm.matmul_packed(x.cuda(), *on_device((codes, s, b)), out=torch.full((M, N), float("nan"), dtype=DT[out], device="cuda"))
    assert torch.isfinite(y).all()
    at = sampled(N)
    want, mag = oracle.matmul_packed(x.double().numpy(), codes[at], s[at], None if b is None else b[at])
    close(y[:, torch.from_numpy(at).cuda()], want, tolerance(mag, K, group), out)


MANY_BUCKETS = [  # T, k, E, N, K, skew: few rows a bucket over many tiles, long buckets among them, tiles of rows
    (3, 2, 300, 1500, 160, 0.0), (40, 4, 64, 160, 608, 1.5), (30, 8, 40, 300, 1120, 2.5), (100, 4, 256, 16, 352, 0.0),
    (60, 5, 100, 80, 736, 0.3), (64, 6, 32, 300, 2048, 0.5), (300, 4, 40, 272, 416, 1.0), (512, 2, 8, 130, 288, 0.5),
    (200, 3, 1000, 50, 192, 0.1),
]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("T,k,E,N,K,skew", MANY_BUCKETS)
def test_many_buckets(fmt, group, T, k, E, N, K, skew):
    K -= K % group
    rng, off, perm, _ = routing(T + N, T, k, E, skew)
    orders = ORDERS[rng.integers(len(ORDERS))]
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
        close(y[r][:, torch.from_numpy(at).cuda()], want, tolerance(mag, K, group), "f32")


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("T,k,E,N", [(1, 6, 8, 1500), (1, 40, 4, 3000), (2, 9, 5, 2100), (3, 5, 24, 800), (5, 7, 16, 600)])
@pytest.mark.parametrize("one", [False, True])
def test_buckets_longer_than_there_are_tokens(fmt, group, T, k, E, N, one):
    """An expert named several times by one token, or by every assignment: more rows than a run is expected to hold."""
    rng = np.random.default_rng(31 * T + k)
    K = 640
    ids = np.full(T * k, E // 2) if one else rng.integers(0, E, T * k)
    off = np.r_[0, np.cumsum(np.bincount(ids, minlength=E))].astype(np.int32)
    perm = np.argsort(ids, kind="stable").astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((T, K))).to(torch.bfloat16)
    codes, s, b = weights(rng, (E, N), K, fmt, group)
    y = qm.grouped_matmul_packed(x.cuda(), *on_device((codes, s, b)), dev(off), perm=dev(perm), top_k=k, x_order="token",
                                 out=torch.full((T * k, N), float("nan"), device="cuda"))
    assert torch.isfinite(y).all()
    rows, at = oracle.source_rows(x.double().numpy(), "token", perm, k), sampled(N)
    for e in np.unique(ids):
        r = slice(off[e], off[e + 1])
        want, mag = oracle.matmul_packed(rows[r], codes[e][at], s[e][at], None if b is None else b[e][at])
        close(y[r][:, torch.from_numpy(at).cuda()], want, tolerance(mag, K, group), "f32")


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_scales_behind_a_row_are_not_its_own(fmt, group):
    """Every second row's scales are no numbers: the rows between, whose blocks of scales reach into them, are as
    without."""
    N, K = 9000, 17 * 128 if group == 128 else 1120
    K -= K % group
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((3, K))).to(torch.bfloat16).cuda()
    codes, s, b = weights(rng, (N,), K, fmt, group)
    clean = qm.matmul_packed(x, *on_device((codes, s, b)), out_dtype="f32")
    s[1::2] = 255 if fmt == "mxfp4" else np.nan
    y = qm.matmul_packed(x, *on_device((codes, s, b)), out_dtype="f32")
    assert torch.equal(y[:, ::2], clean[:, ::2]) and torch.isnan(y[:, 1::2]).all()


def test_quantize_affine_feeds_it():
    """The framework's own converter, its int16 bit patterns passed on as they come."""
    g = torch.Generator().manual_seed(0)
    wt = (torch.randn(96, 512, generator=g) * 0.05).bfloat16()
    x = torch.randn(3, 512, generator=g).bfloat16()
    codes, s, b = qm.quantize_affine(wt.cuda(), bits=4, group=64)
    y = qm.matmul_packed(x.cuda(), codes, s, b, out_dtype="f32")
    want, mag = oracle.matmul_packed(x.double().numpy(), codes.cpu().numpy().view(np.uint32),
                                     s.cpu().numpy().view(np.float16), b.cpu().numpy().view(np.float16))
    close(y, want, tolerance(mag, 512, 64), "f32")
    assert torch.equal(y, qm.matmul_packed(x.cuda(), codes, s.view(torch.float16), b.view(torch.float16), out_dtype="f32"))


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("T", [3, 90])
def test_rows_of_no_bucket_stay_and_nan_does_not_leak(fmt, group, T):
    """The first and last positions belong to no bucket: their rows of x hold NaN, their rows of out stay. So do
    experts without a position hold NaN scales. One row of x with NaN spoils its own results only."""
    k, E, N, K = 4, 6, 40, 640
    rng = np.random.default_rng(T)
    n = T * k
    lo, hi = n // 4, n - n // 4
    off = np.array([lo, lo, lo + 2, (lo + hi) // 2, hi, hi, hi], np.int32)[:E + 1]
    x = torch.from_numpy(rng.standard_normal((n, K))).to(torch.bfloat16)
    x[:lo], x[hi:] = float("nan"), float("inf")
    x[lo + 1, 5] = float("nan")
    codes, s, b = weights(rng, (E, N), K, fmt, group)
    for e in range(E):
        if off[e + 1] == off[e]:
            if fmt == "mxfp4":
                s[e] = 255
            else:
                s[e] = np.nan
    out = torch.full((n, N), 7.0, device="cuda")
    y = qm.grouped_matmul_packed(x.cuda(), *on_device((codes, s, b)), dev(off), out=out).cpu()
    assert (y[:lo] == 7).all() and (y[hi:] == 7).all() and torch.isnan(y[lo + 1]).all()
    keep = [p for p in range(lo, hi) if p != lo + 1]
    assert torch.isfinite(y[keep]).all()
    for e in range(E):
        rows = [p for p in keep if off[e] <= p < off[e + 1]]
        if rows:
            want, mag = oracle.matmul_packed(x[rows].double().numpy(), codes[e], s[e], None if b is None else b[e])
            close(y[rows], want, tolerance(mag, K, group), "f32")


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_values_that_are_not_finite(fmt, group):
    """A row of x with an infinity gives values that are not finite, a scale that is none reaches its row of the matrix
    only; the results next to them are those without it."""
    M, N, K = 6, 40, 384
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.float16)
    w = weights(rng, (N,), K, fmt, group)
    clean = qm.matmul_packed(x.cuda(), *on_device(w), out_dtype="f32")
    x[2, 100] = float("inf")
    y = qm.matmul_packed(x.cuda(), *on_device(w), out_dtype="f32")
    rest = [0, 1, 3, 4, 5]
    assert not torch.isfinite(y[2]).any() and torch.equal(y[rest], clean[rest])
    w[1][7, 1] = 255 if fmt == "mxfp4" else np.nan
    y = qm.matmul_packed(x.cuda(), *on_device(w), out_dtype="f32")
    cols = [n for n in range(N) if n != 7]
    assert torch.isnan(y[:, 7]).all() and torch.equal(y[rest][:, cols], clean[rest][:, cols])


def test_the_smallest_and_largest_mxfp4_scales():
    """Scale bytes 0 (2^-127) and 254 (2^127) are exact powers of two."""
    K, N = 32, 16
    codes = np.full((N, K // 8), 0x22222222, np.uint32)                   # every value 1
    x = torch.zeros(1, K, dtype=torch.bfloat16)
    x[0, 3] = 0.5
    for byte, want in ((0, 2.0 ** -128), (1, 2.0 ** -127), (254, 2.0 ** 126), (127, 0.5)):
        s = np.full((N, 1), byte, np.uint8)
        y = qm.matmul_packed(x.cuda(), *on_device((codes, s, None)), out_dtype="f32")
        assert (y.double() == want).all(), byte


@pytest.mark.parametrize("T", [6, 200])
def test_bad_perm_entries_are_reported_and_write_nothing(T):
    k, E, N, K = 2, 4, 24, 128
    rng, off, perm, _ = routing(3, T, k, E)
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16().cuda()
    w = on_device(weights(rng, (E, N), K, "affine", 32))
    kw = dict(top_k=k, x_order="token", out_order="slot", out_dtype="f32")
    good = qm.grouped_matmul_packed(x, *w, dev(off), perm=dev(perm), **kw)
    for bad in (-1, T * k, 2 ** 31 - 1, -2 ** 31):
        p = perm.copy()
        at = p[5]
        p[5] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((T * k, N), 7.0, device="cuda")
        qm.grouped_matmul_packed(x, *w, dev(off), perm=dev(p), out=out, err=err, **kw)
        assert err.item() == 16 and (out[at] == 7).all()
        rest = [i for i in range(T * k) if i != at]
        assert torch.equal(out[rest], good[rest])
        qm.grouped_matmul_packed(x, *w, dev(off), perm=dev(p), **kw)


def test_offsets_are_clamped():
    T, E, N, K = 20, 3, 16, 64
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16().cuda()
    w = on_device(weights(rng, (E, N), K, "affine", 64))
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    qm.grouped_matmul_packed(x, *w, dev(np.array([-5, 8, 6, 1000], np.int32)), out=out)
    want = torch.full_like(out, 7.0)
    want[:8] = qm.matmul_packed(x[:8], w[0][0], w[1][0], w[2][0])
    want[6:] = qm.matmul_packed(x[6:], w[0][2], w[1][2], w[2][2])
    assert torch.equal(out[8:], want[8:]) and torch.equal(out[:6], want[:6])


def test_empty_calls_and_refusals():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    c, s, off = z(3, 8, 8, d=torch.int32), z(3, 8, 1, d=torch.float16), z(4, d=torch.int32)
    assert qm.matmul_packed(z(0, 64), c[0], s[0], s[0]).shape == (0, 8)
    assert qm.matmul_packed(z(2, 64), c[0, :0], s[0, :0], s[0, :0]).shape == (2, 0)
    assert qm.grouped_matmul_packed(z(0, 64), c, s, s, off).shape == (0, 8)
    out = torch.full((4, 8), 7.0, device="cuda")
    assert (qm.grouped_matmul_packed(z(4, 64), c, s, s, off, out=out) == 7).all()
    for call in (lambda: qm.matmul_packed(z(2, 72), c[0], s[0], s[0]), lambda: qm.matmul_packed(z(2, 0), c[0, :, :0], s[0], s[0]),
                 lambda: qm.matmul_packed(z(2, 128), c[0], s[0], s[0]), lambda: qm.matmul_packed(z(2, 64), c[0], s[1:, 0], s[0]),
                 lambda: qm.matmul_packed(z(2, 64), c[0], s[0].expand(8, 3).contiguous(), s[0]),
                 lambda: qm.matmul_packed(z(2, 64), c[0], s[0, :7], s[0]), lambda: qm.matmul_packed(z(2, 64), c[0], s[0], s[0, :7]),
                 lambda: qm.matmul_packed(z(2, 64), c[0], s[0, :, :0], s[0]),
                 lambda: qm.matmul_packed(z(2, 128)[:, :64], c[0], s[0], s[0]), lambda: qm.matmul_packed(z(2, 64), c[0], s[0], s[0], out=z(2, 7)),
                 lambda: qm.grouped_matmul_packed(z(4, 64), c, s, s, off[:3]), lambda: qm.grouped_matmul_packed(z(5, 64), c, s, s, off, top_k=2),
                 lambda: qm.grouped_matmul_packed(z(4, 64), c, s[:2], s, off), lambda: qm.grouped_matmul_packed(z(4, 64), c, s, s, off, x_order="x")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: qm.matmul_packed(z(2, 64), c[0].short(), s[0], s[0]), lambda: qm.matmul_packed(z(2, 64), c[0], s[0]),
                 lambda: qm.matmul_packed(z(2, 64), c[0], s[0].float(), s[0]), lambda: qm.matmul_packed(z(2, 64), c[0], s[0], s[0].float()),
                 lambda: qm.grouped_matmul_packed(z(4, 64), c, s, s, off.long())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: qm.matmul_packed(z(2, 64), c[0], s[0].expand(8, 4).contiguous(), s[0].expand(8, 4).contiguous()),
                 lambda: qm.grouped_matmul_packed(z(4, 64), c, s, s, off, x_order="slot"),
                 lambda: qm.grouped_matmul_packed(z(4, 64), c, s, s, off, out_order="token")):
        with pytest.raises(qm.MoeError):
            call()


def test_weights_past_32_bits():
    """More than 2^32 bytes of codes; an expert at the far end and one at the front."""
    E, N, K = 600, 4096, 4096                                              # 5.0 GB of codes
    codes = torch.zeros(E, N, K // 8, dtype=torch.int32, device="cuda")
    s = torch.ones(E, N, K // 128, dtype=torch.float16, device="cuda")
    b = torch.zeros_like(s)
    codes[-1], codes[0] = 0x11111111, 0x22222222
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:], off[-1] = 1, 3
    x = torch.ones(3, K, dtype=torch.bfloat16, device="cuda")
    y = qm.grouped_matmul_packed(x, codes, s, b, off, out_dtype="f32")
    assert (y[0] == 2 * K).all() and (y[1:] == K).all()
