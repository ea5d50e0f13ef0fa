"""The block-scaled FP8 product and the products grouped by expert against the
float64 oracle: every type, order and direction, from one row up, ragged and
empty buckets, tails of every kind, masked neighbours that hold NaN, rows of no
bucket left as they were, bad perm entries, graph replays, streams; gradients
against the formula and against differences; and whole runs of them together.

Tolerance of a product of length Q (computed in the test, not tuned): summed in
fp32 in any order with rounding or truncation at each step, |error| <= (Q + 4) *
2^-23 * sum |products|; plus half a step of the output type relative to the
value, and the smallest subnormal's half step for fp16. FP8 with a 16-bit output:
the matrix instruction sums 8 neighbouring products with 13 bits below the
largest, so each of the other 7 loses less than 2^-13 of it, which all groups
together bound by 7 * 2^-13 * sum |products|. Integer inputs small
enough to be exact at every step are compared for equality."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm
from quantized_sparse_moe_amd import _lib

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def close(got, want, mag, Q, out, fp8=False):
    got = got.double().cpu().numpy()
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[out]
    tol = (Q + 4) * 2.0 ** -23 * mag * (1 + half) + half * np.abs(want) + (2.0 ** -25 if out == "f16" else 0.0)
    if fp8 and out != "f32":
        tol = tol + 7 * 2.0 ** -13 * mag * (1 + half)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def buckets(seed, T, k, E, kind):
    """offsets, perm of T tokens' distinct experts: "even", "skew" (few popular experts), "one" (the last k experts
    take everything, the others are empty)."""
    rng = np.random.default_rng(seed)
    w = {"even": np.ones(E), "skew": 1.0 / np.arange(1, E + 1) ** 1.5, "one": np.r_[np.zeros(E - k), np.ones(k)]}[kind]
    ids = np.argsort(-(np.log(np.maximum(w, 1e-30)) + rng.gumbel(size=(T, E))), axis=1)[:, :k].reshape(-1)
    perm = np.argsort(ids, kind="stable").astype(np.int32)
    off = np.r_[0, np.cumsum(np.bincount(ids, minlength=E))].astype(np.int32)
    return off, perm


def ints(rng, *shape, top=4):
    return rng.integers(-top, top + 1, size=shape).astype(np.float32)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


SHAPES = [  # T, k, E, N, K, kind
    (1, 1, 1, 8, 16, "even"), (1, 6, 256, 136, 272, "even"), (5, 2, 7, 72, 144, "skew"), (2, 8, 8, 264, 1040, "even"),
    (33, 4, 9, 264, 400, "one"), (97, 6, 64, 128, 256, "skew"), (130, 3, 16, 520, 128, "skew"),
    (257, 1, 3, 256, 528, "one"), (300, 4, 8, 512, 512, "even"), (700, 2, 5, 776, 656, "skew"),
    (1500, 1, 4, 264, 272, "skew"),
]
ORDERS = [("bucket", "bucket"), ("token", "bucket"), ("bucket", "slot"), ("slot", "slot"), ("token", "slot")]


def place(y, out_order, perm):
    """y (bucket order) as the call lays it out."""
    if out_order == "bucket":
        return y
    z = np.empty_like(y)
    z[perm] = y
    return z


def case_seed(*key):
    return int(np.random.SeedSequence([hash_part(k) for k in key]).generate_state(1)[0])


def hash_part(k):
    return k if isinstance(k, int) else int.from_bytes(str(k).encode(), "little") % (1 << 60)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("orders", ORDERS, ids="-".join)
@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_matmul(shape, orders, transposed):
    T, k, E, N, K, kind = shape
    rng = np.random.default_rng(case_seed(*shape, *orders, int(transposed)))
    off, perm = buckets(T + E, T, k, E, kind)
    dtype = ["bf16", "f16"][rng.integers(2)]
    out = ["f32", dtype][rng.integers(2)]
    Q, C = (N, K) if transposed else (K, N)
    x = torch.from_numpy(rng.standard_normal((T if orders[0] == "token" else T * k, Q))).to(DT[dtype])
    w = torch.from_numpy(rng.standard_normal((E, N, K)) * Q ** -0.5).to(DT[dtype])
    y = qm.grouped_matmul(x.cuda(), w.cuda(), dev(off), perm=dev(perm), top_k=k, x_order=orders[0],
                          out_order=orders[1], transposed=transposed, out_dtype=out)
    w64 = w.double().numpy()
    want, mag = oracle.grouped_matmul(oracle.source_rows(x.double().numpy(), orders[0], perm, k),
                                      w64.transpose(0, 2, 1) if transposed else w64, off)
    assert y.dtype == DT[out] and y.shape == (T * k, C)
    close(y, place(want, orders[1], perm), place(mag, orders[1], perm), Q, out)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("orders", [("bucket", "bucket"), ("token", "slot"), ("slot", "bucket"), ("token", "bucket")],
                         ids="-".join)
def test_grouped_matmul_dw(shape, orders):
    T, k, E, N, K, kind = shape
    rng = np.random.default_rng(case_seed(*shape, *orders))
    off, perm = buckets(T + E, T, k, E, kind)
    dtype = ["bf16", "f16"][rng.integers(2)]
    out = ["f32", dtype][rng.integers(2)]
    x = torch.from_numpy(rng.standard_normal((T if orders[0] == "token" else T * k, K))).to(DT[dtype])
    dy = torch.from_numpy(rng.standard_normal((T * k, N))).to(DT[dtype])
    dw = qm.grouped_matmul_dw(x.cuda(), dy.cuda(), dev(off), perm=dev(perm), top_k=k, x_order=orders[0],
                              dy_order=orders[1], out_dtype=out)
    want, mag = oracle.grouped_matmul_dw(oracle.source_rows(x.double().numpy(), orders[0], perm, k),
                                         oracle.source_rows(dy.double().numpy(), orders[1], perm, k), off)
    assert dw.dtype == DT[out] and dw.shape == (E, N, K)
    close(dw, want, mag, int(np.diff(off).max()), out)
    for e in np.flatnonzero(np.diff(off) == 0):
        assert not dw[e].any()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("orders", ORDERS, ids="-".join)
def test_grouped_matmul_block(shape, orders):
    T, k, E, N, K, kind = shape
    rng = np.random.default_rng(case_seed(*shape, *orders, "block"))
    off, perm = buckets(T + E, T, k, E, kind)
    out = ["bf16", "f32", "f16"][rng.integers(3)]
    x = (rng.standard_normal((T if orders[0] == "token" else T * k, K)) * np.exp(rng.standard_normal(K))).astype(np.float32)
    a, sa = oracle.quantize_block(x, 1, False)
    q = [oracle.quantize_block((rng.standard_normal((N, K)) * K ** -0.5).astype(np.float32), 128, False)
         for _ in range(min(E, 16))]
    w, sw = np.stack([q[e % 16][0] for e in range(E)]), np.stack([q[e % 16][1] * (1 + e) for e in range(E)])
    y = qm.grouped_matmul_block(dev(a), dev(sa), dev(w), dev(sw), dev(off), perm=dev(perm), top_k=k,
                                x_order=orders[0], out_order=orders[1], out_dtype=out,
                                out=torch.full((T * k, N), float("nan"), dtype=DT[out], device="cuda"))
    a64 = oracle.source_rows(oracle.dequant_block(a, sa, 1), orders[0], perm, k)
    w64 = np.stack([oracle.dequant_block(w[e], sw[e], 128) for e in range(E)])
    want, mag = oracle.grouped_matmul(a64, w64, off)
    close(y, place(want, orders[1], perm), place(mag, orders[1], perm), K, out, fp8=True)


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 4096, 4096), (2, 264, 272), (15, 136, 2000), (16, 2048, 144),
                                   (17, 520, 1040), (63, 1032, 528), (200, 776, 656), (513, 264, 1168),
                                   (1100, 1288, 400)])
@pytest.mark.parametrize("out", ["bf16", "f32", "f16"])
def test_matmul_block(M, N, K, out):
    rng = np.random.default_rng(M * N + K)
    a, sa = oracle.quantize_block((rng.standard_normal((M, K)) * 3).astype(np.float32), 1, False)
    b, sb = oracle.quantize_block((rng.standard_normal((N, K)) * K ** -0.5).astype(np.float32), 128, True)
    y = qm.matmul_block(dev(a).view(torch.float8_e4m3fn), dev(sa), dev(b).view(torch.float8_e4m3fn), dev(sb),
                        out_dtype=out)
    a64, b64 = oracle.dequant_block(a, sa, 1), oracle.dequant_block(b, sb, 128)
    close(y, a64 @ b64.T, np.abs(a64) @ np.abs(b64).T, K, out, fp8=True)


# Sizes that reach each tile size and the steps in the middle of a long contraction: rows x columns that fill the chip
# with 256 x 256 tiles, with 128 x 256 (ragged and dense), with 128 x 128 and 64 x 128 ones. Columns, contraction, rows.
FILL = [(4100, 1, 4, 4104, 528, "skew"), (2050, 3, 64, 2056, 656, "even"), (1000, 2, 16, 2056, 1296, "skew"),
        (900, 4, 128, 1032, 400, "skew"), (800, 2, 16, 2056, 1296, "skew")]


@pytest.mark.parametrize("T,k,E,C,Q,kind", FILL)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_grouped_matmul_that_fills_the_chip(T, k, E, C, Q, kind, transposed, dtype):
    rng = np.random.default_rng(case_seed(T, E, C, int(transposed), dtype))
    off, perm = buckets(T, T, k, E, kind)
    x, w = ints(rng, T, Q), ints(rng, E, *((Q, C) if transposed else (C, Q)))
    y = qm.grouped_matmul(dev(x, DT[dtype]), dev(w, DT[dtype]), dev(off), perm=dev(perm), top_k=k, x_order="token",
                          out_order="slot", transposed=transposed, out_dtype="f32")
    # |sums| <= 16 * 1296 < 2^24: exact in float32 on the host too
    want = np.empty((T * k, C), np.float32)
    for e in range(E):
        p = perm[off[e]:off[e + 1]]
        want[p] = x[p // k] @ (w[e] if transposed else w[e].T)
    assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("T,k,E,N,K,kind", FILL)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped_matmul_block_that_fills_the_chip(T, k, E, N, K, kind, out):
    """Codes and scales that make every product and sum exact, with 13 bits below the largest product too: integers up
    to 4, and scales that are powers of two."""
    rng = np.random.default_rng(case_seed(T, E, N, out))
    off, perm = buckets(T, T, k, E, kind)
    nb = -(-K // 128)
    av, wv = ints(rng, T, K), ints(rng, E, N, K)
    sa = np.exp2(rng.integers(-1, 2, (T, nb))).astype(np.float32)
    sw = np.exp2(rng.integers(-1, 2, (E, -(-N // 128), nb))).astype(np.float32)
    y = qm.grouped_matmul_block(dev(oracle.e4m3_encode(av)), dev(sa), dev(oracle.e4m3_encode(wv)), dev(sw), dev(off),
                                perm=dev(perm), top_k=k, x_order="token", out_dtype=out)
    a32 = av * np.repeat(sa, 128, 1)[:, :K]
    want = np.empty((T * k, N), np.float32)
    for e in range(E):
        w32 = wv[e] * np.repeat(np.repeat(sw[e], 128, 0)[:N], 128, 1)[:, :K]
        want[off[e]:off[e + 1]] = a32[perm[off[e]:off[e + 1]] // k] @ w32.T
    want = torch.from_numpy(want).to(DT[out])
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("M,N,K", [(4096, 4104, 528), (2100, 4096, 656), (1100, 4104, 400), (500, 4096, 1296)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_block_that_fills_the_chip(M, N, K, out):
    rng = np.random.default_rng(case_seed(M, N, K, out))
    nb = -(-K // 128)
    av, bv = ints(rng, M, K), ints(rng, N, K)
    sa = np.exp2(rng.integers(-1, 2, (M, nb))).astype(np.float32)
    sb = np.exp2(rng.integers(-1, 2, (-(-N // 128), nb))).astype(np.float32)
    y = qm.matmul_block(dev(oracle.e4m3_encode(av)), dev(sa), dev(oracle.e4m3_encode(bv)), dev(sb), out_dtype=out)
    want = (av * np.repeat(sa, 128, 1)[:, :K]) @ (bv * np.repeat(np.repeat(sb, 128, 0)[:N], 128, 1)[:, :K]).T
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(DT[out]))


# Few tiles and a contraction that is shared out: one, two and four row tiles of 16 at a time. Rows, experts, columns,
# contraction.
@pytest.mark.parametrize("T,E,C,Q", [(40, 2, 520, 1296), (200, 2, 520, 1040), (200, 2, 1000, 1040), (305, 1, 240, 1296),
                                     (200, 1, 1000, 656), (90, 5, 264, 2000)])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_few_tiles_share_the_contraction(T, E, C, Q, out):
    rng = np.random.default_rng(case_seed(T, E, C, out))
    off, perm = buckets(T, T, 1, E, "skew")
    nb = -(-Q // 128)
    av, wv = ints(rng, T, Q), ints(rng, E, C, Q)
    want = np.empty((T, C), np.float32)
    for e in range(E):
        p = perm[off[e]:off[e + 1]]
        want[p] = av[p] @ wv[e].T
    kw = dict(perm=dev(perm), top_k=1, x_order="token", out_order="slot", out_dtype=out)
    if out != "f32":
        y = qm.grouped_matmul(dev(av, DT[out]), dev(wv, DT[out]), dev(off), **kw)
        assert torch.equal(y.cpu(), torch.from_numpy(want).to(DT[out]))
    codes, scales = oracle.e4m3_encode(wv), np.ones((E, -(-C // 128), nb), np.float32)
    y = qm.grouped_matmul_block(dev(oracle.e4m3_encode(av)), dev(np.ones((T, nb), np.float32)), dev(codes),
                                dev(scales), dev(off), **kw)
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(DT[out]))
    if E == 1:
        y = qm.matmul_block(dev(oracle.e4m3_encode(av)), dev(np.ones((T, nb), np.float32)), dev(codes[0]),
                            dev(scales[0]), out_dtype=out)
        assert torch.equal(y.cpu(), torch.from_numpy(want).to(DT[out]))


@pytest.mark.parametrize("T,k,E,N,K,kind", [(2000, 2, 16, 1032, 1032, "skew"), (1500, 1, 3, 520, 264, "even")])
@pytest.mark.parametrize("orders", [("bucket", "bucket"), ("token", "slot"), ("slot", "bucket")], ids="-".join)
def test_weight_gradient_of_long_buckets(T, k, E, N, K, kind, orders):
    rng = np.random.default_rng(case_seed(T, E, N, *orders))
    off, perm = buckets(T, T, k, E, kind)
    x, dy = ints(rng, T if orders[0] == "token" else T * k, K), ints(rng, T * k, N)
    dw = qm.grouped_matmul_dw(dev(x, DT["bf16"]), dev(dy, DT["bf16"]), dev(off), perm=dev(perm), top_k=k,
                              x_order=orders[0], dy_order=orders[1])
    xs, ds = oracle.source_rows(x, orders[0], perm, k), oracle.source_rows(dy, orders[1], perm, k)
    want = np.stack([ds[off[e]:off[e + 1]].T @ xs[off[e]:off[e + 1]] for e in range(E)])
    assert np.array_equal(dw.cpu().numpy(), want)


# ------------------------------------------------------------------ exact on integers

@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_integers_are_exact(shape, dtype):
    """Sums of at most 16 * 1040 stay below 2^24: every step is exact in fp32."""
    T, k, E, N, K, kind = shape
    rng = np.random.default_rng(case_seed(*shape, dtype))
    off, perm = buckets(T + E, T, k, E, kind)
    x, w, dy = ints(rng, T, K), ints(rng, E, N, K), ints(rng, T * k, N)
    kw = dict(perm=dev(perm), top_k=k)
    y = qm.grouped_matmul(dev(x, DT[dtype]), dev(w, DT[dtype]), dev(off), x_order="token", out_dtype="f32", **kw)
    want, _ = oracle.grouped_matmul(x[perm // k].astype(np.float64), w.astype(np.float64), off)
    assert np.array_equal(y.cpu().numpy(), want)
    dx = qm.grouped_matmul(dev(dy, DT[dtype]), dev(w, DT[dtype]), dev(off), x_order="slot", out_order="slot",
                           transposed=True, out_dtype="f32", **kw)
    want, _ = oracle.grouped_matmul(dy[perm].astype(np.float64), w.transpose(0, 2, 1).astype(np.float64), off)
    assert np.array_equal(dx.cpu().numpy()[perm], want)
    dw = qm.grouped_matmul_dw(dev(x, DT[dtype]), dev(dy, DT[dtype]), dev(off), x_order="token", dy_order="slot", **kw)
    want, _ = oracle.grouped_matmul_dw(x[perm // k].astype(np.float64), dy[perm].astype(np.float64), off)
    assert np.array_equal(dw.cpu().numpy(), want)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_integer_codes_with_power_of_two_scales_are_exact(shape):
    T, k, E, N, K, kind = shape
    rng = np.random.default_rng(case_seed(*shape, "pow2"))
    off, perm = buckets(T + E, T, k, E, kind)
    nb = -(-K // 128)
    a, w = oracle.e4m3_encode(ints(rng, T, K)), oracle.e4m3_encode(ints(rng, E, N, K))
    sa = np.exp2(rng.integers(-1, 2, (T, nb))).astype(np.float32)
    sw = np.exp2(rng.integers(-1, 2, (E, -(-N // 128), nb))).astype(np.float32)
    y = qm.grouped_matmul_block(dev(a), dev(sa), dev(w), dev(sw), dev(off), perm=dev(perm), top_k=k, x_order="token",
                                out_order="slot", out_dtype="f32")
    a64 = oracle.dequant_block(a, sa, 1)[perm // k]
    want, _ = oracle.grouped_matmul(a64, np.stack([oracle.dequant_block(w[e], sw[e], 128) for e in range(E)]), off)
    assert np.array_equal(y.cpu().numpy()[perm], want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_equal_differences(dtype):
    """The product is linear in x and in w: with integers, the change of sum(y * g) under an integer change of w (or x)
    equals the gradient's inner product with that change, exactly."""
    T, k, E, N, K = 70, 2, 6, 40, 24
    rng = np.random.default_rng(12)
    off, perm = buckets(3, T, k, E, "skew")
    kw = dict(perm=dev(perm), top_k=k)
    x, w, g = ints(rng, T, K, top=2), ints(rng, E, N, K, top=2), ints(rng, T * k, N, top=2)
    dxx, dww = ints(rng, T, K, top=2), ints(rng, E, N, K, top=2)

    def loss(x, w):
        y = qm.grouped_matmul(dev(x, DT[dtype]), dev(w, DT[dtype]), dev(off), x_order="token", out_order="slot",
                              out_dtype="f32", **kw)
        return (y.double().cpu().numpy() * g).sum()

    gw = qm.grouped_matmul_dw(dev(x, DT[dtype]), dev(g, DT[dtype]), dev(off), x_order="token", dy_order="slot", **kw)
    assert loss(x, w + dww) - loss(x, w) == (gw.double().cpu().numpy() * dww).sum()
    gx = qm.grouped_matmul(dev(g, DT[dtype]), dev(w, DT[dtype]), dev(off), x_order="slot", out_order="slot",
                           transposed=True, out_dtype="f32", **kw)
    gx = qm.combine(gx, torch.ones(T, k, device="cuda"), None, out_dtype="f32")     # a token's slots share its row
    assert loss(x + dxx, w) - loss(x, w) == (gx.double().cpu().numpy() * dxx).sum()


# ------------------------------------------------------------------ what must not leak

BIG = [(40, 3, 5, 264, 272), (600, 2, 6, 520, 272)]


@pytest.mark.parametrize("T,k,E,N,K", BIG)
@pytest.mark.parametrize("transposed", [False, True])
def test_rows_of_no_bucket_stay_and_nan_does_not_leak(T, k, E, N, K, transposed):
    """Positions before offsets[0], behind offsets[E] and of other experts hold NaN, as do the weights of an empty
    expert: the computed rows are exact all the same and the others keep their bytes."""
    rng = np.random.default_rng(T)
    R = T * k
    cuts = np.sort(rng.choice(np.arange(6, R - 5), E - 1, replace=False))
    off = np.r_[5, cuts, R - 5].astype(np.int32)
    off[2] = off[1]                                                        # expert 1 is empty
    Q, C = (N, K) if transposed else (K, N)
    x, w, dy = ints(rng, R, Q), ints(rng, E, N, K), ints(rng, R, N)
    bad = 3                                                                # expert 3's rows and expert 1's weights
    x[:5] = x[-5:] = x[off[bad]:off[bad + 1]] = np.nan
    w[1] = np.nan
    out = torch.full((R, C), 7.0, device="cuda")
    y = qm.grouped_matmul(dev(x, DT["bf16"]), dev(w, DT["bf16"]), dev(off), transposed=transposed, out=out)
    want, _ = oracle.grouped_matmul(np.nan_to_num(x).astype(np.float64),
                                    np.nan_to_num(w.transpose(0, 2, 1) if transposed else w).astype(np.float64), off)
    y = y.cpu().numpy()
    assert np.all(y[:5] == 7) and np.all(y[-5:] == 7)
    keep = np.r_[5:off[bad], off[bad + 1]:R - 5]
    assert np.array_equal(y[keep], want[keep]) and np.isnan(y[off[bad]:off[bad + 1]]).all()
    if not transposed:
        dw = qm.grouped_matmul_dw(dev(x, DT["bf16"]), dev(dy, DT["bf16"]), dev(off)).cpu().numpy()
        ref, _ = oracle.grouped_matmul_dw(np.nan_to_num(x).astype(np.float64), dy.astype(np.float64), off)
        ok = [e for e in range(E) if e != bad]
        assert np.array_equal(dw[ok], ref[ok]) and not dw[1].any()


@pytest.mark.parametrize("T,k,E,N,K", BIG)
def test_block_rows_of_no_bucket_stay_and_nan_does_not_leak(T, k, E, N, K):
    rng = np.random.default_rng(T + 1)
    R, nb = T * k, -(-K // 128)
    cuts = np.sort(rng.choice(np.arange(6, R - 5), E - 1, replace=False))
    off = np.r_[5, cuts, R - 5].astype(np.int32)
    off[2] = off[1]
    a, w = oracle.e4m3_encode(ints(rng, R, K)), oracle.e4m3_encode(ints(rng, E, N, K))
    sa, sw = np.ones((R, nb), np.float32), np.ones((E, -(-N // 128), nb), np.float32)
    want, _ = oracle.grouped_matmul(oracle.e4m3_decode(a), oracle.e4m3_decode(w), off)
    a[:5] = 0x7F
    a[off[3]:off[4]] = 0x7F
    sa[-5:] = np.nan
    w[1], sw[1] = 0x7F, np.nan
    y = qm.grouped_matmul_block(dev(a), dev(sa), dev(w), dev(sw), dev(off),
                                out=torch.full((R, N), 7.0, device="cuda")).cpu().numpy()
    assert np.all(y[:5] == 7) and np.all(y[-5:] == 7)
    keep = np.r_[5:off[3], off[4]:R - 5]
    assert np.array_equal(y[keep], want[keep]) and np.isnan(y[off[3]:off[4]]).all()


def test_infinite_and_nan_scales_reach_only_their_rows():
    """A row whose block has a NaN scale (a non-finite input to the quantiser) is NaN; the others are not."""
    x = torch.randn(40, 256, generator=torch.Generator().manual_seed(1))
    x[3, 5], x[39, 200] = float("inf"), float("nan")
    a, sa = qm.quantize_block(x.cuda())
    b, sb = qm.quantize_block(torch.randn(72, 256, generator=torch.Generator().manual_seed(2)).cuda(), block_rows=128)
    y = qm.matmul_block(a, sa, b, sb).float().cpu()
    assert torch.isnan(y[[3, 39]]).all() and torch.isfinite(y[[i for i in range(40) if i not in (3, 39)]]).all()


@pytest.mark.parametrize("T", [6, 400])
def test_bad_perm_entries_are_reported_and_write_nothing(T):
    k, E, N, K = 2, 4, 72, 80
    rng = np.random.default_rng(T)
    off, perm = buckets(1, T, k, E, "even")
    bad = [1, T, 2 * T - 1]
    broken = perm.copy()
    broken[bad] = [-1, 2 * T, 1 << 30]
    x, w = ints(rng, T * k, K), ints(rng, E, N, K)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((T * k, N), 7.0, device="cuda")
    y = qm.grouped_matmul(dev(x, DT["f16"]), dev(w, DT["f16"]), dev(off), perm=dev(broken), top_k=k, out_order="slot",
                          out=out, err=err).cpu().numpy()
    assert err.item() == _lib.MOE_DEVERR_ROW_INDEX
    want, _ = oracle.grouped_matmul(x.astype(np.float64), w.astype(np.float64), off)
    good = np.setdiff1d(np.arange(T * k), bad)
    assert np.array_equal(y[perm[good]], want[good]) and np.all(y[perm[bad]] == 7)
    for call in (lambda e: qm.grouped_matmul(dev(x[:T], DT["f16"]), dev(w, DT["f16"]), dev(off), perm=dev(broken),
                                             top_k=k, x_order="token", err=e),
                 lambda e: qm.grouped_matmul_dw(dev(x, DT["f16"]), dev(x, DT["f16"]), dev(off), perm=dev(broken),
                                                top_k=k, dy_order="slot", err=e)):
        err.zero_()
        call(err)
        assert err.item() == _lib.MOE_DEVERR_ROW_INDEX
        call(None)
    err.zero_()
    qm.grouped_matmul(dev(x, DT["f16"]), dev(w, DT["f16"]), dev(off), perm=dev(perm), top_k=k, out_order="slot", err=err)
    assert err.item() == 0


def test_offsets_are_clamped():
    """Offsets outside [0, rows] and buckets that do not ascend stay in bounds; sound buckets are computed."""
    rng = np.random.default_rng(2)
    x, w = ints(rng, 60, 64), ints(rng, 4, 40, 64)
    off = np.array([-7, 20, 10, 50, 1 << 30], np.int32)                    # expert 1 runs backwards: empty
    out = torch.full((60, 40), 7.0, device="cuda")
    y = qm.grouped_matmul(dev(x, DT["bf16"]), dev(w, DT["bf16"]), dev(off), out=out).cpu().numpy()
    ref = lambda e, lo, hi: x[lo:hi].astype(np.float64) @ w[e].astype(np.float64).T  # noqa: E731
    assert np.array_equal(y[:10], ref(0, 0, 10)) and np.array_equal(y[50:], ref(3, 50, 60))
    assert np.array_equal(y[20:50], ref(2, 20, 50))


def test_empty_calls():
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert qm.grouped_matmul(z(0, 16), z(3, 8, 16), off).shape == (0, 8)
    assert not qm.grouped_matmul_dw(z(0, 16), z(0, 8), off, out=torch.ones(3, 8, 16, device="cuda")).any()
    assert not qm.grouped_matmul_dw(z(5, 16), z(5, 8), off, out=torch.ones(3, 8, 16, device="cuda")).any()
    full = torch.tensor([0, 2, 2, 5], dtype=torch.int32, device="cuda")
    y = qm.grouped_matmul(z(5, 0), z(3, 8, 0), full, out=torch.ones(5, 8, device="cuda"))
    assert not y.any()                                                     # a contraction of length 0
    q = torch.zeros(5, 0, dtype=torch.uint8, device="cuda")
    s = torch.zeros(5, 0, device="cuda")
    assert not qm.matmul_block(q, s, q[:0].reshape(0, 0).new_zeros(8, 0), s.new_zeros(1, 0),
                               out=torch.ones(5, 8, device="cuda")).any()


def test_refusals_on_the_device():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    off = z(4, d=torch.int32)
    with pytest.raises(ValueError):
        qm.grouped_matmul(z(4, 32)[:, :16], z(3, 8, 16), off)              # strided rows
    with pytest.raises(ValueError):
        qm.grouped_matmul(z(4, 16), z(3, 8, 24), off)
    with pytest.raises(ValueError):
        qm.grouped_matmul(z(5, 16), z(3, 8, 16), off, top_k=2)
    with pytest.raises(ValueError):
        qm.grouped_matmul(z(4, 16), z(3, 8, 16), off, x_order="rows")
    with pytest.raises(ValueError):
        qm.grouped_matmul(z(4, 16), z(3, 8, 16), off[:3])
    with pytest.raises(TypeError):
        qm.grouped_matmul(z(4, 16), z(3, 8, 16, d=torch.float16), off)
    with pytest.raises(_lib.MoeError):
        qm.grouped_matmul(z(4, 16), z(3, 8, 16), off, x_order="slot")      # no perm
    with pytest.raises(_lib.MoeError):
        qm.grouped_matmul(z(4, 16), z(3, 8, 16), off, out_order="token")
    with pytest.raises(_lib.MoeError):
        qm.grouped_matmul(z(4, 12), z(3, 8, 12), off)
    with pytest.raises(ValueError):
        qm.grouped_matmul(z(4, 16), z(3, 8, 16), off, out=z(4, 16))
    with pytest.raises(ValueError):
        qm.matmul_block(z(4, 128, d=torch.uint8), z(4, 2, d=torch.float32), z(8, 128, d=torch.uint8),
                        z(1, 1, d=torch.float32))


def test_sizes_that_32_bits_do_not_hold_are_refused():
    """2^32 rows would reach the ABI as none."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    off, rows = z(4, d=torch.int32), 1 << 32
    with pytest.raises(ValueError):
        qm.grouped_matmul(z(rows, 0), z(3, 8, 0), off)
    with pytest.raises(ValueError):
        qm.grouped_matmul(z(2, 16), z(3, 8, 16), off, x_order="token", top_k=1 << 31)
    with pytest.raises(ValueError):
        qm.grouped_matmul(z(0, 0), z(3, rows, 0), off)
    with pytest.raises(ValueError):
        qm.grouped_matmul_dw(z(4, 0), z(4, 16), off[:0])
    with pytest.raises(ValueError):
        qm.matmul_block(z(rows, 0, d=torch.uint8), z(rows, 0, d=torch.float32), z(8, 0, d=torch.uint8),
                        z(1, 0, d=torch.float32))
    with pytest.raises(ValueError):
        qm.quantize_block(z(0, rows))
    with pytest.raises(ValueError):
        qm.swiglu_quantize_block(z(0, 2 * rows))


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)
    with pytest.raises(ValueError):
        qm.quantize_block(torch.zeros(2, 128, device="cuda"), stream=Stream())


# ------------------------------------------------------------------ streams, graphs, large offsets

def _all(x, w, dy, off, perm, k, a, sa, wq, sw):
    kw = dict(perm=perm, top_k=k)
    return (qm.grouped_matmul(x, w, off, x_order="token", **kw),
            qm.grouped_matmul(dy, w, off, x_order="slot", out_order="slot", transposed=True, out_dtype="f32", **kw),
            qm.grouped_matmul_dw(x, dy, off, x_order="token", dy_order="slot", **kw),
            qm.grouped_matmul_block(a, sa, wq, sw, off, x_order="token", **kw),
            qm.matmul_block(a, sa, wq[0], sw[0], out_dtype="f32"))


def _inputs(seed, T, k, E, N, K):
    off, perm = buckets(seed, T, k, E, "skew")
    g = torch.Generator().manual_seed(seed)
    x, dy = torch.randn(T, K, generator=g), torch.randn(T * k, N, generator=g)
    a, sa = qm.quantize_block(x.cuda())
    return [x.bfloat16().cuda(), dy.bfloat16().cuda(), dev(off), dev(perm), a, sa]


@pytest.mark.parametrize("T,k,E,N,K", [(3, 2, 6, 264, 528), (300, 3, 8, 264, 528)])
def test_graph_replays_equal_eager(T, k, E, N, K):
    """One captured run, replayed with other tokens and another routing between eager work; two graphs at once."""
    g = torch.Generator().manual_seed(0)
    wf = torch.randn(E, N, K, generator=g).cuda()
    w, (wq, sw) = wf.bfloat16(), qm.quantize_block(wf, block_rows=128)
    sets = [_inputs(s, T, k, E, N, K) for s in range(3)]
    bufs = [t.clone() for t in sets[0]]
    eager = [[t.clone() for t in _all(s[0], w, s[1], s[2], s[3], k, s[4], s[5], wq, sw)] for s in sets]
    graphs = []
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            with torch.cuda.graph(graph, stream=stream):
                outs = _all(bufs[0], w, bufs[1], bufs[2], bufs[3], k, bufs[4], bufs[5], wq, sw)
        graphs.append((graph, outs))
    torch.cuda.current_stream().wait_stream(stream)
    for rep in range(4):
        for b, s in zip(bufs, sets[rep % 3]):
            b.copy_(s)
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
        graphs[0][0].replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            for got, want in zip(outs, eager[rep % 3]):
                assert torch.equal(got, want), rep
        torch.randn(1 << 16, device="cuda").sum().item()


def test_two_streams_at_once():
    T, k, E, N, K = 200, 2, 6, 264, 528
    g = torch.Generator().manual_seed(0)
    wf = torch.randn(E, N, K, generator=g).cuda()
    w, (wq, sw) = wf.bfloat16(), qm.quantize_block(wf, block_rows=128)
    sets = [_inputs(s, T, k, E, N, K) for s in range(2)]
    want = [[t.clone() for t in _all(s[0], w, s[1], s[2], s[3], k, s[4], s[5], wq, sw)] for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for s, st in zip(sets, streams):
        with torch.cuda.stream(st):
            got.append(_all(s[0], w, s[1], s[2], s[3], k, s[4], s[5], wq, sw))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    y = qm.grouped_matmul(sets[0][0], w, sets[0][2], perm=sets[0][3], top_k=k, x_order="token", stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(y, want[0][0])


def test_offsets_past_32_bits():
    """x, weights and output each longer than 2^32 bytes; rows and experts at the far end are right."""
    rng = np.random.default_rng(4)
    R, K, N, E = (1 << 19) + 300, 4352, 4352, 128                          # x 4.6 GB, w 4.8 GB, out 4.6 GB
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    xs, ws = ints(rng, 300, K), ints(rng, N, K)
    x[-300:], w[-1] = dev(xs, DT["bf16"]), dev(ws, DT["bf16"])
    off = np.full(E + 1, R - 300, np.int32)
    off[0], off[-1] = R - 400, R                                           # expert 0: 100 rows of zeros
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = qm.grouped_matmul(x, w, dev(off), out=out)
    want = torch.from_numpy(xs).double() @ torch.from_numpy(ws).double().t()
    assert torch.equal(y[-300:].cpu(), want.float().bfloat16())
    assert not y[-400:-300].any() and (y[:16] == 7).all() and (y[-410:-400] == 7).all()
    dx = qm.grouped_matmul(x, w, dev(off), transposed=True, out=out)
    want = torch.from_numpy(xs).double() @ torch.from_numpy(ws).double()
    assert torch.equal(dx[-300:].cpu(), want.float().bfloat16())
    perm = torch.arange(R, dtype=torch.int32, device="cuda")
    dw = qm.grouped_matmul_dw(x, x, dev(off), perm=perm, x_order="slot", out=w)
    want = torch.from_numpy(xs).double().t() @ torch.from_numpy(xs).double()
    assert torch.equal(dw[-1].cpu(), want.float().bfloat16()) and not dw[0].any() and not dw[E // 2].any()


# ------------------------------------------------------------------ together, as they are used

def test_fp8_expert_layer():
    """route -> permute -> quantise -> gate/up product -> SwiGLU + quantise -> down product -> combine, against the
    same chain in float64 from the same codes (each step checked with its own input, so no error accumulates)."""
    T, k, E, d, I = 96, 4, 12, 384, 272
    rng = np.random.default_rng(21)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).bfloat16().cuda()
    gu = torch.from_numpy((rng.standard_normal((E, 2 * I, d)) * d ** -0.5).astype(np.float32)).bfloat16().cuda()
    dn = torch.from_numpy((rng.standard_normal((E, d, I)) * I ** -0.5).astype(np.float32)).bfloat16().cuda()
    wr = torch.from_numpy((rng.standard_normal((E, d)) * 0.1).astype(np.float32)).cuda()
    router = _lib.RouterC(_lib.MOE_ROUTE_TOPK, E, k, d, 0, wr.data_ptr(), None, None, 1.0)
    import ctypes
    from types import SimpleNamespace
    layer = SimpleNamespace(router_c=router, top_k=k)
    ws = torch.empty(256 + 3 * (8 * T * E + 512), dtype=torch.uint8, device="cuda")
    qm.workspace_init(ws)
    ids, rw = qm.route(layer, x, ws=ws)
    offsets, perm = qm.permute(ids, E, ws)
    (wq, sw), (vq, sv) = qm.quantize_block(gu, block_rows=128), qm.quantize_block(dn, block_rows=128)
    a, sa = qm.quantize_block(x)
    h = qm.grouped_matmul_block(a, sa, wq, sw, offsets, perm=perm, top_k=k, x_order="token")
    hq, sh = qm.swiglu_quantize_block(h)
    y_slot = qm.grouped_matmul_block(hq, sh, vq, sv, offsets, perm=perm, top_k=k, out_order="slot", out_dtype="f32")
    y = qm.combine(y_slot, rw, None, out_dtype="f32")

    n = lambda t: t.cpu().view(torch.uint8).numpy()  # noqa: E731
    off, p = offsets.cpu().numpy(), perm.cpu().numpy()
    w64 = np.stack([oracle.dequant_block(n(wq[e]), sw[e].cpu().numpy(), 128) for e in range(E)])
    v64 = np.stack([oracle.dequant_block(n(vq[e]), sv[e].cpu().numpy(), 128) for e in range(E)])
    want, mag = oracle.grouped_matmul(oracle.dequant_block(n(a), sa.cpu().numpy(), 1)[p // k], w64, off)
    close(h, want, mag, d, "bf16", fp8=True)
    _, rs = oracle.swiglu_quantize_block(h.double().cpu().numpy(), False)
    assert np.all(np.abs(sh.cpu().numpy() / rs - 1) <= 2.0 ** -21)
    want, mag = oracle.grouped_matmul(oracle.dequant_block(n(hq), sh.cpu().numpy(), 1), v64, off)
    close(y_slot, place(want, "slot", p), place(mag, "slot", p), I, "f32")
    ref = (y_slot.double().cpu().numpy().reshape(T, k, d) * rw.double().cpu().numpy()[:, :, None]).sum(1)
    assert np.allclose(y.double().cpu().numpy(), ref, rtol=1e-5, atol=1e-5)
    # and the whole chain is the bf16 layer up to the two quantisations of each operand: e4m3's half step is 2^-4, so
    # a value moves by at most 1/16; independent signs keep the norm of a sum's error below a fifth of the sum's norm
    e_of = np.repeat(np.arange(E), np.diff(off))
    full = np.empty((T * k, d))
    for pos in range(T * k):
        g, u = np.split(gu[e_of[pos]].double().cpu().numpy() @ x[p[pos] // k].double().cpu().numpy(), 2)
        full[p[pos]] = dn[e_of[pos]].double().cpu().numpy() @ (oracle.silu(g) * u)
    full = (full.reshape(T, k, d) * rw.double().cpu().numpy()[:, :, None]).sum(1)
    assert np.linalg.norm(y.cpu().numpy() - full) <= 0.2 * np.linalg.norm(full)


def test_training_step_of_one_projection():
    """Forward, the gradient in the tokens and in the weights of loss = sum(c * combine(product)), as a training step
    calls them, against the formula in float64."""
    T, k, E, N, K = 150, 3, 10, 136, 264
    rng = np.random.default_rng(31)
    off, perm = buckets(8, T, k, E, "skew")
    rw = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).bfloat16().cuda()
    w = torch.from_numpy((rng.standard_normal((E, N, K)) * K ** -0.5).astype(np.float32)).bfloat16().cuda()
    c = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).cuda()
    kw = dict(perm=dev(perm), top_k=k)
    y = qm.combine(qm.grouped_matmul(x, w, dev(off), x_order="token", out_order="slot", out_dtype="f32", **kw), rw,
                   None, out_dtype="f32")
    dslot = (rw[:, :, None] * c[:, None, :]).reshape(T * k, N).bfloat16()
    dx = qm.combine(qm.grouped_matmul(dslot, w, dev(off), x_order="slot", out_order="slot", transposed=True,
                                      out_dtype="f32", **kw), torch.ones(T, k, device="cuda"), None, out_dtype="f32")
    dw = qm.grouped_matmul_dw(x, dslot, dev(off), x_order="token", dy_order="slot", **kw)

    x64, w64, d64 = x.double().cpu().numpy(), w.double().cpu().numpy(), dslot.double().cpu().numpy()
    ref, mag = oracle.grouped_matmul(x64[perm // k], w64, off)
    rw64 = rw.double().cpu().numpy()[:, :, None]
    close(y, (place(ref, "slot", perm).reshape(T, k, N) * rw64).sum(1),
          (place(mag, "slot", perm).reshape(T, k, N) * rw64).sum(1), K + k, "f32")
    ref, mag = oracle.grouped_matmul(d64[perm], w64.transpose(0, 2, 1), off)
    close(dx, place(ref, "slot", perm).reshape(T, k, K).sum(1), place(mag, "slot", perm).reshape(T, k, K).sum(1),
          N + k, "f32")
    close(dw, *oracle.grouped_matmul_dw(x64[perm // k], d64[perm], off), int(np.diff(off).max()), "f32")
