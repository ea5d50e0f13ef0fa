"""Products past what other tests reach: contractions beyond 64 blocks of 128
(where the FP8 tile kernels fetch the weights' scales a second time), every pair
of input and output types, and subnormal inputs."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def ints(rng, *shape, top=2):
    return rng.integers(-top, top + 1, size=shape).astype(np.float32)


# rows, columns, contraction: split over 1, 2 and 4 row tiles; 64 x 128 and 128 x 128 tiles; 128 x 256; 256 x 256
LONG = [(3, 136, 16400), (40, 2056, 8208), (120, 1032, 16400), (300, 4104, 8208), (1100, 4104, 8208),
        (2100, 4096, 8208), (4100, 4104, 8320)]


@pytest.mark.parametrize("M,N,K", LONG)
@pytest.mark.parametrize("out,f32_sums", [("f32", False), ("bf16", False), ("bf16", True)])
def test_scales_of_contractions_beyond_64_blocks(M, N, K, out, f32_sums):
    """Integers up to 2 and scales that differ from block to block by powers of two, 2^-2 .. 1 on each side: sums of at
    most 4 * 16400 in steps of 2^-4, 20 bits, are exact in fp32, and every product of a block is within 13 bits of the
    largest. Checked on 64 rows."""
    rng = np.random.default_rng(M + K)
    nb = -(-K // 128)
    a, b = ints(rng, M, K), ints(rng, N, K)
    sa = np.exp2(rng.integers(-2, 1, (M, nb))).astype(np.float32)
    sb = np.exp2(rng.integers(-2, 1, (-(-N // 128), nb))).astype(np.float32)
    y = qm.matmul_block(dev(a).to(torch.float8_e4m3fn), dev(sa), dev(b).to(torch.float8_e4m3fn), dev(sb), out_dtype=out,
                        f32_sums=f32_sums)
    at = np.sort(rng.choice(M, min(M, 64), replace=False))
    want = (a[at] * np.repeat(sa[at], 128, 1)[:, :K]) @ (b * np.repeat(np.repeat(sb, 128, 0)[:N], 128, 1)[:, :K]).T
    assert torch.equal(y[torch.from_numpy(at).cuda()].cpu(), torch.from_numpy(want).to(DT[out]))


@pytest.mark.parametrize("T,k,E,N,K", [(5, 2, 3, 136, 8464), (600, 2, 4, 520, 8464)])
def test_grouped_scales_beyond_64_blocks(T, k, E, N, K):
    rng = np.random.default_rng(T)
    nb, R = -(-K // 128), T * k
    off = np.r_[0, np.sort(rng.integers(0, R + 1, E - 1)), R].astype(np.int32)
    perm = rng.permutation(R).astype(np.int32)
    a, w = ints(rng, T, K), ints(rng, E, N, K)
    sa = np.exp2(rng.integers(-2, 1, (T, nb))).astype(np.float32)
    sw = np.exp2(rng.integers(-2, 1, (E, -(-N // 128), nb))).astype(np.float32)
    for out in ("f32", "bf16"):
        y = qm.grouped_matmul_block(dev(a).to(torch.float8_e4m3fn), dev(sa), dev(w).to(torch.float8_e4m3fn), dev(sw),
                                    dev(off), perm=dev(perm), top_k=k, x_order="token", out_dtype=out).cpu()
        a32 = (a * np.repeat(sa, 128, 1)[:, :K])[perm // k]
        for e in range(E):
            want = a32[off[e]:off[e + 1]] @ (w[e] * np.repeat(np.repeat(sw[e], 128, 0)[:N], 128, 1)[:, :K]).T
            assert torch.equal(y[off[e]:off[e + 1]], torch.from_numpy(want).to(DT[out])), (out, e)


def routed(rng, T, k, E):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).reshape(-1)
    return (np.r_[0, np.cumsum(np.bincount(ids, minlength=E))].astype(np.int32),
            np.argsort(ids, kind="stable").astype(np.int32))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,k,E,N,K", [(3, 2, 6, 136, 264), (300, 2, 5, 264, 520), (2500, 2, 4, 2056, 264)])
def test_every_pair_of_types(T, k, E, N, K, dtype, out):
    """Integers up to 2: every sum is exact in fp32 and rounded once to the output type."""
    rng = np.random.default_rng(T + N)
    off, perm = routed(rng, T, k, E)
    x, w, dy = ints(rng, T, K), ints(rng, E, N, K), ints(rng, T * k, N)
    kw = dict(perm=dev(perm), top_k=k, out_dtype=out)
    xd, wd, dyd = dev(x, DT[dtype]), dev(w, DT[dtype]), dev(dy, DT[dtype])
    y = qm.grouped_matmul(xd, wd, dev(off), x_order="token", **kw).cpu()
    dx = qm.grouped_matmul(dyd, wd, dev(off), x_order="slot", transposed=True, **kw).cpu()
    dw = qm.grouped_matmul_dw(xd, dyd, dev(off), x_order="token", dy_order="slot", **kw).cpu()
    cast = lambda a: torch.from_numpy(a).to(DT[out])  # noqa: E731
    for e in range(E):
        at = np.s_[off[e]:off[e + 1]]
        xs, ds = x[perm[at] // k], dy[perm[at]]
        assert torch.equal(y[at], cast(xs @ w[e].T)), e
        assert torch.equal(dx[at], cast(ds @ w[e])), e
        assert torch.equal(dw[e], cast(ds.T @ xs)), e


@pytest.mark.parametrize("dtype,tiny", [("f16", 2.0 ** -24), ("f16", 2.0 ** -14), ("bf16", 2.0 ** -133),
                                        ("bf16", 2.0 ** -126)])
@pytest.mark.parametrize("T,E,N,K", [(3, 2, 40, 72), (200, 3, 264, 520), (2100, 3, 2056, 264)])
def test_subnormal_inputs(dtype, tiny, T, E, N, K):
    """Multiples of the smallest subnormal (up to 2 of it, or of the smallest normal) times integers up to 2, and for
    bf16 times 2^20, so that sums are exact and normal in fp32."""
    rng = np.random.default_rng(N + T)
    off, perm = routed(rng, T, 1, E)
    xs, ws, ds = ints(rng, T, K), ints(rng, E, N, K), ints(rng, T, N)
    lift = 2.0 ** 20 if dtype == "bf16" else 1.0
    dt = DT[dtype]
    small = lambda a: (torch.from_numpy(a).double() * tiny).to(dt).cuda()  # noqa: E731
    large = lambda a: (torch.from_numpy(a) * lift).to(dt).cuda()  # noqa: E731
    back = lambda t: (t.double().cpu() / (tiny * lift)).numpy()  # noqa: E731
    assert small(xs).double().cpu().abs().max() == 2 * tiny
    kw = dict(perm=dev(perm), x_order="slot")
    for xd, wd, dd in ((small(xs), large(ws), large(ds)), (large(xs), small(ws), small(ds))):
        y = back(qm.grouped_matmul(xd, wd, dev(off), out_dtype="f32", **kw))
        for e in range(E):
            at = np.s_[off[e]:off[e + 1]]
            assert np.array_equal(y[at], xs[perm[at]] @ ws[e].T)
    dx = back(qm.grouped_matmul(small(ds), large(ws), dev(off), transposed=True, out_dtype="f32", **kw))
    dw = back(qm.grouped_matmul_dw(small(xs), large(ds), dev(off), dy_order="slot", **kw))
    for e in range(E):
        at = np.s_[off[e]:off[e + 1]]
        assert np.array_equal(dx[at], ds[perm[at]] @ ws[e])
        assert np.array_equal(dw[e], ds[perm[at]].T @ xs[perm[at]])


@pytest.mark.parametrize("M,N,K", [(2, 40, 144), (300, 4104, 272), (2100, 4096, 144)])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_subnormal_codes(M, N, K, out):
    """E4M3's subnormals 2^-9 and 2^-8 times integers up to 2, scales 2^9."""
    rng = np.random.default_rng(M)
    a, b = ints(rng, M, K), ints(rng, N, K)
    code = lambda v, s: torch.from_numpy(v * s).to(torch.float8_e4m3fn).cuda()  # noqa: E731
    sa, sb = torch.full((M, -(-K // 128)), 2.0 ** 9).cuda(), torch.ones(-(-N // 128), -(-K // 128)).cuda()
    want = torch.from_numpy(a @ b.T).to(DT[out])
    assert torch.equal(qm.matmul_block(code(a, 2.0 ** -9), sa, code(b, 1.0), sb, out_dtype=out).cpu(), want)
    assert torch.equal(qm.matmul_block(code(a, 1.0), sa, code(b, 2.0 ** -9), sb, out_dtype=out).cpu(), want)


@pytest.mark.parametrize("M,N,K", [(2, 40, 144), (300, 4104, 272), (2100, 4096, 144)])
@pytest.mark.parametrize("out,tiny", [("f16", 2.0 ** -24), ("bf16", 2.0 ** -133)])
def test_subnormal_results(M, N, K, out, tiny):
    """Integers up to 2 with scales that make every result a multiple of a quarter of the smallest subnormal: rounded
    once, ties to even, as the reference's conversion from 64 bits does (through fp32, which holds them exactly)."""
    rng = np.random.default_rng(N)
    a, b = ints(rng, M, K), ints(rng, N, K)
    code = lambda v: torch.from_numpy(v).to(torch.float8_e4m3fn).cuda()  # noqa: E731
    sa = torch.full((M, -(-K // 128)), 2.0 ** -20).cuda()
    sb = torch.full((-(-N // 128), -(-K // 128)), tiny / 4 * 2.0 ** 20).cuda()
    want = (torch.from_numpy(a @ b.T).double() * tiny / 4).float().to(DT[out])
    assert torch.equal(qm.matmul_block(code(a), sa, code(b), sb, out_dtype=out).cpu(), want)
    assert (want.double().abs() == tiny).any()
