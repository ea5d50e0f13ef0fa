"""Rows to buckets and back, with weights, and the gradients, against the
float64 oracle: every pair of types, odd widths at odd addresses, from one token
up, dropped assignments, bad entries, NaN in rows that nothing names.

Errors allowed (computed in each test): a weighted row is one fp32 product,
2^-24 of it; a sum of n terms in fp32, in any order, (n + 1) * 2^-24 of the sum
of their magnitudes; each result is rounded once to its type."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm
from tests._steps import DT, HALF, close, dev, routing, shifted

pytestmark = pytest.mark.gpu

TYPES = list(DT)
SHAPES = [(1, 1, 1), (1, 6, 4096), (5, 2, 7), (3, 8, 64), (33, 4, 1003), (130, 3, 520), (64, 1, 8191), (257, 6, 2056),
          (40, 12, 15), (2000, 2, 24), (700, 5, 333)]


@pytest.mark.parametrize("n,size", [(1, 1), (6, 6), (1000, 1000), (1025, 3000), (24576, 24576), (65536, 65536),
                                    (65537, 65537), (300000, 300000), (5, 70000), (70000, 5), (0, 9), (7, 0)])
def test_invert_perm(n, size):
    rng = np.random.default_rng(n + size)
    perm = np.full(n, -1, np.int32)
    held = rng.permutation(n)[:min(n, size) - min(n, size) // 9]        # some positions without an assignment
    perm[held] = rng.permutation(size)[:len(held)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qm.invert_perm(dev(perm), size, err=err)
    assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), oracle.invert_perm(perm, size))
    assert err.item() == 0
    if n == size:
        assert torch.equal(got, qm.invert_perm(dev(perm)))


@pytest.mark.parametrize("n", [50, 70000])
def test_invert_perm_of_entries_named_twice_and_out_of_range(n):
    rng = np.random.default_rng(n)
    perm = rng.integers(0, n, n).astype(np.int32)
    assert np.array_equal(qm.invert_perm(dev(perm)).cpu().numpy(), oracle.invert_perm(perm, n))
    for bad in (n, -2, -2 ** 31, 2 ** 31 - 1):
        perm[n // 2] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert np.array_equal(qm.invert_perm(dev(perm), err=err).cpu().numpy(), oracle.invert_perm(perm, n))
        assert err.item() == 16


@pytest.mark.parametrize("T,k,d", SHAPES)
@pytest.mark.parametrize("x_order", ["token", "slot"])
def test_gather_copies_bits(T, k, d, x_order):
    """Without weights and with one type, NaN and subnormals included."""
    rng, _, perm, _ = routing(T + d, T, k, 16)
    for dtype, ints in ((torch.bfloat16, torch.int16), (torch.float16, torch.int16), (torch.float32, torch.int32)):
        info = torch.iinfo(ints)
        bits = torch.from_numpy(rng.integers(info.min, info.max + 1, (T if x_order == "token" else T * k, d))).to(ints)
        got = qm.gather_rows(bits.view(dtype).cuda(), dev(perm), top_k=k, x_order=x_order)
        assert torch.equal(got.cpu().view(ints), bits[torch.from_numpy(perm // k if x_order == "token" else perm).long()])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("T,k,d", [(1, 6, 256), (33, 4, 1003), (19, 3, 72)])
def test_gather_with_weights_and_types(T, k, d, dtype, out):
    rng, _, perm, w = routing(T + d, T, k, 16)
    x = torch.from_numpy(rng.standard_normal((T, d))).to(DT[dtype])
    for weights in (None, w):
        want = oracle.gather_rows(x.double().numpy(), perm, k, "token", weights)
        got = qm.gather_rows(x.cuda(), dev(perm), top_k=k, weights=None if weights is None else dev(weights), out_dtype=out)
        assert got.dtype == DT[out]
        close(got, want, 2.0 ** -24 * np.abs(want), out)


@pytest.mark.parametrize("dtype", TYPES)
def test_gather_leaves_rows_without_an_assignment(dtype):
    T, k, d = 9, 2, 37
    rng, _, perm, w = routing(5, T, k, 4)
    x = torch.from_numpy(rng.standard_normal((T, d))).to(DT[dtype])
    for entries, code in (([-1, -1, -1], 0), ([-1, 18, -2 ** 31], 16)):   # the second ones are out of range and say so
        perm[[0, 7, 17]] = entries
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((T * k, d), 7.0, dtype=DT[dtype], device="cuda")
        assert qm.gather_rows(x.cuda(), dev(perm), top_k=k, out=out, err=err) is out
        want = oracle.gather_rows(x.double().numpy(), perm, k, "token")
        assert np.array_equal(out.double().cpu().numpy(), np.where(np.isnan(want), 7.0, want))
        assert err.item() == code and (out[[0, 7, 17]] == 7).all()


@pytest.mark.parametrize("n", [0, 1, 4, 60])
def test_gather_of_any_number_of_positions(n):
    """A share of the positions, or more than there are assignments (some of them named twice)."""
    x = torch.arange(40.0, device="cuda").reshape(10, 4)
    perm = np.random.default_rng(n).integers(0, 20, n).astype(np.int32)
    got = qm.gather_rows(x, dev(perm), top_k=2)
    assert got.shape == (n, 4) and torch.equal(got, x[dev(perm // 2).long()])


@pytest.mark.parametrize("T,k,d", SHAPES)
@pytest.mark.parametrize("order", ["bucket", "slot"])
def test_combine(T, k, d, order):
    rng, _, perm, w = routing(T * 3 + d, T, k, 16)
    pos = oracle.invert_perm(perm, T * k) if order == "bucket" else None
    for dtype, out, weighted, shared in (("bf16", "bf16", True, False), ("f16", "f32", False, True), ("f32", "f16", True, True)):
        y = torch.from_numpy(rng.standard_normal((T * k, d))).to(DT[dtype])
        s = torch.from_numpy(rng.standard_normal((T, d))).to(DT[dtype]) if shared else None
        weights = w if weighted else None
        want, mag = oracle.combine_rows(y.double().numpy(), weights, pos, T, k, s.double().numpy() if shared else None)
        got = qm.combine_rows(y.cuda(), dev(w) if weighted else None, None if pos is None else dev(pos), top_k=k,
                              y_shared=s.cuda() if shared else None, out_dtype=out)
        assert got.dtype == DT[out] and got.shape == (T, d)
        close(got, want, (k + 2) * 2.0 ** -24 * mag, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out", TYPES)
def test_combine_types(dtype, out):
    T, k, d = 19, 5, 203
    rng, _, perm, w = routing(1, T, k, 9)
    pos = oracle.invert_perm(perm, T * k)
    y = torch.from_numpy(rng.standard_normal((T * k, d))).to(DT[dtype])
    want, mag = oracle.combine_rows(y.double().numpy(), w, pos, T, k)
    close(qm.combine_rows(y.cuda(), dev(w), dev(pos), out_dtype=out), want, (k + 1) * 2.0 ** -24 * mag, out)


def test_combine_is_combine_for_fp32_slots():
    """What `combine` gives, bit for bit: the same sum in the same order."""
    T, k, d = 30, 6, 256
    g = torch.Generator().manual_seed(0)
    y, w, s = torch.randn(T * k, d, generator=g).cuda(), torch.rand(T, k, generator=g).cuda(), torch.randn(T, d, generator=g).cuda()
    for out in ("f32", "bf16"):
        assert torch.equal(qm.combine_rows(y, w, y_shared=s, out_dtype=out), qm.combine(y, w, s, out_dtype=out))


def test_combine_of_dropped_assignments_reads_nothing_of_them():
    """Rows that no position names hold NaN, as do the weights of dropped assignments; a token may lose all its rows."""
    T, k, d, n = 12, 3, 70, 50
    rng, _, _, w = routing(2, T, k, 9)
    pos = np.full(T * k, -1, np.int32)
    kept = rng.permutation(T * k)[:25]
    pos[kept] = rng.permutation(n)[:25]
    pos[3:6] = -1
    y = rng.standard_normal((n, d)).astype(np.float32)
    y[np.setdiff1d(np.arange(n), pos)] = np.nan
    w.reshape(-1)[pos < 0] = np.nan
    s = rng.standard_normal((T, d)).astype(np.float32)
    for shared in (None, s):
        want, mag = oracle.combine_rows(y, w, pos, T, k, shared)
        got = qm.combine_rows(dev(y), dev(w), dev(pos), y_shared=None if shared is None else dev(s))
        close(got, want, (k + 2) * 2.0 ** -24 * mag, "f32")
    dout = rng.standard_normal((T, d)).astype(np.float32)
    dy = torch.full((n, d), 7.0, device="cuda")
    got, dw = qm.combine_rows_grad(dev(dout), dev(y), dev(w), dev(pos), out=dy)
    wy, ww, mag = oracle.combine_rows_grad(dout, y, w, pos)
    assert got is dy and np.isnan(wy).any()
    close(dw, ww, (d + 1) * 2.0 ** -24 * mag, "f32")
    close(dy, np.where(np.isnan(wy), 7.0, wy), 2.0 ** -24 * np.where(np.isnan(wy), 0, np.abs(wy)), "f32")


def test_positions_out_of_range_are_reported_and_add_nothing():
    T, k, d = 6, 2, 40
    rng, _, perm, w = routing(3, T, k, 5)
    pos = oracle.invert_perm(perm, T * k)
    y, dout = rng.standard_normal((T * k, d)).astype(np.float32), rng.standard_normal((T, d)).astype(np.float32)
    for bad in (T * k, -2, 2 ** 31 - 1, -2 ** 31):
        p = pos.copy()
        p[5] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        want, mag = oracle.combine_rows(y, w, p, T, k)
        close(qm.combine_rows(dev(y), dev(w), dev(p), err=err), want, (k + 1) * 2.0 ** -24 * mag, "f32")
        assert err.item() == 16
        err.zero_()
        dy, dw = qm.combine_rows_grad(dev(dout), dev(y), dev(w), dev(p), err=err, out=torch.full((T * k, d), 7.0, device="cuda"))
        assert err.item() == 16 and (dy[pos[5]] == 7).all() and dw.reshape(-1)[5] == 0
        qm.combine_rows(dev(y), dev(w), dev(p))                        # without an error word


@pytest.mark.parametrize("T,k,d", SHAPES)
@pytest.mark.parametrize("order", ["bucket", "slot"])
def test_combine_grad(T, k, d, order):
    rng, _, perm, w = routing(T * 5 + d, T, k, 16)
    pos = oracle.invert_perm(perm, T * k) if order == "bucket" else None
    for dtype, dt in (("bf16", "bf16"), ("f16", "f32"), ("f32", "f16"), ("bf16", "f32")):
        y = torch.from_numpy(rng.standard_normal((T * k, d))).to(DT[dtype])
        dout = torch.from_numpy(rng.standard_normal((T, d))).to(DT[dt])
        dy, dw = qm.combine_rows_grad(dout.cuda(), y.cuda(), dev(w), None if pos is None else dev(pos))
        wy, ww, mag = oracle.combine_rows_grad(dout.double().numpy(), y.double().numpy(), w, pos)
        assert dy.dtype == DT[dtype] and dw.dtype == torch.float32 and dw.shape == (T, k)
        close(dy, wy, 2.0 ** -24 * np.abs(wy), dtype)
        close(dw, ww, (d + 1) * 2.0 ** -24 * mag, "f32")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dt", TYPES)
def test_combine_grad_types(dtype, dt):
    T, k, d = 19, 5, 203
    rng, _, perm, w = routing(1, T, k, 9)
    pos = oracle.invert_perm(perm, T * k)
    y = torch.from_numpy(rng.standard_normal((T * k, d))).to(DT[dtype])
    dout = torch.from_numpy(rng.standard_normal((T, d))).to(DT[dt])
    dy, dw = qm.combine_rows_grad(dout.cuda(), y.cuda(), dev(w), dev(pos))
    wy, ww, mag = oracle.combine_rows_grad(dout.double().numpy(), y.double().numpy(), w, pos)
    close(dy, wy, 2.0 ** -24 * np.abs(wy), dtype)
    close(dw, ww, (d + 1) * 2.0 ** -24 * mag, "f32")


def test_gradients_equal_differences():
    """combine is linear in rows and in weights: with integers the change of sum(out * g) under an integer change of
    either equals the gradient's inner product with it, exactly (all sums below 2^24). And so for gather, whose
    gradients are combine and combine's gradient with the roles of x and the rows' gradient exchanged."""
    T, k, d = 23, 3, 41
    rng, _, perm, _ = routing(8, T, k, 6)
    pos = dev(oracle.invert_perm(perm, T * k))
    i = lambda *s: rng.integers(-3, 4, s).astype(np.float32)  # noqa: E731
    y, w, g, cy, cw = i(T * k, d), i(T, k), i(T, d), i(T * k, d), i(T, k)
    out = lambda y, w: qm.combine_rows(dev(y), dev(w), pos).double().cpu().numpy()  # noqa: E731
    dy, dw = (t.double().cpu().numpy() for t in qm.combine_rows_grad(dev(g), dev(y), dev(w), pos))
    assert ((out(y + cy, w) - out(y, w)) * g).sum() == (dy * cy).sum()
    assert ((out(y, w + cw) - out(y, w)) * g).sum() == (dw * cw).sum()
    x, cx, r = i(T, d), i(T, d), i(T * k, d)
    rows = lambda x, w: qm.gather_rows(dev(x), dev(perm), top_k=k, weights=dev(w)).double().cpu().numpy()  # noqa: E731
    dx = qm.combine_rows(dev(r), dev(w), pos).double().cpu().numpy()
    dw = qm.combine_rows_grad(dev(x), dev(r), dev(w), pos)[1].double().cpu().numpy()
    assert ((rows(x + cx, w) - rows(x, w)) * r).sum() == (dx * cx).sum()
    assert ((rows(x, w + cw) - rows(x, w)) * r).sum() == (dw * cw).sum()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [8, 13, 264, 2049])
def test_rows_at_odd_addresses(dtype, d):
    """Tensors that start 1 to 7 elements behind an aligned address; what lies around the outputs stays."""
    T, k = 11, 3
    rng, _, perm, w = routing(d, T, k, 6)
    pos = oracle.invert_perm(perm, T * k)
    x, y = rng.integers(-8, 9, (T, d)).astype(np.float32), rng.integers(-8, 9, (T * k, d)).astype(np.float32)
    ww = rng.integers(-2, 3, (T, k)).astype(np.float32)
    for by in (1, 3, 6):
        around = torch.full((T * k * d + 16,), 5.0, dtype=DT[dtype], device="cuda")
        at = around[by:by + T * k * d].view(T * k, d)
        qm.gather_rows(shifted(x, DT[dtype], by), shifted(perm, torch.int32, by), top_k=k, out=at)
        assert np.array_equal(at.double().cpu().numpy(), x[perm // k])
        assert (around[:by] == 5).all() and (around[by + T * k * d:] == 5).all()
        around.fill_(5.0)
        o = around[by:by + T * d].view(T, d)
        qm.combine_rows(shifted(y, DT[dtype], by + 1), shifted(ww, torch.float32, by), shifted(pos, torch.int32, by), out=o)
        assert np.array_equal(o.double().cpu().numpy(), oracle.combine_rows(y, ww, pos, T, k)[0])
        assert (around[:by] == 5).all() and (around[by + T * d:] == 5).all()
        around.fill_(5.0)
        dy, dw = qm.combine_rows_grad(shifted(x, DT[dtype], by), shifted(y, DT[dtype], by), dev(ww), dev(pos), out=at)
        wy, wd, _ = oracle.combine_rows_grad(x, y, ww, pos)
        assert np.array_equal(dy.double().cpu().numpy(), wy) and np.array_equal(dw.double().cpu().numpy(), wd)
        assert (around[:by] == 5).all() and (around[by + T * k * d:] == 5).all()


def test_infinities_and_nan_stay_in_their_rows():
    T, k, d = 4, 2, 24
    y = torch.zeros(T * k, d, device="cuda")
    y[2], y[5, 3] = float("inf"), float("nan")
    w = torch.ones(T, k, device="cuda")
    out = qm.combine_rows(y, w)
    assert torch.isinf(out[1]).all() and torch.isnan(out[2, 3]) and not out[[0, 3]].any() and not out[2, 4:].any()
    dy, dw = qm.combine_rows_grad(y[:T], torch.ones_like(y), w)
    assert torch.isinf(dw[2]).all() and not dw[[0, 1, 3]].any() and torch.isinf(dy[4:6]).all() and not dy[:4].any()


def test_empty_calls():
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i = lambda n: z(n, d=torch.int32)  # noqa: E731
    assert qm.invert_perm(i(0)).shape == (0,)
    assert qm.gather_rows(z(0, 8), i(0), top_k=2).shape == (0, 8) and qm.gather_rows(z(3, 0), i(6), top_k=2).shape == (6, 0)
    assert qm.combine_rows(z(0, 8), z(0, 2)).shape == (0, 8) and qm.combine_rows(z(6, 0), z(3, 2)).shape == (3, 0)
    dy, dw = qm.combine_rows_grad(z(3, 0), z(6, 0), torch.ones(3, 2, device="cuda"))
    assert dy.shape == (6, 0) and dw.shape == (3, 2) and not dw.any()
    err = i(1)
    out = torch.full((2, 4), 7.0, device="cuda")
    qm.gather_rows(z(0, 4), i(2), out=out, err=err)                    # no token at all: both entries are out of range
    assert (out == 7).all() and err.item() == 16
    all_dropped = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    assert not qm.combine_rows(z(0, 4), torch.ones(2, 2, device="cuda"), all_dropped).any()


def test_refusals_on_the_device():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i, w = z(4, d=torch.int32), z(2, 2, d=torch.float32)
    bad = [lambda: qm.gather_rows(z(4, 32)[:, :16], i), lambda: qm.gather_rows(z(4, 8), i, top_k=0),
           lambda: qm.gather_rows(z(4, 8), i, x_order="bucket"), lambda: qm.gather_rows(z(3, 8), i, top_k=2, x_order="slot"),
           lambda: qm.gather_rows(z(2, 8), i, top_k=2, weights=w[:1]), lambda: qm.gather_rows(z(2, 8), i, out_dtype="f64"),
           lambda: qm.gather_rows(z(2, 8), i, out=z(2, 8)), lambda: qm.gather_rows(z(2, 8), i[None]),
           lambda: qm.combine_rows(z(5, 8), w), lambda: qm.combine_rows(z(4, 8), w, top_k=4),
           lambda: qm.combine_rows(z(4, 8), w, y_shared=z(2, 4)), lambda: qm.combine_rows(z(4, 8), w, i[:3]),
           lambda: qm.combine_rows(z(4, 8), w, out=z(4, 8)), lambda: qm.combine_rows(z(4, 8), top_k=0),
           lambda: qm.combine_rows_grad(z(3, 8), z(4, 8), w), lambda: qm.combine_rows_grad(z(2, 8), z(6, 8), w),
           lambda: qm.combine_rows_grad(z(2, 8), z(4, 8), w, out=z(4, 4)), lambda: qm.invert_perm(i, -1),
           lambda: qm.invert_perm(i, 1 << 32), lambda: qm.gather_rows(z(2, 8), i, top_k=1 << 32)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: qm.combine_rows(z(4, 8), w, y_shared=z(2, 8, d=torch.float16)),
                 lambda: qm.combine_rows(z(4, 8), w.bfloat16()), lambda: qm.combine_rows(z(4, 8), w, i.long()),
                 lambda: qm.combine_rows_grad(z(2, 8), z(4, 8), w, out=z(4, 8, d=torch.float32))):
        with pytest.raises(TypeError):
            call()


def test_rows_past_32_bits():
    """Rows, outputs and gradients longer than 2^32 elements; those at the far end are right."""
    n, d = 70000, 65536                                                  # bf16: 9.2 GB
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.tensor([[1.0], [2.0], [3.0]], device="cuda")
    perm = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    perm[-2:] = torch.tensor([n - 1, n - 3], dtype=torch.int32)
    out = torch.full((n, d), 7.0, dtype=torch.bfloat16, device="cuda")
    qm.gather_rows(x, perm, out=out)
    assert (out[-2] == 3).all() and (out[-1] == 1).all() and (out[-3] == 7).all() and (out[0] == 7).all()
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos[-1] = n - 2
    w = torch.full((n, 1), 2.0, device="cuda")
    qm.combine_rows(x, w, pos, out=out)
    assert (out[-1] == 4).all() and not out[-2].any()
    pos.fill_(-1)
    pos[-1] = n - 1
    dy, dw = qm.combine_rows_grad(x, x, w, pos, out=out)
    assert (dy[-1] == 6).all() and not dy[-2].any() and dw[-1] == 9 * d and not dw[:-1].any()
