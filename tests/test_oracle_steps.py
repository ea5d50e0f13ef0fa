"""Pins of the oracle's row steps, SwiGLU and 4-bit products, on the CPU: against other definitions of the same
(matrices, torch's autograd in float64, integer streams) and by worked examples."""
import numpy as np
import torch

import oracle
from tests import _packing


def _routing(seed, T, k, E):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).reshape(-1)
    return rng, np.argsort(ids, kind="stable").astype(np.int32)


def test_invert_perm():
    _, perm = _routing(0, 30, 3, 7)
    pos = oracle.invert_perm(perm, 90)
    assert np.array_equal(perm[pos], np.arange(90)) and np.array_equal(pos, np.argsort(perm))
    assert oracle.invert_perm([3, -1, 0, 3, 9], 5).tolist() == [2, -1, -1, 3, -1]
    assert oracle.invert_perm([], 2).tolist() == [-1, -1]


def test_gather_and_combine_are_transposed_matrices():
    T, k, d = 11, 3, 5
    rng, perm = _routing(1, T, k, 6)
    w = rng.standard_normal((T, k)).astype(np.float32)
    G = np.zeros((T * k, T))
    G[np.arange(T * k), perm // k] = w.reshape(-1)[perm]
    x, y = rng.standard_normal((T, d)), rng.standard_normal((T * k, d))
    assert np.allclose(oracle.gather_rows(x, perm, k, "token", w), G @ x, rtol=1e-15)
    out, mag = oracle.combine_rows(y, w, oracle.invert_perm(perm, T * k), T, k)
    assert np.allclose(out, G.T @ y, rtol=1e-13, atol=1e-13) and np.all(mag >= np.abs(out) - 1e-12)
    assert np.array_equal(oracle.gather_rows(y, perm, k, "slot"), y[perm])


def test_dropped_rows():
    y = np.arange(6.0).reshape(3, 2)
    out, _ = oracle.combine_rows(y, None, np.array([2, -1, -1, -1, 0, 1]), 3, 2, np.ones((3, 2)))
    assert out.tolist() == [[5, 6], [1, 1], [3, 5]]
    got = oracle.gather_rows(y, [1, -1, 5, 6], 2, "token")
    assert np.array_equal(got[[0, 2]], y[[0, 2]]) and np.isnan(got[[1, 3]]).all()


def test_combine_gradient_is_autograds():
    T, k, d = 9, 4, 7
    rng, perm = _routing(2, T, k, 5)
    pos = oracle.invert_perm(perm, T * k)
    y, w, g = rng.standard_normal((T * k, d)), rng.standard_normal((T, k)).astype(np.float32), rng.standard_normal((T, d))
    ty, tw = torch.from_numpy(y).requires_grad_(), torch.from_numpy(w).double().requires_grad_()
    out = (ty[torch.from_numpy(pos).long()].reshape(T, k, d) * tw[..., None]).sum(1)
    (out * torch.from_numpy(g)).sum().backward()
    dy, dw, _ = oracle.combine_rows_grad(g, y, w, pos)
    assert np.allclose(dy, ty.grad, rtol=1e-14) and np.allclose(dw, tw.grad, rtol=1e-13)


def test_swiglu_and_its_gradient_are_autograds():
    rng = np.random.default_rng(3)
    gu, dh = rng.standard_normal((6, 20)) * 8, rng.standard_normal((6, 10))
    t = torch.from_numpy(gu).requires_grad_()
    h = torch.nn.functional.silu(t[:, :10]) * t[:, 10:]
    (h * torch.from_numpy(dh)).sum().backward()
    assert np.allclose(oracle.swiglu(gu), h.detach(), rtol=1e-13)
    grad, mag = oracle.swiglu_grad(gu, dh)
    assert np.allclose(grad, t.grad, rtol=1e-12) and np.all(mag >= np.abs(grad) * (1 - 1e-12))
    step = 1e-5
    for c in (0, 7, 13):
        up, low = gu.copy(), gu.copy()
        up[:, c] += step
        low[:, c] -= step
        diff = ((oracle.swiglu(up) - oracle.swiglu(low)) * dh).sum(1) / (2 * step)
        # third derivatives of silu stay below 1: step^2 / 6 of |u| <= 40 and |dh| <= 4, and roundings of 1e-14 / step
        assert np.all(np.abs(diff - grad[:, c]) <= 2e-8)


def test_swiglu_far_out():
    gu = np.array([[1000.0, 2.0], [-1000.0, 2.0], [-700.0, 1.0], [0.0, 5.0]])
    h, (g, _) = oracle.swiglu(gu), oracle.swiglu_grad(gu, np.ones((4, 1)))
    assert h[0] == 2000 and abs(h[1]) < 1e-300 and h[3] == 0 and g[0].tolist() == [2, 1000] and g[3].tolist() == [2.5, 0]
    assert 0 < -h[2, 0] < 1e-300


def test_packed_weights_by_integer_streams():
    rng = np.random.default_rng(4)
    q = rng.integers(0, 16, (2, 3, 64))
    s, b = rng.standard_normal((2, 3, 2)).astype(np.float16), rng.standard_normal((2, 3, 2)).astype(np.float16)
    codes = np.stack([_packing.pack_codes(m, 4) for m in q])
    w, mag = oracle.packed_weights(codes, s, b)
    for e, r, c in [(0, 0, 0), (1, 2, 63), (0, 1, 31), (1, 0, 32)]:
        sv, bv = float(s[e, r, c // 32]), float(b[e, r, c // 32])
        assert w[e, r, c] == sv * q[e, r, c] + bv and mag[e, r, c] == abs(sv) * q[e, r, c] + abs(bv)
    e8 = rng.integers(100, 140, (2, 3, 2)).astype(np.uint8)
    w, mag = oracle.packed_weights(codes, e8, None)
    table = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for e, r, c in [(0, 0, 0), (1, 2, 63), (0, 1, 31), (1, 0, 32)]:
        v = q[e, r, c]
        assert w[e, r, c] == (-1) ** (v >> 3) * table[v & 7] * 2.0 ** (int(e8[e, r, c // 32]) - 127)
    x = rng.standard_normal((5, 64))
    y, m = oracle.matmul_packed(x, codes[1], e8[1], None)
    assert np.allclose(y, x @ w[1].T) and np.all(m >= np.abs(y) - 1e-12)
