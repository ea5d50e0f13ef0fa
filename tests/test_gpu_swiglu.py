"""SwiGLU and its gradient against the float64 oracle.

Errors allowed: in fp32 the exponential and the reciprocal are off by a step
(2^-23) each, the sum 1 + e^-g and every product by half a step (2^-24). h = u (g
s): 2^-23 (exponential) + 2^-24 (sum) + 2^-23 (reciprocal) + 2 * 2^-24 (products)
< 4 * 2^-23. 1 - s is e^-g s: another 2^-23 + 2^-24; so dg = dh u s (1 + g t) with
four products and a fused one: < 8 * 2^-23 of |dh u s| (1 + |g t|). Then one
rounding to the type. s below 2^-126 is off by up to a subnormal step, 2^-149, and so is every product: (1 + |g|) (1 +
|u|) (1 + |dh|) of them, |g| up to 104, beyond which s is 0."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm
from tests._steps import DT, close, dev, shifted

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 2048), (6, 2048), (33, 17), (257, 144), (100, 1003), (2000, 24), (3, 8195)]


def check(gu, dh, dtype, dh_type):
    a, d = torch.from_numpy(gu).to(DT[dtype]), torch.from_numpy(dh).to(DT[dh_type])
    a64, d64 = a.double().numpy(), d.double().numpy()
    h, g = qm.swiglu(a.cuda()), qm.swiglu_grad(a.cuda(), d.cuda())
    assert h.dtype == g.dtype == DT[dtype] and g.shape == a.shape
    want = oracle.swiglu(a64)
    g64, u64 = np.split(a64, 2, axis=1)
    least = 2.0 ** -149 * (1 + np.minimum(np.abs(g64), 104)) * (1 + np.abs(u64))
    close(h, want, 4 * 2.0 ** -23 * np.abs(want) + least, dtype)
    want, mag = oracle.swiglu_grad(a64, d64)
    close(g, want, 8 * 2.0 ** -23 * mag + np.tile(least * (1 + np.abs(d64)), 2), dtype)


@pytest.mark.parametrize("rows,inner", SHAPES)
@pytest.mark.parametrize("dtype", DT)
def test_swiglu_and_gradient(rows, inner, dtype):
    rng = np.random.default_rng(rows + inner)
    gu = rng.standard_normal((rows, 2 * inner)) * np.exp(rng.standard_normal(2 * inner))
    for dh_type in (dtype, "f32"):
        check(gu, rng.standard_normal((rows, inner)), dtype, dh_type)


@pytest.mark.parametrize("dh_type", DT)
def test_types_of_the_gradient(dh_type):
    rng = np.random.default_rng(1)
    for dtype in DT:
        check(rng.standard_normal((5, 74)), rng.standard_normal((5, 37)), dtype, dh_type)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_far_out(dtype):
    """Gates from -120 to 120 (e^-g leaves fp32 at -88.7, s its normal range at -87.3), and of 1e30."""
    g = np.r_[np.linspace(-120, 120, 4001), -1e30, 1e30, 0.0, -0.0, 1e-30, -1e-30]
    gu = np.stack([np.r_[g, np.full(g.size, 1.25)], np.r_[g, np.full(g.size, -3e-3)]])
    dh = np.full((2, g.size), 0.75)
    check(gu, dh, dtype, dtype)


def test_infinities_and_nan_follow_the_formula():
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([[inf, -inf, nan, 1.0, 1.0, 0.0]], device="cuda")
    u = torch.tensor([[2.0, 2.0, 2.0, inf, nan, inf]], device="cuda")
    h = qm.swiglu(torch.cat([g, u], 1))[0].tolist()
    assert h[0] == inf and h[3] == inf and all(np.isnan(h[i]) for i in (1, 2, 4, 5))
    d = qm.swiglu_grad(torch.cat([g, u], 1), torch.ones(1, 6, device="cuda"))[0]
    assert torch.isnan(d[[1, 2, 4]]).all() and d[3] == inf and d[6] == inf and torch.isnan(d[[7, 8]]).all()
    assert torch.isfinite(d[9:]).all()


def test_gradient_equals_differences():
    """Central differences of swiglu in fp32, step 2^-6: the third derivative of silu is at most 0.5, so they are off by
    |u dh| 2^-12 / 12, and by the roundings of two values (4.5 * 2^-23 of each) over the step; in u the function is
    linear."""
    rng = np.random.default_rng(5)
    gu, dh = rng.uniform(-4, 4, (40, 64)).astype(np.float32), rng.uniform(-2, 2, (40, 32)).astype(np.float32)
    grad = qm.swiglu_grad(dev(gu), dev(dh)).double().cpu().numpy()
    step = np.float32(2.0 ** -6)
    for half in (0, 1):
        low, high = gu.copy(), gu.copy()
        low[:, 32 * half:32 * half + 32] -= step
        high[:, 32 * half:32 * half + 32] += step
        a, b = (qm.swiglu(dev(t)).double().cpu().numpy() for t in (low, high))
        moved = high.astype(np.float64)[:, 32 * half:32 * half + 32] - low[:, 32 * half:32 * half + 32]
        diff = (b - a) / moved * dh
        cut = np.abs(gu[:, 32:] * dh) * 2.0 ** -12 / 12 * 1.01 if half == 0 else 0.0
        tol = cut + np.abs(dh) * (np.abs(a) + np.abs(b)) * 4.5 * 2.0 ** -23 / moved + 9 * 2.0 ** -23 * 8 * np.abs(dh) * 5
        assert np.all(np.abs(diff - grad[:, 32 * half:32 * half + 32]) <= tol)


@pytest.mark.parametrize("dtype", DT)
def test_odd_addresses(dtype):
    rng = np.random.default_rng(3)
    rows, inner = 7, 29
    gu, dh = rng.standard_normal((rows, 2 * inner)), rng.standard_normal((rows, inner))
    a, d = torch.from_numpy(gu).to(DT[dtype]).cuda(), torch.from_numpy(dh).to(DT[dtype]).cuda()
    h, g = qm.swiglu(a), qm.swiglu_grad(a, d)
    for by in (1, 5):
        around = torch.full((g.numel() + 16,), 5.0, dtype=DT[dtype], device="cuda")
        at = around[by:by + h.numel()].view_as(h)
        assert torch.equal(qm.swiglu(shifted(gu, DT[dtype], by), out=at), h)
        assert (around[:by] == 5).all() and (around[by + h.numel():] == 5).all()
        at = around[by:by + g.numel()].view_as(g)
        assert torch.equal(qm.swiglu_grad(shifted(gu, DT[dtype], by), shifted(dh, DT[dtype], by + 1), out=at), g)
        assert (around[:by] == 5).all() and (around[by + g.numel():] == 5).all()


def test_rows_past_32_bits():
    rows, inner = (1 << 17) + 5, 16384                                    # gu: 4.3 G elements
    gu = torch.zeros(rows, 2 * inner, dtype=torch.bfloat16, device="cuda")
    gu[-1, :inner], gu[-1, inner:] = 100.0, 3.0
    h = qm.swiglu(gu)
    assert (h[-1] == 300).all() and not h[-2].any() and not h[0].any()
    dh = h.zero_()
    dh[-1] = 2.0
    dgu = qm.swiglu_grad(gu, dh, out=torch.empty_like(gu))
    assert (dgu[-1, :inner] == 6).all() and (dgu[-1, inner:] == 200).all() and not dgu[-2].any()


def test_empty_calls_and_refusals():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    assert qm.swiglu(z(0, 8)).shape == (0, 4) and qm.swiglu(z(3, 0)).shape == (3, 0)
    assert qm.swiglu_grad(z(0, 8), z(0, 4)).shape == (0, 8) and qm.swiglu_grad(z(3, 0), z(3, 0)).shape == (3, 0)
    for call in (lambda: qm.swiglu(z(2, 7)), lambda: qm.swiglu(z(2, 16)[:, :8]), lambda: qm.swiglu(z(8)),
                 lambda: qm.swiglu(z(2, 8), out=z(2, 8)), lambda: qm.swiglu_grad(z(2, 8), z(2, 8)),
                 lambda: qm.swiglu_grad(z(2, 7), z(2, 3)), lambda: qm.swiglu_grad(z(2, 8), z(2, 4), out=z(2, 4)),
                 lambda: qm.swiglu(z(0, 1 << 32))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: qm.swiglu(z(2, 8), out=z(2, 4, d=torch.float32)),
                 lambda: qm.swiglu_grad(z(2, 8), z(2, 4), out=z(2, 8, d=torch.float32))):
        with pytest.raises(TypeError):
            call()
