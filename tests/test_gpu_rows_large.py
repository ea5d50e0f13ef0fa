"""Gathers whose result no cache holds (over 32 MiB, 8 slices of columns and
more), which go through the slices' kernel: every pair of types, copied and
weighted, token and slot order, last slices and last lanes that are not full,
numbers of slices that are no multiple of 8, positions that do not fill the last
workgroup, odd addresses, with everything around the written rows left alone.

Without weights the value is the input's, rounded once to the output: compared
bit for bit with the conversion. With them one fp32 product, 2^-24 of it, and one
rounding: |got - w x| <= (2^-24 (1 + h) + h) |w x| + half of the smallest
subnormals, h half a step of the output's type."""
import pytest
import torch

import quantized_sparse_moe_amd as qm
from tests._steps import DT, HALF, LEAST

pytestmark = pytest.mark.gpu

SHAPES = [(1639, 5, 2049, "token"), (1366, 6, 2305, "slot"), (1371, 3, 4099, "token"), (2049, 2, 4096, "token"),
          (4101, 1, 4104, "slot")]
LEFT = 7.0


def shifted(n, d, dtype, by):
    """(a matrix whose first element is `by` elements into its memory, all of that memory), filled with LEFT."""
    whole = torch.full((n * d + by + 64,), LEFT, dtype=dtype, device="cuda")
    return whole[by:by + n * d].view(n, d), whole


@pytest.mark.parametrize("T,k,d,order", SHAPES)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("weighted", [False, True])
def test_large_gathers(T, k, d, order, dtype, out, weighted):
    n = T * k
    assert n * d * (4 if out == "f32" else 2) > 32 << 20 and n % 8 != 0
    assert d > 7 * 32 * (4 if "f32" in (dtype, out) else 8)
    g = torch.Generator("cuda").manual_seed(n + d)
    x, _ = shifted(T if order == "token" else n, d, DT[dtype], 1)
    x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    perm[torch.rand(n, generator=g, device="cuda") < 0.05] = -1
    perm[0], perm[-1] = -1, 1
    w = torch.rand(T, k, generator=g, device="cuda") if weighted else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, whole = shifted(n, d, DT[out], 37)
    qm.gather_rows(x, perm, k, order, w, out=y, err=err)
    assert err.item() == 0 and (whole[:37] == LEFT).all() and (whole[37 + n * d:] == LEFT).all()
    there = perm >= 0
    assert (y[~there] == LEFT).all()
    a = perm[there].long()
    rows = x[a // k if order == "token" else a]
    if not weighted:
        assert torch.equal(y[there], rows.to(DT[out]))
        return
    want = rows.double() * w.reshape(-1)[a].double()[:, None]
    h = HALF[out]
    allowed = (2.0 ** -24 * (1 + h) + h) * want.abs() + LEAST[out] + LEAST["f32"]
    assert ((y[there].double() - want).abs() <= allowed).all()


def test_bad_entries_of_a_large_gather_are_reported_and_write_nothing():
    T, k, d = 1500, 6, 2112
    x = torch.randn(T, d, device="cuda").bfloat16()
    perm = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0)
    good = qm.gather_rows(x, perm, k)
    for at, bad in ((0, T * k), (5000, -2), (T * k - 1, 2 ** 31 - 1)):
        p, err = perm.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        p[at] = bad
        y = qm.gather_rows(x, p, k, out=torch.full_like(good, LEFT), err=err)
        assert err.item() == 16 and (y[at] == LEFT).all()
        assert torch.equal(y[:at], good[:at]) and torch.equal(y[at + 1:], good[at + 1:])
