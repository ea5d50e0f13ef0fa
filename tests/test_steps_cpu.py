"""Refusals of the steps around the experts' products, without a GPU: the C
entry points return the documented status before any launch (fake device
addresses, never dereferenced), and the Python calls refuse host tensors, other
types, shapes and operands that require grad before they reach the library."""
import os

import pytest
import torch

import quantized_sparse_moe_amd as qm
from quantized_sparse_moe_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libqsmoe.so not built")

F = 0x10000
OK, INVALID, UNSUPPORTED, ALIGNMENT = (_lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED,
                                       _lib.MOE_ERR_ALIGNMENT)
BIG = (1 << 30) + 1


def invert(perm=F, n=4, size=4, positions=F, err=None):
    return qm.load().moe_invert_perm(perm, n, size, positions, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(size=-1), INVALID), (dict(perm=None), INVALID), (dict(positions=None), INVALID),
    (dict(n=BIG), UNSUPPORTED), (dict(size=BIG), UNSUPPORTED), (dict(perm=F + 2), ALIGNMENT),
    (dict(positions=F + 1), ALIGNMENT), (dict(err=F + 2), ALIGNMENT), (dict(size=0, positions=None), OK),
])
def test_invert_perm_validates(kw, status):
    assert invert(**kw) == status


def gather(x=F, dtype=0, T=2, k=2, d=8, x_order=1, perm=F, n=4, w=None, out_dtype=0, out=F, err=None):
    return qm.load().moe_gather_rows(x, dtype, T, k, d, x_order, perm, n, w, out_dtype, out, err, None)


def combine(y=F, dtype=0, n=4, positions=F, w=None, shared=None, T=2, k=2, d=8, out_dtype=0, out=F, err=None):
    return qm.load().moe_combine_rows(y, dtype, n, positions, w, shared, T, k, d, out_dtype, out, err, None)


def combine_grad(dout=F, out_dtype=0, y=F, dtype=0, n=4, positions=F, w=F, T=2, k=2, d=8, dy=F, dw=F, err=None):
    return qm.load().moe_combine_rows_grad(dout, out_dtype, y, dtype, n, positions, w, T, k, d, dy, dw, err, None)


TOKENS = [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(n=-1), INVALID), (dict(d=-1), INVALID), (dict(dtype=3), INVALID),
    (dict(out_dtype=-1), INVALID), (dict(T=1 << 30, k=2), INVALID), (dict(T=BIG, k=1), UNSUPPORTED),
    (dict(n=BIG), UNSUPPORTED), (dict(d=(1 << 20) + 1), UNSUPPORTED), (dict(err=F + 2), ALIGNMENT), (dict(w=F + 2), ALIGNMENT),
]


@pytest.mark.parametrize("kw,status", TOKENS + [
    (dict(x_order=0), INVALID), (dict(x_order=3), INVALID), (dict(x=None), INVALID), (dict(perm=None), INVALID),
    (dict(out=None), INVALID), (dict(x=F + 1), ALIGNMENT), (dict(x=F + 2, dtype=1), ALIGNMENT), (dict(out=F + 1), ALIGNMENT),
    (dict(perm=F + 2), ALIGNMENT), (dict(n=0, perm=None, out=None), OK), (dict(d=0, x=None), OK),
])
def test_gather_rows_validates(kw, status):
    assert gather(**kw) == status


@pytest.mark.parametrize("kw,status", TOKENS + [
    (dict(positions=None, n=3), INVALID), (dict(y=None), INVALID), (dict(out=None), INVALID), (dict(y=F + 1), ALIGNMENT),
    (dict(shared=F + 1), ALIGNMENT), (dict(shared=F + 2, dtype=1), ALIGNMENT), (dict(positions=F + 2), ALIGNMENT),
    (dict(out=F + 2, out_dtype=1), ALIGNMENT), (dict(T=0, y=None, out=None), OK), (dict(d=0, out=None), OK),
])
def test_combine_rows_validates(kw, status):
    assert combine(**kw) == status


@pytest.mark.parametrize("kw,status", TOKENS + [
    (dict(positions=None, n=5), INVALID), (dict(w=None), INVALID), (dict(dw=None), INVALID), (dict(y=None), INVALID),
    (dict(dy=None), INVALID), (dict(dout=None), INVALID), (dict(dout=F + 2, out_dtype=1), ALIGNMENT),
    (dict(dy=F + 1), ALIGNMENT), (dict(dw=F + 2), ALIGNMENT), (dict(y=F + 1), ALIGNMENT), (dict(T=0, dw=None), OK),
])
def test_combine_rows_grad_validates(kw, status):
    assert combine_grad(**kw) == status


def swiglu(gu=F, dtype=0, rows=2, inner=8, h=F):
    return qm.load().moe_swiglu(gu, dtype, rows, inner, h, None)


def swiglu_grad(gu=F, dtype=0, dh=F, dh_dtype=0, rows=2, inner=8, h=F):
    return qm.load().moe_swiglu_grad(gu, dtype, dh, dh_dtype, rows, inner, h, None)


@pytest.mark.parametrize("call", [swiglu, swiglu_grad])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INVALID), (dict(rows=-1), INVALID), (dict(inner=-1), INVALID), (dict(gu=None), INVALID),
    (dict(h=None), INVALID), (dict(inner=(1 << 20) + 1), UNSUPPORTED), (dict(rows=1 << 60), UNSUPPORTED),
    (dict(gu=F + 1), ALIGNMENT), (dict(h=F + 2, dtype=1), ALIGNMENT), (dict(rows=0, gu=None), OK), (dict(inner=0, h=None), OK),
])
def test_swiglu_validates(call, kw, status):
    assert call(**kw) == status


def test_swiglu_grad_validates_dh():
    assert swiglu_grad(dh=None) == INVALID and swiglu_grad(dh_dtype=4) == INVALID
    assert swiglu_grad(dh=F + 2, dh_dtype=1) == ALIGNMENT


def packed(x=F, dtype=0, codes=F, scales=F, biases=F, format=0, group=64, T=2, N=8, K=64, out_dtype=0, out=F):
    return qm.load().moe_matmul_packed(x, dtype, codes, scales, biases, format, group, T, N, K, out_dtype, out, None)


def grouped(x=F, dtype=0, codes=F, scales=F, biases=F, format=0, group=64, T=2, k=2, N=8, K=64, E=4, offsets=F, perm=F,
            x_order=0, out_order=0, out_dtype=0, out=F, err=None):
    return qm.load().moe_grouped_matmul_packed(x, dtype, codes, scales, biases, format, group, T, k, N, K, E, offsets,
                                               perm, x_order, out_order, out_dtype, out, err, None)


@pytest.mark.parametrize("call", [packed, grouped])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-32), INVALID), (dict(dtype=3), INVALID),
    (dict(out_dtype=3), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(group=16), UNSUPPORTED), (dict(group=0), UNSUPPORTED),
    (dict(format=2, group=32, biases=None), UNSUPPORTED), (dict(format=1), UNSUPPORTED), (dict(K=0), UNSUPPORTED),
    (dict(K=48, group=32), UNSUPPORTED), (dict(K=96), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED),
    (dict(K=(1 << 20) + 64), UNSUPPORTED), (dict(T=BIG // 2 + 1), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(biases=None), INVALID), (dict(out=None), INVALID),
    (dict(format=1, group=32), INVALID), (dict(x=F + 8), ALIGNMENT), (dict(codes=F + 4), ALIGNMENT),
    (dict(scales=F + 1), ALIGNMENT), (dict(biases=F + 1), ALIGNMENT), (dict(out=F + 1), ALIGNMENT),
    (dict(out=F + 2, out_dtype=1), ALIGNMENT), (dict(T=0, x=None, out=None), OK), (dict(N=0, codes=None), OK),
])
def test_packed_products_validate(call, kw, status):
    if call is packed and kw.get("T") == BIG // 2 + 1:
        kw = dict(T=BIG)
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), INVALID), (dict(E=0), INVALID), (dict(E=1025), UNSUPPORTED), (dict(T=1 << 30, k=2), INVALID),
    (dict(x_order=3), INVALID), (dict(out_order=1), INVALID), (dict(offsets=None), INVALID),
    (dict(perm=None, x_order=1), INVALID), (dict(perm=None, out_order=2), INVALID), (dict(offsets=F + 2), ALIGNMENT),
    (dict(perm=F + 1), ALIGNMENT), (dict(err=F + 2), ALIGNMENT),
])
def test_grouped_packed_products_validate_the_groups(kw, status):
    assert grouped(**kw) == status


X, I32 = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
W = torch.ones(2, 2)
CODES, S16 = torch.zeros(3, 8, 8, dtype=torch.int32), torch.zeros(3, 8, 1, dtype=torch.float16)
CALLS = {
    "invert_perm": lambda: qm.invert_perm(I32),
    "gather_rows": lambda: qm.gather_rows(X, I32),
    "combine_rows": lambda: qm.combine_rows(X, W),
    "combine_rows_grad": lambda: qm.combine_rows_grad(X[:2], X, W),
    "swiglu": lambda: qm.swiglu(X),
    "swiglu_grad": lambda: qm.swiglu_grad(X, X[:, :32]),
    "matmul_packed": lambda: qm.matmul_packed(X, CODES[0], S16[0], S16[0]),
    "grouped_matmul_packed": lambda: qm.grouped_matmul_packed(X, CODES, S16, S16, I32),
}


@pytest.mark.parametrize("name", CALLS)
def test_python_calls_refuse_host_tensors(name):
    with pytest.raises(ValueError, match="contiguous device tensor"):
        CALLS[name]()


def test_python_calls_refuse_other_types():
    for call in (lambda: qm.invert_perm(I32.long()), lambda: qm.gather_rows(X.double(), I32),
                 lambda: qm.combine_rows(X.double()), lambda: qm.swiglu(X.double()),
                 lambda: qm.matmul_packed(X.float(), CODES[0], S16[0], S16[0])):
        with pytest.raises(TypeError):
            call()


def test_python_calls_refuse_operands_that_require_grad():
    g = lambda t: t.clone().requires_grad_()  # noqa: E731
    calls = [lambda: qm.gather_rows(g(X), I32), lambda: qm.gather_rows(X, I32, weights=g(W)),
             lambda: qm.combine_rows(g(X), W), lambda: qm.combine_rows(X, g(W)),
             lambda: qm.combine_rows(X, W, y_shared=g(X[:2])), lambda: qm.combine_rows_grad(g(X[:2]), X, W),
             lambda: qm.combine_rows_grad(X[:2], g(X), W), lambda: qm.combine_rows_grad(X[:2], X, g(W)),
             lambda: qm.swiglu(g(X)), lambda: qm.swiglu_grad(g(X), X[:, :32]), lambda: qm.swiglu_grad(X, g(X[:, :32])),
             lambda: qm.matmul_packed(g(X), CODES[0], S16[0], S16[0]),
             lambda: qm.matmul_packed(X, CODES[0], g(S16[0]), S16[0]),
             lambda: qm.grouped_matmul_packed(X, CODES, S16, g(S16), I32)]
    for call in calls:
        with pytest.raises(RuntimeError, match="not recorded by autograd"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="contiguous device tensor"):
            call()
