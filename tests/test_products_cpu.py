"""Refusals of the block-scaled FP8 and grouped products, without a GPU: the C
entry points return the documented status before any launch (fake device
addresses, never dereferenced), and the Python calls refuse host tensors,
other types and shapes before they reach the library."""
import os

import pytest
import torch

import quantized_sparse_moe_amd as qm
from quantized_sparse_moe_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libqsmoe.so not built")

F = 0x10000
OK, INVALID, UNSUPPORTED, ALIGNMENT = (_lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED,
                                       _lib.MOE_ERR_ALIGNMENT)


def quant(x=F, dtype=0, matrices=1, rows=2, cols=128, block_rows=1, codes=F, scales=F, err=None):
    return qm.load().moe_quantize_block(x, dtype, matrices, rows, cols, block_rows, 0, codes, scales, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INVALID), (dict(rows=-1), INVALID), (dict(matrices=-1), INVALID), (dict(cols=-16), INVALID),
    (dict(cols=120), UNSUPPORTED), (dict(block_rows=64), UNSUPPORTED), (dict(rows=1 << 60, cols=1 << 20), UNSUPPORTED),
    (dict(rows=1 << 40), UNSUPPORTED), (dict(rows=1 << 50, block_rows=128), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(x=F + 2), ALIGNMENT), (dict(codes=F + 8), ALIGNMENT), (dict(scales=F + 2), ALIGNMENT),
    (dict(err=F + 1), ALIGNMENT), (dict(rows=0, x=None), OK), (dict(cols=0, x=None), OK),
    (dict(matrices=0, x=None), OK),
])
def test_quantize_block_validates(kw, status):
    assert quant(**kw) == status


def swiglu(gu=F, dtype=0, rows=2, inner=128, codes=F, scales=F, err=None):
    return qm.load().moe_swiglu_quantize_block(gu, dtype, rows, inner, 0, codes, scales, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID), (dict(inner=-16), INVALID), (dict(inner=24), UNSUPPORTED),
    (dict(rows=1 << 40), UNSUPPORTED), (dict(gu=None), INVALID), (dict(codes=F + 4), ALIGNMENT),
    (dict(rows=0, gu=None), OK), (dict(inner=0, gu=None), OK),
])
def test_swiglu_quantize_block_validates(kw, status):
    assert swiglu(**kw) == status


def dense(a=F, sa=F, b=F, sb=F, M=2, N=8, K=16, out_dtype=0, out=F):
    return qm.load().moe_matmul_block(a, sa, b, sb, M, N, K, out_dtype, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(N=-8), INVALID), (dict(K=-16), INVALID), (dict(out_dtype=3), INVALID),
    (dict(K=24), UNSUPPORTED), (dict(N=12), UNSUPPORTED), (dict(N=(1 << 20) + 8), UNSUPPORTED),
    (dict(M=(1 << 30) + 1), UNSUPPORTED),
    (dict(K=(1 << 20) + 16), UNSUPPORTED), (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(b=None), INVALID),
    (dict(sb=None), INVALID), (dict(out=None), INVALID), (dict(a=F + 8), ALIGNMENT), (dict(b=F + 1), ALIGNMENT),
    (dict(sa=F + 2), ALIGNMENT), (dict(sb=F + 2), ALIGNMENT), (dict(out=F + 8), ALIGNMENT),
    (dict(M=0, a=None, out=None), OK), (dict(N=0, b=None, out=None), OK),
])
def test_matmul_block_validates(kw, status):
    assert dense(**kw) == status


def grouped_block(a=F, sa=F, w=F, sw=F, T=2, k=2, N=8, K=16, E=4, offsets=F, perm=F, a_order=0, out_order=0,
                  out_dtype=0, out=F, err=None):
    return qm.load().moe_grouped_matmul_block(a, sa, w, sw, T, k, N, K, E, offsets, perm, a_order, out_order,
                                              out_dtype, out, err, None)


def grouped(x=F, w=F, dtype=0, T=2, k=2, N=8, K=8, E=4, offsets=F, perm=F, x_order=0, out_order=0, transposed=0,
            out_dtype=0, out=F, err=None):
    return qm.load().moe_grouped_matmul(x, w, dtype, T, k, N, K, E, offsets, perm, x_order, out_order, transposed,
                                        out_dtype, out, err, None)


def grouped_dw(x=F, dy=F, dtype=0, T=2, k=2, N=8, K=8, E=4, offsets=F, perm=F, x_order=0, dy_order=0, out_dtype=1,
               out=F, err=None):
    return qm.load().moe_grouped_matmul_dw(x, dy, dtype, T, k, N, K, E, offsets, perm, x_order, dy_order, out_dtype,
                                           out, err, None)


SHARED = [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(N=-8), INVALID), (dict(K=-16), INVALID), (dict(E=0), INVALID),
    (dict(T=1 << 30, k=2), INVALID), (dict(T=(1 << 30) + 1, k=1), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(N=(1 << 20) + 16), UNSUPPORTED),
    (dict(K=(1 << 20) + 16), UNSUPPORTED), (dict(N=12), UNSUPPORTED), (dict(out_dtype=5), INVALID),
    (dict(offsets=None), INVALID), (dict(out=None), INVALID), (dict(offsets=F + 2), ALIGNMENT),
    (dict(perm=F + 2), ALIGNMENT), (dict(out=F + 8), ALIGNMENT), (dict(err=F + 2), ALIGNMENT),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(K=24), UNSUPPORTED), (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(w=None), INVALID),
    (dict(sw=None), INVALID), (dict(a=F + 8), ALIGNMENT), (dict(sw=F + 1), ALIGNMENT),
    (dict(a_order=3), INVALID), (dict(out_order=1), INVALID), (dict(perm=None, a_order=1), INVALID),
    (dict(perm=None, out_order=2), INVALID), (dict(T=0, a=None, offsets=None, out=None), OK), (dict(N=0), OK),
])
def test_grouped_matmul_block_validates(kw, status):
    assert grouped_block(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(K=12), UNSUPPORTED), (dict(dtype=1), UNSUPPORTED), (dict(dtype=4), INVALID), (dict(x=None), INVALID),
    (dict(w=F + 4), ALIGNMENT), (dict(x_order=-1), INVALID), (dict(out_order=1), INVALID),
    (dict(perm=None, x_order=2), INVALID), (dict(T=0, x=None, perm=None, x_order=1), OK), (dict(N=0, w=None), OK),
    (dict(K=0, transposed=1, w=None), OK),
])
def test_grouped_matmul_validates(kw, status):
    assert grouped(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(K=12), UNSUPPORTED), (dict(dtype=1), UNSUPPORTED), (dict(dy=None), INVALID), (dict(x=F + 4), ALIGNMENT),
    (dict(dy_order=1), INVALID), (dict(perm=None, dy_order=2), INVALID), (dict(N=0, out=None), OK),
    (dict(K=0, out=None), OK),
])
def test_grouped_matmul_dw_validates(kw, status):
    assert grouped_dw(**kw) == status


def test_python_calls_refuse_host_tensors_types_and_shapes():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    q, s = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1)
    for call in (lambda: qm.quantize_block(x), lambda: qm.swiglu_quantize_block(x),
                 lambda: qm.matmul_block(q, s, q, s), lambda: qm.grouped_matmul(x, w, off),
                 lambda: qm.grouped_matmul_dw(x, x, off),
                 lambda: qm.grouped_matmul_block(q, s, torch.zeros(2, 8, 16, dtype=torch.uint8), s, off)):
        with pytest.raises(ValueError, match="contiguous device tensor"):
            call()
    with pytest.raises(TypeError):
        qm.quantize_block(x.to(torch.float64))
    with pytest.raises(TypeError):
        qm.grouped_matmul(x.float(), w.float(), off)
    with pytest.raises(TypeError):
        qm.matmul_block(x, s, q, s)


def test_f32_sums_is_a_flag_of_the_fp8_products():
    S = _lib.MOE_SUMS_F32
    for dt in _lib.MOE_DT.values():
        assert dense(M=0, out_dtype=dt | S) == OK and grouped_block(N=0, out_dtype=dt | S) == OK
    for call in (dense, grouped_block):
        for bad in (3 | S, S << 1, -1):
            assert call(out_dtype=bad) == INVALID
    assert grouped(out_dtype=S) == INVALID and grouped_dw(out_dtype=1 | S) == INVALID


def test_products_refuse_operands_that_require_grad():
    """autograd does not record these calls: a result without a grad_fn would lose the gradients in silence. Under
    no_grad and inside an autograd.Function the calls go on (here to the refusal of host tensors)."""
    x, w, dy = torch.zeros(4, 16), torch.zeros(2, 8, 16), torch.zeros(4, 8)
    x, w, dy = (t.bfloat16() for t in (x, w, dy))
    off = torch.zeros(3, dtype=torch.int32)
    q, s = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1)
    g = lambda t: t.clone().requires_grad_()  # noqa: E731
    calls = [lambda: qm.grouped_matmul(g(x), w, off), lambda: qm.grouped_matmul(x, g(w), off),
             lambda: qm.grouped_matmul(dy, g(w), off, transposed=True),
             lambda: qm.grouped_matmul_dw(g(x), dy, off), lambda: qm.grouped_matmul_dw(x, g(dy), off),
             lambda: qm.matmul_block(q, g(s), q, s), lambda: qm.matmul_block(q, s, q, g(s)),
             lambda: qm.grouped_matmul_block(q, g(s), q[None], s[None], off),
             lambda: qm.grouped_matmul_block(q, s, q[None], g(s[None]), off)]
    for call in calls:
        with pytest.raises(RuntimeError, match="not recorded by autograd"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="contiguous device tensor"):
            call()

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            return qm.grouped_matmul(x, w, off)
    with pytest.raises(ValueError, match="contiguous device tensor"):
        Product.apply(g(x), g(w))


@pytest.mark.parametrize("route", ["topk", "hash"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 6), (7, 33, 2), (300, 1000, 8)])
def test_a_router_without_packed_experts_sizes_its_workspace(route, T, E, k):
    """The size is what moe_route asks for: with a byte less it refuses the workspace, with all of them it comes to the
    next check (a misaligned one)."""
    wr, table = torch.zeros(E, 64), torch.zeros(10, k, dtype=torch.int32)
    layer = qm.DeviceLayer(route, k, wr, None, table if route == "hash" else None)
    n = layer.workspace_size(T)
    call = lambda ws, size: qm.load().moe_route(layer.router_c, F, F, T, F, F, ws, size, None)  # noqa: E731
    assert call(F, n - 1) == _lib.MOE_ERR_WORKSPACE and call(F + 64, n) == ALIGNMENT
    assert layer.workspace_size(0) >= 256 and layer.I == 0 and layer.clone().workspace_size(T) == n
    with pytest.raises(_lib.MoeError):
        layer.workspace_size(-1)


def test_a_router_without_packed_experts_is_refused_where_experts_run():
    layer = qm.DeviceLayer("topk", 2, torch.zeros(4, 64), None, None)
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    for call in (lambda: layer.workspace_layout(3), lambda: layer.c, lambda: qm.expert_ffn(layer, x, x, x, x)):
        with pytest.raises(ValueError, match="router without packed experts"):
            call()
    with pytest.raises(ValueError, match="needs routed experts"):
        qm.DeviceLayer("topk", 2, torch.zeros(4, 64), None, None, None, object())


@pytest.mark.parametrize("cols", [(1 << 31) - 16, (1 << 31) - 112, (1 << 31) - 128])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_block_counts_the_blocks_of_the_longest_rows(cols, block_rows):
    """2^24 blocks in a row (one fewer for the last size): 64 rows of them are more workgroups than a grid holds, and a
    count that wraps would not say so."""
    assert quant(cols=cols, block_rows=block_rows, rows=64 if block_rows == 1 else 257) == UNSUPPORTED
