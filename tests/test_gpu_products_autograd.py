"""The grouped product inside a torch.autograd.Function, the way a training
program calls it: gradients against the formula, exact on integers, and no
product that autograd would lose."""
import numpy as np
import pytest
import torch

import quantized_sparse_moe_amd as qm

pytestmark = pytest.mark.gpu


class Grouped(torch.autograd.Function):
    """x in token order -> [T * k][N] in slot order."""

    @staticmethod
    def forward(ctx, x, w, offsets, perm, k):
        ctx.save_for_backward(x, w, offsets, perm)
        ctx.k = k
        return qm.grouped_matmul(x, w, offsets, perm=perm, top_k=k, x_order="token", out_order="slot")

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets, perm = ctx.saved_tensors
        kw = dict(perm=perm, top_k=ctx.k)
        dx = qm.grouped_matmul(dy, w, offsets, x_order="slot", out_order="slot", transposed=True, out_dtype="f32", **kw)
        ones = torch.ones(x.shape[0], ctx.k, device=x.device)
        dw = qm.grouped_matmul_dw(x, dy, offsets, x_order="token", dy_order="slot", **kw)
        return qm.combine(dx, ones, None, out_dtype="f32").to(x.dtype), dw.to(w.dtype), None, None, None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 3, 16, 24), (90, 3, 7, 136, 264)])
def test_gradients_inside_a_function(T, k, E, N, K, dtype):
    """Integers up to 2, and sums of at most 90 * 4 (dw), 136 * 2 * 3 (dx): integers to 256 are exact in bf16, larger
    ones are rounded once, as the reference is."""
    rng = np.random.default_rng(T + E)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).reshape(-1)
    perm = torch.from_numpy(np.argsort(ids, kind="stable").astype(np.int32)).cuda()
    off = torch.from_numpy(np.r_[0, np.cumsum(np.bincount(ids, minlength=E))].astype(np.int32)).cuda()
    i = lambda *s: torch.from_numpy(rng.integers(-2, 3, s).astype(np.float32)).to(dtype).cuda()  # noqa: E731
    x, w, c = i(T, K).requires_grad_(), i(E, N, K).requires_grad_(), i(T * k, N)
    with pytest.raises(RuntimeError, match="not recorded by autograd"):
        qm.grouped_matmul(x, w, off, perm=perm, top_k=k, x_order="token")
    y = Grouped.apply(x, w, off, perm, k)
    (y.float() * c.float()).sum().backward()
    x64, w64, c64 = (t.detach().double().cpu() for t in (x, w, c))
    want = torch.stack([w64[e] @ x64[s // k] for s, e in enumerate(ids)])
    assert torch.equal(y.detach().cpu(), want.float().to(dtype))
    dx, dw = torch.zeros_like(x64), torch.zeros_like(w64)
    for s, e in enumerate(ids):
        dx[s // k] += w64[e].t() @ c64[s]
        dw[e] += c64[s][:, None] * x64[s // k]
    assert torch.equal(x.grad.cpu(), dx.float().to(dtype)) and torch.equal(w.grad.cpu(), dw.float().to(dtype))
