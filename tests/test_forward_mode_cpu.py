"""Forward-mode derivatives, without a GPU: the calls that autograd does not
record refuse an operand with a tangent, whose derivative they would drop, and
take the primals of such an operand and operands without a tangent."""
import os

import pytest
import torch
from torch.autograd import forward_ad

import quantized_sparse_moe_amd as qm
from quantized_sparse_moe_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libqsmoe.so not built")

BF16 = torch.bfloat16
X, W, I32 = torch.zeros(4, 64, dtype=BF16), torch.ones(2, 2), torch.zeros(4, dtype=torch.int32)
W16 = torch.zeros(3, 64, 64, dtype=BF16)
CODES, S16 = torch.zeros(3, 8, 8, dtype=torch.int32), torch.zeros(3, 8, 1, dtype=torch.float16)
E4M3, S32 = torch.zeros(4, 128, dtype=torch.uint8), torch.ones(4, 1)
CALLS = {  # the call, its operands that may have a tangent
    "matmul_block": (lambda s, t: qm.matmul_block(E4M3, s, E4M3, t), (S32, S32[:1])),
    "grouped_matmul_block": (lambda s, t: qm.grouped_matmul_block(E4M3, s, E4M3[None], t, I32[:2]), (S32, S32[None, :1])),
    "grouped_matmul": (lambda x, w: qm.grouped_matmul(x, w, I32), (X, W16)),
    "grouped_matmul_dw": (lambda x, dy: qm.grouped_matmul_dw(x, dy, I32), (X, X)),
    "gather_rows": (lambda x, w: qm.gather_rows(x, I32, 2, weights=w), (X[:2], W)),
    "combine_rows": (lambda y, w, s: qm.combine_rows(y, w, y_shared=s), (X, W, X[:2])),
    "combine_rows_grad": (qm.combine_rows_grad, (X[:2], X, W)),
    "swiglu": (qm.swiglu, (X,)),
    "swiglu_grad": (qm.swiglu_grad, (X, X[:, :32])),
    "matmul_packed": (lambda x, s, b: qm.matmul_packed(x, CODES[0], s, b), (X, S16[0], S16[0])),
    "grouped_matmul_packed": (lambda x, s, b: qm.grouped_matmul_packed(x, CODES, s, b, I32), (X, S16, S16)),
}


@pytest.mark.parametrize("name", CALLS)
def test_tangents_are_refused(name):
    call, operands = CALLS[name]
    with forward_ad.dual_level():
        for i in range(len(operands)):
            args = list(operands)
            args[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(RuntimeError, match=f"{name} is not recorded by autograd.*tangent"):
                call(*args)
            with torch.no_grad(), pytest.raises(RuntimeError, match="tangent"):   # no_grad keeps forward mode
                call(*args)
            args[i] = forward_ad.unpack_dual(args[i]).primal
            with pytest.raises(ValueError, match="contiguous device tensor"):
                call(*args)


@pytest.mark.parametrize("name", CALLS)
def test_other_calls_in_a_dual_level_are_taken(name):
    call, operands = CALLS[name]
    with forward_ad.dual_level(), pytest.raises(ValueError, match="contiguous device tensor"):
        call(*operands)


@pytest.mark.parametrize("name", CALLS)
def test_an_autograd_function_may_make_the_call(name):
    """Inside a Function's forward the operands have no tangent: its own jvp gives the result's."""
    call, operands = CALLS[name]

    class Op(torch.autograd.Function):
        @staticmethod
        def forward(ctx, *args):
            with pytest.raises(ValueError, match="contiguous device tensor"):
                call(*args)
            return args[0] * 2

        @staticmethod
        def jvp(ctx, *tangents):
            return tangents[0] * 2

    with forward_ad.dual_level():
        duals = [forward_ad.make_dual(t, torch.ones_like(t)) for t in operands]
        assert (forward_ad.unpack_dual(Op.apply(*duals)).tangent == 2).all()
