"""The SwiGLU quantiser value by value: every scale, code and sign is the
64-bit one, or its neighbour where the value lies on the boundary between them."""
import numpy as np
import pytest
import torch

import quantized_sparse_moe_amd as qm
from tests._quant import check_swiglu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,inner", [(1, 16), (6, 2048), (33, 272), (257, 144), (2000, 1408)])
def test_every_code_scale_and_sign(rows, inner, dtype, pow2):
    g = torch.Generator().manual_seed(rows + inner)
    gu = torch.randn(rows, 2 * inner, generator=g) * torch.exp(torch.randn(2 * inner, generator=g))
    gu = gu.to(dtype)
    codes, scales = qm.swiglu_quantize_block(gu.cuda(), pow2=pow2)
    check_swiglu(codes.cpu().view(torch.uint8).numpy(), scales.cpu().numpy(), gu.double().numpy(), pow2)


def test_scales_near_a_power_of_two():
    """Blocks whose largest |h| is 448 times a power of two, up to the last bits on either side."""
    rng = np.random.default_rng(2)
    rows, inner = 400, 128
    gu = np.zeros((rows, 2 * inner), np.float32)
    gu[:, :inner] = rng.uniform(40, 80, (rows, inner))        # silu is the identity but for e^-40
    top = 448.0 * np.exp2(rng.integers(-9, 10, rows)) * (1 + rng.integers(-6, 7, rows) * 2.0 ** -23)
    gu[:, inner:] = rng.uniform(-0.9, 0.9, (rows, inner)) * top[:, None] / 80
    gu[:, inner + 5] = top / gu[:, 5]
    for pow2 in (False, True):
        codes, scales = qm.swiglu_quantize_block(torch.from_numpy(gu).cuda(), pow2=pow2)
        check_swiglu(codes.cpu().view(torch.uint8).numpy(), scales.cpu().numpy(), gu.astype(np.float64), pow2)
