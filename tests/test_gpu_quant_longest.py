"""The block-scaled quantiser on the longest rows: 2^24 blocks of 128."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm
from quantized_sparse_moe_amd import _lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block_rows,cols", [(1, (1 << 31) - 16), (1, (1 << 31) - 128), (128, (1 << 31) - 128)])
def test_the_longest_rows(block_rows, cols):
    x = torch.zeros(1, cols, dtype=torch.bfloat16, device="cuda")
    part = torch.randn(1, 1040, generator=torch.Generator().manual_seed(block_rows)).bfloat16()
    at = cols - cols % 128 - (1024 if cols % 128 else 1152)        # the last blocks, from a block's first column on
    n = min(1040, cols - at)
    x[:, at:at + n] = part[:, :n].cuda()
    codes, scales = qm.quantize_block(x, block_rows=block_rows)
    rc, rs = oracle.quantize_block(part[:, :n].float().numpy(), block_rows, False)
    assert np.array_equal(codes[:, at:at + n].cpu().view(torch.uint8).numpy(), rc)
    assert scales.shape == (1, -(-cols // 128))
    assert np.array_equal(scales[:, at // 128:at // 128 + rs.shape[1]].cpu().numpy(), rs)
    assert (scales[:, :at // 128] == 2.0 ** -126).all() and not codes[:, :4096].view(torch.uint8).any()


def test_one_workgroup_too_many_is_refused():
    x = torch.zeros(1, (1 << 31) - 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(_lib.MoeError):
        qm.quantize_block(x, block_rows=128)
