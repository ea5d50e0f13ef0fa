"""The block-scaled FP8 quantisers against the oracle: codes and scales bit for
bit (the SwiGLU's h differs in its last fp32 bits, so its codes may be one step
apart where h lies that close to a boundary), ragged edges, every type, special
blocks, the error word, graph replays, and offsets past 32 bits."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm
from quantized_sparse_moe_amd import _lib

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def gen(seed, *shape, dtype="bf16", spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(spread * torch.randn(shape[-1], generator=g))
    return x.clamp(-6e4, 6e4).to(DT[dtype])


def bits(t):
    return t.cpu().view(torch.uint8).numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (3, 144), (129, 400), (300, 128), (128, 1136)])
def test_codes_and_scales(rows, cols, dtype, block_rows, pow2):
    x = gen(rows * cols, rows, cols, dtype=dtype)
    codes, scales = qm.quantize_block(x.cuda(), block_rows=block_rows, pow2=pow2)
    rc, rs = oracle.quantize_block(x.float().numpy(), block_rows, pow2)
    assert codes.dtype == torch.float8_e4m3fn and codes.shape == x.shape
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(bits(codes), rc)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_stack_of_matrices_keeps_blocks_apart(block_rows):
    x = gen(5, 3, 130, 272)
    codes, scales = qm.quantize_block(x.cuda(), block_rows=block_rows)
    for m in range(3):
        rc, rs = oracle.quantize_block(x[m].float().numpy(), block_rows, False)
        assert np.array_equal(scales[m].cpu().numpy(), rs) and np.array_equal(bits(codes[m]), rc)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_special_blocks_and_error_word(block_rows, pow2):
    x = gen(6, 256, 512, dtype="f32")
    x[0:128, 0:128] = 0.0
    x[0:128, 128:256] = 1e-41                      # subnormal
    x[128:, 0:128] = 3.0e38
    x[5, 300] = float("inf")
    x[200, 400] = float("nan")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = qm.quantize_block(x.cuda(), block_rows=block_rows, pow2=pow2, err=err)
    rc, rs = oracle.quantize_block(x.numpy(), block_rows, pow2)
    assert np.array_equal(scales.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(bits(codes) & 0x7F, rc & 0x7F)
    assert err.item() == _lib.MOE_DEVERR_QUANT_INPUT
    err.zero_()
    qm.quantize_block(x[128:, :256].contiguous().cuda(), block_rows=block_rows, err=err)
    assert err.item() == 0


def test_ties_go_to_even():
    v = oracle.e4m3_decode(np.arange(127, dtype=np.uint8))
    mid = ((v[:-1] + v[1:]) / 2).astype(np.float32)
    x = np.zeros((3, 128), np.float32)
    x[:, :126] = mid
    x[:, 127] = 448.0                              # makes the scale 1
    x[1, :126] = np.nextafter(mid, np.float32(1e9))
    x[2, :126] = np.nextafter(mid, np.float32(0))
    codes, scales = qm.quantize_block(torch.from_numpy(x).cuda())
    assert np.all(scales.cpu().numpy() == 1.0)
    assert np.array_equal(bits(codes), oracle.e4m3_encode(x))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,inner", [(1, 16), (6, 2048), (33, 272), (257, 144)])
def test_swiglu(rows, inner, dtype, pow2):
    gu = gen(rows + inner, rows, 2 * inner, dtype=dtype)
    codes, scales = qm.swiglu_quantize_block(gu.cuda(), pow2=pow2)
    rc, rs = oracle.swiglu_quantize_block(gu.double().numpy(), pow2)
    # h = g / (1 + e^-g) * u: at most 2 ulp of the exponential and half an ulp for each of four roundings
    # -> relative 2^-21; a power of two moves only if the quotient crosses one, which a scale factor of 2 shows
    rel = np.abs(scales.cpu().numpy() / rs - 1)
    assert np.all((rel <= 2.0 ** -21) | (pow2 & ((rel == 1.0) | (rel == 0.5))))
    same = np.repeat(rel <= 2.0 ** -21, 128, axis=1)[:, :inner]
    g, w = bits(codes).astype(int), rc.astype(int)
    moved = (g != w) & same
    assert np.all(np.abs((g & 127) - (w & 127))[moved] <= 1)
    # only values within 2^-20 of a boundary may move: 8 boundaries an octave makes that about 2^-17 of all
    assert moved.mean() <= 4 / moved.size + 2.0 ** -10


def test_swiglu_extremes_and_error_word():
    gu = torch.zeros(4, 256)
    gu[0, :128], gu[0, 128:] = -200.0, 3.0         # silu underflows to -0
    gu[1, :128], gu[1, 128:] = 90.0, 0.5
    gu[2, 7] = float("nan")
    gu[3, 128 + 9], gu[3, 9] = float("inf"), 1.0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = qm.swiglu_quantize_block(gu.cuda(), err=err)
    s = scales.cpu().numpy().ravel()
    assert s[0] == np.float32(2.0 ** -126) and s[1] == np.float32(45.0) / np.float32(448)
    assert np.isnan(s[2]) and np.isnan(s[3]) and err.item() == _lib.MOE_DEVERR_QUANT_INPUT
    c = bits(codes)
    assert not (c[0] & 127).any() and np.all(c[1] == 126) and not c[2:].any()


def test_graph_replays_equal_eager():
    x, y = gen(1, 70, 544).cuda(), gen(2, 70, 544).cuda()
    w = gen(3, 260, 400).cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            a = qm.quantize_block(buf)
            b = qm.swiglu_quantize_block(buf, pow2=True)
            c = qm.quantize_block(w, block_rows=128)
    torch.cuda.current_stream().wait_stream(stream)
    for src in (x, y, x):
        buf.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        want = (*qm.quantize_block(src), *qm.swiglu_quantize_block(src, pow2=True),
                *qm.quantize_block(w, block_rows=128))
        for got, ref in zip((*a, *b, *c), want):
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_offsets_past_32_bits(block_rows):
    """2^32 + 2^21 elements: the last rows equal those of a small matrix."""
    rows, cols = (1 << 17) + 64, 32768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = gen(8, 64, cols)
    x[-64:] = tail.cuda()
    codes, scales = qm.quantize_block(x, block_rows=block_rows)
    rc, rs = oracle.quantize_block(tail[:, :512].float().numpy(), block_rows, False)
    assert np.array_equal(bits(codes[-64:, :512].contiguous()), rc)
    n = 64 if block_rows == 1 else 1
    assert np.array_equal(scales[-n:, :4].cpu().numpy(), rs)
    assert not codes[:8].view(torch.uint8).any()


def test_other_stream():
    x = gen(4, 513, 2048).cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = qm.quantize_block(x, stream=s)
    s.synchronize()
    want = qm.quantize_block(x)
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
