"""Helpers of the GPU tests of the row steps, SwiGLU and 4-bit products."""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}    # half a step, relative to the value
LEAST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}  # half of the smallest subnormal


def close(got, want, fp32, out):
    """|got - want| <= the fp32 computation's error `fp32` (an array), and one rounding to `out`."""
    got = got.double().cpu().numpy()
    tol = fp32 * (1 + HALF[out]) + HALF[out] * np.abs(want) + LEAST[out] + LEAST["f32"]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def routing(seed, T, k, E, skew=0.7):
    """(rng, offsets, perm, weights) of distinct experts per token."""
    rng = np.random.default_rng(seed)
    score = -skew * np.log(np.arange(1, E + 1)) + rng.gumbel(size=(T, E))
    ids = np.argsort(-score, axis=1)[:, :k].reshape(-1)
    off = np.r_[0, np.cumsum(np.bincount(ids, minlength=E))].astype(np.int32)
    return rng, off, np.argsort(ids, kind="stable").astype(np.int32), rng.random((T, k)).astype(np.float32)


def shifted(a, dtype, by):
    """The array on the device, its first element `by` elements behind an aligned address."""
    t = torch.empty(a.size + by, dtype=dtype, device="cuda")
    t[by:] = torch.from_numpy(np.ascontiguousarray(a)).reshape(-1).cuda()
    return t[by:].view(a.shape)
