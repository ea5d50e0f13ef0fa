"""A router without packed experts in front of the grouped products: routing and
buckets against the oracle, and the whole FP8 and bf16 chains from it."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm
from tests._gpu import check_topk_ids, stable_sort_perm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,d", [(1, 8, 2, 64), (70, 24, 3, 256), (130, 256, 6, 128)])
@pytest.mark.parametrize("kind", ["topk", "hash"])
def test_route_and_permute(kind, T, E, k, d):
    rng = np.random.default_rng(T + E)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).bfloat16()
    wr = (rng.standard_normal((E, d)) * d ** -0.5).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    table = rng.integers(0, E, (50, k)).astype(np.int32)
    tokens = rng.integers(0, 50, T).astype(np.int32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    layer = qm.DeviceLayer(kind, k, dev(wr), dev(bias), dev(table) if kind == "hash" else None)
    ws = layer.workspace(T)
    assert ws.numel() == layer.workspace_size(T)
    ids, w = qm.route(layer, x.cuda(), dev(tokens) if kind == "hash" else None, ws=ws)
    offsets, perm = qm.permute(ids, E, ws)
    assert qm.device_error(ws) == 0
    got = ids.cpu().numpy()
    if kind == "hash":
        want, ww, _ = oracle.route_hash(x.double().numpy(), wr, table, tokens)
        assert np.array_equal(got, want)
    else:
        _, _, key, s = oracle.route_topk(oracle.router_logits(x.double().numpy(), wr), bias, k)
        check_topk_ids(got, oracle.route_topk(oracle.router_logits(x.double().numpy(), wr), bias, k)[0], key, k)
        ww = oracle.combine_weights_for_ids(s, got)
    assert np.allclose(w.cpu().numpy(), ww, rtol=1e-5, atol=1e-6)
    off, p = stable_sort_perm(got, E)
    assert np.array_equal(offsets.cpu().numpy(), off) and np.array_equal(perm.cpu().numpy(), p)


def test_chains_from_a_router_alone():
    """The FP8 and the bf16 expert layer as a user without packed experts runs them: each product equals the one over
    buckets made on the host."""
    T, E, k, d, inner = 45, 9, 2, 128, 144
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, gu, dn = r(T, d).bfloat16(), (r(E, 2 * inner, d) * 0.1).bfloat16(), (r(E, d, inner) * 0.1).bfloat16()
    layer = qm.DeviceLayer("topk", k, r(E, d) * 0.1, None, None)
    ws = layer.workspace(T)
    ids, weights = qm.route(layer, x, ws=ws)
    offsets, perm = qm.permute(ids, E, ws)
    off, p = (torch.from_numpy(a.astype(np.int32)).cuda() for a in stable_sort_perm(ids.cpu().numpy(), E))
    (wq, sw), (vq, sv), (a, sa) = qm.quantize_block(gu, 128), qm.quantize_block(dn, 128), qm.quantize_block(x)

    def chain(offsets, perm):
        kw = dict(perm=perm, top_k=k)
        h, sh = qm.swiglu_quantize_block(qm.grouped_matmul_block(a, sa, wq, sw, offsets, x_order="token", **kw))
        y = qm.grouped_matmul_block(h, sh, vq, sv, offsets, out_order="slot", out_dtype="f32", **kw)
        z = qm.grouped_matmul(x, gu, offsets, x_order="token", out_order="slot", **kw)
        return qm.combine(y, weights, None, out_dtype="f32"), z

    for got, want in zip(chain(offsets, perm), chain(off, p)):
        assert torch.equal(got, want) and torch.isfinite(got).all()
