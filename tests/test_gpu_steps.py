"""The steps around the experts' products together, as they are used: a packed
expert layer served step by step, a training step of 16-bit experts with every
gradient, both captured in graphs, on several streams, and where a call may be
made that no other test makes.

Whole runs are compared step by step: each step's result with the float64 oracle
on that step's own inputs as the GPU has them, so that the bounds are those of one
step (tests/test_gpu_rows.py, _swiglu.py, _packed.py, _products.py)."""
import numpy as np
import pytest
import torch

import oracle
import quantized_sparse_moe_amd as qm
from tests._steps import DT, close, dev, routing

pytestmark = pytest.mark.gpu


def packed(rng, E, N, K, group=64):
    codes = rng.integers(0, 1 << 32, (E, N, K // 8), dtype=np.uint64).astype(np.uint32)
    s = (np.exp(0.5 * rng.standard_normal((E, N, K // group))) * 0.15 * K ** -0.5).astype(np.float16)
    return codes, s, (-7.5 * s * (1 + 0.2 * rng.standard_normal(s.shape))).astype(np.float16)


def upload(w):
    return dev(w[0].view(np.int32)), dev(w[1]), dev(w[2])


def np64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("T", [1, 5, 40])
def test_a_packed_expert_layer_step_by_step(T):
    """route, permute, gate/up product, SwiGLU, down product, combine with a shared expert's output."""
    E, k, d, inner = 12, 3, 256, 128
    rng = np.random.default_rng(T)
    gu_w, down_w = packed(rng, E, 2 * inner, d), packed(rng, E, d, inner)
    sh_w = packed(rng, 1, d, d)
    x = torch.from_numpy(rng.standard_normal((T, d))).bfloat16().cuda()
    layer = qm.DeviceLayer("topk", k, dev(rng.standard_normal((E, d)).astype(np.float32)), None, None)
    ws = layer.workspace(T)
    ids, weights = qm.route(layer, x, ws=ws)
    offsets, perm = qm.permute(ids, E, ws)
    positions = qm.invert_perm(perm)
    gu = qm.grouped_matmul_packed(x, *upload(gu_w), offsets, perm=perm, top_k=k, x_order="token", out_dtype="f32")
    h = qm.swiglu(gu.bfloat16())
    y = qm.grouped_matmul_packed(h, *upload(down_w), offsets, perm=perm, top_k=k, out_dtype="f32")
    shared = qm.matmul_packed(x, *(t[0] for t in upload(sh_w)), out_dtype="f32")
    out = qm.combine_rows(y, weights, positions, y_shared=shared, out_dtype="f32")
    y_slot = qm.grouped_matmul_packed(h, *upload(down_w), offsets, perm=perm, top_k=k, out_order="slot", out_dtype="f32")
    assert torch.equal(out, qm.combine_rows(y_slot, weights, y_shared=shared, out_dtype="f32"))
    assert torch.equal(out, qm.combine(y_slot, weights, shared, out_dtype="f32"))
    # a gather in front of the product gives what the product's own look-up gives
    assert torch.equal(gu, qm.grouped_matmul_packed(qm.gather_rows(x, perm, top_k=k), *upload(gu_w), offsets, out_dtype="f32"))

    off, pm = offsets.cpu().numpy(), perm.cpu().numpy()
    assert np.array_equal(positions.cpu().numpy(), oracle.invert_perm(pm, T * k))

    def product(rows, w, K):
        want, mag = np.empty((T * k, w[0].shape[1])), np.empty((T * k, w[0].shape[1]))
        for e in range(E):
            s = slice(off[e], off[e + 1])
            want[s], mag[s] = oracle.matmul_packed(rows[s], w[0][e], w[1][e], w[2][e])
        return want, (K + 2 * K // 64 + 8) * 2.0 ** -23 * mag

    want, tol = product(oracle.source_rows(np64(x), "token", pm, k), gu_w, d)
    close(gu, want, tol, "f32")
    want = oracle.swiglu(np64(gu.bfloat16()))
    close(h, want, 4 * 2.0 ** -23 * np.abs(want), "bf16")
    want, tol = product(np64(h), down_w, inner)
    close(y, want, tol, "f32")
    want, mag = oracle.combine_rows(np64(y), weights.cpu().numpy(), positions.cpu().numpy(), T, k, np64(shared))
    close(out, want, (k + 2) * 2.0 ** -24 * mag, "f32")
    assert qm.device_error(ws) == 0


class Experts(torch.autograd.Function):
    """x, weights of the two projections and the router's weights -> the layer's output, in bf16 with fp32 weights'
    gradients: the way a training program calls the steps."""

    @staticmethod
    def forward(ctx, x, w1, w2, weights, offsets, perm):
        k = weights.shape[1]
        positions = qm.invert_perm(perm)
        xb = qm.gather_rows(x, perm, top_k=k)
        gu = qm.grouped_matmul(xb, w1, offsets)
        h = qm.swiglu(gu)
        y = qm.grouped_matmul(h, w2, offsets)
        ctx.save_for_backward(xb, gu, h, y, w1, w2, weights, offsets, positions)
        return qm.combine_rows(y, weights, positions, out_dtype="f32")

    @staticmethod
    def backward(ctx, dout):
        xb, gu, h, y, w1, w2, weights, offsets, positions = ctx.saved_tensors
        dy, dweights = qm.combine_rows_grad(dout.contiguous(), y, weights, positions)
        dw2 = qm.grouped_matmul_dw(h, dy, offsets)
        dh = qm.grouped_matmul(dy, w2, offsets, transposed=True)
        dgu = qm.swiglu_grad(gu, dh)
        dw1 = qm.grouped_matmul_dw(xb, dgu, offsets)
        dxb = qm.grouped_matmul(dgu, w1, offsets, transposed=True)
        dx = qm.combine_rows(dxb, None, positions, top_k=weights.shape[1])
        Experts.seen = dict(xb=xb, gu=gu, h=h, y=y, dy=dy, dh=dh, dgu=dgu, dxb=dxb)
        return dx, dw1.to(w1.dtype), dw2.to(w2.dtype), dweights, None, None


def training_inputs(seed, T, k, E, d, inner):
    rng, off, perm, weights = routing(seed, T, k, E)
    x = torch.from_numpy(rng.standard_normal((T, d))).bfloat16().cuda()
    w1 = torch.from_numpy(rng.standard_normal((E, 2 * inner, d)) * d ** -0.5).bfloat16().cuda()
    w2 = torch.from_numpy(rng.standard_normal((E, d, inner)) * inner ** -0.5).bfloat16().cuda()
    return rng, x, w1, w2, dev(weights), dev(off), dev(perm)


@pytest.mark.parametrize("T,k,E,d,inner", [(1, 1, 1, 16, 8), (37, 3, 6, 72, 40), (300, 4, 16, 128, 64)])
def test_training_step_and_its_gradients(T, k, E, d, inner):
    rng, x, w1, w2, weights, off, perm = training_inputs(T, T, k, E, d, inner)
    leaves = [t.clone().requires_grad_() for t in (x, w1, w2, weights)]
    out = Experts.apply(*leaves, off, perm)
    g = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda()
    (out * g).sum().backward()
    s, o, pm = Experts.seen, off.cpu().numpy(), perm.cpu().numpy()
    pos, w = oracle.invert_perm(pm, T * k), weights.cpu().numpy()
    half = 2.0 ** -23

    def product(got, rows, m, Q):
        want, mag = oracle.grouped_matmul(np64(rows), m, o)
        close(got, want, (Q + 4) * half * mag, "bf16")

    assert np.array_equal(np64(s["xb"]), np64(x)[pm // k])
    product(s["gu"], s["xb"], np64(w1), d)
    want = oracle.swiglu(np64(s["gu"]))
    close(s["h"], want, 4 * half * np.abs(want), "bf16")
    product(s["y"], s["h"], np64(w2), inner)
    want, mag = oracle.combine_rows(np64(s["y"]), w, pos, T, k)
    close(out.detach(), want, (k + 1) * 2.0 ** -24 * mag, "f32")
    # and back
    dy, dw, mag = oracle.combine_rows_grad(np64(g), np64(s["y"]), w, pos)
    close(s["dy"], dy, 2.0 ** -24 * np.abs(dy), "bf16")
    close(leaves[3].grad, dw, (d + 1) * 2.0 ** -24 * mag, "f32")
    product(s["dh"], s["dy"], np64(w2).transpose(0, 2, 1), d)
    want, mag = oracle.swiglu_grad(np64(s["gu"]), np64(s["dh"]))
    close(s["dgu"], want, 8 * half * mag, "bf16")
    product(s["dxb"], s["dgu"], np64(w1).transpose(0, 2, 1), 2 * inner)
    want, mag = oracle.combine_rows(np64(s["dxb"]), None, pos, T, k)
    close(leaves[0].grad, want, (k + 1) * 2.0 ** -24 * mag, "bf16")
    for leaf, rows, dr in ((leaves[1], "xb", "dgu"), (leaves[2], "h", "dy")):
        want, mag = oracle.grouped_matmul_dw(np64(s[rows]), np64(s[dr]), o)
        most = int(np.diff(o).max())
        # rounded to fp32 by the product, then to bf16 by the program
        close(leaf.grad, want, (most + 4) * half * mag + 2.0 ** -24 * np.abs(want), "bf16")


def all_steps(x, y, w, off, perm, gu, dh, pk, pk1):
    k = w.shape[1]
    pos = qm.invert_perm(perm)
    rows = qm.gather_rows(x, perm, top_k=k)
    dy, dw = qm.combine_rows_grad(x, y, w, pos)
    return (pos, rows, qm.gather_rows(x, perm, top_k=k, weights=w, out_dtype="f32"), qm.combine_rows(y, w, pos),
            qm.combine_rows(y, None, top_k=k, y_shared=x, out_dtype="f32"), dy, dw, qm.swiglu(gu), qm.swiglu_grad(gu, dh),
            qm.matmul_packed(x, *pk1), qm.grouped_matmul_packed(rows, *pk, off, out_dtype="f32"),
            qm.grouped_matmul_packed(x, *pk, off, perm=perm, top_k=k, x_order="token", out_order="slot"))


def step_inputs(seed, T, k, E, d, inner):
    rng, off, perm, w = routing(seed, T, k, E)
    b = lambda *s: torch.from_numpy(rng.standard_normal(s)).bfloat16().cuda()  # noqa: E731
    return [b(T, d), b(T * k, d), dev(w), dev(off), dev(perm), b(T * k, 2 * inner), b(T * k, inner)]


# few rows: the product's small kernel and, over 12 buckets of 100 tiles, its streaming one; many: its tiles
SIZES = [(2, 2, 5, 128, 40, 96), (9, 2, 12, 640, 72, 1600), (130, 3, 6, 256, 64, 200)]


@pytest.mark.parametrize("T,k,E,d,inner,N", SIZES)
def test_graph_replays_equal_eager(T, k, E, d, inner, N):
    """One captured run replayed with other inputs and routings between eager work; two graphs of it at once."""
    rng = np.random.default_rng(1)
    pk = upload(packed(rng, E, N, d))
    pk1 = tuple(t[0] for t in pk)
    sets = [step_inputs(s, T, k, E, d, inner) for s in range(3)]
    bufs = [t.clone() for t in sets[0]]
    eager = [[t.clone() for t in all_steps(*s, pk, pk1)] for s in sets]
    graphs, stream = [], torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            with torch.cuda.graph(graph, stream=stream):
                outs = all_steps(*bufs, pk, pk1)
        graphs.append((graph, outs))
    torch.cuda.current_stream().wait_stream(stream)
    for rep in range(4):
        for buf, s in zip(bufs, sets[rep % 3]):
            buf.copy_(s)
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
        graphs[0][0].replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            for i, (got, want) in enumerate(zip(outs, eager[rep % 3])):
                assert torch.equal(got, want), (rep, i)
        torch.randn(1 << 16, device="cuda").sum().item()


def test_a_training_step_is_captured_beside_an_eager_one():
    """Forward and backward of the whole step in a graph (the calls allocate and keep nothing of their own), replayed
    between eager steps on the same inputs."""
    T, k, E, d, inner = 60, 2, 5, 64, 32
    _, x, w1, w2, weights, off, perm = training_inputs(3, T, k, E, d, inner)

    class Context:
        def save_for_backward(self, *tensors):
            self.saved_tensors = tensors

    def step():
        ctx = Context()
        out = Experts.forward(ctx, x, w1, w2, weights, off, perm)
        return [out, *[t for t in Experts.backward(ctx, out) if t is not None]]

    with torch.no_grad():
        eager = [t.clone() for t in step()]
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            with torch.cuda.graph(graph, stream=stream):
                outs = step()
        torch.cuda.current_stream().wait_stream(stream)
        for _ in range(3):
            for t in outs:
                t.fill_(7)
            graph.replay()
            again = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(outs, eager, again))


@pytest.mark.parametrize("T,k,E,d,inner,N", SIZES)
def test_two_streams_at_once_and_a_given_stream(T, k, E, d, inner, N):
    rng = np.random.default_rng(2)
    pk = upload(packed(rng, E, N, d))
    pk1 = tuple(t[0] for t in pk)
    sets = [step_inputs(s, T, k, E, d, inner) for s in range(2)]
    want = [[t.clone() for t in all_steps(*s, pk, pk1)] for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for s, st in zip(sets, streams):
        with torch.cuda.stream(st):
            got.append(all_steps(*s, pk, pk1))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    x, y, w, off, perm, gu, dh = sets[0]
    st, kk = streams[0], w.shape[1]
    pos = want[0][0]
    given = (qm.invert_perm(perm, stream=st), qm.gather_rows(x, perm, top_k=kk, stream=st),
             qm.combine_rows(y, w, pos, stream=st), *qm.combine_rows_grad(x, y, w, pos, stream=st),
             qm.swiglu(gu, stream=st), qm.swiglu_grad(gu, dh, stream=st), qm.matmul_packed(x, *pk1, stream=st),
             qm.grouped_matmul_packed(want[0][1], *pk, off, out_dtype="f32", stream=st))
    st.synchronize()
    for a, i in zip(given, (0, 1, 3, 5, 6, 7, 8, 9, 10)):
        assert torch.equal(a, want[0][i]), i


def test_a_stream_of_another_device_and_mixed_devices_are_refused():
    class Stream:
        device = torch.device("cuda", 1)
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i, w = z(4, d=torch.int32), z(2, 2, d=torch.float32)
    c, s = z(8, 8, d=torch.int32), z(8, 1, d=torch.float16)
    for call in (lambda **kw: qm.invert_perm(i, **kw), lambda **kw: qm.gather_rows(z(2, 8), i, top_k=2, **kw),
                 lambda **kw: qm.combine_rows(z(4, 8), w, **kw), lambda **kw: qm.combine_rows_grad(z(2, 8), z(4, 8), w, **kw),
                 lambda **kw: qm.swiglu(z(2, 8), **kw), lambda **kw: qm.swiglu_grad(z(2, 8), z(2, 4), **kw),
                 lambda **kw: qm.matmul_packed(z(2, 64), c, s, s, **kw),
                 lambda **kw: qm.grouped_matmul_packed(z(2, 64), c[None], s[None], s[None], i[:2], **kw)):
        with pytest.raises(ValueError, match="the stream is on"):
            call(stream=Stream())
    for call in (lambda: qm.gather_rows(z(2, 8), i.cpu(), top_k=2), lambda: qm.combine_rows(z(4, 8), w.cpu()),
                 lambda: qm.combine_rows(z(4, 8), w, i.cpu()), lambda: qm.combine_rows_grad(z(2, 8), z(4, 8).cpu(), w),
                 lambda: qm.swiglu_grad(z(2, 8), z(2, 4).cpu()), lambda: qm.matmul_packed(z(2, 64), c.cpu(), s, s),
                 lambda: qm.matmul_packed(z(2, 64), c, s, s.cpu()), lambda: qm.invert_perm(i, err=i[:1].cpu())):
        with pytest.raises(ValueError):
            call()


def test_results_do_not_change_from_call_to_call():
    T, k, E, d, inner, N = SIZES[2]
    pk = upload(packed(np.random.default_rng(5), E, N, d))
    pk1 = tuple(t[0] for t in pk)
    s = step_inputs(4, T, k, E, d, inner)
    first = [t.clone() for t in all_steps(*s, pk, pk1)]
    for _ in range(5):
        torch.randn(1 << 20, device="cuda")
        assert all(torch.equal(a, b) for a, b in zip(all_steps(*s, pk, pk1), first))
