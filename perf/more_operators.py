"""The measured cases of the steps around the experts' products.

Six operators, each in a plain form (elementary torch operations in 32 bits) and, where ``own`` is true, as the
framework's call:

  gather_rows            rows of tokens brought into bucket order (expert by expert), times their weight where asked
  combine_rows           rows back to tokens: the weighted sum over a token's rows
  combine_rows_grad      its gradient in the rows and in the weights
  swiglu                 silu(gate) * up, and its gradient in gate and up
  matmul_packed          few rows times a matrix held in 4 bits with group scales (affine or MXFP4)
  grouped_matmul_packed  the same, rows grouped by expert

Sizes follow the layer this framework computes: hidden 4096, intermediate 2048, 256 experts, top-6, 1 to 4096 tokens,
vocabulary 129280.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's hidden state on its way to six experts: latency
        dict(name="gather 1 token", op="gather_rows", T=1, k=6, E=256, d=4096, weighted=False, dtype="bf16", out="bf16",
             skew=0.5),
        # dispatch of a 4096-token training step
        dict(name="gather 4096 tokens", op="gather_rows", T=4096, k=6, E=256, d=4096, weighted=False, dtype="bf16",
             out="bf16", skew=0.5),
        # a small step of an odd width: fp32 rows in slot order with a shared expert's output, fp16 result
        dict(name="combine odd width", op="combine_rows", T=137, k=4, E=24, d=1003, order="slot", weighted=True,
             shared=True, dtype="f32", out="f16", skew=0.8),
        # the experts' outputs of a 4096-token step from bucket order back to tokens, the positions found on the way
        dict(name="combine 4096 tokens", op="combine_rows", T=4096, k=6, E=256, d=4096, order="bucket", weighted=True,
             shared=False, dtype="bf16", out="bf16", skew=0.5),
        # fine-tuning on a short prompt of odd length
        dict(name="combine grad 61 tokens", op="combine_rows_grad", T=61, k=6, E=64, d=4096, order="bucket",
             dtype="bf16", dout="f32", skew=0.5),
        # backward pass of the 4096-token step
        dict(name="combine grad 4096 tokens", op="combine_rows_grad", T=4096, k=6, E=256, d=4096, order="bucket",
             dtype="bf16", dout="bf16", skew=0.5),
        # between the two products of one token's six experts: latency
        dict(name="swiglu 6 rows", op="swiglu", rows=6, inner=2048, grad=False, dtype="bf16"),
        # backward pass of the activation, 4096 tokens at top-6
        dict(name="swiglu grad 24576 rows", op="swiglu", rows=24576, inner=2048, grad=True, dtype="bf16"),
        # one token through a head over the vocabulary
        dict(name="4-bit head 1 token", op="matmul_packed", M=1, N=129280, K=4096, format="affine", group=64,
             dtype="bf16", out="f32"),
        # a few sequences decoded together through a dense projection of odd size
        dict(name="4-bit dense 13 tokens", op="matmul_packed", M=13, N=2053, K=4000, format="affine", group=32,
             dtype="f16", out="f16"),
        # single-token decode: six of 256 experts, gate and up stacked
        dict(name="4-bit experts 1 token", op="grouped_matmul_packed", T=1, k=6, E=256, N=4096, K=4096, format="affine",
             group=64, x="token", y="bucket", dtype="bf16", out="bf16", skew=0.5),
        # the down projection of a 64-token decode batch, back in slot order in fp32 for the combine
        dict(name="4-bit experts 64 tokens", op="grouped_matmul_packed", T=64, k=6, E=256, N=4096, K=2048, format="mxfp4",
             group=32, x="bucket", y="slot", dtype="bf16", out="f32", skew=0.5),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gather_rows", "combine_rows", "combine_rows_grad", "swiglu", "matmul_packed",
                     "grouped_matmul_packed"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "swiglu":
        c = dict(op=op, rows=_log_uniform(rng, 1, 24576), grad=rng.random() < 0.6, dtype=dtype)
        c["inner"] = rng.choice([1, 8]) * _log_uniform(rng, 16, 352)
        while c["rows"] * c["inner"] * SIZE[dtype] > 24576 * 2048 * 2:
            c["rows"] = (c["rows"] + 1) // 2
        return c
    if op in ("gather_rows", "combine_rows", "combine_rows_grad"):
        E = _log_uniform(rng, 8, 256)
        c = dict(op=op, T=_log_uniform(rng, 1, 4096), k=rng.randint(1, 8), E=E, d=rng.choice([1, 8]) * _log_uniform(rng, 16, 1024),
                 dtype=dtype, skew=rng.choice([0.0, 0.5, 1.0]))
        if op == "gather_rows":
            c.update(weighted=rng.random() < 0.4, out=rng.choice([dtype, dtype, "f32"]))
        elif op == "combine_rows":
            c.update(order=rng.choice(["bucket", "slot"]), weighted=rng.random() < 0.7, shared=rng.random() < 0.3,
                     out=rng.choice([dtype, "bf16"]))
        else:
            c.update(order=rng.choice(["bucket", "slot"]), dout=rng.choice([dtype, "f32"]))
        while c["T"] * c["k"] * c["d"] * max(SIZE[dtype], SIZE[c.get("out", "bf16")]) > 24576 * 4096 * 2:
            c["T"] = (c["T"] + 1) // 2
        return c
    fmt, group = rng.choice([("affine", 32), ("affine", 64), ("affine", 128), ("mxfp4", 32)])
    c = dict(op=op, K=128 * _log_uniform(rng, 1, 64) if rng.random() < 0.6 else group * _log_uniform(rng, 2, 8192 // group),
             format=fmt, group=group, dtype=rng.choice(["bf16", "f16"]))
    c["out"] = rng.choice([c["dtype"], "f32"])
    if op == "matmul_packed":
        c.update(M=_log_uniform(rng, 1, 64), N=_log_uniform(rng, 64, 32768))
        return c
    E = _log_uniform(rng, 8, 256)
    c.update(T=_log_uniform(rng, 1, 512), k=rng.randint(1, 8), E=E, N=_log_uniform(rng, 64, 4096),
             x=rng.choice(["bucket", "slot", "token"]), y=rng.choice(["bucket", "slot"]), skew=rng.choice([0.0, 0.5, 1.0]))
    while c["E"] * c["N"] * c["K"] > 256 * 4096 * 2048:
        c["N"] = (c["N"] + 1) // 2
    while c["T"] * c["k"] * c["N"] * c["K"] > 2 * 512 * 4096 * 4096:
        c["T"] = (c["T"] + 1) // 2
    return c


def _experts_used(c):
    """How many experts have a row, expected."""
    share = [(e + 1) ** -c["skew"] for e in range(c["E"])]
    total = sum(share)
    used = sum(1 - (1 - min(1.0, c["k"] * s / total)) ** c["T"] for s in share)
    return min(max(used, 1), c["T"] * c["k"])


def work(case):
    c = case
    if c["op"] == "swiglu":
        n, s = c["rows"] * c["inner"], SIZE[c["dtype"]]
        return {"bytes": n * s * (5 if c["grad"] else 3), "flops": n * (12 if c["grad"] else 6)}
    if c["op"] in ("matmul_packed", "grouped_matmul_packed"):
        N, K = c["N"], c["K"]
        matrix = N * K / 2 + N * (K // c["group"]) * (4 if c["format"] == "affine" else 1)
        if c["op"] == "matmul_packed":
            M, rows, used = c["M"], c["M"], 1
        else:
            M, used = c["T"] * c["k"], _experts_used(c)
            rows = c["T"] if c["x"] == "token" else M
        return {"bytes": used * matrix + 2 * rows * K + M * N * SIZE[c["out"]], "flops": 2 * M * N * K}
    T, d, s = c["T"], c["d"], SIZE[c["dtype"]]
    R = T * c["k"]
    if c["op"] == "gather_rows":
        return {"bytes": T * d * s + R * d * SIZE[c["out"]] + R * (8 if c["weighted"] else 4),
                "flops": R * d if c["weighted"] else 0}
    if c["op"] == "combine_rows":
        b = R * d * s + T * d * SIZE[c["out"]] + (T * d * s if c["shared"] else 0) + (4 * R if c["weighted"] else 0)
        return {"bytes": b + (8 * R if c["order"] == "bucket" else 0), "flops": 2 * R * d}
    return {"bytes": 2 * R * d * s + T * d * SIZE[c["dout"]] + (12 if c["order"] == "bucket" else 8) * R, "flops": 3 * R * d}


# ------------------------------------------------------------------ inputs

def _activations(g, rows, cols, dtype):
    """Normal values with channels of unequal size, as a transformer's hidden state has them."""
    gain = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return (torch.randn(rows, cols, generator=g, device="cuda") * gain).to(dtype)


def _routing(g, T, k, E, skew):
    """(perm, offsets, weights): distinct experts per token with popularity (rank + 1) ** -skew, bucketed by expert in
    stable order, and each token's weights, which sum to 1."""
    rank = torch.randperm(E, generator=g, device="cuda")
    logits = -skew * torch.log(rank.float() + 1)
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-12, 1 - 1e-7)))
    top = torch.topk(logits + noise, k, dim=1)
    ids = top.indices.reshape(-1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0)
    weights = torch.rand(T, k, generator=g, device="cuda") + 0.1
    return torch.argsort(ids, stable=True).to(torch.int32), offsets, (weights / weights.sum(1, keepdim=True)).contiguous()


# The magnitudes of a 4-bit floating code without its sign bit, and the borders between them.
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


def _packed(g, E, N, K, fmt, group):
    """(codes int32 [E][N][K / 8], scales [E][N][K / group], biases): normal weights converted group by group, by
    smallest and largest value (affine) or by the largest one's power of two (MXFP4)."""
    codes = torch.empty(E, N, K // 8, dtype=torch.int32, device="cuda")
    scales = torch.empty(E, N, K // group, dtype=torch.float16 if fmt == "affine" else torch.uint8, device="cuda")
    biases = torch.empty_like(scales) if fmt == "affine" else None
    shifts = 4 * torch.arange(8, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 26) // (N * K))  # matrices at a time, or rows of one
    rows = N if N * K <= 1 << 27 else (1 << 27) // K
    for e in range(0, E, step):
        for r in range(0, N, rows):
            part = codes[e:e + step, r:r + rows]
            w = torch.randn(part.shape[0], part.shape[1], K // group, group, generator=g, device="cuda") * K ** -0.5
            if fmt == "affine":
                low, high = w.amin(-1), w.amax(-1)
                s, b = ((high - low) / 15).half(), low.half()
                scales[e:e + step, r:r + rows], biases[e:e + step, r:r + rows] = s, b
                q = ((w - b.float()[..., None]) / s.float()[..., None]).round_().clamp_(0, 15).to(torch.int32)
            else:
                top = torch.frexp(w.abs().amax(-1)).exponent - 3  # the largest lies in [4, 8) of its unit
                scales[e:e + step, r:r + rows] = (top + 127).clamp(0, 254).to(torch.uint8)
                w = torch.ldexp(w, -top[..., None])
                q = torch.bucketize(w.abs(), torch.tensor(BORDERS, device="cuda"), out_int32=True) + 8 * (w < 0).to(torch.int32)
            part.copy_((q.reshape(*part.shape, 8) << shifts).sum(-1, dtype=torch.int32))
    return codes, scales, biases


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "swiglu":
        s["gu"] = _activations(g, c["rows"], 2 * c["inner"], DTYPES[c["dtype"]])
        s["dh"] = (torch.randn(c["rows"], c["inner"], generator=g, device="cuda") * 0.1).to(DTYPES[c["dtype"]])
        return s
    if c["op"] == "matmul_packed":
        s["x"] = _activations(g, c["M"], c["K"], DTYPES[c["dtype"]])
        codes, scales, biases = _packed(g, 1, c["N"], c["K"], c["format"], c["group"])
        s["codes"], s["scales"], s["biases"] = codes[0], scales[0], None if biases is None else biases[0]
        return s
    T, k, E = c["T"], c["k"], c["E"]
    s["perm"], s["offsets"], s["weights"] = _routing(g, T, k, E, c["skew"])
    if c["op"] == "gather_rows":
        s["x"] = _activations(g, T, c["d"], DTYPES[c["dtype"]])
    elif c["op"] == "combine_rows":
        s["y"] = _activations(g, T * k, c["d"], DTYPES[c["dtype"]])
        s["shared"] = _activations(g, T, c["d"], DTYPES[c["dtype"]]) if c["shared"] else None
    elif c["op"] == "combine_rows_grad":
        s["y"] = _activations(g, T * k, c["d"], DTYPES[c["dtype"]])
        s["dout"] = (torch.randn(T, c["d"], generator=g, device="cuda") * 0.1).to(DTYPES[c["dout"]])
        # where the forward pass found each assignment's row
        s["positions"] = torch.argsort(s["perm"]).to(torch.int32) if c["order"] == "bucket" else None
    else:
        s["codes"], s["scales"], s["biases"] = _packed(g, E, c["N"], c["K"], c["format"], c["group"])
        s["x"] = _activations(g, T if c["x"] == "token" else T * k, c["K"], DTYPES[c["dtype"]])
        # where the plain form finds the rows of its padded batch: the experts in use, each row's bucket and place
        counts = (s["offsets"][1:] - s["offsets"][:-1]).long()
        active = torch.nonzero(counts).reshape(-1)
        group = torch.repeat_interleave(torch.arange(active.numel(), device="cuda"), counts[active])
        place = torch.arange(T * k, device="cuda") - s["offsets"][active].long()[group]
        s["plan"] = dict(active=active, group=group, place=place, longest=int(counts.max()))
    return s


# ------------------------------------------------------------------ plain forms (32 bits)

def _dequantize(codes, scales, biases, fmt, group):
    shifts = 4 * torch.arange(8, dtype=torch.int32, device=codes.device)
    q = ((codes[..., None] >> shifts) & 15).reshape(*codes.shape[:-1], -1, group)
    if fmt == "affine":
        w = q.float().mul_(scales.float()[..., None]).add_(biases.float()[..., None])
    else:
        table = torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device)
        w = table[q].mul_(torch.exp2(scales.float() - 127)[..., None])
    return w.reshape(*codes.shape[:-1], -1)


def run(state):
    c = state["case"]
    if own:
        return _run_own(state)
    if c["op"] == "swiglu":
        gate, up = state["gu"].float().chunk(2, dim=1)
        sig = 1 / (1 + torch.exp(-gate))
        if not c["grad"]:
            return (gate * sig * up).to(DTYPES[c["dtype"]])
        dh = state["dh"].float()
        return torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], dim=1).to(DTYPES[c["dtype"]])
    if c["op"] == "matmul_packed":
        w = _dequantize(state["codes"], state["scales"], state["biases"], c["format"], c["group"])
        return (state["x"].float() @ w.t()).to(DTYPES[c["out"]])
    k, perm, weights = c["k"], state["perm"].long(), state["weights"]
    if c["op"] == "gather_rows":
        rows = state["x"].float()[perm // k]
        return (rows * weights.reshape(-1)[perm][:, None] if c["weighted"] else rows).to(DTYPES[c["out"]])
    if c["op"] == "combine_rows":
        y, out = state["y"].float(), []
        if c["order"] == "bucket":
            positions = torch.empty_like(perm)
            positions[perm] = torch.arange(perm.numel(), device=perm.device)
            y = y[positions]
            out = [positions.to(torch.int32)]
        y = y.reshape(c["T"], k, c["d"])
        y = (y * weights[..., None] if c["weighted"] else y).sum(1)
        return [(y + state["shared"].float() if c["shared"] else y).to(DTYPES[c["out"]])] + out
    if c["op"] == "combine_rows_grad":
        dout, y = state["dout"].float(), state["y"].float()
        if c["order"] == "bucket":
            positions = state["positions"].long()
            y = y[positions]
        dw = (y.reshape(c["T"], k, c["d"]) * dout[:, None]).sum(-1)
        dy = (weights[..., None] * dout[:, None]).reshape(-1, c["d"]).to(DTYPES[c["dtype"]])
        if c["order"] == "bucket":
            dy, slots = torch.empty_like(dy), dy
            dy[positions] = slots
        return dy, dw
    plan = state["plan"]
    x = state["x"].float()
    if c["x"] != "bucket":
        x = x[perm // k if c["x"] == "token" else perm]
    padded = torch.zeros(plan["active"].numel(), plan["longest"], c["K"], device=x.device)
    padded[plan["group"], plan["place"]] = x
    used = [None if t is None else t[plan["active"]] for t in (state["codes"], state["scales"], state["biases"])]
    y = torch.bmm(padded, _dequantize(*used, c["format"], c["group"]).transpose(1, 2))[plan["group"], plan["place"]]
    if c["y"] == "slot":
        y, rows = torch.empty_like(y), y
        y[perm] = rows
    return y.to(DTYPES[c["out"]])


# ------------------------------------------------------------------ the framework's calls

def _run_own(state):
    import quantized_sparse_moe_amd as qm
    c = state["case"]
    if c["op"] == "swiglu":
        return qm.swiglu_grad(state["gu"], state["dh"]) if c["grad"] else qm.swiglu(state["gu"])
    if c["op"] == "matmul_packed":
        return qm.matmul_packed(state["x"], state["codes"], state["scales"], state["biases"], out_dtype=c["out"])
    if c["op"] == "grouped_matmul_packed":
        return qm.grouped_matmul_packed(state["x"], state["codes"], state["scales"], state["biases"], state["offsets"],
                                      perm=state["perm"], top_k=c["k"], x_order=c["x"], out_order=c["y"],
                                      out_dtype=c["out"])
    if c["op"] == "gather_rows":
        return qm.gather_rows(state["x"], state["perm"], top_k=c["k"],
                              weights=state["weights"] if c["weighted"] else None, out_dtype=c["out"])
    if c["op"] == "combine_rows":
        positions = qm.invert_perm(state["perm"]) if c["order"] == "bucket" else None
        y = qm.combine_rows(state["y"], state["weights"] if c["weighted"] else None, positions, top_k=c["k"],
                            y_shared=state["shared"], out_dtype=c["out"])
        return [y] if positions is None else [y, positions]
    return qm.combine_rows_grad(state["dout"], state["y"], state["weights"], state["positions"])


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_weights(codes, scales, biases, fmt, group):
    """[N][K] of one matrix in 64 bits, nibble by nibble."""
    N, words = codes.shape
    w = torch.empty(N, words, 8, dtype=torch.float64, device=codes.device)
    unsigned = codes.long() % (1 << 32)
    for j in range(8):
        q = torch.div(unsigned, 16 ** j, rounding_mode="floor") % 16
        if fmt == "affine":
            w[..., j] = q.double()
        else:
            m, e = q % 2, torch.div(q, 2, rounding_mode="floor") % 4
            v = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * torch.exp2(e.double() - 1))
            w[..., j] = torch.where(q >= 8, -v, v)
    w = w.reshape(N, words * 8)
    spread = lambda t: t.repeat_interleave(group, dim=1)  # noqa: E731
    if fmt == "affine":
        return w.mul_(spread(scales.double())).add_(spread(biases.double()))
    return w.mul_(spread(torch.exp2(scales.double() - 127)))


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "swiglu":
        gate, up = s["gu"].double().chunk(2, dim=1)
        sig = torch.sigmoid(gate)
        if not c["grad"]:
            return gate * sig * up
        dh = s["dh"].double()
        return torch.cat([dh * up * (sig + gate * sig * torch.sigmoid(-gate)), dh * gate * sig], dim=1)
    if c["op"] == "matmul_packed":
        parts = []
        for r in range(0, c["N"], 16384):
            w = _exact_weights(s["codes"][r:r + 16384], s["scales"][r:r + 16384],
                               None if s["biases"] is None else s["biases"][r:r + 16384], c["format"], c["group"])
            parts.append(s["x"].double() @ w.t())
        return torch.cat(parts, dim=1)
    k, perm, weights = c["k"], s["perm"].long(), s["weights"].double().reshape(-1)
    tokens = torch.div(perm, k, rounding_mode="floor")
    if c["op"] == "gather_rows":
        rows = s["x"].double().index_select(0, tokens)
        return rows * weights[perm].unsqueeze(1) if c["weighted"] else rows
    if c["op"] == "combine_rows":
        slot = perm if c["order"] == "bucket" else torch.arange(perm.numel(), device=perm.device)
        out = s["shared"].double().clone() if c["shared"] else torch.zeros(c["T"], c["d"], dtype=torch.float64, device="cuda")
        rows = s["y"].double()
        out.index_add_(0, torch.div(slot, k, rounding_mode="floor"), rows * weights[slot].unsqueeze(1) if c["weighted"] else rows)
        return [out, None] if c["order"] == "bucket" else [out]
    if c["op"] == "combine_rows_grad":
        slot = perm if c["order"] == "bucket" else torch.arange(perm.numel(), device=perm.device)
        dout = s["dout"].double().index_select(0, torch.div(slot, k, rounding_mode="floor"))
        dw = torch.empty(c["T"] * k, dtype=torch.float64, device="cuda")
        dw[slot] = torch.linalg.vecdot(dout, s["y"].double())
        return dout * weights[slot].unsqueeze(1), dw.reshape(c["T"], k)
    bounds = s["offsets"].tolist()
    y = torch.zeros(c["T"] * k, c["N"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi == lo:
            continue
        rows = torch.arange(lo, hi, device="cuda") if c["x"] == "bucket" else tokens[lo:hi] if c["x"] == "token" else perm[lo:hi]
        w = _exact_weights(s["codes"][e], s["scales"][e], None if s["biases"] is None else s["biases"][e], c["format"], c["group"])
        y[perm[lo:hi] if c["y"] == "slot" else torch.arange(lo, hi, device="cuda")] = s["x"][rows].double() @ w.t()
    return y
