"""Python front end of the library: device copies of a layer's weights and thin
wrappers around the C entry points.

torch provides device memory and the current stream only; every computation
happens in libqsmoe.so's HIP kernels (argument marshalling here, nothing else).
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from . import _lib
from ._lib import ExpertsC, LayerC, QTensorC, RouterC, check


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _to_device(a: np.ndarray, device) -> torch.Tensor:
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    elif a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


def _bits_tensor(x: torch.Tensor) -> torch.Tensor:
    if x.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"activations must be bf16 (or its int16 bit pattern), got {x.dtype}")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("activations must be a contiguous device tensor")
    return x


class DeviceQTensor:
    """A stacked quantised projection resident on the device."""

    def __init__(self, fmt: str, bits: int, group: int, rows: int, cols: int, codes: torch.Tensor,
                 scales: torch.Tensor, biases: Optional[torch.Tensor]):
        self.fmt, self.bits, self.group, self.rows, self.cols = fmt, bits, group, rows, cols
        self.codes, self.scales, self.biases = codes, scales, biases
        self.num_experts = codes.shape[0]
        fmt_c = {"affine": _lib.MOE_FMT_AFFINE, "mxfp4": _lib.MOE_FMT_MXFP4, "mxfp8": _lib.MOE_FMT_MXFP8}[fmt]
        self.c = QTensorC(fmt_c, bits, group, rows, cols,
                          self.num_experts, codes.data_ptr(), scales.data_ptr(),
                          biases.data_ptr() if biases is not None else None)

    @classmethod
    def from_host(cls, q, device) -> "DeviceQTensor":
        """From an object with spec.{fmt,bits,group}, rows, cols, codes, scales, biases (numpy)."""
        return cls(q.spec.fmt, q.spec.bits, q.spec.group, q.rows, q.cols, _to_device(q.codes, device),
                   _to_device(q.scales, device), None if q.biases is None else _to_device(q.biases, device))

    def clone(self) -> "DeviceQTensor":
        return DeviceQTensor(self.fmt, self.bits, self.group, self.rows, self.cols, self.codes.clone(),
                             self.scales.clone(), None if self.biases is None else self.biases.clone())

    def nbytes_per_expert(self) -> int:
        b = (self.codes[0].numel() * 4 + self.scales[0].numel() * self.scales.element_size())
        if self.biases is not None:
            b += self.biases[0].numel() * 2
        return b


class DeviceExperts:
    def __init__(self, gate: DeviceQTensor, up: DeviceQTensor, down: DeviceQTensor):
        self.gate, self.up, self.down = gate, up, down
        self.c = ExpertsC(gate.c, up.c, down.c)

    @classmethod
    def from_host(cls, ew, device) -> "DeviceExperts":
        return cls(DeviceQTensor.from_host(ew.gate, device), DeviceQTensor.from_host(ew.up, device),
                   DeviceQTensor.from_host(ew.down, device))

    def clone(self) -> "DeviceExperts":
        return DeviceExperts(self.gate.clone(), self.up.clone(), self.down.clone())

    def nbytes_per_expert(self) -> int:
        return sum(q.nbytes_per_expert() for q in (self.gate, self.up, self.down))


class DeviceLayer:
    """Router, routed experts and optional shared expert of one MoE layer. With
    `routed` None it is a router alone, for experts that the layer's packed
    formats do not hold (the grouped products): router_logits, route and
    workspace take it, the calls that run experts refuse it."""

    def __init__(self, route: str, top_k: int, wr: torch.Tensor, bias: Optional[torch.Tensor],
                 tid2eid: Optional[torch.Tensor], routed: Optional[DeviceExperts] = None,
                 shared: Optional[DeviceExperts] = None, routed_scale: float = 1.0):
        if routed is None and shared is not None:
            raise ValueError("a shared expert needs routed experts beside it")
        self.route, self.top_k = route, top_k
        self.wr, self.bias, self.tid2eid = wr, bias, tid2eid
        self.routed, self.shared = routed, shared
        self.E, self.d = wr.shape
        self.I = 0 if routed is None else routed.gate.rows
        self.vocab = 0 if tid2eid is None else tid2eid.shape[0]
        self.router_c = RouterC(_lib.MOE_ROUTE_HASH if route == "hash" else _lib.MOE_ROUTE_TOPK, self.E, top_k,
                                self.d, self.vocab, wr.data_ptr(), bias.data_ptr() if bias is not None else None,
                                tid2eid.data_ptr() if tid2eid is not None else None, routed_scale)
        self._shared_c = shared.c if shared is not None else None
        self._c = None if routed is None else LayerC(
            self.router_c, routed.c, ctypes.pointer(self._shared_c) if shared is not None else ctypes.POINTER(ExpertsC)())

    @property
    def c(self) -> LayerC:
        if self._c is None:
            raise ValueError("this layer is a router without packed experts")
        return self._c

    @classmethod
    def from_host(cls, layer, device="cuda", routed=None) -> "DeviceLayer":
        """From a host layer (cfg.route, cfg.top_k, wr, bias, tid2eid, routed, shared as numpy)."""
        cfg = layer.cfg
        r = routed if routed is not None else DeviceExperts.from_host(layer.routed, device)
        sh = DeviceExperts.from_host(layer.shared, device) if layer.shared is not None else None
        return cls(cfg.route, cfg.top_k, _to_device(layer.wr, device),
                   None if layer.bias is None or cfg.route == "hash" else _to_device(layer.bias, device),
                   None if layer.tid2eid is None else _to_device(layer.tid2eid, device), r, sh)

    def clone(self) -> "DeviceLayer":
        """An independent device copy of every weight (same values, new memory)."""
        c = lambda t: None if t is None else t.clone()
        return DeviceLayer(self.route, self.top_k, c(self.wr), c(self.bias), c(self.tid2eid), c(self.routed),
                           c(self.shared), self.router_c.routed_scale)

    # -- workspace ---------------------------------------------------------
    def workspace_size(self, max_tokens: int) -> int:
        if self._c is None:  # what moe_route needs by its documentation; moe_permute needs the first 256 bytes
            if max_tokens < 0:
                raise _lib.MoeError(_lib.MOE_ERR_INVALID_ARG, "workspace_size")
            words = 4 * max_tokens * self.E if self.route == "topk" else 0
            return 256 + sum(-(-n // 256) * 256 for n in (words, 2 * words, words))
        n = _lib.load().moe_workspace_size(ctypes.byref(self.c), max_tokens)
        if n == 0:
            raise _lib.MoeError(_lib.MOE_ERR_INVALID_ARG, "moe_workspace_size")
        return n

    def workspace(self, max_tokens: int) -> torch.Tensor:
        ws = torch.empty(self.workspace_size(max_tokens), dtype=torch.uint8, device=self.wr.device)
        workspace_init(ws)
        return ws

    def workspace_layout(self, T: int) -> dict:
        """moe_workspace_layout: byte offsets of moe_forward's intermediates in
        the workspace for T tokens (0: not written), plus 'total' and 'fused'."""
        out = _lib.WsLayoutC()
        check(_lib.load().moe_workspace_layout(ctypes.byref(self.c), T, ctypes.byref(out)), "moe_workspace_layout")
        return {name: getattr(out, name) for name, _ in _lib.WsLayoutC._fields_}


def workspace_init(ws: torch.Tensor, stream=None) -> None:
    check(_lib.load().moe_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "moe_workspace_init")


def device_error(ws: torch.Tensor, stream=None) -> int:
    code = ctypes.c_int32(0)
    check(_lib.load().moe_device_error(_ptr(ws), ctypes.byref(code), _stream(stream)), "moe_device_error")
    return code.value


def router_logits(layer: DeviceLayer, x: torch.Tensor, stream=None) -> torch.Tensor:
    x = _bits_tensor(x)
    T = x.shape[0]
    out = torch.empty((T, layer.E), dtype=torch.float32, device=x.device)
    check(_lib.load().moe_router_logits(ctypes.byref(layer.router_c), _ptr(x), T, _ptr(out), _stream(stream)),
          "moe_router_logits")
    return out


def route(layer: DeviceLayer, x: torch.Tensor, token_ids: Optional[torch.Tensor] = None,
          ws: Optional[torch.Tensor] = None, stream=None):
    x = _bits_tensor(x)
    T, k = x.shape[0], layer.top_k
    if ws is None:
        ws = layer.workspace(T)
    ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    check(_lib.load().moe_route(ctypes.byref(layer.router_c), _ptr(x), _ptr(token_ids), T, _ptr(ids), _ptr(w),
                                _ptr(ws), ws.numel(), _stream(stream)), "moe_route")
    return ids, w


def quantize_affine(w: torch.Tensor, bits: int, group: int, err: Optional[torch.Tensor] = None, stream=None):
    """Plain min/max affine quantisation of bf16 weights [rows][cols] (moe_quantize_affine):
    returns (codes uint32 [rows][cols*bits/32], scales fp16, biases fp16 [rows][cols/group])
    as device tensors (the fp16 ones as int16 bit patterns)."""
    w = _bits_tensor(w)
    rows, cols = w.shape
    codes = torch.empty((rows, cols * bits // 32), dtype=torch.int32, device=w.device)
    scales = torch.empty((rows, cols // group), dtype=torch.int16, device=w.device)
    biases = torch.empty_like(scales)
    check(_lib.load().moe_quantize_affine(_ptr(w), rows, cols, bits, group, _ptr(codes), _ptr(scales), _ptr(biases),
                                          None if err is None else _ptr(err), _stream(stream)), "moe_quantize_affine")
    return codes, scales, biases


def mhc_sinkhorn(logits: torch.Tensor, iters: int = 10, eps: float = 0.0, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """mHC mix matrices (moe_mhc_sinkhorn): logits fp32 [T][n][n] -> fp32 [T][n][n]."""
    if logits.dtype != torch.float32 or not logits.is_cuda or not logits.is_contiguous() or logits.dim() != 3:
        raise ValueError("logits must be a contiguous fp32 device tensor [T][n][n]")
    T, n, n2 = logits.shape
    if n != n2:
        raise ValueError("mix matrices must be square")
    out = torch.empty_like(logits) if out is None else out
    check(_lib.load().moe_mhc_sinkhorn(_ptr(logits), T, n, iters, eps, _ptr(out), _stream(stream)),
          "moe_mhc_sinkhorn")
    return out


def permute(ids: torch.Tensor, num_experts: int, ws: torch.Tensor, stream=None):
    T, k = ids.shape
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=ids.device)
    perm = torch.empty(T * k, dtype=torch.int32, device=ids.device)
    check(_lib.load().moe_permute(_ptr(ids), T, k, num_experts, _ptr(offsets), _ptr(perm), _ptr(ws), ws.numel(),
                                  _stream(stream)), "moe_permute")
    return offsets, perm


def expert_ffn(layer: DeviceLayer, x: torch.Tensor, offsets: torch.Tensor, perm: torch.Tensor,
               ws: torch.Tensor, stream=None):
    if layer.routed is None:
        raise ValueError("this layer is a router without packed experts")
    x = _bits_tensor(x)
    T, k, d = x.shape[0], layer.top_k, layer.d
    y_slot = torch.empty((T * k, d), dtype=torch.float32, device=x.device)
    y_sh = torch.empty((T, d), dtype=torch.float32, device=x.device) if layer.shared is not None else None
    sh = ctypes.byref(layer._shared_c) if layer.shared is not None else None
    check(_lib.load().moe_expert_ffn(ctypes.byref(layer.routed.c), sh, _ptr(x), T, k, _ptr(offsets), _ptr(perm),
                                     _ptr(y_slot), _ptr(y_sh), _ptr(ws), ws.numel(), _stream(stream)),
          "moe_expert_ffn")
    return y_slot, y_sh


def combine(y_slot: torch.Tensor, w: torch.Tensor, y_shared: Optional[torch.Tensor], out_dtype: str = "bf16",
            stream=None) -> torch.Tensor:
    T, k = w.shape
    d = y_slot.shape[1]
    f32 = out_dtype == "f32"
    out = torch.empty((T, d), dtype=torch.float32 if f32 else torch.bfloat16, device=y_slot.device)
    check(_lib.load().moe_combine(_ptr(y_slot), _ptr(w), _ptr(y_shared), T, k, d,
                                  _lib.MOE_OUT_F32 if f32 else _lib.MOE_OUT_BF16, _ptr(out), _stream(stream)),
          "moe_combine")
    return out


def forward(layer: DeviceLayer, x: torch.Tensor, token_ids: Optional[torch.Tensor] = None,
            out_dtype: str = "bf16", ws: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    x = _bits_tensor(x)
    T = x.shape[0]
    if ws is None:
        ws = layer.workspace(T)
    if out is None:
        f32 = out_dtype == "f32"
        out = torch.empty((T, layer.d), dtype=torch.float32 if f32 else torch.bfloat16, device=x.device)
    else:  # a given output buffer decides the output type
        if out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (T, layer.d):
            raise ValueError(f"out must be float32 or bfloat16 of shape ({T}, {layer.d})")
        f32 = out.dtype == torch.float32
    check(_lib.load().moe_forward(ctypes.byref(layer.c), _ptr(x), _ptr(token_ids), T,
                                  _lib.MOE_OUT_F32 if f32 else _lib.MOE_OUT_BF16, _ptr(out), _ptr(ws), ws.numel(),
                                  _stream(stream)), "moe_forward")
    return out


def forward_noalloc(layer: DeviceLayer, x: torch.Tensor, token_ids: Optional[torch.Tensor], out: torch.Tensor,
                    stream=None) -> torch.Tensor:
    """moe_forward_noalloc: moe_forward on the library's own per-GPU workspace
    (no workspace argument; calls on one GPU must not overlap in time). The
    output type follows `out` (float32 or bfloat16)."""
    x = _bits_tensor(x)
    f32 = out.dtype == torch.float32
    check(_lib.load().moe_forward_noalloc(ctypes.byref(layer.c), _ptr(x), _ptr(token_ids), x.shape[0],
                                          _lib.MOE_OUT_F32 if f32 else _lib.MOE_OUT_BF16, _ptr(out),
                                          _stream(stream)), "moe_forward_noalloc")
    return out


def forward_probed(layer: DeviceLayer, x: torch.Tensor, token_ids: Optional[torch.Tensor], out: torch.Tensor,
                   ws: torch.Tensor, events, stream=None):
    """moe_forward with a (start, stop) event pair per kernel, timestamped by
    the dispatch itself: kernel i runs between events[2i] and events[2i+1].
    Returns the kernels' names. ``events`` are torch.cuda.Event(enable_timing=True),
    already created on the device (record them once first)."""
    x = _bits_tensor(x)
    n = len(events)
    evs = (ctypes.c_void_p * n)(*[ctypes.c_void_p(e.cuda_event) for e in events])
    names = (ctypes.c_char_p * n)()
    count = ctypes.c_int32(0)
    f32 = out.dtype == torch.float32
    check(_lib.load().moe_forward_probed(ctypes.byref(layer.c), _ptr(x), _ptr(token_ids), x.shape[0],
                                         _lib.MOE_OUT_F32 if f32 else _lib.MOE_OUT_BF16, _ptr(out), _ptr(ws),
                                         ws.numel(), _stream(stream), evs, n, names, ctypes.byref(count)),
          "moe_forward_probed")
    return [names[i].decode() for i in range(count.value)]


def ws_region(ws: torch.Tensor, offset: int, dtype: torch.dtype, shape) -> torch.Tensor:
    """A view of `shape` elements of `dtype` at byte `offset` of a workspace
    (for reading the intermediates moe_workspace_layout locates)."""
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.tensor([], dtype=dtype).element_size()
    if offset <= 0 or offset + nbytes > ws.numel():
        raise ValueError(f"region [{offset}, {offset + nbytes}) outside the workspace")
    return ws[offset:offset + nbytes].view(dtype).view(*shape)


def probe_stream(buf: torch.Tensor, mode: int, sink: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_probe_stream over all of `buf` (a contiguous device tensor):
    mode 0 dense read, 1 the first 32 bytes of every 128-byte line, 2 write.
    Reads need `sink`: 2048 int32 words on the device (one per workgroup)."""
    check(_lib.load().moe_probe_stream(_ptr(buf), buf.numel() * buf.element_size(), mode, _ptr(sink),
                                       _stream(stream)), "moe_probe_stream")


def probe_mfma(workgroups: int, iters: int, out: torch.Tensor, stream=None) -> None:
    """moe_probe_mfma into `out` (int64 [5] on the device, zeroed by the caller)."""
    check(_lib.load().moe_probe_mfma(workgroups, iters, _ptr(out), _stream(stream)), "moe_probe_mfma")


@dataclass
class Intermediates:
    ids: torch.Tensor
    w: torch.Tensor
    offsets: torch.Tensor
    perm: torch.Tensor
    y_slot: torch.Tensor
    y_shared: Optional[torch.Tensor]
    out: torch.Tensor


def forward_staged(layer: DeviceLayer, x: torch.Tensor, token_ids: Optional[torch.Tensor] = None,
                   out_dtype: str = "f32", ws: Optional[torch.Tensor] = None, stream=None) -> Intermediates:
    """The four entry points called one after another, keeping every intermediate."""
    T = x.shape[0]
    if ws is None:
        ws = layer.workspace(T)
    ids, w = route(layer, x, token_ids, ws, stream)
    offsets, perm = permute(ids, layer.E, ws, stream)
    y_slot, y_sh = expert_ffn(layer, x, offsets, perm, ws, stream)
    out = combine(y_slot, w, y_sh, out_dtype, stream)
    return Intermediates(ids, w, offsets, perm, y_slot, y_sh, out)


# -- block-scaled FP8 and products grouped by expert ---------------------------
#
# The smallest of these calls take a few microseconds on the GPU, so what the
# host spends per call shows: arguments go to ctypes as plain integers, and the
# current stream's handle is asked for directly (0.06 us; a Stream object takes
# 2.6), as is the current device (0.06; 0.25), and empty() gets its sizes one by
# one (1.0 us; 1.35 as a tuple).

_DT = {torch.bfloat16: _lib.MOE_DT["bf16"], torch.float32: _lib.MOE_DT["f32"], torch.float16: _lib.MOE_DT["f16"]}
_TORCH_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}
_E4M3 = torch.float8_e4m3fn
_FP8 = (_E4M3, torch.uint8)
_B16 = (torch.bfloat16, torch.float16)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_forward_ad = torch.autograd.forward_ad  # _current_level: -1 outside of every dual level (0.06 us)


def _operand(t: torch.Tensor, name: str, dtypes, dims, device=None) -> torch.Tensor:
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous() or t.dim() not in dims:
        raise ValueError(f"{name} must be a contiguous device tensor of {' or '.join(str(d) for d in dims)} dimensions")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the first operand on {device}")
    return t


def _unrecorded(call: str, *operands: Optional[torch.Tensor]) -> None:
    """Refuse a call that autograd would have to record: its result would look
    like a constant, and the operands' gradients, or tangents in forward mode,
    would be lost in silence."""
    given = [t for t in operands if t is not None]
    if torch.is_grad_enabled() and any(t.requires_grad for t in given):
        raise RuntimeError(f"{call} is not recorded by autograd, but an operand requires grad: call it under "
                           "torch.no_grad(), with detached operands, or inside a torch.autograd.Function")
    if any(_forward_ad.unpack_dual(t).tangent is not None for t in given):
        raise RuntimeError(f"{call} is not recorded by autograd, but an operand has a forward-mode tangent: call it "
                           "with the operands' primals, or inside a torch.autograd.Function that has a jvp")


def _shape(t: torch.Tensor, name: str, shape) -> None:
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")


def _sides(*sizes: int) -> None:
    """ctypes would pass on the low 32 bits of a size that the ABI takes in 32."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"sizes must be below 2^31, got {sizes}")


def _elsewhere(device: torch.device, stream) -> bool:
    """Whether a call has to make another device or stream current first."""
    return stream is not None or device.index != _current_device()


@contextlib.contextmanager
def _on(device: torch.device, stream):
    """`device` current and, if a stream is given, that stream too, so that what
    a call allocates belongs to the stream its kernels run on."""
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the operands on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _err_ptr(err: Optional[torch.Tensor], device) -> Optional[int]:
    return None if err is None else _operand(err, "err", _I32, (1,), device).data_ptr()


def _out_type(name: str) -> torch.dtype:
    if name not in _TORCH_DT:
        raise ValueError(f"output type must be one of {', '.join(_TORCH_DT)}, got {name!r}")
    return _TORCH_DT[name]


def _out(out: Optional[torch.Tensor], shape, dtype: torch.dtype, device) -> torch.Tensor:
    if out is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    _shape(_operand(out, "out", tuple(_DT), (len(shape),), device), "out", shape)
    return out


def _block_out(y: torch.Tensor, f32_sums: bool) -> int:
    return _DT[y.dtype] | (_lib.MOE_SUMS_F32 if f32_sums else 0)


def _blocks(n: int) -> int:
    return -(-n // 128)


def quantize_block(x: torch.Tensor, block_rows: int = 1, pow2: bool = False, err: Optional[torch.Tensor] = None,
                   stream=None):
    """E4M3 codes with an fp32 scale per block of `block_rows` (1 or 128) rows
    and 128 columns (moe_quantize_block): x bf16, fp16 or fp32 [rows][cols], or
    [matrices][rows][cols] -> (codes float8_e4m3fn of x's shape, scales). A
    quantised copy: codes and scales are constants to autograd."""
    dev = _operand(x, "x", _DT, (2, 3)).device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return quantize_block(x, block_rows, pow2, err)
    *lead, rows, cols = x.shape
    _sides(cols, block_rows)
    codes = torch.empty_like(x, dtype=_E4M3)
    scales = torch.empty(*lead, -(-rows // max(block_rows, 1)), _blocks(cols), dtype=torch.float32, device=dev)
    check(_lib.load().moe_quantize_block(x.data_ptr(), _DT[x.dtype], lead[0] if lead else 1, rows, cols, block_rows,
                                         1 if pow2 else 0, codes.data_ptr(), scales.data_ptr(), _err_ptr(err, dev),
                                         _raw_stream(dev.index)), "moe_quantize_block")
    return codes, scales


def swiglu_quantize_block(gu: torch.Tensor, pow2: bool = False, err: Optional[torch.Tensor] = None, stream=None):
    """silu(gate) * up of gu [rows][gate | up], quantised per 1 x 128 block
    (moe_swiglu_quantize_block) -> (codes [rows][inner], scales), constants to
    autograd."""
    dev = _operand(gu, "gu", _DT, (2,)).device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return swiglu_quantize_block(gu, pow2, err)
    rows, two = gu.shape
    if two % 2:
        raise ValueError("gu must hold gate and up columns in equal number")
    inner = two // 2
    _sides(inner)
    codes = torch.empty(rows, inner, dtype=_E4M3, device=dev)
    scales = torch.empty(rows, _blocks(inner), dtype=torch.float32, device=dev)
    check(_lib.load().moe_swiglu_quantize_block(gu.data_ptr(), _DT[gu.dtype], rows, inner, 1 if pow2 else 0,
                                                codes.data_ptr(), scales.data_ptr(), _err_ptr(err, dev),
                                                _raw_stream(dev.index)), "moe_swiglu_quantize_block")
    return codes, scales


def matmul_block(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                 out_dtype: str = "bf16", out: Optional[torch.Tensor] = None, stream=None,
                 f32_sums: bool = False) -> torch.Tensor:
    """a @ b^T of block-scaled FP8 matrices (moe_matmul_block): a [M][K] with
    1 x 128 scales, b [N][K] with 128 x 128 scales -> [M][N]. A given `out`
    decides the output type. A bf16 result is summed by the FP8 matrix
    instruction, which drops the low bits of small products next to large ones;
    `f32_sums` makes its sums fp32, as those of the other types always are.
    Not recorded by autograd: operands that require grad are refused."""
    if (a.requires_grad or a_scales.requires_grad or b.requires_grad or b_scales.requires_grad
            or _forward_ad._current_level >= 0):
        _unrecorded("matmul_block", a, a_scales, b, b_scales)
    dev = _operand(a, "a", _FP8, (2,)).device
    M, K = a.shape
    N = _operand(b, "b", _FP8, (2,), dev).shape[0]
    _shape(b, "b", (N, K))
    _sides(M, N, K)
    _shape(_operand(a_scales, "a_scales", _F32, (2,), dev), "a_scales", (M, _blocks(K)))
    _shape(_operand(b_scales, "b_scales", _F32, (2,), dev), "b_scales", (_blocks(N), _blocks(K)))
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return matmul_block(a, a_scales, b, b_scales, out_dtype, out, None, f32_sums)
    y = _out(out, (M, N), _out_type(out_dtype), dev)
    check(_lib.load().moe_matmul_block(a.data_ptr(), a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(), M, N, K,
                                       _block_out(y, f32_sums), y.data_ptr(), _raw_stream(dev.index)), "moe_matmul_block")
    return y


def _groups(rows: int, order: str, top_k: int, offsets: torch.Tensor, perm: Optional[torch.Tensor], E: int, N: int,
            K: int, dev):
    """Checks of sizes, offsets and perm, and the token count of a matrix of `rows` rows in `order`."""
    if order not in _lib.MOE_ROWS:
        raise ValueError(f"row order must be one of {', '.join(_lib.MOE_ROWS)}, got {order!r}")
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    if order != "token" and rows % top_k:
        raise ValueError(f"{rows} rows in {order} order are no multiple of top_k = {top_k}")
    T = rows if order == "token" else rows // top_k
    _sides(T * top_k, E, N, K)
    _shape(_operand(offsets, "offsets", _I32, (1,), dev), "offsets", (E + 1,))
    if perm is not None:
        _shape(_operand(perm, "perm", _I32, (1,), dev), "perm", (T * top_k,))
    return T


def grouped_matmul_block(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                         offsets: torch.Tensor, perm: Optional[torch.Tensor] = None, top_k: int = 1,
                         x_order: str = "bucket", out_order: str = "bucket", out_dtype: str = "bf16",
                         out: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                         stream=None, f32_sums: bool = False) -> torch.Tensor:
    """Rows grouped by expert times their expert's weights, block-scaled FP8
    (moe_grouped_matmul_block): a [rows][K] with 1 x 128 scales in `x_order`
    ("bucket", "token" or "slot"), w [E][N][K] with 128 x 128 scales, offsets
    and perm as `permute` gives them -> [T * top_k][N] in `out_order` ("bucket"
    or "slot"). Rows of no bucket are not written. `f32_sums` and operands that
    require grad as in matmul_block."""
    if (a.requires_grad or a_scales.requires_grad or w.requires_grad or w_scales.requires_grad
            or _forward_ad._current_level >= 0):
        _unrecorded("grouped_matmul_block", a, a_scales, w, w_scales)
    dev = _operand(a, "a", _FP8, (2,)).device
    E, N, K = _operand(w, "w", _FP8, (3,), dev).shape
    rows = a.shape[0]
    _shape(a, "a", (rows, K))
    _shape(_operand(a_scales, "a_scales", _F32, (2,), dev), "a_scales", (rows, _blocks(K)))
    _shape(_operand(w_scales, "w_scales", _F32, (3,), dev), "w_scales", (E, _blocks(N), _blocks(K)))
    T = _groups(rows, x_order, top_k, offsets, perm, E, N, K, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return grouped_matmul_block(a, a_scales, w, w_scales, offsets, perm, top_k, x_order, out_order, out_dtype,
                                        out, err, None, f32_sums)
    y = _out(out, (T * top_k, N), _out_type(out_dtype), dev)
    check(_lib.load().moe_grouped_matmul_block(
        a.data_ptr(), a_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), T, top_k, N, K, E, offsets.data_ptr(),
        None if perm is None else perm.data_ptr(), _lib.MOE_ROWS[x_order], _lib.MOE_ROWS.get(out_order, -1),
        _block_out(y, f32_sums), y.data_ptr(), _err_ptr(err, dev), _raw_stream(dev.index)), "moe_grouped_matmul_block")
    return y


def grouped_matmul(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, perm: Optional[torch.Tensor] = None,
                   top_k: int = 1, x_order: str = "bucket", out_order: str = "bucket", transposed: bool = False,
                   out_dtype: Optional[str] = None, out: Optional[torch.Tensor] = None,
                   err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows grouped by expert times their expert's bf16 or fp16 weights
    (moe_grouped_matmul): w [E][N][K]; y = x w^T, or with `transposed` y = x w
    (the gradient in the rows of a product with w^T). Orders as in
    grouped_matmul_block; the output type is x's unless `out_dtype` or `out`
    says otherwise. Not recorded by autograd (operands that require grad are
    refused): the gradients are this call with `transposed` and
    grouped_matmul_dw."""
    if x.requires_grad or w.requires_grad or _forward_ad._current_level >= 0:
        _unrecorded("grouped_matmul", x, w)
    dev = _operand(x, "x", _B16, (2,)).device
    E, N, K = _operand(w, "w", (x.dtype,), (3,), dev).shape
    rows = x.shape[0]
    _shape(x, "x", (rows, N if transposed else K))
    T = _groups(rows, x_order, top_k, offsets, perm, E, N, K, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return grouped_matmul(x, w, offsets, perm, top_k, x_order, out_order, transposed, out_dtype, out, err)
    y = _out(out, (T * top_k, K if transposed else N), x.dtype if out_dtype is None else _out_type(out_dtype), dev)
    check(_lib.load().moe_grouped_matmul(
        x.data_ptr(), w.data_ptr(), _DT[x.dtype], T, top_k, N, K, E, offsets.data_ptr(),
        None if perm is None else perm.data_ptr(), _lib.MOE_ROWS[x_order], _lib.MOE_ROWS.get(out_order, -1),
        1 if transposed else 0, _DT[y.dtype], y.data_ptr(), _err_ptr(err, dev), _raw_stream(dev.index)),
        "moe_grouped_matmul")
    return y


def grouped_matmul_dw(x: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor, perm: Optional[torch.Tensor] = None,
                      top_k: int = 1, x_order: str = "bucket", dy_order: str = "bucket", out_dtype: str = "f32",
                      out: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """The gradient of grouped_matmul in the weights (moe_grouped_matmul_dw):
    x [rows][K] in `x_order`, dy [T * top_k][N] in `dy_order` ("bucket" or
    "slot") -> [E][N][K], the sum over each expert's positions of dy x^T. Not
    recorded by autograd either."""
    if x.requires_grad or dy.requires_grad or _forward_ad._current_level >= 0:
        _unrecorded("grouped_matmul_dw", x, dy)
    dev = _operand(x, "x", _B16, (2,)).device
    rows, K = x.shape
    N = _operand(dy, "dy", (x.dtype,), (2,), dev).shape[1]
    E = max(offsets.shape[0] - 1, 0) if offsets.dim() == 1 else 0
    T = _groups(rows, x_order, top_k, offsets, perm, E, N, K, dev)
    _shape(dy, "dy", (T * top_k, N))
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return grouped_matmul_dw(x, dy, offsets, perm, top_k, x_order, dy_order, out_dtype, out, err)
    dw = _out(out, (E, N, K), _out_type(out_dtype), dev)
    check(_lib.load().moe_grouped_matmul_dw(
        x.data_ptr(), dy.data_ptr(), _DT[x.dtype], T, top_k, N, K, E, offsets.data_ptr(),
        None if perm is None else perm.data_ptr(), _lib.MOE_ROWS[x_order], _lib.MOE_ROWS.get(dy_order, -1),
        _DT[dw.dtype], dw.data_ptr(), _err_ptr(err, dev), _raw_stream(dev.index)), "moe_grouped_matmul_dw")
    return dw


# -- rows to buckets and back, SwiGLU, 4-bit products ---------------------------

_WEIGHT16 = (torch.float16, torch.int16)  # fp16 scales and biases, as such or as quantize_affine's bit patterns


def _rows(T: int, k: int, n: int, *sizes: int) -> None:
    if k < 1:
        raise ValueError("top_k must be at least 1")
    _sides(T * k, n, *sizes)


def _weights(weights: Optional[torch.Tensor], T: int, k: int, dev) -> Optional[int]:
    if weights is None:
        return None
    _shape(_operand(weights, "weights", _F32, (2,), dev), "weights", (T, k))
    return weights.data_ptr()


def invert_perm(perm: torch.Tensor, size: Optional[int] = None, err: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """The bucket position of every assignment (moe_invert_perm): positions
    int32 [size] with positions[perm[p]] = p, -1 where perm names none; size is
    perm's length unless given."""
    dev = _operand(perm, "perm", _I32, (1,)).device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return invert_perm(perm, size, err)
    n = perm.shape[0]
    if size is None:
        size = n
    if size < 0:
        raise ValueError("size must not be negative")
    _sides(n, size)
    positions = torch.empty(size, dtype=torch.int32, device=dev)
    check(_lib.load().moe_invert_perm(perm.data_ptr(), n, size, positions.data_ptr(), _err_ptr(err, dev),
                                      _raw_stream(dev.index)), "moe_invert_perm")
    return positions


def gather_rows(x: torch.Tensor, perm: torch.Tensor, top_k: int = 1, x_order: str = "token",
                weights: Optional[torch.Tensor] = None, out_dtype: Optional[str] = None,
                out: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows in bucket order (moe_gather_rows): out[p] = x[perm[p] // top_k]
    (`x_order` "token") or x[perm[p]] ("slot"), times weights[T][top_k] at
    perm[p] if given. Rows of entries -1 are not written. The output type is x's
    unless `out_dtype` or `out` says otherwise. Not recorded by autograd
    (operands that require grad are refused): with perm naming no assignment
    twice, the gradient in x is combine_rows of the rows' gradient, the one in
    the weights (token order) combine_rows_grad's second result for (x, the
    rows' gradient, weights)."""
    if x.requires_grad or (weights is not None and weights.requires_grad) or _forward_ad._current_level >= 0:
        _unrecorded("gather_rows", x, weights)
    dev = _operand(x, "x", _DT, (2,)).device
    if x_order not in ("token", "slot"):
        raise ValueError(f"row order must be token or slot, got {x_order!r}")
    rows, d = x.shape
    n = _operand(perm, "perm", _I32, (1,), dev).shape[0]
    T = rows if x_order == "token" else rows // max(top_k, 1)
    _rows(T, top_k, n, d)
    if x_order == "slot" and rows != T * top_k:
        raise ValueError(f"{rows} rows in slot order are no multiple of top_k = {top_k}")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return gather_rows(x, perm, top_k, x_order, weights, out_dtype, out, err)
    w = _weights(weights, T, top_k, dev)
    y = _out(out, (n, d), x.dtype if out_dtype is None else _out_type(out_dtype), dev)
    check(_lib.load().moe_gather_rows(x.data_ptr(), _DT[x.dtype], T, top_k, d, _lib.MOE_ROWS[x_order],
                                      perm.data_ptr(), n, w, _DT[y.dtype], y.data_ptr(), _err_ptr(err, dev),
                                      _raw_stream(dev.index)), "moe_gather_rows")
    return y


def _slots(rows: int, positions: Optional[torch.Tensor], weights: Optional[torch.Tensor], top_k: Optional[int], dev):
    """(T, top_k) of rows in slot order, or of rows in bucket order by their positions."""
    if top_k is None:
        top_k = weights.shape[1] if weights is not None and weights.dim() == 2 else 1
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    slots = rows if positions is None else _operand(positions, "positions", _I32, (1,), dev).shape[0]
    if slots % top_k:
        raise ValueError(f"{slots} {'rows in slot order' if positions is None else 'positions'} are no multiple of "
                         f"top_k = {top_k}")
    return slots // top_k, top_k


def combine_rows(y: torch.Tensor, weights: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 top_k: Optional[int] = None, y_shared: Optional[torch.Tensor] = None,
                 out_dtype: Optional[str] = None, out: Optional[torch.Tensor] = None,
                 err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The weighted sum over each token's rows, and y_shared (moe_combine_rows):
    y [rows][d] in slot order, or in bucket order with `positions` from
    invert_perm (-1: no row); weights fp32 [T][top_k], None for ones (then
    `top_k` tells the slots of a token) -> [T][d] of y's type unless `out_dtype`
    or `out` says otherwise. `combine` is the same for fp32 rows in slot order.
    Not recorded by autograd (operands that require grad are refused): the
    gradients are combine_rows_grad's."""
    if y.requires_grad or (weights is not None and weights.requires_grad) or (
            y_shared is not None and y_shared.requires_grad) or _forward_ad._current_level >= 0:
        _unrecorded("combine_rows", y, weights, y_shared)
    dev = _operand(y, "y", _DT, (2,)).device
    n, d = y.shape
    T, top_k = _slots(n, positions, weights, top_k, dev)
    _rows(T, top_k, n, d)
    if y_shared is not None:
        _shape(_operand(y_shared, "y_shared", (y.dtype,), (2,), dev), "y_shared", (T, d))
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return combine_rows(y, weights, positions, top_k, y_shared, out_dtype, out, err)
    w = _weights(weights, T, top_k, dev)
    o = _out(out, (T, d), y.dtype if out_dtype is None else _out_type(out_dtype), dev)
    check(_lib.load().moe_combine_rows(y.data_ptr(), _DT[y.dtype], n, None if positions is None else positions.data_ptr(),
                                       w, None if y_shared is None else y_shared.data_ptr(), T, top_k, d, _DT[o.dtype],
                                       o.data_ptr(), _err_ptr(err, dev), _raw_stream(dev.index)), "moe_combine_rows")
    return o


def combine_rows_grad(dout: torch.Tensor, y: torch.Tensor, weights: torch.Tensor,
                      positions: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      err: Optional[torch.Tensor] = None, stream=None):
    """The gradients of combine_rows (moe_combine_rows_grad): dout [T][d], y and
    weights as there -> (dy of y's shape and type, dweights fp32 [T][top_k]).
    Rows of dy that no position names are not written, one that several name is
    not their sum. `out` takes dy."""
    if dout.requires_grad or y.requires_grad or weights.requires_grad or _forward_ad._current_level >= 0:
        _unrecorded("combine_rows_grad", dout, y, weights)
    dev = _operand(dout, "dout", _DT, (2,)).device
    n, d = _operand(y, "y", _DT, (2,), dev).shape
    T, top_k = _slots(n, positions, _operand(weights, "weights", _F32, (2,), dev), None, dev)
    _rows(T, top_k, n, d)
    _shape(dout, "dout", (T, d))
    _shape(weights, "weights", (T, top_k))
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return combine_rows_grad(dout, y, weights, positions, out, err)
    dy = _out(out, (n, d), y.dtype, dev)
    if dy.dtype != y.dtype:
        raise TypeError(f"out must be {y.dtype} as y, got {dy.dtype}")
    dw = torch.empty(T, top_k, dtype=torch.float32, device=dev)
    check(_lib.load().moe_combine_rows_grad(
        dout.data_ptr(), _DT[dout.dtype], y.data_ptr(), _DT[y.dtype], n,
        None if positions is None else positions.data_ptr(), weights.data_ptr(), T, top_k, d, dy.data_ptr(), dw.data_ptr(),
        _err_ptr(err, dev), _raw_stream(dev.index)), "moe_combine_rows_grad")
    return dy, dw


def swiglu(gu: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """silu(gate) * up of gu [rows][gate | up] (moe_swiglu) -> [rows][inner] of
    gu's type. Not recorded by autograd (a gu that requires grad is refused): the
    gradient is swiglu_grad."""
    if gu.requires_grad or _forward_ad._current_level >= 0:
        _unrecorded("swiglu", gu)
    dev = _operand(gu, "gu", _DT, (2,)).device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return swiglu(gu, out)
    rows, two = gu.shape
    if two % 2:
        raise ValueError("gu must hold gate and up columns in equal number")
    _sides(two)
    h = _out(out, (rows, two // 2), gu.dtype, dev)
    if h.dtype != gu.dtype:
        raise TypeError(f"out must be {gu.dtype} as gu, got {h.dtype}")
    check(_lib.load().moe_swiglu(gu.data_ptr(), _DT[gu.dtype], rows, two // 2, h.data_ptr(), _raw_stream(dev.index)),
          "moe_swiglu")
    return h


def swiglu_grad(gu: torch.Tensor, dh: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of swiglu (moe_swiglu_grad): gu [rows][gate | up], dh
    [rows][inner] -> dgu of gu's shape and type."""
    if gu.requires_grad or dh.requires_grad or _forward_ad._current_level >= 0:
        _unrecorded("swiglu_grad", gu, dh)
    dev = _operand(gu, "gu", _DT, (2,)).device
    rows, two = gu.shape
    if two % 2:
        raise ValueError("gu must hold gate and up columns in equal number")
    _sides(two)
    _shape(_operand(dh, "dh", _DT, (2,), dev), "dh", (rows, two // 2))
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return swiglu_grad(gu, dh, out)
    dgu = _out(out, (rows, two), gu.dtype, dev)
    if dgu.dtype != gu.dtype:
        raise TypeError(f"out must be {gu.dtype} as gu, got {dgu.dtype}")
    check(_lib.load().moe_swiglu_grad(gu.data_ptr(), _DT[gu.dtype], dh.data_ptr(), _DT[dh.dtype], rows, two // 2,
                                      dgu.data_ptr(), _raw_stream(dev.index)), "moe_swiglu_grad")
    return dgu


def _packed(codes: torch.Tensor, scales: torch.Tensor, biases: Optional[torch.Tensor], lead: tuple, K: int, dev):
    """(format, group, biases' address) of 4-bit weights [*lead][K], after checks of their three parts."""
    dims = (len(lead) + 1,)
    if K % 32 or K == 0:
        raise ValueError(f"the contraction must be a positive multiple of 32, got {K}")
    _shape(_operand(codes, "codes", _I32, dims, dev), "codes", (*lead, K // 8))
    _operand(scales, "scales", (torch.uint8,) if biases is None else _WEIGHT16, dims, dev)
    groups = scales.shape[-1]
    if groups == 0 or K % groups:
        raise ValueError(f"{groups} groups do not divide {K} columns")
    _shape(scales, "scales", (*lead, groups))
    if biases is None:
        return _lib.MOE_FMT_MXFP4, K // groups, None
    _shape(_operand(biases, "biases", _WEIGHT16, dims, dev), "biases", (*lead, groups))
    return _lib.MOE_FMT_AFFINE, K // groups, biases.data_ptr()


def _grad_of_packed(x, scales, biases) -> bool:
    return (x.requires_grad or scales.requires_grad or (biases is not None and biases.requires_grad)
            or _forward_ad._current_level >= 0)


def matmul_packed(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: Optional[torch.Tensor] = None,
                out_dtype: Optional[str] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [M][K] (bf16 or fp16) times W^T of 4-bit weights (moe_matmul_packed): codes
    int32 [N][K / 8] with scales and biases [N][K / group] as quantize_affine
    gives them (fp16, or their int16 bit patterns), or MXFP4 with uint8 scales
    [N][K / 32] and no biases -> [M][N] of x's type unless `out_dtype` or `out`
    says otherwise. For few rows. Not recorded by autograd: operands that require
    grad are refused."""
    if _grad_of_packed(x, scales, biases):
        _unrecorded("matmul_packed", x, scales, biases)
    dev = _operand(x, "x", _B16, (2,)).device
    M, K = x.shape
    N = _operand(codes, "codes", _I32, (2,), dev).shape[0]
    _sides(M, N, K)
    fmt, group, b = _packed(codes, scales, biases, (N,), K, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return matmul_packed(x, codes, scales, biases, out_dtype, out)
    y = _out(out, (M, N), x.dtype if out_dtype is None else _out_type(out_dtype), dev)
    check(_lib.load().moe_matmul_packed(x.data_ptr(), _DT[x.dtype], codes.data_ptr(), scales.data_ptr(), b, fmt, group,
                                      M, N, K, _DT[y.dtype], y.data_ptr(), _raw_stream(dev.index)), "moe_matmul_packed")
    return y


def grouped_matmul_packed(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: Optional[torch.Tensor],
                        offsets: torch.Tensor, perm: Optional[torch.Tensor] = None, top_k: int = 1,
                        x_order: str = "bucket", out_order: str = "bucket", out_dtype: Optional[str] = None,
                        out: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Rows grouped by expert times their expert's 4-bit weights
    (moe_grouped_matmul_packed): codes int32 [E][N][K / 8], scales and biases as in
    matmul_packed with E in front, orders, offsets and perm as in grouped_matmul ->
    [T * top_k][N] in `out_order`. Rows of no bucket are not written."""
    if _grad_of_packed(x, scales, biases):
        _unrecorded("grouped_matmul_packed", x, scales, biases)
    dev = _operand(x, "x", _B16, (2,)).device
    rows, K = x.shape
    E, N, _ = _operand(codes, "codes", _I32, (3,), dev).shape
    T = _groups(rows, x_order, top_k, offsets, perm, E, N, K, dev)
    fmt, group, b = _packed(codes, scales, biases, (E, N), K, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return grouped_matmul_packed(x, codes, scales, biases, offsets, perm, top_k, x_order, out_order, out_dtype,
                                       out, err)
    y = _out(out, (T * top_k, N), x.dtype if out_dtype is None else _out_type(out_dtype), dev)
    check(_lib.load().moe_grouped_matmul_packed(
        x.data_ptr(), _DT[x.dtype], codes.data_ptr(), scales.data_ptr(), b, fmt, group, T, top_k, N, K, E,
        offsets.data_ptr(), None if perm is None else perm.data_ptr(), _lib.MOE_ROWS[x_order],
        _lib.MOE_ROWS.get(out_order, -1), _DT[y.dtype], y.data_ptr(), _err_ptr(err, dev), _raw_stream(dev.index)),
        "moe_grouped_matmul_packed")
    return y
