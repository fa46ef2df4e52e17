"""The embedding at the other end of the policy, and the norm of all gradients.

``embedding_fwd`` turns tokens into the rows a model begins with and
``embedding_bwd`` adds up their gradients by token, into a gradient of its own
or into the fused loss's grad_weight where the head shares the weight;
``grad_norm`` gives the global norm over many gradients and the factor that
clips them, which ``adamw_step`` takes as grad_scale; ``clip_grads`` applies it
in place for optimizers that take none. Bindings over include/plp.h, enqueued
on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Union

import torch

from . import _abi
from ._marshal import _check_vec, _dtype_code, _on, _one_device, _ptr, _stream_on, _workspace
from .operators import _fits, _out


def embedding_fwd(tokens: torch.Tensor, weight: torch.Tensor, *, scale: float = 1.0,
                  out: Optional[dict] = None) -> dict:
    """Rows of weight [V, H] (float32 or bfloat16) by int64 tokens [...], times
    scale (plp_embedding_fwd); a token outside [0, V) gives zeros. Returns
    {"y": [..., H]}, written into out's tensor where it has one."""
    dev = _one_device((("tokens", tokens), ("weight", weight)))
    if weight.dim() != 2:
        raise ValueError(f"weight: expected [V, H], got {tuple(weight.shape)}")
    if tokens.dtype != torch.int64:
        raise ValueError(f"tokens: expected torch.int64, got {tokens.dtype}")
    V, H = (int(n) for n in weight.shape)
    _fits(V, "V")
    _fits(H, "H")
    with _on(dev):
        y = _out(out, "y", (*tokens.shape, H), weight.dtype, dev)
        _abi.check(_abi.lib().plp_embedding_fwd(_ptr(tokens), _ptr(weight), tokens.numel(), H, V, _dtype_code(weight),
                                                float(scale), _ptr(y), _stream_on(dev)))
    return {"y": y}


def embedding_bwd(grad_y: torch.Tensor, tokens: torch.Tensor, V: int, *, scale: float = 1.0,
                  grad_dtype: Optional[torch.dtype] = None, accumulate: bool = False,
                  workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """The gradient of embedding_fwd's weight from grad_y [..., H] and its
    tokens [...] (plp_embedding_bwd), summed in fp32 in a fixed order. Returns
    {"grad_weight": [V, H]} of grad_dtype (grad_y's by default, or float32),
    written into out's tensor where it has one. accumulate=True adds to
    out["grad_weight"], such as the fused loss's where the head shares the
    weight, and leaves rows without tokens alone."""
    dev = _one_device((("grad_y", grad_y), ("tokens", tokens), ("workspace", workspace)))
    if tokens.dtype != torch.int64:
        raise ValueError(f"tokens: expected torch.int64, got {tokens.dtype}")
    if grad_y.dim() < 1 or grad_y.shape[:-1] != tokens.shape:
        raise ValueError(f"grad_y: expected {(*tokens.shape, 'H')}, got {tuple(grad_y.shape)}")
    if accumulate and (out is None or out.get("grad_weight") is None):
        raise ValueError("accumulate=True adds to out['grad_weight'], which is missing")
    H, V, N = int(grad_y.shape[-1]), int(V), tokens.numel()
    if V < 1:
        raise ValueError(f"V must be >= 1, got {V}")
    _fits(V, "V")
    _fits(H, "H")
    dtype = grad_y.dtype if grad_dtype is None else grad_dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"unsupported grad_dtype {dtype}: float32 or bfloat16")
    wdt = _abi.DTYPE_F32 if dtype == torch.float32 else _abi.DTYPE_BF16
    L = _abi.lib()
    n = ctypes.c_size_t()
    gdt, acc = _dtype_code(grad_y), 1 if accumulate else 0
    _abi.check(L.plp_embedding_bwd_workspace_size(N, H, V, gdt, ctypes.byref(n)))
    with _on(dev):
        gw = _out(out, "grad_weight", (V, H), dtype, dev)
        ws = _workspace(n.value, dev, workspace)
        _abi.check(L.plp_embedding_bwd(_ptr(tokens), _ptr(grad_y), N, H, V, gdt, wdt, float(scale), acc, _ptr(gw),
                                       _ptr(ws), ws.numel() * ws.element_size(), _stream_on(dev)))
    return {"grad_weight": gw}


class GradTable:
    """A checked list of gradients for grad_norm and clip_grads. It holds the
    tensors; a call refuses it where one of them has other memory than when it
    was built (.data). It does not see that a parameter has a new gradient
    tensor, and then goes on with the one it was given."""

    def __init__(self, grads, entries, device, overlap: str):
        self.grads = grads
        self.count = len(grads)
        self.device = device
        self._array = (_abi.PlpGradTensor * max(1, self.count))(*entries)
        self._at = [g.data_ptr() for g in grads]
        self._overlap = overlap
        n = ctypes.c_size_t()
        _abi.check(_abi.lib().plp_grad_norm_workspace_size(self._array, self.count, ctypes.byref(n)))
        self._bytes = n.value

    def _check_current(self) -> None:
        if list(map(torch.Tensor.data_ptr, self.grads)) != self._at:
            raise ValueError("a gradient has other memory than when the table was built: build it again")


def grad_table(grads: Sequence[torch.Tensor]) -> GradTable:
    """The gradients of a norm or a clipping, checked once for all steps:
    float32 or bfloat16 in any mixture, contiguous, on one GPU. Meant for
    gradients in buffers that stay, as adamw_table is."""
    grads = list(grads)
    entries, ranges, dev = [], [], None
    for i, g in enumerate(grads):
        d = _one_device(((f"grads[{i}]", g),))
        if dev is not None and d != dev:
            raise ValueError(f"grads[{i}] is on {d}, the first on {dev}")
        dev = d
        entries.append(_abi.PlpGradTensor(_ptr(g), g.numel(), _dtype_code(g), 0))
        if g.numel():
            ranges.append((g.data_ptr(), g.data_ptr() + g.numel() * g.element_size(), i))
    ranges.sort()
    overlap, end, who = "", 0, 0
    for a, b, i in ranges:
        if a < end:
            overlap = f"grads[{i}] overlaps grads[{who}]"
            break
        end, who = b, i
    return GradTable(grads, entries, dev, overlap)


def _scalar(t: torch.Tensor, name: str, table: GradTable) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor of one torch.float32, got {t!r}")
    _check_vec(t, 1, torch.float32, name)
    _one_device(((name, t), ("grads[0]", table.grads[0] if table.count else None)))
    return t


def grad_norm(grads: Union[GradTable, Sequence[torch.Tensor]], *, max_norm: Optional[float] = None, eps: float = 1e-6,
              grad_scale: Optional[torch.Tensor] = None, norms: bool = False,
              workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """The global 2-norm over many gradients, a grad_table or a list (checked
    at each call), and the factor that clips it to max_norm (None: no limit)
    (plp_grad_norm). grad_scale (fp32 [1] on the device) is a factor that the
    gradients still lack; norm and scale have it in them. Returns {"norm": fp32
    [1], "scale": fp32 [1], NaN where the norm is not finite} and with
    norms=True {"norms": fp32 [count]}, written into out's tensors where it has
    them. Pass "scale" to adamw_step as grad_scale, or to clip_grads."""
    table = grads if isinstance(grads, GradTable) else grad_table(grads)
    table._check_current()
    if table.device is None:
        raise ValueError("no gradients: an empty list has no device")
    if grad_scale is not None:
        _scalar(grad_scale, "grad_scale", table)
    dev = table.device
    if workspace is not None:
        _one_device((("workspace", workspace), ("gradients", table.grads[0])))
    limit = math.inf if max_norm is None else float(max_norm)
    with _on(dev):
        norm = _out(out, "norm", (1,), torch.float32, dev, grad_scale if grad_scale is not None and grad_scale.dim() == 1 else None)
        res = {"norm": norm, "scale": _out(out, "scale", (1,), torch.float32, dev, norm)}
        if norms:
            res["norms"] = _out(out, "norms", (table.count,), torch.float32, dev)
        ws = _workspace(table._bytes, dev, workspace)
        _abi.check(_abi.lib().plp_grad_norm(table._array, table.count, limit, float(eps), _ptr(grad_scale),
                                            _ptr(res["norm"]), _ptr(res["scale"]), _ptr(res.get("norms")), _ptr(ws),
                                            ws.numel() * ws.element_size(), _stream_on(dev)))
    return res


def clip_grads(grads: Union[GradTable, Sequence[torch.Tensor]], scale: torch.Tensor) -> None:
    """Multiplies every gradient by scale (fp32 [1] on the device, grad_norm's)
    in place (plp_clip_grads); a scale of 1, or one that is not finite, leaves
    them as they are. No two of them may overlap."""
    table = grads if isinstance(grads, GradTable) else grad_table(grads)
    table._check_current()
    if table._overlap:
        raise ValueError(table._overlap)
    _scalar(scale, "scale", table)
    if table.device is None:
        return
    with _on(table.device):
        _abi.check(_abi.lib().plp_clip_grads(table._array, table.count, _ptr(scale), _stream_on(table.device)))
