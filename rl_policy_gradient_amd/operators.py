"""The operators around the fused loss in a policy's training loop.

``layer_norm_fwd`` gives the hidden states the fused loss takes and
``layer_norm_bwd`` takes its grad_hidden back. Like the rest of the package
these are bindings: the work is done by HIP kernels behind include/plp.h,
enqueued on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _abi
from ._marshal import _check_vec, _dtype_code, _one_device, _ptr, _stream, _workspace


def _out(out: Optional[dict], name: str, shape, dtype, dev) -> torch.Tensor:
    """out[name], checked, or a new tensor."""
    t = None if out is None else out.get(name)
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != dev:
        raise ValueError(f"out[{name!r}]: expected {tuple(shape)} {dtype} on {dev}, got {tuple(t.shape)} {t.dtype} "
                         f"on {t.device}")
    return t


def _norm_sizes(x, weight, bias):
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    H = int(x.shape[-1])
    N = 1
    for n in x.shape[:-1]:
        N *= int(n)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and (tuple(t.shape) != (H,) or t.dtype != x.dtype):
            raise ValueError(f"{name}: expected ({H},) {x.dtype}, got {tuple(t.shape)} {t.dtype}")
    return N, H


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
                   rms: bool = False, out: Optional[dict] = None) -> dict:
    """Layer norm over the last dimension of x [..., H] (plp_layer_norm_fwd);
    rms=True leaves the mean out (root-mean-square norm). weight and bias [H]
    of x's dtype (float32 or bfloat16). Returns {"y": like x, "mean" (not with
    rms), "rstd": fp32 [...]}, written into out's tensors where it has them."""
    dev = _one_device(x=x, weight=weight, bias=bias)
    N, H = _norm_sizes(x, weight, bias)
    with torch.cuda.device(dev):
        res = {"y": _out(out, "y", x.shape, x.dtype, dev), "rstd": _out(out, "rstd", x.shape[:-1], torch.float32, dev)}
        if not rms:
            res["mean"] = _out(out, "mean", x.shape[:-1], torch.float32, dev)
        _abi.check(_abi.lib().plp_layer_norm_fwd(_ptr(x), _ptr(weight), _ptr(bias), N, H, _dtype_code(x),
                                                 1 if rms else 0, float(eps), _ptr(res["y"]), _ptr(res.get("mean")),
                                                 _ptr(res["rstd"]), _stream(dev)))
    return res


def layer_norm_bwd(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                   mean: Optional[torch.Tensor] = None, *, rms: bool = False, grad_x: bool = True,
                   grad_weight: bool = True, grad_bias: bool = True, workspace: Optional[torch.Tensor] = None,
                   out: Optional[dict] = None) -> dict:
    """The gradients of layer_norm_fwd from its input and statistics
    (plp_layer_norm_bwd); mean is required unless rms. Returns the asked-for
    ones of {"grad_x": like x, "grad_weight": [H], "grad_bias": [H]} in x's
    dtype, written into out's tensors where it has them."""
    dev = _one_device(grad_y=grad_y, x=x, weight=weight, rstd=rstd, mean=mean)
    N, H = _norm_sizes(x, weight, None)
    if grad_y.shape != x.shape or grad_y.dtype != x.dtype:
        raise ValueError(f"grad_y: expected {tuple(x.shape)} {x.dtype}, got {tuple(grad_y.shape)} {grad_y.dtype}")
    _check_vec(rstd, N, torch.float32, "rstd")
    _check_vec(mean, N, torch.float32, "mean")
    if (mean is None) != bool(rms):
        raise ValueError("pass the forward's mean, and none with rms=True")
    L = _abi.lib()
    n = ctypes.c_size_t()
    dt = _dtype_code(x)
    _abi.check(L.plp_layer_norm_bwd_workspace_size(N, H, dt, ctypes.byref(n)))
    with torch.cuda.device(dev):
        res = {}
        if grad_x:
            res["grad_x"] = _out(out, "grad_x", x.shape, x.dtype, dev)
        for name, wanted in (("grad_weight", grad_weight), ("grad_bias", grad_bias)):
            if wanted:
                res[name] = _out(out, name, (H,), x.dtype, dev)
        ws = _workspace(n.value if grad_weight or grad_bias else 0, dev, workspace)
        _abi.check(L.plp_layer_norm_bwd(_ptr(grad_y), _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), N, H, dt,
                                        1 if rms else 0, _ptr(res.get("grad_x")), _ptr(res.get("grad_weight")),
                                        _ptr(res.get("grad_bias")), ws.data_ptr(), ws.numel() * ws.element_size(),
                                        _stream(dev)))
    return res
