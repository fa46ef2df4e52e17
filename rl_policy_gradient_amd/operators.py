"""The operators around the fused loss in a policy's training loop.

``sample_tokens`` draws the completions, with the log-probs the loss takes as
old_logp; ``layer_norm_fwd`` gives the hidden states the fused loss takes and
``layer_norm_bwd`` takes its grad_hidden back; ``adamw_step`` takes the
gradients of the weights, over every tensor of the model at once. Like the
rest of the package these are bindings: the work is done by HIP kernels behind
include/plp.h, enqueued on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import operator
from typing import Optional, Sequence, Union

import torch

from . import _abi
from ._marshal import _check_vec, _dtype_code, _on, _one_device, _ptr, _stream_on, _workspace


def _out(out: Optional[dict], name: str, shape, dtype, dev, like: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[name], checked, or a new tensor. like: a contiguous tensor of that
    shape and type, if there is one (half the time of describing it)."""
    if out is None or (t := out.get(name)) is None:
        return torch.empty(shape, dtype=dtype, device=dev) if like is None else torch.empty_like(like)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != dev:
        raise ValueError(f"out[{name!r}]: expected {tuple(shape)} {dtype} on {dev}, got {tuple(t.shape)} {t.dtype} "
                         f"on {t.device}")
    return t


_INT32_MAX = 2 ** 31 - 1


def _fits(n: int, name: str) -> None:
    """The C ABI holds row lengths in 32 bits."""
    if n > _INT32_MAX:
        raise ValueError(f"{name}={n} is above {_INT32_MAX}")


def sample_tokens(logits: torch.Tensor, uniforms: torch.Tensor, *, temperature: Union[float, torch.Tensor] = 1.0,
                  top_k: Union[int, torch.Tensor] = 0, top_p: Union[float, torch.Tensor] = 1.0,
                  min_p: Union[float, torch.Tensor] = 0.0, workspace: Optional[torch.Tensor] = None,
                  out: Optional[dict] = None) -> dict:
    """One token a row of logits [N, V] (float32 or bfloat16; rows contiguous,
    any distance apart) from uniforms fp32 [N] in [0, 1) (plp_sample_tokens).
    temperature, top_p, min_p (fp32) and top_k (int32) are one value or a
    device tensor [N]; 0 temperature is greedy, top_k 0, top_p 1 and min_p 0
    do not limit. Returns {"token": int64 [N], "logp": fp32 [N] under the
    whole tempered distribution, "kept_logp": fp32 [N] among the kept
    tokens}, written into out's tensors where it has them; token -1 and NaN
    for a row without a distribution."""
    if logits.dim() != 2:
        raise ValueError(f"logits: expected [N, V], got {tuple(logits.shape)}")
    N, V = (int(n) for n in logits.shape)
    rows = {k: t for k, t in (("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p)) if
            isinstance(t, torch.Tensor)}
    dev = _one_device((("logits", logits), ("uniforms", uniforms), ("workspace", workspace), *rows.items()))
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("plp needs each row of logits contiguous")
    _fits(V, "V")
    _check_vec(uniforms, N, torch.float32, "uniforms")
    for k, t in rows.items():
        _check_vec(t, N, torch.int32 if k == "top_k" else torch.float32, k)
    a = _abi.PlpSampleArgs()
    a.struct_size, a.dtype = ctypes.sizeof(a), _dtype_code(logits)
    a.N, a.V, a.row_stride = N, V, int(logits.stride(0)) if N > 1 else V
    a.logits, a.uniforms = logits.data_ptr(), _ptr(uniforms)
    if "temperature" in rows:
        a.temperature_rows = _ptr(temperature)
    else:
        a.temperature = float(temperature)
    if "top_k" in rows:
        a.top_k_rows = _ptr(top_k)
    else:
        a.top_k = max(-1, min(int(top_k), _INT32_MAX))
    if "top_p" in rows:
        a.top_p_rows = _ptr(top_p)
    else:
        a.top_p = float(top_p)
    if "min_p" in rows:
        a.min_p_rows = _ptr(min_p)
    else:
        a.min_p = float(min_p)
    L = _abi.lib()
    n = ctypes.c_size_t()
    _abi.check(L.plp_sample_tokens_workspace_size(N, V, ctypes.byref(n)))
    with _on(dev):
        like = uniforms if uniforms.dim() == 1 else None
        res = {"token": _out(out, "token", (N,), torch.int64, dev),
               "logp": _out(out, "logp", (N,), torch.float32, dev, like),
               "kept_logp": _out(out, "kept_logp", (N,), torch.float32, dev, like)}
        a.token_out, a.logp_out, a.kept_logp_out = _ptr(res["token"]), _ptr(res["logp"]), _ptr(res["kept_logp"])
        ws = _workspace(n.value, dev, workspace)
        _abi.check(L.plp_sample_tokens(ctypes.byref(a), _ptr(ws), ws.numel() * ws.element_size(), _stream_on(dev)))
    return res


def _norm_sizes(x, weight, bias):
    H = x.shape[-1]
    N = x.numel() // H if H else 0
    _fits(H, "H")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and (t.shape != (H,) or t.dtype != x.dtype):
            raise ValueError(f"{name}: expected ({H},) {x.dtype}, got {tuple(t.shape)} {t.dtype}")
    return N, H


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
                   rms: bool = False, out: Optional[dict] = None) -> dict:
    """Layer norm over the last dimension of x [..., H] (plp_layer_norm_fwd);
    rms=True leaves the mean out (root-mean-square norm). weight and bias [H]
    of x's dtype (float32 or bfloat16). Returns {"y": like x, "mean" (not with
    rms), "rstd": fp32 [...]}, written into out's tensors where it has them."""
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    dev = _one_device((("x", x), ("weight", weight), ("bias", bias)))
    N, H = _norm_sizes(x, weight, bias)
    with _on(dev):
        res = {"y": _out(out, "y", x.shape, x.dtype, dev, x)}
        rstd = res["rstd"] = _out(out, "rstd", x.shape[:-1], torch.float32, dev)
        if not rms:
            res["mean"] = _out(out, "mean", x.shape[:-1], torch.float32, dev, rstd)
        _abi.check(_abi.lib().plp_layer_norm_fwd(_ptr(x), _ptr(weight), _ptr(bias), N, H, _dtype_code(x),
                                                 1 if rms else 0, float(eps), _ptr(res["y"]), _ptr(res.get("mean")),
                                                 _ptr(res["rstd"]), _stream_on(dev)))
    return res


def layer_norm_bwd(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                   mean: Optional[torch.Tensor] = None, *, rms: bool = False, grad_x: bool = True,
                   grad_weight: bool = True, grad_bias: bool = True, workspace: Optional[torch.Tensor] = None,
                   out: Optional[dict] = None) -> dict:
    """The gradients of layer_norm_fwd from its input and statistics
    (plp_layer_norm_bwd); mean is required unless rms. Returns the asked-for
    ones of {"grad_x": like x, "grad_weight": [H], "grad_bias": [H]} in x's
    dtype, written into out's tensors where it has them."""
    dev = _one_device((("grad_y", grad_y), ("x", x), ("weight", weight), ("rstd", rstd), ("mean", mean),
                       ("workspace", workspace)))
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
    with _on(dev):
        res = {}
        if grad_x:
            res["grad_x"] = _out(out, "grad_x", x.shape, x.dtype, dev, x)
        for name, wanted in (("grad_weight", grad_weight), ("grad_bias", grad_bias)):
            if wanted:
                res[name] = _out(out, name, (H,), x.dtype, dev, weight)
        ws = _workspace(n.value if grad_weight or grad_bias else 0, dev, workspace)
        _abi.check(L.plp_layer_norm_bwd(_ptr(grad_y), _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), N, H, dt,
                                        1 if rms else 0, _ptr(res.get("grad_x")), _ptr(res.get("grad_weight")),
                                        _ptr(res.get("grad_bias")), _ptr(ws), ws.numel() * ws.element_size(),
                                        _stream_on(dev)))
    return res


ADAMW_BLOCK = 256  # elements of one scale of the 8-bit states
_SCALED = {"exp_avg": "exp_avg_scale", "exp_rms": "exp_rms_scale"}


def adamw_state(param: torch.Tensor, *, bits: int = 32, master: bool = False) -> dict:
    """The state of one parameter before its first step. bits=32: "exp_avg"
    and "exp_avg_sq" in fp32; bits=8: "exp_avg" and "exp_rms" (the second
    moment's root) as float8_e4m3fn codes with an fp32 scale per 256 elements
    in "exp_avg_scale" and "exp_rms_scale"; with a beta above 0.95 they are
    right in the mean over steps numbered one after the other (plp_adamw_step).
    master=True adds an fp32 copy of a bfloat16 parameter, on which the step
    then works."""
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    new = lambda n, dt: torch.zeros(n, dtype=dt, device=param.device)  # noqa: E731
    if bits == 32:
        st = {"exp_avg": new(param.shape, torch.float32), "exp_avg_sq": new(param.shape, torch.float32)}
    else:
        blocks = -(-param.numel() // ADAMW_BLOCK)
        st = {k: new(param.shape, torch.uint8).view(torch.float8_e4m3fn) for k in _SCALED}
        st.update({k: new(blocks, torch.float32) for k in _SCALED.values()})
    if master:
        if param.dtype != torch.bfloat16:
            raise ValueError("a master copy is for bfloat16 parameters")
        st["master"] = param.detach().float()
    return st


class AdamWTable:
    """A checked list of tensors for adamw_step. It holds the memory that its
    pointers name, whatever becomes of the tensors. Build it again when a
    tensor is replaced: a step refuses the table where a state's dict holds
    another tensor or a parameter has other memory (.data, a checkpoint put
    in its place). It does not see that there is a new gradient tensor, or
    other memory behind a gradient or a state's tensor, and then goes on with
    the ones it was given."""

    def __init__(self, entries, tensors, names, device):
        self.count = len(entries)
        self.device = device
        self.tensors = tensors
        self._array = (_abi.PlpAdamwTensor * max(1, self.count))(*entries)
        self._params = [p for p, _, _ in tensors]
        self._at = [p.data_ptr() for p in self._params]
        # the states by name: what reads it, the dicts that have it, what they held
        self._held = []
        for k in dict.fromkeys(k for ks in names for k in ks):
            dicts = [st for (_, _, st), ks in zip(tensors, names) if k in ks]
            self._held.append((operator.itemgetter(k), dicts, [st[k] for st in dicts], k))
        self._memory = [t.untyped_storage() for p, g, st in tensors for t in (p, g)]
        self._memory += [t.untyped_storage() for _, _, held, _ in self._held for t in held]

    def _check_current(self) -> None:
        """A few microseconds for a dozen tensors: identities and pointers, in
        one pass of C code each."""
        for get, dicts, held, k in self._held:
            try:
                same = all(map(operator.is_, map(get, dicts), held))
            except KeyError:
                same = False
            if not same:
                raise ValueError(f"a state's {k!r} has been replaced since the table was built: build it again")
        if list(map(torch.Tensor.data_ptr, self._params)) != self._at:
            raise ValueError("a parameter has other memory than when the table was built: build it again")


def adamw_table(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], states: Sequence[dict], *,
                weight_decay: Union[float, Sequence[float]] = 0.0) -> AdamWTable:
    """The tensors of an AdamW step, checked once for all steps: params and
    grads float32 or bfloat16 in any combination, states as adamw_state makes
    them (8 and 32 bits may be mixed), weight_decay one value or one per
    tensor. All are contiguous, on one GPU, and no two overlap but for
    gradients, which are only read. The checks take 6 to 8 microseconds a
    tensor: meant for gradients in buffers that stay (out= of the calls that
    give them), rather than a table a step."""
    params, grads, states = list(params), list(grads), list(states)
    if not len(params) == len(grads) == len(states):
        raise ValueError(f"{len(params)} params, {len(grads)} grads and {len(states)} states")
    decay = [float(weight_decay)] * len(params) if not hasattr(weight_decay, "__len__") else [float(w) for w in
                                                                                              weight_decay]
    if len(decay) != len(params):
        raise ValueError(f"{len(decay)} weight decays for {len(params)} tensors")
    entries, keep, held, ranges, dev = [], [], [], [], None
    for i, (p, g, st, wd) in enumerate(zip(params, grads, states, decay)):
        bits = 8 if "exp_rms" in st else 32
        n = p.numel()
        names = list(_SCALED) + list(_SCALED.values()) if bits == 8 else ["exp_avg", "exp_avg_sq"]
        want = {k: (n, torch.float8_e4m3fn if bits == 8 else torch.float32) for k in names}
        want.update({k: (-(-n // ADAMW_BLOCK), torch.float32) for k in _SCALED.values() if k in want})
        if st.get("master") is not None:
            want["master"] = (n, torch.float32)
        for k, (m, dt) in want.items():
            if k not in st:
                raise ValueError(f"states[{i}] has no {k!r}")
            _check_vec(st[k], m, dt, f"states[{i}][{k!r}]")
        if g.numel() != n:
            raise ValueError(f"grads[{i}]: {g.numel()} elements, the parameter has {n}")
        written = {"params": p, **{k: st[k] for k in want}}
        d = _one_device((("grads", g), *written.items()))
        if dev is not None and d != dev:
            raise ValueError(f"tensor {i} is on {d}, the first on {dev}")
        dev = d
        e = _abi.PlpAdamwTensor()
        e.param, e.grad, e.master = _ptr(p), _ptr(g), _ptr(st.get("master"))
        e.exp_avg, e.exp_avg_sq = _ptr(st["exp_avg"]), _ptr(st["exp_rms" if bits == 8 else "exp_avg_sq"])
        if bits == 8:
            e.exp_avg_scale, e.exp_avg_sq_scale = _ptr(st["exp_avg_scale"]), _ptr(st["exp_rms_scale"])
        e.numel, e.state_bits, e.weight_decay = n, bits, wd
        e.param_dtype, e.grad_dtype = _dtype_code(p), _dtype_code(g)
        entries.append(e)
        keep.append((p, g, st))
        held.append(tuple(want))
        ranges += [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), f"{k} of tensor {i}", True)
                   for k, t in written.items() if t.numel()]
        ranges += [(g.data_ptr(), g.data_ptr() + g.numel() * g.element_size(), f"grad of tensor {i}", False)] * (n > 0)
    ranges.sort()
    end, end_w, who, who_w = 0, 0, "", ""  # the furthest end so far, of all and of what is written
    for a, b, name, w in ranges:
        if a < (end if w else end_w):
            raise ValueError(f"{name} overlaps {who if w else who_w}")
        if b > end:
            end, who = b, name
        if w and b > end_w:
            end_w, who_w = b, name
    return AdamWTable(entries, keep, held, dev)


_ARGS_SIZE, _TENSOR_SIZE = ctypes.sizeof(_abi.PlpAdamwArgs), ctypes.sizeof(_abi.PlpAdamwTensor)


def _on_device(t, dtype, name: str, table: AdamWTable) -> Optional[int]:
    """The address of a step's scalar in device memory; None if it is none."""
    if not isinstance(t, torch.Tensor):
        return None
    _check_vec(t, 1, dtype, name)
    if table.device is not None and t.device != table.device:
        raise ValueError(f"{name} is on {t.device}, the tensors on {table.device}")
    return _ptr(t)


def adamw_step(table: AdamWTable, *, lr: Union[float, torch.Tensor], step: Union[int, torch.Tensor],
               betas=(0.9, 0.999), eps: float = 1e-8, grad_scale: Optional[torch.Tensor] = None) -> None:
    """One AdamW step over a table's tensors, in place (plp_adamw_step). step
    counts from 1. lr (fp32 [1]) and step (int64 [1]) may be device tensors,
    read when the step runs, so that a captured graph can be replayed.
    grad_scale (fp32 [1] on the device) multiplies every gradient; where it is
    not finite the step changes nothing."""
    table._check_current()
    lr_at = _on_device(lr, torch.float32, "lr", table)
    step_at = _on_device(step, torch.int64, "step", table)
    scale_at = _on_device(grad_scale, torch.float32, "grad_scale", table)
    if scale_at is None and grad_scale is not None:
        raise ValueError(f"grad_scale: expected a tensor of one torch.float32, got {grad_scale!r}")
    a = _abi.PlpAdamwArgs(_ARGS_SIZE, _TENSOR_SIZE, float(lr) if lr_at is None else 0.0, float(betas[0]), float(betas[1]),
                          float(eps), int(step) if step_at is None else 0, step_at, lr_at, scale_at)
    L = _abi.lib()
    if table.count == 0:
        _abi.check(L.plp_adamw_step(ctypes.byref(a), table._array, 0, None))
        return
    with _on(table.device):
        _abi.check(L.plp_adamw_step(ctypes.byref(a), table._array, table.count, _stream_on(table.device)))
