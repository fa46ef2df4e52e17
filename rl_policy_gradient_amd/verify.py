"""Verification of drafted tokens: a rollout in which a smaller model, or a copy
of the prompt, proposes several tokens and the policy takes as many of them as
its own distribution allows. ``verify_tokens`` is the counterpart of
``sample_tokens`` there; a binding over include/plp.h, enqueued on the current
stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Union

import torch

from . import _abi
from ._marshal import _check_vec, _dtype_code, _on, _one_device, _ptr, _stream_on, _workspace
from .operators import _INT32_MAX, _fits, _out

_Float = Union[float, torch.Tensor]
_Int = Union[int, torch.Tensor]


def _limits(t: _abi.PlpTokenLimits, B: int, who: str, temperature, top_k, top_p, min_p) -> None:
    """The settings of one side: values, or checked tensors of one a sequence."""
    for name, v in (("temperature", temperature), ("top_p", top_p), ("min_p", min_p)):
        if isinstance(v, torch.Tensor):
            setattr(t, name + "_rows", _ptr(_check_vec(v, B, torch.float32, who + name)))
        else:
            setattr(t, name, float(v))
    if isinstance(top_k, torch.Tensor):
        t.top_k_rows = _ptr(_check_vec(top_k, B, torch.int32, who + "top_k"))
    else:
        t.top_k = max(-1, min(int(top_k), _INT32_MAX))


def verify_tokens(logits: torch.Tensor, draft_tokens: torch.Tensor, uniforms: torch.Tensor, *,
                  draft_logits: Optional[torch.Tensor] = None, num_drafts: Optional[torch.Tensor] = None,
                  temperature: _Float = 1.0, top_k: _Int = 0, top_p: _Float = 1.0, min_p: _Float = 0.0,
                  draft_temperature: _Float = 1.0, draft_top_k: _Int = 0, draft_top_p: _Float = 1.0,
                  draft_min_p: _Float = 0.0, workspace: Optional[torch.Tensor] = None,
                  out: Optional[dict] = None) -> dict:
    """Takes drafted tokens [B, K] (int64) as far as the target's logits
    [B, K+1, V] allow and adds one token of its own (plp_verify_tokens), from
    uniforms fp32 [B, K+1] in [0, 1). draft_logits [B, K, V] of the logits' dtype
    (float32 or bfloat16; rows contiguous, any distances) are what the drafts
    were sampled from, with the draft_ settings; without them each draft is
    certain (copied from the prompt, or a draft's likeliest token). num_drafts
    (int32 [B]) says how many drafts a sequence has, where not K. Settings are
    those of sample_tokens, one value or a device tensor [B]. Returns {"tokens":
    int64 [B, K+1] the accepted drafts, one token more, then -1, "accepted":
    int32 [B], "logp" and "kept_logp": fp32 [B, K+1] of the tokens as
    sample_tokens gives them, 0 after the last}, written into out's tensors
    where it has them; token -1 and NaN where a sequence comes to a row without
    a distribution."""
    if logits.dim() != 3 or logits.shape[1] < 1:
        raise ValueError(f"logits: expected [B, K+1, V], got {tuple(logits.shape)}")
    B, K, V = int(logits.shape[0]), int(logits.shape[1]) - 1, int(logits.shape[2])
    settings = (("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p))
    if draft_logits is not None:
        settings += (("draft_temperature", draft_temperature), ("draft_top_k", draft_top_k),
                     ("draft_top_p", draft_top_p), ("draft_min_p", draft_min_p))
    dev = _one_device((("logits", logits), ("draft_tokens", draft_tokens), ("uniforms", uniforms),
                       ("draft_logits", draft_logits), ("num_drafts", num_drafts), ("workspace", workspace),
                       *((k, t) for k, t in settings if isinstance(t, torch.Tensor))))
    _fits(V, "V")
    _fits(K, "K")
    for name, t, shape, dtype in (("draft_tokens", draft_tokens, (B, K), torch.int64),
                                  ("uniforms", uniforms, (B, K + 1), torch.float32)):
        if tuple(t.shape) != shape or t.dtype != dtype:
            raise ValueError(f"{name}: expected {shape} {dtype}, got {tuple(t.shape)} {t.dtype}")
    _check_vec(num_drafts, B, torch.int32, "num_drafts")
    a = _abi.PlpVerifyArgs()
    a.struct_size, a.dtype = ctypes.sizeof(a), _dtype_code(logits)
    a.B, a.K, a.V = B, K, V
    for name, t in (("logits", logits), ("draft_logits", draft_logits)):
        if t is not None and V > 1 and t.stride(2) != 1:
            raise ValueError(f"plp needs each row of {name} contiguous")
    a.logits, a.seq_stride, a.row_stride = logits.data_ptr(), int(logits.stride(0)), int(logits.stride(1))
    if draft_logits is not None:
        if tuple(draft_logits.shape) != (B, K, V) or draft_logits.dtype != logits.dtype:
            raise ValueError(f"draft_logits: expected {(B, K, V)} {logits.dtype}, got {tuple(draft_logits.shape)} "
                             f"{draft_logits.dtype}")
        a.draft_logits = draft_logits.data_ptr()
        a.draft_seq_stride, a.draft_row_stride = int(draft_logits.stride(0)), int(draft_logits.stride(1))
        _limits(a.draft, B, "draft_", draft_temperature, draft_top_k, draft_top_p, draft_min_p)
    _limits(a.target, B, "", temperature, top_k, top_p, min_p)
    a.draft_tokens, a.num_drafts, a.uniforms = _ptr(draft_tokens), _ptr(num_drafts), _ptr(uniforms)
    L = _abi.lib()
    n = ctypes.c_size_t()
    _abi.check(L.plp_verify_tokens_workspace_size(B, K, V, 0 if draft_logits is None else 1, ctypes.byref(n)))
    with _on(dev):
        res = {"tokens": _out(out, "tokens", (B, K + 1), torch.int64, dev),
               "accepted": _out(out, "accepted", (B,), torch.int32, dev),
               "logp": _out(out, "logp", (B, K + 1), torch.float32, dev, uniforms),
               "kept_logp": _out(out, "kept_logp", (B, K + 1), torch.float32, dev, uniforms)}
        a.tokens_out, a.accepted_out = _ptr(res["tokens"]), _ptr(res["accepted"])
        a.logp_out, a.kept_logp_out = _ptr(res["logp"]), _ptr(res["kept_logp"])
        ws = _workspace(n.value, dev, workspace)
        _abi.check(L.plp_verify_tokens(ctypes.byref(a), _ptr(ws), ws.numel() * ws.element_size(), _stream_on(dev)))
    return res
