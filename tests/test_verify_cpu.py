"""Verification of drafted tokens without a GPU: sizes and refusals. Every call
here is answered by the host checks before any launch; the pointers are made up
and never followed."""
import ctypes
import math
import os

import pytest
import torch

abi = pytest.importorskip("rl_policy_gradient_amd._abi")


def _lib():
    if not os.path.exists(abi.LIB_PATH):
        pytest.skip("libplp.so not built")
    return abi.lib()


def _err():
    return _lib().plp_last_error().decode()


AT = [0x100000000 * (i + 1) for i in range(16)]  # far apart: nothing overlaps
WS = AT[15]


def verify(n=1 << 24, ws=WS, target=None, draft=None, **kw):
    a = abi.PlpVerifyArgs()
    a.struct_size, a.dtype = ctypes.sizeof(a), abi.DTYPE_BF16
    a.B, a.K, a.V = 4, 3, 1000
    a.logits, a.seq_stride, a.row_stride = AT[0], 4000, 1000
    a.draft_logits, a.draft_seq_stride, a.draft_row_stride = AT[1], 3000, 1000
    a.draft_tokens, a.num_drafts, a.uniforms = AT[2], AT[3], AT[4]
    a.tokens_out, a.accepted_out, a.logp_out, a.kept_logp_out = AT[5:9]
    for side, more in ((a.target, target), (a.draft, draft)):
        side.temperature = side.top_p = 1.0
        for k, v in (more or {}).items():
            setattr(side, k, v)
    for k, v in kw.items():
        setattr(a, k, v)
    return _lib().plp_verify_tokens(ctypes.byref(a), ws, n, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(struct_size=16), abi.PLP_E_INVALID, "struct_size"), (dict(dtype=2), abi.PLP_E_INVALID, "dtype"),
    (dict(B=-1), abi.PLP_E_INVALID, "B=-1"), (dict(B=1 << 31), abi.PLP_E_INVALID, "B="),
    (dict(K=-1), abi.PLP_E_INVALID, "K must"), (dict(K=1025), abi.PLP_E_UNSUPPORTED, "K=1025"),
    (dict(V=0), abi.PLP_E_INVALID, "V must"), (dict(V=(1 << 20) + 1), abi.PLP_E_UNSUPPORTED, "V="),
    (dict(seq_stride=-1), abi.PLP_E_INVALID, "strides"), (dict(row_stride=-1), abi.PLP_E_INVALID, "strides"),
    (dict(draft_row_stride=-4), abi.PLP_E_INVALID, "strides"), (dict(draft_seq_stride=-4), abi.PLP_E_INVALID, "strides"),
    (dict(seq_stride=1 << 61), abi.PLP_E_INVALID, "address space"), (dict(row_stride=1 << 62), abi.PLP_E_INVALID, "address space"),
    (dict(draft_seq_stride=1 << 62), abi.PLP_E_INVALID, "address space"),
    (dict(target=dict(temperature=-0.5)), abi.PLP_E_INVALID, "target's temperature"),
    (dict(target=dict(temperature=math.inf)), abi.PLP_E_INVALID, "target's temperature"),
    (dict(target=dict(top_k=-2)), abi.PLP_E_INVALID, "target's top_k"), (dict(target=dict(top_p=1.1)), abi.PLP_E_INVALID, "target's top_p"),
    (dict(target=dict(min_p=math.nan)), abi.PLP_E_INVALID, "target's min_p"), (dict(draft=dict(top_p=-0.1)), abi.PLP_E_INVALID, "draft's top_p"),
    (dict(draft=dict(temperature=math.nan)), abi.PLP_E_INVALID, "draft's temperature"),
    (dict(draft=dict(top_k=-1)), abi.PLP_E_INVALID, "draft's top_k"), (dict(draft=dict(min_p=2.0)), abi.PLP_E_INVALID, "draft's min_p"),
    (dict(target=dict(temperature_rows=AT[9] + 1)), abi.PLP_E_INVALID, "aligned"),
    (dict(draft=dict(top_k_rows=AT[9] + 2)), abi.PLP_E_INVALID, "aligned"),
    (dict(logits=None), abi.PLP_E_INVALID, "required"), (dict(draft_tokens=None), abi.PLP_E_INVALID, "required"),
    (dict(uniforms=None), abi.PLP_E_INVALID, "required"), (dict(tokens_out=None), abi.PLP_E_INVALID, "required"),
    (dict(accepted_out=None), abi.PLP_E_INVALID, "required"), (dict(logits=AT[0] + 1), abi.PLP_E_INVALID, "aligned"),
    (dict(draft_logits=AT[1] + 1), abi.PLP_E_INVALID, "aligned"), (dict(draft_tokens=AT[2] + 4), abi.PLP_E_INVALID, "aligned"),
    (dict(tokens_out=AT[5] + 4), abi.PLP_E_INVALID, "aligned"), (dict(accepted_out=AT[6] + 2), abi.PLP_E_INVALID, "aligned"),
    (dict(num_drafts=AT[3] + 1), abi.PLP_E_INVALID, "aligned"), (dict(kept_logp_out=AT[8] + 3), abi.PLP_E_INVALID, "aligned"),
    (dict(tokens_out=AT[0] + 4 * 4000 * 2 - 8), abi.PLP_E_INVALID, "overlap an input"),
    (dict(tokens_out=AT[2] + 88), abi.PLP_E_INVALID, "overlap an input"), (dict(logp_out=AT[4]), abi.PLP_E_INVALID, "overlap an input"),
    (dict(logp_out=AT[1] + 40), abi.PLP_E_INVALID, "overlap an input"), (dict(accepted_out=AT[3] + 12), abi.PLP_E_INVALID, "overlap an input"),
    (dict(target=dict(min_p_rows=AT[8])), abi.PLP_E_INVALID, "overlap an input"),
    (dict(draft=dict(top_p_rows=AT[7] + 60)), abi.PLP_E_INVALID, "overlap an input"),
    (dict(kept_logp_out=AT[7] + 60), abi.PLP_E_INVALID, "overlap each other"), (dict(ws=AT[5]), abi.PLP_E_INVALID, "overlap each other"),
    (dict(ws=AT[0]), abi.PLP_E_INVALID, "overlap an input"), (dict(ws=None), abi.PLP_E_WORKSPACE, "NULL"),
    (dict(n=1000), abi.PLP_E_WORKSPACE, "too small"), (dict(ws=WS + 16), abi.PLP_E_WORKSPACE, "aligned"),
])
def test_refuses(kw, code, msg):
    assert verify(**kw) == code
    assert msg in _err()


def test_settings_that_are_not_read_are_not_checked():
    """The draft's where there are no draft logits; values beside arrays. (Refused
    by the workspace's size, the last check.)"""
    bad = dict(temperature=-1.0, top_k=-1, top_p=7.0, min_p=-1.0)
    assert verify(draft_logits=None, draft=bad, draft_seq_stride=-1, n=0) == abi.PLP_E_WORKSPACE
    rows = dict(temperature_rows=AT[9], top_k_rows=AT[10], top_p_rows=AT[11], min_p_rows=AT[12])
    assert verify(target={**bad, **rows}, n=0) == abi.PLP_E_WORKSPACE
    assert verify(K=0, draft_tokens=None, draft=bad, n=0) == abi.PLP_E_WORKSPACE


def test_of_nothing_and_workspace():
    assert verify(B=0, logits=None, ws=None, n=0) == abi.PLP_OK
    L, n = _lib(), ctypes.c_size_t()
    for B in (0, 1, 64, (1 << 31) - 1):
        for K in (0, 1, 8, 1024):
            for V in (1, 256, 257, 151936, 1 << 20):
                for drafts in (0, 1):
                    assert L.plp_verify_tokens_workspace_size(B, K, V, drafts, ctypes.byref(n)) == abi.PLP_OK
                    rows, blocks = B * (K + 1 + (K if drafts else 0)), (V + 255) // 256
                    # 12 bytes a block and 40 a row; a sequence's two chances a draft, verdict, mark and blocks' sums
                    least = rows * (blocks * 12 + 40) + B * (16 * K + 112 + 4 + blocks * 8)
                    # a row may begin within a block of 256: up to one more
                    assert n.value % 256 == 0 and least <= n.value <= least + rows * 12 + 7 * 256
    assert L.plp_verify_tokens_workspace_size(1, 1, 1, 0, None) == abi.PLP_E_INVALID
    assert L.plp_verify_tokens_workspace_size(1, 2000, 1, 0, ctypes.byref(n)) == abi.PLP_E_UNSUPPORTED


def test_binding_refuses_cpu_tensors():
    import rl_policy_gradient_amd as plp
    z, t, u = torch.zeros(2, 3, 5), torch.zeros(2, 2, dtype=torch.int64), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="GPU"):
        plp.verify_tokens(z, t, u)
    with pytest.raises(ValueError, match="B, K"):
        plp.verify_tokens(z[0], t, u)
