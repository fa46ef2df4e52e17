"""The embedding and the gradients' norm without a GPU: sizes and refusals.
Every call here is answered by the host checks before any launch; the pointers
are made up and never followed."""
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


T, W, Y, WS = (0x100000000 * (i + 1) for i in range(4))  # far apart: nothing overlaps


def fwd(**kw):
    a = dict(t=T, w=W, N=8, H=64, V=100, dtype=abi.DTYPE_BF16, scale=1.0, y=Y)
    a.update(kw)
    return _lib().plp_embedding_fwd(a["t"], a["w"], a["N"], a["H"], a["V"], a["dtype"], a["scale"], a["y"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(N=-1), abi.PLP_E_INVALID, "N=-1"), (dict(N=1 << 31), abi.PLP_E_INVALID, "N="),
    (dict(H=0), abi.PLP_E_INVALID, "H must"), (dict(V=0), abi.PLP_E_INVALID, "V must"),
    (dict(H=65537), abi.PLP_E_UNSUPPORTED, "H=65537"), (dict(dtype=2), abi.PLP_E_INVALID, "dtype"),
    (dict(scale=math.inf), abi.PLP_E_INVALID, "scale"), (dict(scale=math.nan), abi.PLP_E_INVALID, "scale"),
    (dict(t=None), abi.PLP_E_INVALID, "required"), (dict(w=None), abi.PLP_E_INVALID, "required"),
    (dict(y=None), abi.PLP_E_INVALID, "required"), (dict(t=T + 4), abi.PLP_E_INVALID, "aligned"),
    (dict(w=W + 1), abi.PLP_E_INVALID, "aligned"), (dict(y=Y + 1), abi.PLP_E_INVALID, "aligned"),
    (dict(dtype=abi.DTYPE_F32, y=Y + 2), abi.PLP_E_INVALID, "aligned"),
    (dict(y=W + 100 * 64 * 2 - 2), abi.PLP_E_INVALID, "overlap"), (dict(y=T - 8 * 64 * 2 + 2), abi.PLP_E_INVALID, "overlap"),
])
def test_embedding_forward_refuses(kw, code, msg):
    assert fwd(**kw) == code
    assert msg in _err()


def need(N=8, H=64, V=100, dt=abi.DTYPE_BF16):
    n = ctypes.c_size_t()
    return _lib().plp_embedding_bwd_workspace_size(N, H, V, dt, ctypes.byref(n)), n.value


def bwd(**kw):
    a = dict(t=T, gy=Y, N=8, H=64, V=100, gdt=abi.DTYPE_BF16, wdt=abi.DTYPE_BF16, scale=1.0, acc=0, gw=W, ws=WS, n=1 << 24)
    a.update(kw)
    return _lib().plp_embedding_bwd(a["t"], a["gy"], a["N"], a["H"], a["V"], a["gdt"], a["wdt"], a["scale"], a["acc"],
                                    a["gw"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(N=-1), abi.PLP_E_INVALID, "N=-1"), (dict(H=0), abi.PLP_E_INVALID, "H must"),
    (dict(V=-5), abi.PLP_E_INVALID, "V must"), (dict(H=1 << 20), abi.PLP_E_UNSUPPORTED, "H="),
    (dict(gdt=7), abi.PLP_E_INVALID, "dtype"), (dict(wdt=-1), abi.PLP_E_INVALID, "dtype"),
    (dict(gdt=abi.DTYPE_F32), abi.PLP_E_UNSUPPORTED, "fp32"), (dict(scale=math.nan), abi.PLP_E_INVALID, "scale"),
    (dict(gw=None), abi.PLP_E_INVALID, "grad_weight"), (dict(t=None), abi.PLP_E_INVALID, "required"),
    (dict(gy=None), abi.PLP_E_INVALID, "required"), (dict(gw=W + 1), abi.PLP_E_INVALID, "aligned"),
    (dict(wdt=abi.DTYPE_F32, gw=W + 2), abi.PLP_E_INVALID, "aligned"), (dict(t=T + 1), abi.PLP_E_INVALID, "aligned"),
    (dict(gw=Y), abi.PLP_E_INVALID, "overlap"), (dict(gw=T + 56), abi.PLP_E_INVALID, "overlap"),
    (dict(ws=W), abi.PLP_E_INVALID, "overlap each other"), (dict(ws=Y), abi.PLP_E_INVALID, "overlap an input"),
    (dict(n=100), abi.PLP_E_WORKSPACE, "too small"), (dict(ws=None), abi.PLP_E_WORKSPACE, "NULL"),
    (dict(ws=WS + 64), abi.PLP_E_WORKSPACE, "aligned"),
])
def test_embedding_backward_refuses(kw, code, msg):
    assert bwd(**kw) == code
    assert msg in _err()


def test_embedding_of_nothing_and_workspace():
    assert fwd(N=0, t=None, y=None) == abi.PLP_OK
    assert bwd(N=0, t=None, gy=None, ws=None, n=0, acc=1) == abi.PLP_OK
    assert need(N=0) == (abi.PLP_OK, 0)
    for N in (1, 4096, 4097, 70000, 1 << 20, (1 << 31) - 1):
        for H in (1, 896, 65536):
            for V in (1, 1000, 151936, (1 << 31) - 1):
                for dt in (abi.DTYPE_BF16, abi.DTYPE_F32):
                    rc, n = need(N, H, V, dt)
                    assert rc == abi.PLP_OK and n % 256 == 0
                    # two pairs of 32-bit words a token, a table of 256 x 1024, partial sums of some 8192 waves'
                    # columns on either side (512 or 256 of them) and 12 bytes a range
                    assert 8 * N <= n <= 16 * N + (1 << 20) + 2 * 4 * (8192 + 256) * 512 + 12 * 8448 + 4096
    assert need(H=0)[0] == abi.PLP_E_INVALID and need(dt=3)[0] == abi.PLP_E_INVALID
    assert _lib().plp_embedding_bwd_workspace_size(1, 1, 1, 0, None) == abi.PLP_E_INVALID


def grads(n=3, **kw):
    t = (abi.PlpGradTensor * n)()
    for i in range(n):
        t[i] = abi.PlpGradTensor(0x10000000 * (i + 1), 1000, i % 2, 0)
    for k, v in kw.items():
        setattr(t[1], k, v)
    return t


def norm(t=None, count=3, **kw):
    a = dict(max_norm=1.0, eps=1e-6, given=None, norm=T, scale=T + 4, norms=None, ws=WS, n=1 << 20)
    a.update(kw)
    return _lib().plp_grad_norm(grads() if t is None else t, count, a["max_norm"], a["eps"], a["given"], a["norm"],
                                a["scale"], a["norms"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(count=-1), abi.PLP_E_INVALID, "count"), (dict(count=(1 << 20) + 1), abi.PLP_E_INVALID, "count"),
    (dict(max_norm=-1.0), abi.PLP_E_INVALID, "max_norm"), (dict(max_norm=math.nan), abi.PLP_E_INVALID, "max_norm"),
    (dict(eps=-1e-9), abi.PLP_E_INVALID, "eps"), (dict(eps=math.inf), abi.PLP_E_INVALID, "eps"),
    (dict(norm=None), abi.PLP_E_INVALID, "required"), (dict(scale=None), abi.PLP_E_INVALID, "required"),
    (dict(norm=T + 1), abi.PLP_E_INVALID, "aligned"), (dict(given=W + 2), abi.PLP_E_INVALID, "aligned"),
    (dict(norms=Y + 3), abi.PLP_E_INVALID, "aligned"), (dict(scale=T), abi.PLP_E_INVALID, "overlap each other"),
    (dict(given=T), abi.PLP_E_INVALID, "overlap an input"), (dict(norm=0x10000000), abi.PLP_E_INVALID, "tensor 0 overlaps"),
    (dict(scale=0x20000000 + 1996), abi.PLP_E_INVALID, "tensor 1 overlaps"),
    (dict(norms=0x30000000 - 8), abi.PLP_E_INVALID, "tensor 2 overlaps"),
    (dict(ws=0x10000000), abi.PLP_E_INVALID, "tensor 0 overlaps"), (dict(ws=None), abi.PLP_E_WORKSPACE, "NULL"),
    (dict(n=8), abi.PLP_E_WORKSPACE, "too small"), (dict(ws=WS + 8), abi.PLP_E_WORKSPACE, "aligned"),
    (dict(t=grads(numel=-1)), abi.PLP_E_INVALID, "tensor 1"), (dict(t=grads(numel=(1 << 40) + 1)), abi.PLP_E_INVALID, "numel"),
    (dict(t=grads(numel=1 << 40)), abi.PLP_E_INVALID, "in all"), (dict(t=grads(dtype=2)), abi.PLP_E_INVALID, "dtype"),
    (dict(t=grads(grad=None)), abi.PLP_E_INVALID, "required"), (dict(t=grads(grad=0x20000001)), abi.PLP_E_INVALID, "aligned"),
])
def test_grad_norm_refuses(kw, code, msg):
    assert norm(**kw) == code
    assert msg in _err()


@pytest.mark.parametrize("scale,t,msg", [
    (None, None, "required"), (T + 2, None, "aligned"), (0x10000000 + 4, None, "tensor 0 overlaps"),
    (T, grads(dtype=5), "dtype"), (T, grads(numel=-3), "numel"),
])
def test_clip_refuses(scale, t, msg):
    assert _lib().plp_clip_grads(grads() if t is None else t, 3, scale, None) == abi.PLP_E_INVALID
    assert msg in _err()


def test_nothing_to_clip_and_workspace():
    assert _lib().plp_clip_grads(None, 0, T, None) == abi.PLP_OK
    n = ctypes.c_size_t()
    t = (abi.PlpGradTensor * 300)()
    for numel in (0, 1, 2048, 2049, 1 << 20, 1 << 31):
        for i in range(300):
            t[i] = abi.PlpGradTensor(0x10000000, numel, 0, 0)
        assert _lib().plp_grad_norm_workspace_size(t, 300, ctypes.byref(n)) == abi.PLP_OK
        assert n.value % 256 == 0 and 300 * 12 <= n.value <= (8192 + 300) * 8 + 300 * 4 + 512
    assert _lib().plp_grad_norm_workspace_size(t, 300, None) == abi.PLP_E_INVALID


def test_binding_refuses():
    import rl_policy_gradient_amd as plp
    t, w = torch.zeros(4, dtype=torch.int64), torch.ones(8, 4)
    with pytest.raises(ValueError, match="GPU"):
        plp.embedding_fwd(t, w)
    with pytest.raises(ValueError, match="GPU"):
        plp.embedding_bwd(torch.ones(4, 4), t, 8)
    with pytest.raises(ValueError, match="GPU"):
        plp.grad_norm([w])
    with pytest.raises(ValueError, match="GPU"):
        plp.clip_grads([w], torch.ones(1))
    with pytest.raises(ValueError, match="empty list"):
        plp.grad_norm([])
