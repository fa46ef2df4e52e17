"""The operators around the fused loss without a GPU: sizes and refusals. Every
call here is answered by the host checks before any launch; the pointers are
made up and never followed."""
import ctypes
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


X, W, B, Y, M, R, G, WS = (0x10000000 * (i + 1) for i in range(8))  # far apart: nothing overlaps


def norm_fwd(**kw):
    a = dict(x=X, w=W, b=B, N=8, H=64, dtype=abi.DTYPE_BF16, rms=0, eps=1e-5, y=Y, mean=M, rstd=R)
    a.update(kw)
    return _lib().plp_layer_norm_fwd(a["x"], a["w"], a["b"], a["N"], a["H"], a["dtype"], a["rms"], a["eps"], a["y"],
                                     a["mean"], a["rstd"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(N=-1), abi.PLP_E_INVALID, "N=-1"),
    (dict(N=1 << 31), abi.PLP_E_INVALID, "N="),
    (dict(H=0), abi.PLP_E_INVALID, "H must"),
    (dict(H=65537), abi.PLP_E_UNSUPPORTED, "H=65537"),
    (dict(dtype=2), abi.PLP_E_INVALID, "dtype"),
    (dict(eps=-1.0), abi.PLP_E_INVALID, "eps"),
    (dict(eps=float("nan")), abi.PLP_E_INVALID, "eps"),
    (dict(w=None), abi.PLP_E_INVALID, "weight"),
    (dict(x=None), abi.PLP_E_INVALID, "x and y"),
    (dict(y=None), abi.PLP_E_INVALID, "x and y"),
    (dict(rms=1), abi.PLP_E_INVALID, "mean_out"),
    (dict(x=X + 1), abi.PLP_E_INVALID, "aligned"),
    (dict(y=X), abi.PLP_E_INVALID, "overlap"),
    (dict(y=X + 8 * 64 * 2 - 2), abi.PLP_E_INVALID, "overlap"),
    (dict(y=W - 2), abi.PLP_E_INVALID, "overlap"),
    (dict(mean=Y), abi.PLP_E_INVALID, "overlap each other"),
    (dict(rstd=X + 8), abi.PLP_E_INVALID, "overlap an input"),
    (dict(rstd=M + 28), abi.PLP_E_INVALID, "overlap each other"),
    (dict(mean=M + 2), abi.PLP_E_INVALID, "aligned"),
])
def test_norm_forward_refuses(kw, code, msg):
    assert norm_fwd(**kw) == code
    assert msg in _err()


def norm_bwd(**kw):
    a = dict(gy=Y, x=X, w=W, mean=M, rstd=R, N=8, H=64, dtype=abi.DTYPE_F32, rms=0, gx=G, gw=B, gb=B + 4096, ws=WS,
             n=1 << 20)
    a.update(kw)
    return _lib().plp_layer_norm_bwd(a["gy"], a["x"], a["w"], a["mean"], a["rstd"], a["N"], a["H"], a["dtype"],
                                     a["rms"], a["gx"], a["gw"], a["gb"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(N=-1), abi.PLP_E_INVALID, "N=-1"),
    (dict(H=-3), abi.PLP_E_INVALID, "H must"),
    (dict(gy=None), abi.PLP_E_INVALID, "required"),
    (dict(rstd=None), abi.PLP_E_INVALID, "required"),
    (dict(mean=None), abi.PLP_E_INVALID, "required"),
    (dict(w=None), abi.PLP_E_INVALID, "weight"),
    (dict(gx=X + 2), abi.PLP_E_INVALID, "aligned"),
    (dict(gx=Y), abi.PLP_E_INVALID, "overlap an input"),
    (dict(gw=W), abi.PLP_E_INVALID, "overlap an input"),
    (dict(gb=B), abi.PLP_E_INVALID, "overlap each other"),
    (dict(gx=M), abi.PLP_E_INVALID, "overlap an input"),
    (dict(gw=R + 16), abi.PLP_E_INVALID, "overlap an input"),
    (dict(rstd=R + 1), abi.PLP_E_INVALID, "aligned"),
    (dict(n=16), abi.PLP_E_WORKSPACE, "too small"),
    (dict(ws=None), abi.PLP_E_WORKSPACE, "NULL"),
    (dict(ws=WS + 128), abi.PLP_E_WORKSPACE, "aligned"),
])
def test_norm_backward_refuses(kw, code, msg):
    assert norm_bwd(**kw) == code
    assert msg in _err()


def test_norm_of_nothing_and_workspace():
    assert norm_fwd(N=0, x=None, y=None) == abi.PLP_OK
    L, n, m = _lib(), ctypes.c_size_t(), ctypes.c_size_t()
    for N, H in ((0, 5), (1, 1), (65536, 896), ((1 << 31) - 1, 65536)):
        assert L.plp_layer_norm_bwd_workspace_size(N, H, abi.DTYPE_BF16, ctypes.byref(n)) == 0
        assert n.value >= 2 * H * 4 and n.value % 256 == 0
        assert L.plp_layer_norm_bwd_workspace_size(N, H, abi.DTYPE_F32, ctypes.byref(m)) == 0 and m.value == n.value
    assert n.value <= 2 * 1024 * 65536 * 4 + 256  # bounded whatever N is
    assert L.plp_layer_norm_bwd_workspace_size(8, 8, 9, ctypes.byref(n)) == abi.PLP_E_INVALID
    assert L.plp_layer_norm_bwd_workspace_size(8, 8, 0, None) == abi.PLP_E_INVALID


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import rl_policy_gradient_amd as plp
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(ValueError, match="GPU"):
        plp.layer_norm_fwd(x, w)
    with pytest.raises(ValueError, match="GPU"):
        plp.layer_norm_bwd(x, x, w, torch.ones(4), torch.ones(4))


def adamw(count=1, tensor=None, **kw):
    t = (abi.PlpAdamwTensor * 1)()
    for i, k in enumerate(("param", "grad", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")):
        setattr(t[0], k, 0x10000000 * (i + 1))
    t[0].numel, t[0].state_bits, t[0].weight_decay = 1000, 8, 0.1
    t[0].param_dtype = t[0].grad_dtype = abi.DTYPE_BF16
    for k, v in (tensor or {}).items():
        setattr(t[0], k, v)
    a = abi.PlpAdamwArgs()
    a.struct_size, a.tensor_size = ctypes.sizeof(a), ctypes.sizeof(abi.PlpAdamwTensor)
    a.lr, a.beta1, a.beta2, a.eps, a.step = 1e-3, 0.9, 0.999, 1e-8, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return _lib().plp_adamw_step(ctypes.byref(a), t, count, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(struct_size=8), "struct_size"), (dict(tensor_size=72), "tensor_size"), (dict(count=-1), "count"),
    (dict(lr=-1.0), "lr"), (dict(lr=float("inf")), "lr"), (dict(beta1=1.0), "beta1"), (dict(beta2=-0.1), "beta1"),
    (dict(beta2=float("nan")), "beta1"), (dict(eps=-1e-8), "eps"), (dict(step=0), "step"),
    (dict(step_dev=0x1004), "aligned"), (dict(lr_dev=0x1002), "aligned"), (dict(grad_scale=0x1001), "aligned"),
    (dict(tensor=dict(numel=-1)), "numel"), (dict(tensor=dict(numel=(1 << 35) + 1)), "numel"),
    (dict(tensor=dict(param_dtype=2)), "dtype"), (dict(tensor=dict(grad_dtype=-1)), "dtype"),
    (dict(tensor=dict(state_bits=4)), "state_bits"), (dict(tensor=dict(weight_decay=-0.1)), "weight_decay"),
    (dict(tensor=dict(weight_decay=float("nan"))), "weight_decay"),
    (dict(tensor=dict(param_dtype=abi.DTYPE_F32)), "master"),
    (dict(tensor=dict(param=None)), "required"), (dict(tensor=dict(grad=None)), "required"),
    (dict(tensor=dict(exp_avg=None)), "required"), (dict(tensor=dict(exp_avg_sq=None)), "required"),
    (dict(tensor=dict(exp_avg_scale=None)), "scales"), (dict(tensor=dict(exp_avg_sq_scale=None)), "scales"),
    (dict(tensor=dict(state_bits=32)), "scales"), (dict(tensor=dict(param=0x10000001)), "aligned"),
    (dict(tensor=dict(master=0x30000002)), "aligned"), (dict(tensor=dict(grad=0x10000000)), "overlap"),
    (dict(tensor=dict(exp_avg_sq=0x40000000 + 999)), "overlap"), (dict(tensor=dict(exp_avg_scale=0x70000008)), "overlap"),
])
def test_adamw_refuses(kw, msg):
    assert adamw(**kw) == abi.PLP_E_INVALID
    assert msg in _err()


def test_adamw_of_nothing():
    assert adamw(count=0) == abi.PLP_OK
    assert adamw(tensor=dict(numel=0, param=None, grad=None)) == abi.PLP_OK


def test_operator_structs_match_header(tmp_path):
    """sizeof and every offsetof of the operators' structs against the ctypes mirror."""
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    structs = {"plp_adamw_tensor": abi.PlpAdamwTensor, "plp_adamw_args": abi.PlpAdamwArgs,
               "plp_sample_args": abi.PlpSampleArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "plp.h"', "int main(void){"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} . %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    c = tmp_path / "probe.c"
    c.write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "probe"
    r = subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(root, "include"), "-I", "/opt/rocm/include",
                        str(c), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    for ln in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines():
        name, field, n = ln.split()
        cls = structs[name]
        assert int(n) == (ctypes.sizeof(cls) if field == "." else getattr(cls, field).offset), ln


def sample(ws=WS, ws_bytes=1 << 24, **kw):
    a = abi.PlpSampleArgs()
    a.struct_size, a.dtype = ctypes.sizeof(a), abi.DTYPE_BF16
    a.N, a.V, a.row_stride = 4, 1000, 1000
    a.logits, a.uniforms, a.token_out = X, W, Y
    a.temperature, a.top_p = 1.0, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return _lib().plp_sample_tokens(ctypes.byref(a), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(struct_size=8), abi.PLP_E_INVALID, "struct_size"),
    (dict(dtype=2), abi.PLP_E_INVALID, "dtype"),
    (dict(N=-1), abi.PLP_E_INVALID, "N="),
    (dict(N=1 << 31), abi.PLP_E_INVALID, "N="),
    (dict(V=0), abi.PLP_E_INVALID, "V must"),
    (dict(V=(1 << 20) + 1), abi.PLP_E_UNSUPPORTED, "V="),
    (dict(row_stride=-1), abi.PLP_E_INVALID, "row_stride"),
    (dict(temperature=-0.5), abi.PLP_E_INVALID, "temperature"),
    (dict(temperature=float("nan")), abi.PLP_E_INVALID, "temperature"),
    (dict(temperature=float("inf")), abi.PLP_E_INVALID, "temperature"),
    (dict(top_k=-1), abi.PLP_E_INVALID, "top_k"),
    (dict(top_p=1.5), abi.PLP_E_INVALID, "top_p"),
    (dict(top_p=float("nan")), abi.PLP_E_INVALID, "top_p"),
    (dict(min_p=-0.1), abi.PLP_E_INVALID, "min_p"),
    (dict(logits=None), abi.PLP_E_INVALID, "required"),
    (dict(uniforms=None), abi.PLP_E_INVALID, "required"),
    (dict(token_out=None), abi.PLP_E_INVALID, "required"),
    (dict(logits=X + 1), abi.PLP_E_INVALID, "aligned"),
    (dict(token_out=Y + 4), abi.PLP_E_INVALID, "aligned"),
    (dict(logp_out=M + 2), abi.PLP_E_INVALID, "aligned"),
    (dict(token_out=X), abi.PLP_E_INVALID, "overlap an input"),
    (dict(logp_out=X + 7996), abi.PLP_E_INVALID, "overlap an input"),
    (dict(row_stride=0, logp_out=X + 1996), abi.PLP_E_INVALID, "overlap an input"),
    (dict(logp_out=W), abi.PLP_E_INVALID, "overlap an input"),
    (dict(kept_logp_out=G, temperature_rows=G + 12), abi.PLP_E_INVALID, "overlap an input"),
    (dict(logp_out=M, kept_logp_out=M + 8), abi.PLP_E_INVALID, "overlap each other"),
    (dict(row_stride=1 << 62), abi.PLP_E_INVALID, "address space"),
    (dict(row_stride=(1 << 63) - 1), abi.PLP_E_INVALID, "address space"),
    (dict(ws_bytes=64), abi.PLP_E_WORKSPACE, "too small"),
    (dict(ws=None), abi.PLP_E_WORKSPACE, "NULL"),
    (dict(ws=WS + 8), abi.PLP_E_WORKSPACE, "aligned"),
])
def test_sampling_refuses(kw, code, msg):
    assert sample(**kw) == code
    assert msg in _err()


def test_sampling_of_nothing_and_workspace():
    assert sample(N=0, logits=None, uniforms=None, token_out=None, ws=None, ws_bytes=0) == abi.PLP_OK
    L, n = _lib(), ctypes.c_size_t()
    for N, V in ((1, 1), (512, 151936), ((1 << 31) - 1, 1 << 20)):
        assert L.plp_sample_tokens_workspace_size(N, V, ctypes.byref(n)) == 0
        # a maximum and a sum for each 256 logits, never a copy of them
        assert N * ((V + 255) // 256) * 12 <= n.value <= N * ((V + 262) // 256) * 12 + 512
    assert L.plp_sample_tokens_workspace_size(1, 1, None) == abi.PLP_E_INVALID


def test_row_lengths_past_32_bits_are_refused():
    """The C ABI's row lengths have 32 bits: a longer one must not wrap."""
    from rl_policy_gradient_amd import operators
    with pytest.raises(ValueError, match="H=4294967304"):
        x = torch.empty(1, dtype=torch.bfloat16).expand(1, 2 ** 32 + 8)
        operators._norm_sizes(x, x[0], None)
    with pytest.raises(ValueError, match="V="):
        operators._fits(2 ** 31, "V")
    operators._fits(2 ** 31 - 1, "V")
