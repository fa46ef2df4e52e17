"""The AdamW list's own life without a GPU: which memory it holds and which
replaced tensors it sees. Only the checks that ask for a GPU are stood in for;
no step is launched."""
import contextlib

import pytest
import torch

pytest.importorskip("rl_policy_gradient_amd._abi")


@pytest.fixture(autouse=True)
def float32_default():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


class Launched(Exception):
    pass


@pytest.fixture
def plp(monkeypatch):
    import rl_policy_gradient_amd as plp
    from rl_policy_gradient_amd import _abi, operators

    class Lib:
        @staticmethod
        def plp_adamw_step(*args):
            raise Launched

    monkeypatch.setattr(operators, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(operators, "_one_device", lambda pairs: torch.device("cpu"))
    monkeypatch.setattr(operators, "_on", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(operators, "_stream_on", lambda dev: 0)
    monkeypatch.setattr(_abi, "lib", lambda: Lib)
    return plp


def make(plp, bits=8, master=True, n=4096, count=3):
    ps = [torch.randn(n).bfloat16() if master else torch.randn(n) for _ in range(count)]
    gs = [torch.randn_like(p) for p in ps]
    sts = [plp.adamw_state(p, bits=bits, master=master) for p in ps]
    return ps, gs, sts, plp.adamw_table(ps, gs, sts)


def step(plp, table, **kw):
    plp.adamw_step(table, lr=1e-3, step=1, **kw)


@pytest.mark.parametrize("bits,master,key", [(8, True, "exp_avg"), (8, True, "exp_rms"), (8, True, "exp_avg_scale"),
                                             (8, False, "exp_rms_scale"), (32, True, "master"), (32, False, "exp_avg_sq")])
def test_a_replaced_state_is_refused(plp, bits, master, key):
    _, _, sts, table = make(plp, bits, master)
    with pytest.raises(Launched):
        step(plp, table)
    old = sts[1][key]
    sts[1][key] = old.clone()  # as a checkpoint's tensors put in
    with pytest.raises(ValueError, match=key):
        step(plp, table)
    del sts[1][key]
    with pytest.raises(ValueError, match=key):
        step(plp, table)
    sts[1][key] = old
    with pytest.raises(Launched):
        step(plp, table)


def test_a_parameter_with_other_memory_is_refused(plp):
    ps, gs, sts, table = make(plp)
    ps[2].data = ps[2].clone()
    with pytest.raises(ValueError, match="parameter"):
        step(plp, table)
    with pytest.raises(Launched):
        step(plp, plp.adamw_table(ps, gs, sts))


def test_states_with_entries_of_their_own(plp):
    """What a program keeps beside the state may change; mixed 8 and 32 bits."""
    ps = [torch.randn(300), torch.randn(5), torch.randn(0)]
    gs = [torch.randn_like(p) for p in ps]
    sts = [plp.adamw_state(ps[0], bits=8), plp.adamw_state(ps[1]), plp.adamw_state(ps[2], bits=8)]
    sts[0]["seen"] = 0
    table = plp.adamw_table(ps, gs, sts)
    sts[0]["seen"] = 1
    with pytest.raises(Launched):
        step(plp, table)
    sts[1]["exp_avg"] = torch.zeros(5)
    with pytest.raises(ValueError, match="exp_avg"):
        step(plp, table)


def test_the_memory_of_every_pointer_is_held(plp):
    """Every tensor dropped or given other memory: nothing allocated later
    lies where the list's pointers point."""
    ps, gs, sts, table = make(plp, n=1 << 16)
    held = []
    for e in table._array:
        held += [(e.param, 2 << 16), (e.grad, 2 << 16), (e.master, 4 << 16), (e.exp_avg, 1 << 16),
                 (e.exp_avg_sq, 1 << 16), (e.exp_avg_scale, 1024), (e.exp_avg_sq_scale, 1024)]
    for p, g, st in zip(ps, gs, sts):
        p.data, g.data = torch.zeros(1).bfloat16(), torch.zeros(1).bfloat16()
        for t in st.values():
            t.data = torch.zeros(1, dtype=t.dtype)
        st.clear()
    del ps, gs, sts, p, g, st, t
    later = [torch.zeros(n, dtype=torch.uint8) for n in (2 << 16, 4 << 16, 1 << 16, 1024) for _ in range(20)]
    for t in later:
        a, b = t.data_ptr(), t.data_ptr() + t.numel()
        assert all(b <= at or a >= at + n for at, n in held)


def test_a_scale_that_is_no_tensor_is_refused(plp):
    _, _, _, table = make(plp)
    with pytest.raises(ValueError, match="grad_scale"):
        step(plp, table, grad_scale=0.5)
