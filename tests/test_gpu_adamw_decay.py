"""The AdamW step's weight decay at the rates of fine-tuning, where a step's
decay is smaller than a rounding of the parameter: the new value has to be the
exact one rounded once.

What is formed before that rounding is off by at most e: the update's own 16
roundings of 2^-24 (as derived in test_gpu_adamw.py) and five of the decay
(weight_decay, lr, their product, the product with p, the sum). Rounding does
not fall as its argument rises, so the result lies between the exact value
less e and the exact value plus e, each rounded to fp32: one number, but for
the few elements next to a tie. (The errors of the one rounding cannot be
taken to average out: from a new state every update is lr c sign(g), so the
elements of a binade are all rounded alike.)"""
import math

import pytest
import torch

from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def float32_default():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


@pytest.mark.parametrize("lr,wd", [(1e-6, 0.1), (1e-6, 0.01), (3e-6, 0.01), (1e-5, 0.1), (1e-3, 0.1)])
@pytest.mark.parametrize("on_device", [False, True])
@pytest.mark.parametrize("bits,master", [(32, False), (32, True), (8, True)])
def test_mean_decay(bits, master, on_device, lr, wd):
    require_gpu()
    import rl_policy_gradient_amd as plp
    n, b1, b2, eps, t = 1 << 20, 0.9, 0.95, 1e-8, 9
    g = torch.Generator().manual_seed(17)
    p32 = torch.randn(n, generator=g) * 0.05
    p = (p32.bfloat16() if master else p32).cuda()
    grad = (torch.randn(n, generator=g) * 1e-3).cuda()
    st = plp.adamw_state(p, bits=bits, master=master)
    w = st["master"] if master else p
    w.copy_(p32)
    old, gd = w.double().cpu(), grad.double().cpu()
    table = plp.adamw_table([p], [grad], [st], weight_decay=wd)
    rate = torch.tensor([lr], device="cuda")
    plp.adamw_step(table, lr=rate if on_device else lr, step=t, betas=(b1, b2), eps=eps)
    rate = rate.double().item() if on_device else lr
    # from zero states: m = (1 - b1) g, v = (1 - b2) g^2
    update = (1 - b1) / (1 - b1 ** t) * gd / (math.sqrt((1 - b2) / (1 - b2 ** t)) * gd.abs() + eps)
    exact = old - rate * (update + wd * old)
    e = U * rate * (16 * update.abs() + 5 * wd * old.abs()) + 2.0 ** -50 * old.abs()
    lo, hi = (exact - e).float(), (exact + e).float()
    new = w.cpu()
    assert ((lo <= new) & (new <= hi)).all(), ((new < lo) | (new > hi)).sum().item()
    # a factor of 1 - lr wd in fp32 does not pass at rates like these
    keep = torch.tensor(1 - rate * wd, dtype=torch.float64).float().double()
    other = (old * keep - rate * update).float()
    assert lr > 1e-5 or ((other < lo) | (other > hi)).sum() > 1000


@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_infinite_parameters_stay(wd):
    """-inf as a mask among the parameters, without a gradient."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    p = torch.randn(600, device="cuda")
    p[::7] = -math.inf
    p[3] = math.inf
    g = torch.randn(600, device="cuda")
    g[::7] = 0.0
    g[3] = 0.0
    before = p.clone()
    plp.adamw_step(plp.adamw_table([p], [g], [plp.adamw_state(p)], weight_decay=wd), lr=1e-3, step=1)
    assert torch.equal(torch.isinf(p), torch.isinf(before)) and torch.equal(p[torch.isinf(p)], before[torch.isinf(before)])
    assert not torch.isnan(p).any()
