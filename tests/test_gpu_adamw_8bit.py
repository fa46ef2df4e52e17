"""The 8-bit moments the AdamW step stores, where a beta is above 0.95 and at
it: code for code against the rule in plain operations (tests/adamw_8bit.py),
and over many steps beside fp32 moments."""
import pytest
import torch

from tests import adamw_8bit as rule
from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def float32_default():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


def held(st, n):
    """The stored moments as (codes, scales) in fp32 [blocks, 256], padded with zeros."""
    out = []
    for k in ("exp_avg", "exp_rms"):
        c = torch.zeros(-(-n // 256) * 256)
        c[:n] = st[k].float().cpu().view(-1)
        out.append((c.view(-1, 256), st[k + "_scale"].cpu()[:, None]))
    return out


def new_state(plp, p, seed, **kw):
    """A mid-training state: moments of sizes a factor e apart, by the rule."""
    st = plp.adamw_state(p, bits=8, **kw)
    n = p.numel()
    g = torch.Generator().manual_seed(seed)
    r = torch.zeros(-(-n // 256) * 256)
    r[:n] = torch.exp(torch.randn(n, generator=g)) * 1e-3
    m = r * torch.randn(r.shape, generator=g)
    for k, x, first in (("exp_avg", m, True), ("exp_rms", r, False)):
        c, s = rule.store(x.view(-1, 256), 0, 0.0, first)
        st[k].copy_(c.view(-1)[:n].view(p.shape).to(torch.float8_e4m3fn))
        st[k + "_scale"].copy_(s[:, 0])
    return st


@pytest.mark.parametrize("b1,b2", [(0.9, 0.999), (0.95, 0.95), (0.99, 0.9999), (0.96, 0.5), (0.0, 0.999)])
@pytest.mark.parametrize("kind", ["f32", "bf16 master"])
@pytest.mark.parametrize("on_device", [False, True])
def test_codes_are_the_rules(b1, b2, kind, on_device):
    """Eight steps, each from what is stored: every operation is rounded once
    on either side, so codes and scales are equal."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    n = 256 * 37 + 129
    g = torch.Generator().manual_seed(5)
    p = torch.randn(n, generator=g).to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()
    st = new_state(plp, p, 6, master=kind != "f32")
    grad = torch.zeros(n, device="cuda")
    table = plp.adamw_table([p], [grad], [st], weight_decay=0.1)
    for t in (1, 2, 3, 1000, 1001, 2 ** 31 + 7, 2 ** 32 + 8, 10 ** 12):
        gr = torch.zeros(-(-n // 256) * 256)
        gr[:n] = torch.randn(n, generator=g) * 1e-3
        grad.copy_(gr[:n])
        (mc, ms), (rc, rs) = held(st, n)
        m, r = rule.moments(mc * ms, rc * rs, gr.view(-1, 256), b1, b2)
        plp.adamw_step(table, lr=1e-4, step=torch.tensor([t], device="cuda") if on_device else t, betas=(b1, b2))
        for (c, s), x, beta, first in zip(held(st, n), (m, r), (b1, b2), (True, False)):
            want, ws = rule.store(x, t, beta, first)
            assert torch.equal(s, ws), t
            assert torch.equal(c.view(-1)[:n], want.view(-1)[:n]), (t, first, (c != want).sum().item())


@pytest.mark.parametrize("b2,steps", [(0.96, 149), (0.99, 599), (0.999, 5999)])
def test_stored_roots_follow(b2, steps):
    """Half the elements' gradients fall to 0.03: their stored roots, beside a
    tensor with fp32 states of the same gradients, are within 6 % in the mean
    and nine in ten within a factor of two (as the rule's are on the CPU)."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    n = 64 * 256
    g = torch.Generator(device="cuda").manual_seed(3)
    size = torch.exp(torch.randn(n, generator=g, device="cuda"))
    ps = [torch.zeros(n, device="cuda") for _ in range(2)]
    grad = torch.zeros(n, device="cuda")
    sts = [plp.adamw_state(ps[0], bits=8), plp.adamw_state(ps[1])]
    c, s = rule.store(size.cpu().view(-1, 256), 0, 0.0, False)
    sts[0]["exp_rms"].copy_(c.view(-1).to(torch.float8_e4m3fn))
    sts[0]["exp_rms_scale"].copy_(s[:, 0])
    sts[1]["exp_avg_sq"].copy_(size ** 2)
    table = plp.adamw_table(ps, [grad, grad], sts)
    half = torch.arange(n, device="cuda") % 2 == 0
    now = torch.where(half, size * 0.03, size)
    for t in range(1, steps + 1):
        grad.copy_(torch.randn(n, generator=g, device="cuda") * now)
        plp.adamw_step(table, lr=0.0, step=t, betas=(0.9, b2))
    (_, _), (c, s) = held(sts[0], n)
    x = ((c * s).view(-1) / sts[1]["exp_avg_sq"].sqrt().cpu())[half.cpu()]
    q = torch.quantile(x, torch.tensor([0.05, 0.95]))
    assert 0.94 <= x.mean() <= 1.06 and q[0] >= 0.5 and q[1] <= 2.0, (x.mean(), q)


def test_first_moments_follow():
    """The same of the first moment at beta1 0.99: after the gradients fall,
    the stored moments' size is the fp32 ones'."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    n = 64 * 256
    g = torch.Generator(device="cuda").manual_seed(4)
    size = torch.exp(torch.randn(n, generator=g, device="cuda"))
    ps = [torch.zeros(n, device="cuda") for _ in range(2)]
    grad = torch.zeros(n, device="cuda")
    sts = [plp.adamw_state(ps[0], bits=8), plp.adamw_state(ps[1])]
    table = plp.adamw_table(ps, [grad, grad], sts)
    mean = 0.3 * torch.randn(n, generator=g, device="cuda")
    half = torch.arange(n, device="cuda") % 2 == 0
    a = b = 0.0
    for t in range(1, 1201):
        now = torch.where(half, size * 0.03, size) if t > 30 else size
        grad.copy_((torch.randn(n, generator=g, device="cuda") + mean) * now)
        plp.adamw_step(table, lr=0.0, step=t, betas=(0.99, 0.95))
        if t > 600 and t % 20 == 0:
            (c, s), _ = held(sts[0], n)
            x, y = ((c * s).view(-1) / size.cpu())[half.cpu()], (sts[1]["exp_avg"].cpu() / size.cpu())[half.cpu()]
            a, b = a + (x * y).sum().item(), b + (y * y).sum().item()
    assert 0.9 <= a / b <= 1.1, a / b  # rounded to the nearest code it is 2.7
