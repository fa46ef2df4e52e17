"""The rule by which the AdamW step stores moments in 8 bits, over many steps
beside fp32 moments, on the CPU. (That the kernel stores by this rule, code for
code, is tested on the GPU.)"""
import pytest
import torch

from tests import adamw_8bit as rule


@pytest.fixture(autouse=True)
def float32_default():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


def test_either_code_is_a_neighbour_and_right_in_the_mean():
    """Every code stays itself; what lies between two takes the upper one in
    as many phases as its distance from the lower asks for."""
    codes = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).float()  # 0 .. 448
    for phase in (0, 1, 1 << 19, (1 << 20) - 1):
        for c in (codes, -codes):
            assert torch.equal(rule.either_code(c, torch.full(c.shape, phase, dtype=torch.int32)), c)
    g = torch.Generator().manual_seed(1)
    lo = codes[:-1].repeat_interleave(8)
    gap = (codes[1:] - codes[:-1]).repeat_interleave(8)
    y = lo + gap * torch.rand(lo.shape, generator=g)
    share = ((y.double() - lo.double()) / gap.double())
    n = 4096
    up = torch.zeros_like(share)
    for i in range(n):
        z = rule.either_code(y, torch.full(y.shape, (i << 20) // n, dtype=torch.int32))
        assert ((z == lo) | (z == lo + gap)).all()
        up += z > lo
    # n phases in even steps: within one of them, and y + 2^-6 is rounded by 2^-30 where codes are 2^-9 apart
    assert ((up / n - share).abs() <= 1.0 / n + 2.0 ** -20).all()


@pytest.mark.parametrize("i", [0, 1, 77, 255])
@pytest.mark.parametrize("start", [0, 12345])
def test_phases_are_even_over_the_steps(i, start):
    """The share of steps whose phase lies below any bound, over as few as 50
    steps: a golden rotation's discrepancy is below (2 + 1.5 ln n) / n."""
    for n in (50, 1000, 4000):
        p = torch.sort(torch.tensor([rule.phases(start + t, False)[i].item() for t in range(1, n + 1)])).values
        off = (p.double() / 2 ** 20 - torch.arange(n, dtype=torch.float64) / n).abs().max().item()
        assert off <= (3 + 1.5 * torch.log(torch.tensor(float(n))).item()) / n


def roots(b2, fall, steps, blocks=16, seed=0, nearest=False):
    """Stored roots over fp32 ones after `steps`, of the elements whose
    gradients (noise, sizes a factor e apart) fall to `fall` at the start."""
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn(blocks, 256, generator=g))
    v = size ** 2
    m = torch.zeros_like(v)
    codes, s = rule.store(size, 0, 0.0 if nearest else b2, False)
    half = torch.arange(256).expand(blocks, 256) % 2 == 0
    now = torch.where(half, size * fall, size)
    for t in range(1, steps + 1):
        grad = torch.randn(blocks, 256, generator=g) * now
        v = b2 * v + (1 - b2) * grad * grad
        _, x = rule.moments(m, codes * s, grad, 0.9, b2)
        codes, s = rule.store(x, t, 0.0 if nearest else b2, False)
    return ((codes * s) / v.sqrt())[half]


@pytest.mark.parametrize("b2,fall,steps,low,high", [
    (0.95, 1.0, 600, 0.85, 1.20), (0.95, 0.03, 3000, 0.85, 1.20),  # the nearest code
    (0.96, 1.0, 600, 0.80, 1.25), (0.96, 0.03, 149, 0.60, 1.50),
    (0.99, 1.0, 600, 0.75, 1.35), (0.99, 0.03, 599, 0.55, 1.65),
    (0.999, 1.0, 3000, 0.70, 1.40), (0.999, 0.03, 5999, 0.50, 1.75), (0.9999, 0.03, 6000, 0.60, 1.50)])
def test_stored_roots_follow(b2, fall, steps, low, high):
    """In the mean within 6 % of the fp32 roots, and nine in ten between low
    and high: codes are up to 1/8 apart, a step of the rule's is one code, and
    where gradients fall by 30 a root passes through some forty of them."""
    x = roots(b2, fall, steps)
    q = torch.quantile(x, torch.tensor([0.05, 0.95]))
    assert 0.94 <= x.mean() <= 1.06 and q[0] >= low and q[1] <= high, (x.mean(), q)


@pytest.mark.parametrize("b2,steps", [(0.98, 299), (0.99, 599)])
def test_nearest_codes_would_not_follow(b2, steps):
    """What the rule is for: rounded to the nearest code, falling roots stay
    several times too large."""
    assert roots(b2, 0.03, steps, nearest=True).median() > 5
