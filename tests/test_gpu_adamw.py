"""The AdamW step on the GPU against the formula in 64 bits.

Tolerances count roundings, u = 2^-24 of fp32 and eps_t / 2 of a bfloat16
parameter. m = b1 m + c1 g' with g' = scale g: the two constants, the scaled
gradient, two products and a sum, at most 5 u of |b1 m| + |c1 g'|; v has one
product more, 6 u. The update is m over a root (half of v's error, and u), a
product, a sum with eps, two constants, a quotient and a product: 16 u of its
size. An 8-bit state is the nearest e4m3 code of x / scale: off by at most
2^-4 |x|, or below exponent -6 by 2^-10 scale, and by the fp32 value's own
error; a root above zero is at least the code 2^-9."""
import math

import pytest
import torch

from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def float32_default():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HP = dict(betas=(0.9, 0.95), eps=1e-8)


def make(n, param="f32", grad="f32", bits=32, master=False, seed=0, lead=0):
    """One tensor's parameter, gradient and a mid-training state; lead: that
    many elements into larger storage, with guards on both sides."""
    import rl_policy_gradient_amd as plp
    g = torch.Generator().manual_seed(seed)

    def place(t):
        store = torch.zeros(lead + t.numel() + 3, dtype=t.dtype, device="cuda")
        store[lead:lead + t.numel()].copy_(t)
        return store[lead:lead + t.numel()]

    p32 = torch.randn(n, generator=g) * 0.05
    p = place(p32.to(DT[param]))
    gr = place((torch.randn(n, generator=g) * 10 ** (-4 * torch.rand(n, generator=g))).to(DT[grad]))
    st = plp.adamw_state(p, bits=bits, master=master)
    if master:
        st["master"] = place(p32)
    m = torch.randn(n, generator=g) * 1e-3 * 10 ** (-3 * torch.rand(n, generator=g))
    r = (m.abs() + 1e-4) * (0.5 + torch.rand(n, generator=g))
    if bits == 8:
        for k, x in (("exp_avg", m), ("exp_rms", r)):
            nb = -(-n // 256)
            pad = torch.zeros(nb * 256)
            pad[:n] = x
            s = pad.view(nb, 256).abs().amax(1) / 448
            st[k + "_scale"] = place(s)
            st[k] = place((pad.view(nb, 256) / s[:, None]).view(-1)[:n].to(torch.float8_e4m3fn).view(torch.uint8)).view(
                torch.float8_e4m3fn)
    else:
        st["exp_avg"], st["exp_avg_sq"] = place(m), place(r * r)
    return p, gr, st


def values(p, gr, st):
    """(p, g, m, v) in 64 bits on the CPU."""
    n = p.numel()
    base = st.get("master", p).double().cpu().reshape(-1)
    if "exp_rms" in st:
        sc = {k: st[k + "_scale"].double().cpu().repeat_interleave(256)[:n] for k in ("exp_avg", "exp_rms")}
        m = st["exp_avg"].float().cpu().double().reshape(-1) * sc["exp_avg"]
        v = (st["exp_rms"].float().cpu().double().reshape(-1) * sc["exp_rms"]) ** 2
    else:
        m, v = (st[k].double().cpu().reshape(-1) for k in ("exp_avg", "exp_avg_sq"))
    return base, gr.double().cpu().reshape(-1), m, v


def check_step(before, p, gr, st, lr, step, wd, scale=1.0, where=None):
    """One step from `before` (values()) against what the tensors hold now."""
    b1, b2 = HP["betas"]
    w, g, m, v = before
    g = g * scale
    m1, am = b1 * m + (1 - b1) * g, (b1 * m).abs() + ((1 - b1) * g).abs()
    v1 = b2 * v + (1 - b2) * g * g
    denom = v1.sqrt() / math.sqrt(1 - b2 ** step) + HP["eps"]
    k = lr / (1 - b1 ** step)
    new = w * (1 - lr * wd) - k * m1 / denom
    tol = 4 * U * w.abs() + 16 * U * k * am / denom
    sel = slice(None) if where is None else where

    def near(got, want, tol, what):
        off = ((got - want).abs() - tol)[sel]
        assert not torch.isnan(got[sel]).any(), what
        assert off.numel() == 0 or off.max().item() <= 0, (what, off.max().item())

    if "master" in st:
        near(st["master"].double().cpu().reshape(-1), new, tol, "master")
        assert torch.equal(p.cpu().reshape(-1)[sel], st["master"].to(p.dtype).cpu().reshape(-1)[sel])
    h = torch.finfo(p.dtype).eps / 2 if p.dtype == torch.bfloat16 else 0.0
    near(p.double().cpu().reshape(-1), new, tol + h * (new.abs() + tol), "param")
    if "exp_rms" not in st:
        near(st["exp_avg"].double().cpu().reshape(-1), m1, 5 * U * am, "exp_avg")
        near(st["exp_avg_sq"].double().cpu().reshape(-1), v1, 6 * U * v1, "exp_avg_sq")
        return
    n = p.numel()
    for name, x, ax in (("exp_avg", m1, am), ("exp_rms", v1.sqrt(), v1.sqrt())):
        pad = torch.zeros(-(-n // 256) * 256, dtype=torch.float64)
        pad[:n] = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs()
        want = pad.view(-1, 256).amax(1) / 448
        got = st[name + "_scale"].double().cpu()
        pad[:n] = torch.where(torch.isfinite(ax), ax, torch.zeros_like(ax))
        # the largest value's own error and a quotient
        assert ((got - want).abs() <= 6 * U * pad.view(-1, 256).amax(1) / 448 + U * want).all(), name
        s = got.repeat_interleave(256)[:n]
        y = st[name].float().cpu().double().reshape(-1) * s
        half = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s)
        if name == "exp_rms":
            half = torch.where(x.abs() < 2.0 ** -9 * s, 2.0 ** -9 * s, half)
            assert (y[sel][(x[sel] > 0) & (s[sel] > 0)] > 0).all()
        near(y, x, half * (1 + 8 * U) + 8 * U * ax, name)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False),
                                               ("bf16", "f32", True), ("bf16", "bf16", True)])
def test_one_step(param, grad, master, bits):
    """Every combination of types, lengths around a block, a tile and a wave,
    aligned and one element off, all in one call."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    sizes = [1, 2, 15, 16, 17, 255, 256, 257, 1023, 4095, 4096, 4097, 10007, 70001]
    sets = [make(n, param, grad, bits, master, seed=n + lead, lead=lead) for n in sizes for lead in (0, 1)]
    wds = [0.1 * (i % 3) for i in range(len(sets))]
    before = [values(*s) for s in sets]
    table = plp.adamw_table([s[0] for s in sets], [s[1] for s in sets], [s[2] for s in sets], weight_decay=wds)
    plp.adamw_step(table, lr=3e-3, step=7, **HP)
    for b, s, wd in zip(before, sets, wds):
        check_step(b, *s, 3e-3, 7, wd)
        for t in [s[0], *s[2].values()]:
            raw = torch.empty(0, dtype=torch.uint8, device="cuda").set_(t.untyped_storage())
            lo = t.storage_offset() * t.element_size()
            assert (raw[:lo] == 0).all() and (raw[lo + t.numel() * t.element_size():] == 0).all()


def test_mixed_list_with_empty_tensors():
    """States of 8 and 32 bits, every type and empty tensors in one list of
    more tensors than a launch takes, over several steps."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    kinds = [("f32", "f32", 32, False), ("bf16", "bf16", 8, True), ("bf16", "f32", 8, False), ("f32", "bf16", 8, False),
             ("bf16", "bf16", 32, True)]
    sets = [make([0, 5, 300, 5000][i % 4], *kinds[i % 5][:2], kinds[i % 5][2], kinds[i % 5][3], seed=i, lead=i % 3)
            for i in range(97)]
    table = plp.adamw_table(*zip(*sets), weight_decay=0.05)
    for step in (1, 2, 3):
        before = [values(*s) for s in sets]
        plp.adamw_step(table, lr=1e-2, step=step, **HP)
        for b, s in zip(before, sets):
            check_step(b, *s, 1e-2, step, 0.05)


@pytest.mark.parametrize("bits", [8, 32])
def test_first_steps_from_a_new_state(bits):
    """From zero states; elements whose gradient is zero do not move but for
    the decay, and a zero block keeps zero scales."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    n = 1000
    p = torch.randn(n, device="cuda")
    g = torch.randn(n, device="cuda")
    g[256:512] = 0
    st = plp.adamw_state(p, bits=bits)
    table = plp.adamw_table([p], [g], [st], weight_decay=0.0)
    p0 = p.clone()
    for step in range(1, 6):
        before = values(p, g, st)
        plp.adamw_step(table, lr=1e-3, step=step, **HP)
        check_step(before, p, g, st, 1e-3, step, 0.0)
        g.copy_(torch.randn(n, device="cuda"))
        g[256:512] = 0
    assert torch.equal(p[256:512], p0[256:512])
    if bits == 8:
        assert st["exp_avg_scale"][1] == 0 and st["exp_rms_scale"][1] == 0


def test_every_code_is_read():
    """Each of the 256 codes as a first and as a second moment."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    p = torch.randn(512, device="cuda")
    g = torch.randn(512, device="cuda") * 1e-3
    st = plp.adamw_state(p, bits=8)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    st["exp_avg"].view(torch.uint8)[:256] = codes
    st["exp_rms"].view(torch.uint8)[:256] = 0x30
    st["exp_avg"].view(torch.uint8)[256:] = 0x28
    st["exp_rms"].view(torch.uint8)[256:] = codes
    st["exp_avg_scale"].fill_(1e-5)
    st["exp_rms_scale"].fill_(2e-5)
    before = values(p, g, st)
    ok = torch.isfinite(before[2]) & torch.isfinite(before[3])
    assert ok.sum() == 512 - 4  # 0x7f and 0xff are NaN
    plp.adamw_step(plp.adamw_table([p], [g], [st]), lr=1e-3, step=10, **HP)
    check_step(before, p, g, st, 1e-3, 10, 0.0, where=ok)
    assert torch.isnan(p.cpu()[~ok]).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_not_finite_gradients_stay_in_their_elements(bits):
    require_gpu()
    import rl_policy_gradient_amd as plp
    p, g, st = make(2000, "f32", "f32", bits, seed=3)
    g[[5, 300, 1999]] = torch.tensor([float("inf"), float("nan"), -float("inf")], device="cuda")
    before = values(p, g, st)
    plp.adamw_step(plp.adamw_table([p], [g], [st]), lr=1e-3, step=4, **HP)
    ok = torch.ones(2000, dtype=torch.bool)
    ok[[5, 300, 1999]] = False
    check_step(before, p, g, st, 1e-3, 4, 0.0, where=ok)
    assert torch.isnan(p.cpu()[~ok]).all()
    if bits == 8:
        assert (st["exp_rms"].view(torch.uint8).cpu()[~ok] == 0x7f).all()
        assert torch.isfinite(st["exp_rms_scale"]).all() and torch.isfinite(st["exp_avg_scale"]).all()


def test_grad_scale_and_a_step_left_out():
    require_gpu()
    import rl_policy_gradient_amd as plp
    p, g, st = make(5000, "bf16", "bf16", 8, True, seed=8)
    table = plp.adamw_table([p], [g], [st], weight_decay=0.1)
    before = values(p, g, st)
    scale = torch.tensor([0.37], device="cuda")
    plp.adamw_step(table, lr=1e-3, step=3, grad_scale=scale, **HP)
    check_step(before, p, g, st, 1e-3, 3, 0.1, scale=scale.double().item())
    kept = [t.clone() for t in (p, *[x.view(torch.uint8) for x in st.values()])]
    for bad in (float("nan"), float("inf"), -float("inf")):
        plp.adamw_step(table, lr=1e-3, step=4, grad_scale=torch.tensor([bad], device="cuda"), **HP)
    for a, b in zip(kept, (p, *[x.view(torch.uint8) for x in st.values()])):
        assert torch.equal(a, b)


def test_tiny_and_huge_magnitudes():
    """Blocks whose values span the type: a largest value too small for a
    scale stores zeros, gradients whose square overflows leave a NaN root."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    p = torch.ones(768, device="cuda")
    g = torch.full((768,), 1e-38, device="cuda")
    g[256:512] = torch.logspace(-18, 0, 256, device="cuda")
    g[512:] = 1e20
    st = plp.adamw_state(p, bits=8)
    before = values(p, g, st)
    plp.adamw_step(plp.adamw_table([p], [g], [st]), lr=1e-3, step=1, **HP)
    assert st["exp_avg_scale"][0] == 0 and (st["exp_avg"].float()[:256] == 0).all()
    keep = torch.zeros(768, dtype=torch.bool)
    keep[256:512] = True
    part = lambda t: t[256:512]  # noqa: E731
    cut = {k: part(v) if v.numel() == 768 else v[1:2] for k, v in st.items()}
    check_step(tuple(part(b) for b in before), part(p), part(g), cut, 1e-3, 1, 0.0)
    assert torch.isfinite(p[:512]).all()
    assert (st["exp_rms"].view(torch.uint8)[512:] == 0x7f).all()


def test_replayed_with_new_steps_and_rates():
    """Captured once with the step, the rate and the scale in device memory."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    sets = [make(3000, "bf16", "bf16", 8, True, seed=1), make(700, "f32", "f32", 32, seed=2)]
    table = plp.adamw_table(*zip(*sets), weight_decay=0.1)
    step = torch.tensor([1], device="cuda")
    lr = torch.tensor([1e-3], device="cuda")
    scale = torch.ones(1, device="cuda")
    run = lambda: plp.adamw_step(table, lr=lr, step=step, grad_scale=scale, **HP)  # noqa: E731
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(1, 5):
        step.fill_(k)
        lr.fill_(1e-3 / k)
        for _, g, _ in sets:
            g.copy_(torch.randn(g.shape, device="cuda"))
        before = [values(*s) for s in sets]
        graph.replay()
        torch.cuda.synchronize()
        for b, s in zip(before, sets):
            # one rounding more: the rate is an fp32 number
            check_step(b, *s, lr.double().item(), k, 0.1)


def test_host_and_device_scalars_agree():
    require_gpu()
    import rl_policy_gradient_amd as plp
    a, b = (make(4000, "bf16", "bf16", 32, True, seed=5) for _ in range(2))
    lr = torch.tensor([2e-3], device="cuda")
    plp.adamw_step(plp.adamw_table([a[0]], [a[1]], [a[2]], weight_decay=0.0), lr=lr.item(), step=12, **HP)
    plp.adamw_step(plp.adamw_table([b[0]], [b[1]], [b[2]], weight_decay=0.0), lr=lr,
                   step=torch.tensor([12], device="cuda"), **HP)
    # the same doubles rounded once on either side; expm1 may differ in its last place
    assert (a[2]["master"].double() - b[2]["master"].double()).abs().max() <= 2 * U * a[2]["master"].abs().max()
    assert torch.equal(a[2]["exp_avg"], b[2]["exp_avg"])


def test_table_refuses():
    require_gpu()
    import rl_policy_gradient_amd as plp
    p, g, st = make(1000, seed=1)
    q, h, su = make(1000, "bf16", "bf16", 8, True, seed=2)
    bad = [
        (lambda: plp.adamw_table([p, p], [g, g], [st, st]), "overlaps"),
        (lambda: plp.adamw_table([p], [p], [st]), "overlaps"),
        (lambda: plp.adamw_table([p, p[500:]], [g, g[500:]], [st, plp.adamw_state(p[500:])]), "overlaps"),
        (lambda: plp.adamw_table([p], [g[:5]], [st]), "elements"),
        (lambda: plp.adamw_table([p], [g], [{"exp_avg": st["exp_avg"]}]), "exp_avg_sq"),
        (lambda: plp.adamw_table([q], [h], [{**su, "exp_rms_scale": su["exp_rms_scale"][:-1]}]), "exp_rms_scale"),
        (lambda: plp.adamw_table([p], [g], [st, st]), "states"),
        (lambda: plp.adamw_table([p], [g], [st], weight_decay=[0.1, 0.2]), "decays"),
        (lambda: plp.adamw_table([p.view(500, 2).t()], [g], [st]), "contiguous"),
        (lambda: plp.adamw_table([p.cpu()], [g], [st]), "GPU"),
        (lambda: plp.adamw_state(p, master=True), "master"),
        (lambda: plp.adamw_state(p, bits=16), "bits"),
        (lambda: plp.adamw_table([p.half()], [g], [st]), "dtype"),
    ]
    for call, msg in bad:
        with pytest.raises(ValueError, match=msg):
            call()
    plp.adamw_table([p, q], [g, g[:1000]], [st, su])  # a gradient read twice is fine
    table = plp.adamw_table([p], [g], [st])
    for kw in (dict(lr=-1.0, step=1), dict(lr=1e-3, step=0), dict(lr=1e-3, step=1, betas=(1.0, 0.9)),
               dict(lr=1e-3, step=1, eps=-1.0), dict(lr=float("nan"), step=1)):
        with pytest.raises(plp.PlpError):
            plp.adamw_step(table, **kw)
    plp.adamw_step(plp.adamw_table([], [], []), lr=1e-3, step=1)


def test_more_than_2_to_the_32_elements():
    """One tensor of 2^32 + 777 elements: its blocks repeat every 2^20, and so
    do the results."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    n, period = 2 ** 32 + 777, 2 ** 20
    g = torch.Generator().manual_seed(5)
    p1, g1 = (torch.randn(period, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    reps = -(-n // period)
    p, gr = p1.repeat(reps)[:n], g1.repeat(reps)[:n]
    st, st1 = plp.adamw_state(p, bits=8), plp.adamw_state(p1, bits=8)
    for a, b, s in ((p, gr, st), (p1, g1, st1)):
        table = plp.adamw_table([a], [b], [s], weight_decay=0.01)
        for step in (1, 2):
            plp.adamw_step(table, lr=1e-2, step=step)
    whole = (n // period) * period
    assert (p[:whole].view(-1, period) == p1).all()
    assert torch.equal(p[whole:whole + 768], p1[:768])  # whole blocks of the last 777
    for k in ("exp_avg", "exp_rms"):
        a, b = st[k].view(torch.uint8), st1[k].view(torch.uint8)
        assert (a[:whole].view(-1, period) == b).all(), k
        assert torch.equal(a[whole:whole + 768], b[:768]), k
        s, s1 = st[k + "_scale"], st1[k + "_scale"]
        assert (s[:whole // 256].view(-1, period // 256) == s1).all() and torch.equal(s[whole // 256:][:3], s1[:3]), k
