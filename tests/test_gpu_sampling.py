"""Token sampling on the GPU against a plain 80-bit implementation on the CPU.

Tokens have to be equal: kernel and reference form each weight to far better
than the spacing of two running sums that a test's uniforms could fall
between. Log-probs are one rounding to fp32 of a value good to 1e-12."""
import numpy as np
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


def reference_row(z, u, tau, k, p, mp):
    """(token, logp, kept_logp, kept indices) of one row."""
    z = np.asarray(z, np.float64).astype(np.longdouble)
    bad = (-1, np.nan, np.nan, [])
    if np.isnan(z).any() or not np.isfinite(z.max()) or not (tau >= 0 and np.isfinite(tau)):
        return bad
    if np.isnan(p) or np.isnan(mp) or np.isnan(u):
        return bad
    if tau == 0:
        t = int(np.argmax(z))
        return t, 0.0, 0.0, [t]
    x = (z - z.max()) / np.longdouble(tau)
    w = np.exp(x)
    order = np.argsort(-z, kind="stable")
    order = order[np.isfinite(z[order])]
    if 0 < k < len(z):
        order = order[:k]
    if p < 1:
        c = np.cumsum(w[order])
        before = c - w[order]
        n = int((before < np.longdouble(max(p, 0.0)) * c[-1]).sum())
        order = order[:max(1, n)]
    if mp > 0:
        order = order[:max(1, int((w[order] >= min(mp, 1.0)).sum()))]
    ids = np.sort(order)
    c = np.cumsum(w[ids])
    u = min(max(u, 0.0), 1 - 2.0 ** -24)
    t = int(ids[min(int((c <= np.longdouble(u) * c[-1]).sum()), len(ids) - 1)])
    return t, float(x[t] - np.log(w.sum())), float(x[t] - np.log(c[-1])), ids


def f32(v, n):
    if torch.is_tensor(v):
        return v.double().cpu().numpy()
    return np.full(n, np.float32(v), np.float64)


def check(z, u, tau=1.0, k=0, p=1.0, mp=0.0, **kw):
    """Runs the call on logits z (any device layout) and compares every row."""
    import rl_policy_gradient_amd as plp
    dev = lambda v: v.cuda() if torch.is_tensor(v) else v  # noqa: E731
    out = plp.sample_tokens(z.cuda() if not z.is_cuda else z, u.cuda(), temperature=dev(tau), top_k=dev(k),
                            top_p=dev(p), min_p=dev(mp), **kw)
    N = z.shape[0]
    zs, us = z.double().cpu().numpy(), u.double().cpu().numpy()
    taus, ps, mps = f32(tau, N), f32(p, N), f32(mp, N)
    ks = k.cpu().numpy() if torch.is_tensor(k) else np.full(N, k)
    tok, lp, kp = (out[n].cpu().numpy() for n in ("token", "logp", "kept_logp"))
    for n in range(N):
        t, a, b, _ = reference_row(zs[n], us[n], taus[n], int(ks[n]), ps[n], mps[n])
        assert tok[n] == t, (n, tok[n], t, taus[n], ks[n], ps[n], mps[n], us[n])
        for got, want in ((lp[n], a), (kp[n], b)):
            if np.isnan(want):
                assert np.isnan(got), (n, got)
            else:
                assert abs(got - want) <= U * abs(want) + 1e-12, (n, got, want)
    return out


def logits(N, V, dtype, seed, peaked=True):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g) * 2
    if peaked:
        n = min(V, 60)
        ids = torch.randint(0, V, (N, n), generator=g)
        top = 15 - 2.5 * torch.rand(N, 1, generator=g) * torch.log(torch.arange(1, n + 1).float())
        z.scatter_reduce_(1, ids, top, "amax")
    return z.to(DT[dtype]), torch.rand(N, generator=g)


LIMITS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.9, 40, 0.95, 0.02),
          (1.0, 1, 1.0, 0.0), (1.5, 3000, 0.99, 0.0), (2.0, 0, 0.5, 0.01), (0.0, 5, 0.5, 0.5)]


@pytest.mark.parametrize("peaked", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau,k,p,mp", LIMITS)
@pytest.mark.parametrize("N,V", [(3, 1), (5, 2), (4, 7), (9, 255), (9, 256), (3, 257), (40, 1000), (7, 8193), (5, 32000),
                                 (3, 151936)])
def test_against_reference(N, V, tau, k, p, mp, dtype, peaked):
    require_gpu()
    z, u = logits(N, V, dtype, 13 * V + N, peaked)
    check(z, u, tau, k, p, mp)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_settings_of_each_row(dtype):
    require_gpu()
    z, u = logits(64, 20001, dtype, 5)
    g = torch.Generator().manual_seed(3)
    pick = lambda v, t: torch.tensor(v, dtype=t)[torch.randint(0, len(v), (64,), generator=g)]  # noqa: E731
    check(z, u, pick([0.0, 0.5, 1.0, 1.0, 3.0], torch.float32), pick([0, -3, 1, 7, 100, 20001, 30000], torch.int32),
          pick([0.0, 0.3, 0.9, 1.0, 1.5, -1.0], torch.float32), pick([0.0, 0.1, 1.0, 2.0, -0.5], torch.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 256, 3000, 40000])
def test_equal_logits(V, dtype):
    """All equal: which are kept and taken is whole-number arithmetic."""
    require_gpu()
    N = 16
    z = torch.full((N, V), 3.25).to(DT[dtype])
    u = torch.arange(N) / N
    import rl_policy_gradient_amd as plp
    for k, p in ((0, 1.0), (3, 1.0), (V // 2, 1.0), (0, 0.5), (V // 2, 0.5), (0, 2.0 ** -20), (0, 0.0)):
        kept = V if k == 0 else min(k, V)
        kept = max(1, int(np.ceil(p * kept))) if p < 1 else kept
        out = check(z, u, 1.0, k, p, 0.0)
        want = torch.floor(u.double() * kept).long()
        assert torch.equal(out["token"].cpu(), want), (k, p)
        assert torch.allclose(out["kept_logp"].cpu(), torch.full((N,), -float(np.log(kept))), rtol=2 * U, atol=1e-12)
    out = plp.sample_tokens(z.cuda(), u.cuda(), min_p=1.0)  # every one weighs the most
    assert torch.equal(out["token"].cpu(), torch.floor(u.double() * V).long())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau,k,p,mp", LIMITS)
def test_few_values_many_ties(tau, k, p, mp, dtype):
    """Logits of a handful of values, so that every cut falls among ties."""
    require_gpu()
    g = torch.Generator().manual_seed(1)
    z = torch.randint(-3, 4, (6, 5001), generator=g).float() * 0.5
    z[2] *= -0.0  # signed zeros tie
    check(z.to(DT[dtype]), torch.rand(6, generator=g), tau, k, p, mp)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau,k,p,mp", LIMITS)
def test_masked_rows(tau, k, p, mp, dtype):
    """-inf in most places, in all, in all but one, the type's lowest value
    as a mask, NaN and +inf."""
    require_gpu()
    z, u = logits(12, 3001, dtype, 8)
    inf = float("inf")
    g = torch.Generator().manual_seed(2)
    z[0, torch.rand(3001, generator=g) < 0.99] = -inf
    z[1] = -inf
    z[2] = -inf
    z[2, 3000] = -7.0
    z[3, 17] = float("nan")
    z[4, 100] = inf
    low = torch.finfo(DT[dtype]).min
    z[5, 5:] = low
    z[6] = low  # every logit is the mask: an even row
    z[7, ::2] = -inf
    z[8, :1500] = -inf
    z[9, 0] = torch.finfo(DT[dtype]).max
    z[10] = -inf
    z[10, :4] = torch.tensor([1.0, 1.0, -inf, 1.0])
    check(z, u, tau, k, p, mp)


def test_settings_that_are_none():
    require_gpu()
    z, u = logits(8, 500, "f32", 4)
    nan = float("nan")
    row = lambda *v: torch.tensor(v, dtype=torch.float32)  # noqa: E731
    check(z, u, row(1, nan, -1, float("inf"), 1, 1, 1, 1e-30), 0, row(1, 1, 1, 1, nan, 0.9, 1, 1),
          row(0, 0, 0, 0, 0, nan, 0.1, 0))
    u[3] = nan
    check(z, u)


def test_uniforms_at_the_ends():
    require_gpu()
    z, _ = logits(6, 70000, "bf16", 2)
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, 2.0 ** -149])
    for lim in LIMITS:
        check(z, u, *lim)


@pytest.mark.parametrize("tau", [1e-3, 0.05, 20.0, 1e6])
def test_extreme_temperatures(tau):
    require_gpu()
    for dtype in ("f32", "bf16"):
        z, u = logits(6, 9000, dtype, 6)
        for k, p, mp in ((0, 1.0, 0.0), (100, 0.9, 0.0), (0, 0.95, 0.0), (0, 1.0, 0.3)):
            check(z, u, tau, k, p, mp)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_alignment(dtype):
    """Rows apart, rows that begin at odd elements, one row for all."""
    require_gpu()
    g = torch.Generator().manual_seed(9)
    store = (torch.randn(40 * 1013 + 50, generator=g) * 3).to(DT[dtype]).cuda()
    u = torch.rand(40, generator=g)
    for lead in (0, 1, 3, 7):
        for V, stride in ((1013, 1013), (1000, 1013), (999, 1001), (37, 1012)):
            z = store[lead:].as_strided((40, V), (stride, 1), lead)
            for lim in LIMITS[:5]:
                check(z, u, *lim)
    check(store[5:5 + 1013].view(1, 1013).expand(40, 1013), u, 1.0, 20, 0.9, 0.0)


def test_long_rows_and_far_offsets():
    """The longest vocabulary, and rows beyond 2^32 bytes and 2^31 elements."""
    require_gpu()
    z, u = logits(2, 1 << 20, "bf16", 3)
    for lim in LIMITS[:5]:
        check(z, u, *lim)
    stride = 600_000_011
    z, u = logits(5, 4001, "bf16", 7)
    far = torch.empty(4 * stride + 4001, dtype=torch.bfloat16, device="cuda").as_strided((5, 4001), (stride, 1))
    far.copy_(z)
    for lim in LIMITS[:5]:
        check(far, u, *lim)


def test_rows_do_not_depend_on_each_other():
    """A row alone, in a batch and at another place: the same bits."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    z, u = logits(300, 5000, "bf16", 12)
    z, u = z.cuda(), u.cuda()
    kw = dict(temperature=0.8, top_k=30, top_p=0.9)
    a = plp.sample_tokens(z, u, **kw)
    b = plp.sample_tokens(z.flip(0), u.flip(0), **kw)
    for k in a:
        assert torch.equal(a[k], b[k].flip(0)), k
    one = plp.sample_tokens(z[77:78], u[77:78], **kw)
    for k in a:
        assert torch.equal(a[k][77:78], one[k]), k


def test_log_probs_are_the_loss_stages():
    """logp is what selective_entropy and the losses take: the log-softmax of
    the logits over the temperature."""
    require_gpu()
    z, u = logits(33, 1500, "f32", 21)
    out = check(z, u, 0.8, 10, 0.9, 0.0)
    want = torch.log_softmax(z.double() / float(np.float32(0.8)), -1).gather(1, out["token"].cpu()[:, None])[:, 0]
    assert ((out["logp"].double().cpu() - want).abs() <= U * want.abs() + 1e-12).all()
    assert (out["kept_logp"] >= out["logp"]).all()


def test_empty_batch_outputs_and_refusals():
    require_gpu()
    import rl_policy_gradient_amd as plp
    z = torch.empty(0, 100, device="cuda")
    out = plp.sample_tokens(z, torch.empty(0, device="cuda"))
    assert out["token"].shape == (0,)
    z, u = (t.cuda() for t in logits(4, 100, "bf16", 1))
    o = {"token": torch.empty(4, dtype=torch.int64, device="cuda")}
    res = plp.sample_tokens(z, u, out=o)
    assert res["token"] is o["token"]
    bad = [
        (lambda: plp.sample_tokens(z.t(), u), "contiguous|uniforms"),
        (lambda: plp.sample_tokens(z[0], u), "logits"),
        (lambda: plp.sample_tokens(z, u[:3]), "uniforms"),
        (lambda: plp.sample_tokens(z, u.double()), "uniforms"),
        (lambda: plp.sample_tokens(z, u, top_k=torch.ones(4, device="cuda")), "top_k"),
        (lambda: plp.sample_tokens(z, u, temperature=torch.ones(3, device="cuda")), "temperature"),
        (lambda: plp.sample_tokens(z.half(), u), "dtype"),
        (lambda: plp.sample_tokens(z, u.cpu()), "GPU"),
        (lambda: plp.sample_tokens(z, u, out={"token": torch.empty(4, dtype=torch.int32, device="cuda")}), "token"),
        (lambda: plp.sample_tokens(z, u, workspace=torch.empty(1, device="cuda")), "workspace"),
    ]
    for call, msg in bad:
        with pytest.raises(ValueError, match=msg):
            call()
    for kw in (dict(temperature=-1.0), dict(temperature=float("nan")), dict(top_k=-1), dict(top_p=1.1),
               dict(top_p=-0.1), dict(min_p=2.0)):
        with pytest.raises(plp.PlpError):
            plp.sample_tokens(z, u, **kw)


def test_captured_and_replayed():
    """One capture, new logits and settings each replay, eager calls between."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    z, u = (t.cuda() for t in logits(20, 30000, "bf16", 1))
    tau, k = torch.ones(20, device="cuda"), torch.full((20,), 50, dtype=torch.int32, device="cuda")
    out = plp.sample_tokens(z, u, temperature=tau, top_k=k, top_p=0.9)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plp.sample_tokens(z, u, temperature=tau, top_k=k, top_p=0.9, out=out, workspace=ws)
    for i in range(3):
        z2, u2 = logits(20, 30000, "bf16", 50 + i)
        z.copy_(z2)
        u.copy_(u2)
        tau.fill_(0.5 + 0.5 * i)
        k.fill_(10 ** (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        want = plp.sample_tokens(z, u, temperature=tau, top_k=k, top_p=0.9)
        for n in want:
            assert torch.equal(out[n], want[n]), (i, n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_huge_magnitudes(dtype):
    """Logits up to the type's largest and lowest, whose differences overflow fp32."""
    require_gpu()
    g = torch.Generator().manual_seed(31)
    for V in (700, 9000, 40000):
        z = (torch.rand(6, V, generator=g, dtype=torch.float64) * 2 - 1) * 3.38e38
        z[1, ::2] = torch.finfo(DT[dtype]).max
        z[2] = torch.finfo(DT[dtype]).min
        z[3, : V // 2] = torch.finfo(DT[dtype]).min
        z[4, 5:] = -1e30
        z = z.to(DT[dtype])
        u = torch.rand(6, generator=g)
        for tau in (1.0, 1e37, 3e38):
            for k, p, mp in ((0, 1.0, 0.0), (50, 1.0, 0.0), (0, 0.9, 0.0), (3000, 0.5, 0.0), (0, 1.0, 0.3), (20, 0.9, 0.1)):
                check(z, u, tau, k, p, mp)


def test_many_rows_and_a_top_k_past_32_bits():
    """More rows than one launch takes (32768), settings of each row, and a k
    that a 32-bit argument does not hold (no limit)."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    z, u = logits(70001, 37, "f32", 4)
    g = torch.Generator().manual_seed(4)
    k = torch.randint(0, 40, (70001,), generator=g, dtype=torch.int32)
    check(z, u, 0.9, k, 0.9, 0.0)
    a, b = plp.sample_tokens(z.cuda(), u.cuda(), top_k=2 ** 32 + 5), plp.sample_tokens(z.cuda(), u.cuda())
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_calls_side_by_side():
    """Two streams at once, each with its own workspace and outputs."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    zs = [tuple(t.cuda() for t in logits(64, 30000, "bf16", s)) for s in (1, 2)]
    kws = [dict(top_p=0.9), dict(top_k=50, temperature=0.7)]
    want = [plp.sample_tokens(*z, **kw) for z, kw in zip(zs, kws)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in zs]
    got = [[] for _ in zs]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(plp.sample_tokens(*zs[i], **kws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            for n in o:
                assert torch.equal(o[n], want[i][n]), (i, n)


def test_workspace_has_to_be_contiguous():
    require_gpu()
    import rl_policy_gradient_amd as plp
    z, u = (t.cuda() for t in logits(4, 100, "bf16", 1))
    with pytest.raises(ValueError, match="contiguous"):
        plp.sample_tokens(z, u, workspace=torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 20))


@pytest.mark.parametrize("V,k,tau,peaked", [(1697, 300, 1.0, False), (1797, 300, 2.5, True), (28755, 1000, 2.5, False)])
def test_what_is_listed_ends_between_two_values(V, k, tau, peaked):
    """Rows among which some list exactly k candidates above a bound that lies
    between two neighbouring bf16 values: the lower one is not kept."""
    require_gpu()
    z, u = logits(340 if V > 10000 else 1000, V, "bf16", 7, peaked)
    check(z, u, tau, k, 1.0, 0.0)
