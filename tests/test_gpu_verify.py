"""Verification of drafted tokens on the GPU against a plain implementation on
the CPU in 80 bits.

Tokens and counts have to be equal: kernel and reference form each probability
to far better than the spacing of what a test's uniforms could fall between.
Log-probs are one rounding to fp32 of a value good to 1e-12."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def float32_default():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


def distribution(z, tau, k, p, mp):
    """(probabilities, log-prob and kept log-prob of each token) or None."""
    z = np.asarray(z, np.float64).astype(np.longdouble)
    if np.isnan(z).any() or not np.isfinite(z.max()) or not (tau >= 0 and np.isfinite(tau)):
        return None
    if np.isnan(p) or np.isnan(mp):
        return None
    if tau == 0:
        one = np.zeros(len(z), np.longdouble)
        one[int(np.argmax(z))] = 1
        return one, np.zeros(len(z)), np.zeros(len(z))
    x = (z - z.max()) / np.longdouble(tau)
    w = np.exp(x)
    order = np.argsort(-z, kind="stable")
    order = order[np.isfinite(z[order])]
    if 0 < k < len(z):
        order = order[:k]
    if p < 1:
        c = np.cumsum(w[order])
        order = order[:max(1, int((c - w[order] < np.longdouble(max(p, 0.0)) * c[-1]).sum()))]
    if mp > 0:
        order = order[:max(1, int((w[order] >= min(mp, 1.0)).sum()))]
    kept = np.zeros(len(z), np.longdouble)
    kept[order] = w[order]
    return kept / kept.sum(), x - np.log(w.sum()), x - np.log(kept.sum())


def reference(target, draft, tokens, u, n, settings, draft_settings):
    """One sequence: (tokens, accepted, logp, kept_logp), -1 and 0 after the last."""
    K = len(tokens)
    out, lps, kps = np.full(K + 1, -1, np.int64), np.zeros(K + 1), np.zeros(K + 1)
    clamp = lambda v: min(max(float(v), 0.0), 1 - 2.0 ** -24)  # noqa: E731
    for k in range(n + 1):
        d = distribution(target[k], *settings)
        bad = d is None or (k == n and np.isnan(u[K]))
        q, t, V = None, -1, len(target[k])
        if k < n:
            bad = bad or np.isnan(u[k])
            t = int(tokens[k])
            if draft is not None:
                q = distribution(draft[k], *draft_settings)
                bad = bad or q is None
                q = None if q is None else q[0]
            else:
                q = np.zeros(V, np.longdouble)
                if 0 <= t < V:
                    q[t] = 1
        if bad:
            lps[k] = kps[k] = np.nan
            return out, k, lps, kps
        p, lp, kp = d
        took = k < n and 0 <= t < V and np.longdouble(clamp(u[k])) * q[t] < p[t]
        if not took:
            if np.isnan(u[K]):
                lps[k] = kps[k] = np.nan
                return out, k, lps, kps
            rest = np.maximum(p - q, 0) if k < n else p
            rest = rest if rest.any() else p  # a draft that neither side could give, where p is q
            run = np.cumsum(rest)
            t = min(int((run <= np.longdouble(clamp(u[K])) * run[-1]).sum()), int(np.flatnonzero(rest)[-1]))
        out[k], lps[k], kps[k] = t, lp[t], kp[t]
        if not took:
            return out, k, lps, kps
    raise AssertionError


def each(v, B):
    if torch.is_tensor(v):
        return v.double().cpu().numpy()
    return np.full(B, np.float32(v), np.float64)


NAMES = ("temperature", "top_k", "top_p", "min_p")


def check(z, tokens, u, draft=None, n=None, target=None, drafts=None, **kw):
    """Runs the call (any device layout) and compares every sequence. target and
    drafts: the settings of the two sides."""
    import rl_policy_gradient_amd as plp
    target, drafts = target or {}, drafts or {}
    dev = lambda v: v.cuda() if torch.is_tensor(v) and not v.is_cuda else v  # noqa: E731
    settings = {k: dev(v) for k, v in target.items()}
    if draft is not None:
        settings.update({"draft_" + k: dev(v) for k, v in drafts.items()})
    r = plp.verify_tokens(dev(z), dev(tokens), dev(u), draft_logits=dev(draft), num_drafts=dev(n), **settings, **kw)
    B, K = z.shape[0], z.shape[1] - 1
    default = dict(zip(NAMES, (1.0, 0, 1.0, 0.0)))
    ts = [each({**default, **target}[k], B) for k in NAMES]
    ds = [each({**default, **drafts}[k], B) for k in NAMES]
    zs, us, toks = z.double().cpu().numpy(), u.double().cpu().numpy(), tokens.cpu().numpy()
    qs = None if draft is None else draft.double().cpu().numpy()
    got = {k: v.cpu().numpy() for k, v in r.items()}
    for b in range(B):
        nb = K if n is None else min(max(int(n[b]), 0), K)
        row = lambda s: (s[0][b], int(s[1][b]), s[2][b], s[3][b])  # noqa: E731
        want = reference(zs[b], None if qs is None else qs[b], toks[b], us[b], nb, row(ts), row(ds))
        assert got["accepted"][b] == want[1], (b, got["accepted"][b], want[1])
        assert np.array_equal(got["tokens"][b], want[0]), (b, got["tokens"][b], want[0])
        for name, w in (("logp", want[2]), ("kept_logp", want[3])):
            g = got[name][b].astype(np.float64)
            assert np.array_equal(np.isnan(g), np.isnan(w)), (b, name, g, w)
            fine = ~np.isnan(w)
            assert (np.abs(g - w)[fine] <= U * np.abs(w[fine]) + 1e-12).all(), (b, name, g, w)
    return r


def inputs(B, K, V, dtype, seed, peaked=True, noise=0.7, certain=False):
    """Target and draft logits, drafts drawn from the draft's whole distribution
    (some of them any token), uniforms."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(B, K + 1, V, generator=g) * 2
    if peaked:
        m = min(V, 60)
        ids = torch.randint(0, V, (B, K + 1, m), generator=g)
        top = 15 - 2.5 * torch.rand(B, K + 1, 1, generator=g) * torch.log(torch.arange(1, m + 1).float())
        z.scatter_reduce_(2, ids, top.expand(B, K + 1, m), "amax")
    q = z[:, :K] + noise * torch.randn(B, K, V, generator=g)
    z, q = z.to(DT[dtype]), q.to(DT[dtype])
    if K:
        w = torch.softmax(q.double(), -1).view(B * K, V)
        tokens = torch.multinomial(w, 1, generator=g).view(B, K)
        tokens = torch.where(torch.rand(B, K, generator=g) < 0.15, torch.randint(0, V, (B, K), generator=g), tokens)
    else:
        tokens = torch.zeros(B, 0, dtype=torch.int64)
    return z, tokens, torch.rand(B, K + 1, generator=g), None if certain else q


LIMITS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.9, 40, 0.95, 0.02),
          (1.0, 1, 1.0, 0.0), (2.0, 0, 0.5, 0.01), (0.0, 5, 0.5, 0.5)]


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("limits", LIMITS, ids=str)
@pytest.mark.parametrize("B,K,V", [(1, 0, 5), (2, 1, 1), (3, 2, 2), (5, 3, 7), (6, 4, 255), (6, 1, 256), (5, 2, 257),
                                   (20, 3, 1000), (4, 5, 8193), (5, 2, 32000)])
def test_against_reference(B, K, V, limits, dtype, certain):
    require_gpu()
    s = dict(zip(NAMES, limits))
    for peaked in (True, False):
        z, tokens, u, q = inputs(B, K, V, dtype, 7 * V + K, peaked, certain=certain)
        check(z, tokens, u, q, target=s, drafts=s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("one,other", [((1.0, 0, 1.0, 0.0), (1.0, 20, 1.0, 0.0)), ((0.8, 50, 0.95, 0.0), (0.0, 0, 1.0, 0.0)),
                                       ((0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0)), ((0.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0)),
                                       ((1.2, 0, 0.9, 0.0), (0.6, 3, 1.0, 0.1))], ids=str)
def test_sides_of_different_settings(one, other, dtype):
    """The draft samples otherwise than the target, so that a draft may have had
    no chance there, or none here."""
    require_gpu()
    for V in (300, 5000):
        z, tokens, u, q = inputs(24, 3, V, dtype, V)
        check(z, tokens, u, q, target=dict(zip(NAMES, one)), drafts=dict(zip(NAMES, other)))


def test_full_vocabulary():
    require_gpu()
    for dtype, limits in (("bf16", (1.0, 0, 1.0, 0.0)), ("bf16", (0.8, 50, 0.95, 0.0)), ("f32", (1.0, 0, 0.9, 0.0))):
        s = dict(zip(NAMES, limits))
        z, tokens, u, q = inputs(3, 4, 151936, dtype, 1)
        check(z, tokens, u, q, target=s, drafts=s)
    z, tokens, u, q = inputs(2, 1, 1 << 20, "bf16", 2)
    check(z, tokens, u, q)
    check(z, tokens, u, q, target=dict(top_k=100, top_p=0.95), drafts=dict(top_p=0.9))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_settings_and_drafts_of_each_sequence(dtype):
    require_gpu()
    B, K, V = 64, 4, 3001
    z, tokens, u, q = inputs(B, K, V, dtype, 5)
    g = torch.Generator().manual_seed(3)
    pick = lambda v, t: torch.tensor(v, dtype=t)[torch.randint(0, len(v), (B,), generator=g)]  # noqa: E731

    def some():
        return dict(temperature=pick([0.0, 0.5, 1.0, 1.0, 3.0], torch.float32),
                    top_k=pick([0, -3, 1, 7, 100, 3001, 9000], torch.int32),
                    top_p=pick([0.0, 0.3, 0.9, 1.0, 1.5, -1.0], torch.float32),
                    min_p=pick([0.0, 0.1, 1.0, 2.0, -0.5], torch.float32))

    n = pick([0, 1, 2, 4, 4, 9, -2], torch.int32)
    check(z, tokens, u, q, n, some(), some())
    check(z, tokens, u, None, n, some())
    check(z, tokens, u, q, n, dict(temperature=0.9, top_k=30))


def test_the_same_distribution_takes_every_draft():
    """Where p and q are one row under one setting no draft that it can give is
    refused, at the largest uniform below 1 either."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    B, K, V = 64, 6, 2000
    z, _, u, _ = inputs(B, K, V, "bf16", 8)
    for s in (dict(), dict(temperature=0.7, top_k=40), dict(top_p=0.9), dict(temperature=1.4, min_p=0.02)):
        rows = z[:, :K].reshape(B * K, V).cuda()
        drawn = plp.sample_tokens(rows, torch.rand(B * K, generator=torch.Generator().manual_seed(4)).cuda(), **s)
        tokens = drawn["token"].view(B, K)
        u[:, :K] = 1 - 2.0 ** -24
        r = plp.verify_tokens(z.cuda(), tokens, u.cuda(), draft_logits=z[:, :K].contiguous().cuda(), **s,
                              **{"draft_" + k: v for k, v in s.items()})
        assert (r["accepted"] == K).all() and torch.equal(r["tokens"][:, :K], tokens)
        # the log-probs are those that sampling gave, and the token after them is sampling's own
        assert torch.equal(r["logp"][:, :K].reshape(-1), drawn["logp"])
        assert torch.equal(r["kept_logp"][:, :K].reshape(-1), drawn["kept_logp"])
        last = plp.sample_tokens(z[:, K].cuda(), u[:, K].cuda().contiguous(), **s)
        assert torch.equal(r["tokens"][:, K], last["token"]) and torch.equal(r["logp"][:, K], last["logp"])
        assert torch.equal(r["kept_logp"][:, K], last["kept_logp"])


def test_no_drafts_is_sampling():
    require_gpu()
    import rl_policy_gradient_amd as plp
    z, tokens, u, _ = inputs(40, 0, 4001, "f32", 11)
    for s in (dict(), dict(top_k=10), dict(top_p=0.8, temperature=1.5), dict(temperature=0.0)):
        a = plp.verify_tokens(z.cuda(), tokens.cuda(), u.cuda(), **s)
        b = plp.sample_tokens(z[:, 0].cuda(), u[:, 0].cuda().contiguous(), **s)
        assert torch.equal(a["tokens"][:, 0], b["token"]) and torch.equal(a["logp"][:, 0], b["logp"])
        assert torch.equal(a["kept_logp"][:, 0], b["kept_logp"]) and (a["accepted"] == 0).all()


@pytest.mark.parametrize("certain", [False, True])
def test_tokens_are_distributed_as_the_targets(certain):
    """The first and the second token of many sequences over one pair of rows: the
    counts of each within five standard deviations of p's."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    B, K, V = 200000, 2, 6
    g = torch.Generator().manual_seed(0)
    z = torch.randn(1, K + 1, V, generator=g)
    q = torch.randn(1, K, V, generator=g)
    p = torch.softmax(z[0, :2].double(), -1)
    draft = torch.multinomial(torch.softmax(q[0], -1), B, replacement=True, generator=g).t().contiguous()
    r = plp.verify_tokens(z.cuda().expand(B, K + 1, V), draft.cuda(), torch.rand(B, K + 1, generator=g).cuda(),
                          draft_logits=None if certain else q.cuda().expand(B, K, V))
    tokens, count = r["tokens"].cpu(), r["accepted"].cpu()
    for k in range(2):
        seen = tokens[count >= k, k]
        n = len(seen)
        got = torch.bincount(seen, minlength=V).double()
        if certain and k == 1:
            continue  # whether there is a second token depends on the first, but not on what it is
        assert ((got - n * p[k]).abs() <= 5 * (n * p[k] * (1 - p[k])).sqrt()).all(), (k, got / n, p[k])
    assert (count > 0).any() and (count == 0).any()


def test_the_token_after_a_certain_draft_is_distributed_as_the_targets():
    """Whether a sequence has a second token depends on the first draft and its
    uniform; what it is on the second draft, its uniform and the last one, which
    are independent of those: so it is distributed as p_1, its draft taken or not."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    B, K, V = 200000, 2, 6
    g = torch.Generator().manual_seed(5)
    z, q = torch.randn(1, K + 1, V, generator=g), torch.randn(1, K, V, generator=g)
    p = torch.softmax(z[0].double(), -1)
    draft = torch.multinomial(torch.softmax(q[0], -1), B, replacement=True, generator=g).t().contiguous()
    r = plp.verify_tokens(z.cuda().expand(B, K + 1, V), draft.cuda(), torch.rand(B, K + 1, generator=g).cuda())
    tokens, count = r["tokens"].cpu(), r["accepted"].cpu()
    for k in range(K + 1):
        seen = tokens[count >= k, k]
        n, got = len(seen), torch.bincount(seen, minlength=V).double()
        assert n > 1000 and ((got - n * p[k]).abs() <= 5 * (n * p[k] * (1 - p[k])).sqrt()).all(), (k, got / n, p[k])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,tail,limits", [(151936, -13.0, dict(top_p=0.9999)), (151936, -13.0, dict(min_p=1e-12)),
                                           (151936, -20.0, dict(min_p=1e-12)), (151936, -20.0, dict(top_k=100000)),
                                           (1 << 20, -20.0, dict(min_p=1e-12)), (1 << 20, -24.0, dict(top_k=1000000))])
def test_masses_of_long_tails(V, tail, limits, dtype):
    """One likely token and all others equal, whose weights are all rounded the
    same way: a limited row's mass is a sum of weights that are each off by up to
    2^-51 of the whole mass, k of the V in all by up to k 2^-51 of it, of which the
    largest k hold k / V at least; the log of a mass is off by as much of itself:
    V 2^-51. The mass is sampling's to the last bit."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    B, K, top = 3, 1, V // 2
    z = torch.full((B, K + 1, V), tail).to(DT[dtype])
    z[:, :, top] = 0.0
    tokens, u = torch.tensor([[top], [top], [5]]), torch.tensor([[0.125, 0.0], [0.125, 0.25], [0.5, 0.25]])
    r = plp.verify_tokens(z.cuda(), tokens.cuda(), u.cuda(), **limits)
    settings = tuple({**dict(zip(NAMES, (1.0, 0, 1.0, 0.0))), **limits}[k] for k in NAMES)
    settings = (settings[0], settings[1], float(np.float32(settings[2])), float(np.float32(settings[3])))
    for b in range(B):
        want = reference(z[b].double().numpy(), None, tokens[b].numpy(), u[b].double().numpy(), K, settings, None)
        assert r["accepted"][b] == want[1] == (b < 2)
        assert np.array_equal(r["tokens"][b].cpu().numpy(), want[0])
        for name, w, off in (("logp", want[2], 0.0), ("kept_logp", want[3], V * 2.0 ** -51)):
            got = r[name][b].double().cpu().numpy()
            assert (np.abs(got - w) <= U * np.abs(w) + off + 1e-12).all(), (b, name, got, w)
    one = plp.sample_tokens(z[:2, K].cuda(), u[:2, K].cuda().contiguous(), **limits)
    assert torch.equal(r["tokens"][:2, K], one["token"]) and torch.equal(r["kept_logp"][:2, K], one["kept_logp"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_that_weigh_next_to_nothing(dtype):
    """A token has its chance down to 2^-1000 (e^-693.1) of the row's largest, also
    where sampling's rounding of the weights leaves nothing of it; below there is none."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    logits = [-36.0, -40.0, -300.0, -692.0, -696.0, -700.0]
    B, K, V = 2, len(logits), 300
    for s in (dict(), dict(top_k=200)):
        z = torch.full((B, K + 1, V), -800.0)
        z[:, :, 7] = 0.0
        tokens = torch.arange(10, 10 + K).expand(B, K).contiguous()
        for k, x in enumerate(logits):
            z[:, k, 10 + k] = x
        u = torch.tensor([0.0, 0.5])[:, None].expand(B, K + 1).contiguous()
        r = plp.verify_tokens(z.to(DT[dtype]).cuda(), tokens.cuda(), u.cuda(), **s)
        assert r["accepted"].tolist() == [4, 0]
        assert r["tokens"].tolist() == [[10, 11, 12, 13, 7, -1, -1], [7] + [-1] * K]
        # each log-prob is z - log(1 + e^x), x the row's drafted logit, e^x at most e^-36 =
        # 2.3e-16 (not 0): a value good to 1e-12 like the others, and one rounding
        want = torch.tensor([logits[:4] + [0.0] * 3, [0.0] * (K + 1)], dtype=torch.float64)
        for name in ("logp", "kept_logp"):
            assert ((r[name].cpu().double() - want).abs() <= U * want.abs() + 1e-12).all(), (name, r[name])


def test_drafts_that_are_no_token():
    require_gpu()
    z, tokens, u, q = inputs(40, 3, 500, "f32", 21)
    tokens[::3, 0] = -1
    tokens[1::3, 1] = 500
    tokens[2::7, 0] = 2 ** 40
    check(z, tokens, u, q)
    check(z, tokens, u, None, target=dict(top_p=0.9))
    u[:] = 0.0
    check(z, tokens, u, q)


def test_rows_without_a_distribution():
    """They end a sequence that comes to them, and no other."""
    require_gpu()
    nan, inf = float("nan"), float("inf")
    B, K, V = 48, 3, 700
    for certain in (False, True):
        z, tokens, u, q = inputs(B, K, V, "f32", 31, noise=0.1, certain=certain)
        z[0, 0, 5], z[1, 1, 699], z[2, 3, 0], z[3, 2] = nan, inf, nan, -inf
        u[4, 0], u[5, 2], u[6, 3], u[7, 0], u[8, 3], u[9, 1] = nan, nan, nan, -3.0, 7.0, inf
        if q is not None:
            q[10, 0, 3], q[11, 2], q[12, 1, 4] = nan, -inf, inf
        z[13, 0, 100:], z[14, 1, :699] = -inf, -inf  # masked, but not wholly
        n = torch.full((B,), K, dtype=torch.int32)
        n[15:20] = torch.tensor([0, 1, 2, 3, 3]).int()
        z[15, 1], z[16, 2], z[17, 3] = nan, nan, nan  # past their drafts
        check(z, tokens, u, q, n)
        check(z, tokens, u, q, n, dict(top_k=20, top_p=0.9), dict(top_k=20))
        tau = torch.ones(B)
        tau[20], tau[21], tau[22] = nan, inf, -1.0
        check(z, tokens, u, q, n, dict(temperature=tau))
        if q is not None:
            check(z, tokens, u, q, n, dict(), dict(temperature=tau))


def test_ties_and_huge_logits():
    require_gpu()
    g = torch.Generator().manual_seed(1)
    B, K, V = 30, 2, 900
    z = torch.randint(0, 4, (B, K + 1, V), generator=g).float()
    q = torch.randint(0, 4, (B, K, V), generator=g).float()
    tokens, u = torch.randint(0, V, (B, K), generator=g), torch.rand(B, K + 1, generator=g)
    z[0, 0], q[0, 0] = 0.0, -0.0
    for s in (dict(top_k=100), dict(top_p=0.4), dict(temperature=0.0), dict(min_p=0.1), dict()):
        check(z, tokens, u, q, target=s, drafts=s)
    check(z * 1e37, tokens, u, q * 1e37)
    check(z - 3e38, tokens, u, q + 3e38, target=dict(top_k=50))


@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_alignment(dtype, shift):
    """Rows anywhere in a larger buffer, sequences that share rows, and what lies
    around the outputs."""
    require_gpu()
    B, K, V = 5, 3, 517
    z, tokens, u, q = inputs(B, K, V, dtype, 2)

    def placed(x, s0, s1):
        buf = torch.full((shift + s0 * B + s1 * 5,), float("nan"), dtype=x.dtype, device="cuda")
        view = buf.as_strided(x.shape, (s0, s1, 1), shift)
        view.copy_(x)
        return view

    zd, qd = placed(z, 7 * 523, 523), placed(q, 6 * 519 + 1, 519)
    s = dict(top_k=40, top_p=0.95)
    bufs = {k: torch.full((B * (K + 1) + 8,), -7, dtype=t, device="cuda") for k, t in
            (("tokens", torch.int64), ("logp", torch.float32), ("kept_logp", torch.float32))}
    out = {k: b[shift:shift + B * (K + 1)].view(B, K + 1) for k, b in bufs.items()}
    count = torch.full((B + 8,), -7, dtype=torch.int32, device="cuda")
    out["accepted"] = count[shift:shift + B]
    r = check(zd, tokens, u, qd, target=s, drafts=s, out=out)
    assert all(r[k] is out[k] for k in out)
    for b in (*bufs.values(), count):
        assert (b[:shift] == -7).all() and (b[-8 + shift:] == -7).all()
    one = z[:1].cuda().expand(B, K + 1, V)
    check(one, tokens, u, qd)


def test_many_rows_and_many_drafts():
    """More rows than one launch takes, and as many drafts as a call may have."""
    require_gpu()
    g = torch.Generator().manual_seed(7)
    B, K, V = 12000, 2, 9
    z, q = torch.randn(B, K + 1, V, generator=g), torch.randn(B, K, V, generator=g)
    check(z, torch.randint(0, V, (B, K), generator=g), torch.rand(B, K + 1, generator=g), q,
          torch.randint(0, K + 1, (B,), generator=g).int(), dict(top_k=4))
    B, K, V = 3, 1024, 40
    z = torch.randn(B, K + 1, V, generator=g)
    q = z[:, :K] + 1e-3 * torch.randn(B, K, V, generator=g)
    tokens = torch.multinomial(torch.softmax(q, -1).view(B * K, V), 1, generator=g).view(B, K)
    u = 0.99 * torch.rand(B, K + 1, generator=g)
    r = check(z, tokens, u, q)
    assert (r["accepted"] > 256).any()  # past what one workgroup looks at in a step


@pytest.mark.parametrize("certain", [False, True])
def test_batches_that_leave_rows_out(certain):
    """So many rows with limits that those after a refused draft are left out, in
    an order that changes with the launch: the same bits at every call."""
    require_gpu()
    for B, K, V in ((300, 4, 1500), (700, 3, 600), (150, 2, 1000)):
        z, tokens, u, q = inputs(B, K, V, "bf16", 77, certain=certain)
        n = torch.randint(0, K + 1, (B,), generator=torch.Generator().manual_seed(1)).int()
        for s in (dict(top_p=0.9), dict(top_k=20, temperature=0.7)):
            first = check(z, tokens, u, q, n, s, s)
            for _ in range(3):
                again = check(z, tokens, u, q, n, s, s)
                assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [700, 9000, 140000, 300000])
def test_a_sequence_does_not_depend_on_the_batch(V, dtype):
    """A batch of more rows than CUs, whose workgroups are smaller, against its
    sequences a few at a time: the same bits."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    g = torch.Generator(device="cuda").manual_seed(V)
    B, K, few = 63, 2, 21
    for flat in (False, True):
        z = torch.randn(B, K + 1, V, generator=g, device="cuda") * (0.3 if flat else 3.0)
        q = (z[:, :K] + 0.3 * torch.randn(B, K, V, generator=g, device="cuda")).to(DT[dtype])
        z = z.to(DT[dtype])
        u = torch.rand(B, K + 1, generator=g, device="cuda")
        for s in (dict(), dict(top_p=0.9), dict(top_p=0.3, temperature=0.7), dict(top_k=50), dict(top_k=3000, top_p=0.8),
                  dict(min_p=0.1), dict(top_k=400, min_p=0.001, temperature=1.5)):
            drafts = torch.stack([plp.sample_tokens(q[:, k], torch.rand(B, generator=g, device="cuda"), **s)["token"]
                                  for k in range(K)], 1)
            kw = dict(s, **{"draft_" + k: v for k, v in s.items()})
            whole = plp.verify_tokens(z, drafts, u, draft_logits=q, **kw)
            assert (whole["tokens"][:, 0] >= 0).all()
            for b in range(0, B, few):
                part = plp.verify_tokens(z[b:b + few], drafts[b:b + few], u[b:b + few], draft_logits=q[b:b + few], **kw)
                assert all(torch.equal(part[k], whole[k][b:b + few]) for k in part), (s, b)


@pytest.mark.parametrize("certain,B,K,V", [(True, 2200, 1, 40000), (True, 230, 2, 110000), (False, 240, 1, 200000),
                                           (False, 260, 3, 160000)])
def test_rows_in_several_launches(certain, B, K, V):
    """So many logits that a sequence's first rows, or its first and its second,
    go ahead of the others: as a few sequences at a time, and as a graph."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    g = torch.Generator(device="cuda").manual_seed(B)
    z = (torch.randn(B, K + 1, V, generator=g, device="cuda") * 3).bfloat16()
    q = None if certain else (z[:, :K].float() + 0.5 * torch.randn(B, K, V, generator=g, device="cuda")).bfloat16()
    n = torch.randint(0, K + 1, (B,), generator=g, device="cuda").int()
    u = torch.rand(B, K + 1, generator=g, device="cuda")
    for s in (dict(), dict(top_p=0.9, min_p=0.001)):
        drafts = torch.stack([plp.sample_tokens((z if certain else q)[:, k], torch.rand(B, generator=g, device="cuda"), **s)["token"]
                              for k in range(K)], 1)
        side = {} if certain else dict(draft_logits=q, **{"draft_" + k: v for k, v in s.items()})
        whole = plp.verify_tokens(z, drafts, u, num_drafts=n, **s, **side)
        assert (whole["tokens"][:, 0] >= 0).all() and (whole["accepted"] <= n).all()
        for b in range(0, B, 10):
            c = slice(b, b + 10)
            if not certain:
                side["draft_logits"] = q[c]
            part = plp.verify_tokens(z[c], drafts[c], u[c], num_drafts=n[c], **s, **side)
            assert all(torch.equal(part[k], whole[k][c]) for k in part), (s, b)
        if not certain:
            side["draft_logits"] = q
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = plp.verify_tokens(z, drafts, u, num_drafts=n, **s, **side)
        for _ in range(3):
            out["tokens"].fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(out[k], whole[k]) for k in out)


@pytest.mark.parametrize("certain,B,K,V", [(False, 260, 3, 160000), (True, 230, 2, 200000), (False, 900, 2, 700),
                                           (True, 900, 2, 700), (True, 60, 3, 700)])
def test_settings_of_each_sequence_in_large_batches(certain, B, K, V):
    """Large batches whose sequences have settings of their own, in one launch over
    rows or several, against their sequences a few at a time: the same bits."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    g = torch.Generator(device="cuda").manual_seed(B + V)
    z = (torch.randn(B, K + 1, V, generator=g, device="cuda") * 3).bfloat16()
    q = None if certain else (z[:, :K].float() + 0.5 * torch.randn(B, K, V, generator=g, device="cuda")).bfloat16()
    n, u = (torch.randint(0, K + 1, (B,), generator=g, device="cuda").int(), torch.rand(B, K + 1, generator=g, device="cuda"))
    pick = lambda v, t: torch.tensor(v, dtype=t, device="cuda")[  # noqa: E731
        torch.randint(0, len(v), (B,), generator=g, device="cuda")]
    s = dict(temperature=pick([0.0, 0.7, 1.0, 1.3], torch.float32), top_k=pick([0, 0, 20, 400], torch.int32),
             top_p=pick([1.0, 0.9, 0.99], torch.float32), min_p=pick([0.0, 0.0, 0.05], torch.float32))
    drafts = torch.stack([plp.sample_tokens((z if certain else q)[:, k], torch.rand(B, generator=g, device="cuda"), **s)["token"]
                          for k in range(K)], 1)

    def some(c):
        side = {} if certain else dict(draft_logits=q[c], **{"draft_" + k: v[c] for k, v in s.items()})
        return plp.verify_tokens(z[c], drafts[c], u[c], num_drafts=n[c], **{k: v[c] for k, v in s.items()}, **side)

    whole = some(slice(None))
    assert (whole["tokens"][:, 0] >= 0).all() and (whole["accepted"] <= n).all()
    for b in range(0, B, 20):
        part = some(slice(b, b + 20))
        assert all(torch.equal(part[k], whole[k][b:b + 20]) for k in part), b


@pytest.mark.parametrize("certain", [False, True])
def test_what_a_workspace_holds_and_two_streams(certain):
    """The same results whatever the workspace held, of batches that leave rows
    out and of others, from two calls at once and from a captured graph."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    for B, K, V, s in ((700, 3, 600, dict(top_p=0.9)), (300, 4, 1500, dict(top_k=20)), (8, 3, 3000, dict()), (9, 0, 70, dict())):
        z, tokens, u, q = (None if t is None else t.cuda() for t in inputs(B, K, V, "bf16", 78, certain=certain))
        n = torch.randint(0, K + 1, (B,), generator=torch.Generator().manual_seed(2)).int().cuda()
        kw = dict(s, draft_logits=q, num_drafts=n, **({} if q is None else {"draft_" + k: v for k, v in s.items()}))
        want = check(z, tokens, u, q, n, s, s)
        same = lambda r: all(torch.equal(r[k], want[k]) for k in want)  # noqa: E731
        size = (B * (2 * K + 1) * ((V + 255) // 256 + 1) * 12 + B * ((2 * K + 1) * 40 + (K + 40) * 16 + V // 8)) + 65536
        for byte in (0x00, 0x3f, 0x7f, 0xbf, 0xff):  # zeros, a half, large, minus a half, NaN
            ws = torch.full((size,), byte, dtype=torch.uint8, device="cuda")
            assert same(plp.verify_tokens(z, tokens, u, workspace=ws, **kw)), byte
        sides, got = (torch.cuda.Stream(), torch.cuda.Stream()), []
        for side in sides:
            side.wait_stream(torch.cuda.current_stream())
        for i in range(6):
            with torch.cuda.stream(sides[i % 2]):
                got.append(plp.verify_tokens(z, tokens, u, **kw))
        for side in sides:
            torch.cuda.current_stream().wait_stream(side)
        assert all(map(same, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = plp.verify_tokens(z, tokens, u, **kw)
        for _ in range(3):
            for t in out.values():
                t.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert same(out) and same(plp.verify_tokens(z, tokens, u, **kw))


def test_offsets_past_32_bits():
    require_gpu()
    B, K, V = 5, 1, 1000
    z, tokens, u, q = inputs(B, K, V, "bf16", 3)
    buf = torch.zeros(4 * 2 ** 29 + 2 ** 28 + 5000, dtype=torch.bfloat16, device="cuda")
    zd = buf.as_strided((B, K + 1, V), (2 ** 29, 2 ** 28, 1), 1)
    zd.copy_(z)
    check(zd, tokens, u, q)
    zd = buf.as_strided((B, K + 1, V), (2 ** 29 + 11, 1003, 1), 3)
    zd.copy_(z)
    check(zd, tokens, u, q, target=dict(top_p=0.9))


def test_streams_graphs_and_repeats():
    """The same bits at every call, on a stream of its own, and from two graphs
    over separate memory replayed in turn between eager calls."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    made = []
    for seed, s in ((1, dict()), (2, dict(top_k=50, top_p=0.9, temperature=0.8))):
        z, tokens, u, q = (t.cuda() for t in inputs(16, 3, 4000, "bf16", seed))
        kw = dict(s, **{"draft_" + k: v for k, v in s.items()})

        def run(z=z, tokens=tokens, u=u, q=q, kw=kw):
            return plp.verify_tokens(z, tokens, u, draft_logits=q, **kw)

        want = run()
        same = lambda a, b: all(torch.equal(a[k], b[k]) for k in b)  # noqa: E731
        assert all(same(run(), want) for _ in range(3))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = run()
        torch.cuda.current_stream().wait_stream(side)
        assert same(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        made.append((graph, out, run, u))
    g = torch.Generator(device="cuda").manual_seed(0)
    for _ in range(4):
        for graph, out, run, u in made:
            u.copy_(torch.rand(u.shape, generator=g, device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            assert same(out, run())


def test_refuses():
    require_gpu()
    import rl_policy_gradient_amd as plp
    z, tokens, u, q = (t.cuda() for t in inputs(4, 2, 50, "f32", 0))

    def call(**kw):
        a = dict(logits=z, draft_tokens=tokens, uniforms=u, draft_logits=q)
        a.update(kw)
        return plp.verify_tokens(a.pop("logits"), a.pop("draft_tokens"), a.pop("uniforms"), **a)

    for kw, match in ((dict(logits=z[0]), "B, K"), (dict(logits=z[:, :0]), "B, K"), (dict(draft_tokens=tokens.int()), "draft_tokens"),
                      (dict(draft_tokens=tokens[:, :1]), "draft_tokens"), (dict(uniforms=u[:, :2]), "uniforms"),
                      (dict(uniforms=u.double()), "uniforms"), (dict(draft_logits=q.bfloat16()), "draft_logits"),
                      (dict(draft_logits=q[:, :, :49]), "draft_logits"), (dict(num_drafts=torch.ones(4, device="cuda")), "num_drafts"),
                      (dict(num_drafts=torch.ones(4, dtype=torch.int32)), "GPU"), (dict(logits=z.transpose(1, 2).contiguous().transpose(1, 2)), "contiguous"),
                      (dict(draft_top_k=torch.ones(3, dtype=torch.int32, device="cuda")), "draft_top_k"),
                      (dict(temperature=torch.ones(4)), "GPU"), (dict(workspace=torch.empty(8, device="cuda")), "workspace"),
                      (dict(out={"tokens": torch.empty(4, 2, dtype=torch.int64, device="cuda")}), "tokens"),
                      (dict(logits=z.half(), draft_logits=q.half()), "dtype")):
        with pytest.raises(ValueError, match=match):
            call(**kw)
    for kw, match in ((dict(temperature=-1.0), "target's temperature"), (dict(draft_temperature=float("nan")), "draft's temperature"),
                      (dict(top_p=1.5), "top_p"), (dict(draft_min_p=2.0), "draft's min_p"), (dict(top_k=-1), "top_k"),
                      (dict(out={"logp": u}), "overlap"), (dict(out={"kept_logp": z.view(-1)[:12].view(4, 3)}), "overlap")):
        with pytest.raises(plp.PlpError, match=match):
            call(**kw)
    none = plp.verify_tokens(z[:0], tokens[:0], u[:0], draft_logits=q[:0])
    assert none["tokens"].shape == (0, 3) and none["accepted"].shape == (0,)
