"""The operators as a training loop uses them, with an embedding that shares the
head's weight: tokens -> embedding -> norm -> logits -> drafts verified ->
fused loss -> norm backward -> embedding gradient added to the head's ->
global norm -> AdamW."""
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


def setup(dtype, B=6, K=3, H=128, V=500, seed=0, std=0.3):
    """B sequences, each K + 1 positions whose input tokens are given."""
    g = torch.Generator().manual_seed(seed)
    t = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype).cuda()  # noqa: E731
    R = K + 1
    tokens = torch.randint(0, V, (B, R), generator=g)
    tokens[0, 0] = -1  # a place that holds no token
    return dict(B=B, K=K, R=R, V=V, tokens=tokens.cuda(), W=t(V, H, std=std), w=(1 + 0.1 * torch.randn(H, generator=g)).to(dtype).cuda(),
                draft=torch.randint(0, V, (B, K), generator=g).cuda(), noise=(0.3 * torch.randn(B, K, V, generator=g)).cuda(),
                u=torch.rand(B, R, generator=g).cuda(), ud=torch.rand(B * K, generator=g).cuda(),
                adv=torch.randn(B, generator=g).cuda(), scale=H ** 0.5)


def one_pass(d, tau=0.8, logits=None):
    """Up to the gradients; the rollout's tokens and log-probs come from the
    verification of drafts that a noisier head sampled."""
    import rl_policy_gradient_amd as plp
    B, R, V = d["B"], d["R"], d["V"]
    x = plp.embedding_fwd(d["tokens"], d["W"], scale=d["scale"])["y"].view(B * R, -1)
    f = plp.layer_norm_fwd(x, d["w"], rms=True)
    z = (f["y"].float() @ d["W"].float().t()).view(B, R, V) if logits is None else logits
    q = (z[:, :-1] + d["noise"]).contiguous()
    s = plp.sample_tokens(q.view(-1, V), d["ud"], temperature=tau, top_p=0.95)
    v = plp.verify_tokens(z, s["token"].view(B, -1), d["u"], draft_logits=q, temperature=tau, draft_temperature=tau,
                          draft_top_p=0.95)
    mask = (v["tokens"] >= 0).to(torch.uint8)
    targets = v["tokens"].clamp_min(0).view(-1)
    r = plp.fused_lmhead_policy_loss_fwd_bwd(f["y"], d["W"], targets, mask.view(-1), d["adv"], B=B, T=R,
                                             old_logp=v["logp"].view(-1), temperature=tau, epsilon_low=0.4,
                                             epsilon_high=0.4, diagnostics=True)
    n = plp.layer_norm_bwd(r["grad_hidden"], x, d["w"], f["rstd"], rms=True, grad_bias=False)
    head = r["grad_weight"].clone()
    plp.embedding_bwd(n["grad_x"].view(B, R, -1), d["tokens"], V, scale=d["scale"], accumulate=True,
                      out={"grad_weight": r["grad_weight"]})
    return dict(x=x, v=v, r=r, n=n, head=head, targets=targets, mask=mask)


@pytest.mark.parametrize("std", [0.3, 0.05])
def test_gradients_through_the_chain(std):
    """fp32: the verified log-probs are the loss's own, and the shared weight's
    gradient is that of sum(dlogp * logp) through both of its uses in 64 bits.
    With std 0.3 each position is all but certain to give its own token back, so
    that the gradients are what roundings leave of them."""
    require_gpu()
    d = setup(torch.float32, std=std)
    tau, H = 0.8, 128
    o = one_pass(d, tau)
    used = o["mask"].view(-1).bool()
    assert used.sum().item() == int(o["v"]["accepted"].sum()) + d["B"]
    # the fp32 logits of a 128-term product, on either side: 2 * 136 roundings of
    # terms that add up to below 40 in magnitude, over the temperature
    delta = 2 * 136 * 2.0 ** -24 * 40 / tau
    off = (o["v"]["logp"].view(-1) - o["r"]["logp"]).abs()[used].max().item()
    assert off <= delta
    leaves = {k: d[k].double().cpu().requires_grad_() for k in ("W", "w")}
    t = d["tokens"].cpu().view(-1)
    x = leaves["W"][t.clamp_min(0)] * (t >= 0)[:, None] * float(torch.tensor(d["scale"]))
    rstd = 1 / torch.sqrt((x ** 2).mean(-1, keepdim=True) + 1e-5)
    y = x * rstd * leaves["w"]
    lp = torch.log_softmax(y @ leaves["W"].t() / tau, -1).gather(1, o["targets"].cpu()[:, None])[:, 0]
    g = o["r"]["dlogp"].double().cpu()
    (lp * g).sum().backward()
    # Beside the fused path's own 1e-4 (of gradients that are not roundings): logits off by delta make
    # every p_v off by at most 2 delta p_v, so d z_v = g / tau ([v = y] - p_v), over all v, by 2 delta |g| / tau.
    # That goes into W's gradient times |y_t|, into grad_hidden times |W_v| at most, from there into the
    # norm's weight times |x rstd| <= sqrt(H), and through the norm (a projection times rstd w) and the
    # embedding's scale into W's again.
    with torch.no_grad():
        dz = 2 * delta * g.abs() / tau
        dh = dz * leaves["W"].norm(dim=1).max()
        through = (dh * rstd[:, 0] * leaves["w"].abs().max() * d["scale"])[t >= 0].sum()
        most = {"W": float((dz * y.norm(dim=1)).sum() + through), "w": float(dh.sum() * H ** 0.5)}
    for got, k in ((o["r"]["grad_weight"], "W"), (o["n"]["grad_weight"], "w")):
        want = leaves[k].grad
        err = (got.double().cpu() - want).norm().item()
        assert err <= 1e-4 * want.norm().item() + (most[k] if std > 0.1 else 0.0), (k, err, want.norm().item())
    untouched = torch.ones(d["V"], dtype=torch.bool)
    untouched[t[t >= 0]] = False
    assert torch.equal(o["r"]["grad_weight"].cpu()[untouched], o["head"].cpu()[untouched])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clipped_steps(dtype):
    """Three steps by the norm's factor, and the same steps with the gradients
    clipped in place: what is stepped with differs by the rounding of a product."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    ends = []
    for in_place in (False, True):
        d = setup(dtype, seed=3)
        names = ["W", "w"]
        grads = {k: torch.zeros_like(d[k]) for k in names}
        states = [plp.adamw_state(d[k], master=dtype == torch.bfloat16) for k in names]
        adam = plp.adamw_table([d[k] for k in names], list(grads.values()), states)
        table = plp.grad_table(list(grads.values()))
        for step in (1, 2, 3):
            o = one_pass(d)
            grads["W"].copy_(o["r"]["grad_weight"])
            grads["w"].copy_(o["n"]["grad_weight"])
            norm = float(plp.grad_norm(table)["norm"])
            r = plp.grad_norm(table, max_norm=norm / 3, norms=True)
            want = torch.sqrt(sum(g.double().square().sum() for g in grads.values()))
            assert abs(norm - float(want)) <= 2.0 ** -24 * float(want) * 1.01
            assert abs(float(r["norms"].double().square().sum().sqrt()) - norm) <= 3 * 2.0 ** -24 * norm
            if in_place:
                plp.clip_grads(table, r["scale"])
                half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
                # each element off by half a step, the limit and the factor by one rounding each, and eps
                assert abs(float(plp.grad_norm(table)["norm"]) - norm / 3) <= norm / 3 * (half + 5 * 2.0 ** -24) + 1e-6
                plp.adamw_step(adam, lr=1e-3, step=step)
            else:
                plp.adamw_step(adam, lr=1e-3, step=step, grad_scale=r["scale"])
            if step == 1:
                ends.append([(s.get("master") if s.get("master") is not None else d[k]).clone() for s, k in zip(states, names)])
    # the first step is lr m^ / (sqrt(v^) + eps) = lr sign(g), whatever the rounding, where |g| is far above eps
    for a, b in zip(*ends):
        moved = (a.double() - b.double()).abs()
        assert moved.max().item() <= 2 * 1e-3 and (moved > 1e-5).double().mean().item() < 0.05


def test_captured_chain():
    """The chain without torch's own matrix product, captured twice over separate
    memory and replayed in turn."""
    require_gpu()
    import rl_policy_gradient_amd as plp

    def record(seed):
        d = setup(torch.bfloat16, seed=seed)
        z = torch.randn(d["B"], d["R"], d["V"], generator=torch.Generator().manual_seed(seed)).mul(2).cuda()
        grads = [torch.zeros_like(d["W"]), torch.zeros_like(d["w"])]
        adam = plp.adamw_table([d["W"], d["w"]], grads, [plp.adamw_state(d[k], bits=8, master=True) for k in ("W", "w")])
        table, step = plp.grad_table(grads), torch.ones(1, dtype=torch.int64, device="cuda")

        def run():
            o = one_pass(d, logits=z)
            grads[0].copy_(o["r"]["grad_weight"])
            grads[1].copy_(o["n"]["grad_weight"])
            r = plp.grad_norm(table, max_norm=1e-3)
            plp.adamw_step(adam, lr=1e-2, step=step, grad_scale=r["scale"])
            return {"tokens": o["v"]["tokens"], "loss": o["r"]["loss"], "norm": r["norm"], "W": d["W"], "gW": grads[0]}

        return run

    eager, captured = [], []
    for seed in (1, 2):
        run = record(seed)
        eager.append([{k: v.clone() for k, v in run().items()} for _ in range(3)])
        run = record(seed)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        captured.append((graph, out, run))  # run holds the tensors that the graph reads
    for i in range(3):
        for c in (0, 1):
            captured[c][0].replay()
            torch.cuda.synchronize()
            for k, v in captured[c][1].items():
                assert torch.equal(v, eager[c][i][k]), (c, i, k)
