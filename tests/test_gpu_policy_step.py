"""The operators as a training loop uses them: norm -> logits -> sampled
completions -> fused loss -> norm backward -> AdamW over the head's tensors,
captured into one graph from the sampling on and by hand."""
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


def setup(dtype, B=4, T=24, H=128, V=700, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype).cuda()  # noqa: E731
    return dict(B=B, T=T, x=t(B * T, H), w=(1 + 0.1 * torch.randn(H, generator=g)).to(dtype).cuda(), b=t(H, std=0.1),
                W=t(V, H, std=0.1), bias=t(V, std=0.1), u=torch.rand(B * T, generator=g).cuda(),
                mask=(torch.rand(B * T, generator=g) < 0.8).cuda(), adv=torch.randn(B, generator=g).cuda())


def loss_and_gradients(d, tau=0.9):
    """One pass up to the gradients; also returns what was sampled."""
    import rl_policy_gradient_amd as plp
    f = plp.layer_norm_fwd(d["x"], d["w"], d["b"])
    logits = f["y"].float() @ d["W"].float().t() + d["bias"].float()
    s = plp.sample_tokens(logits, d["u"], temperature=tau, top_k=200, top_p=0.95)
    r = plp.fused_lmhead_policy_loss_fwd_bwd(f["y"], d["W"], s["token"], d["mask"], d["adv"], B=d["B"], T=d["T"],
                                             bias=d["bias"], old_logp=s["logp"], temperature=tau, epsilon_low=0.4,
                                             epsilon_high=0.4, diagnostics=True)
    n = plp.layer_norm_bwd(r["grad_hidden"], d["x"], d["w"], f["rstd"], f["mean"])
    return f, s, r, n


def test_gradients_through_the_chain():
    """fp32: the sampled log-probs are the loss's own, and every gradient is
    that of sum(dlogp * logp) through the head and the norm in 64 bits."""
    require_gpu()
    d = setup(torch.float32)
    tau = 0.9
    f, s, r, n = loss_and_gradients(d, tau)
    # the fp32 logits of a 128-term product, on either side: 2 * 136 roundings
    # of terms that add up to below 16 in magnitude, over the temperature
    assert (s["logp"] - r["logp"]).abs().max().item() <= 2 * 136 * 2.0 ** -24 * 16 / tau
    leaves = {k: d[k].double().cpu().requires_grad_() for k in ("x", "w", "b", "W", "bias")}
    x = leaves["x"]
    xc = x - x.mean(-1, keepdim=True)
    y = xc / torch.sqrt((xc ** 2).mean(-1, keepdim=True) + 1e-5) * leaves["w"] + leaves["b"]
    lp = torch.log_softmax((y @ leaves["W"].t() + leaves["bias"]) / tau, -1)
    lp = lp.gather(1, s["token"].cpu()[:, None])[:, 0]
    (lp * r["dlogp"].double().cpu()).sum().backward()
    for got, k in ((n["grad_x"], "x"), (n["grad_weight"], "w"), (n["grad_bias"], "b"), (r["grad_weight"], "W"),
                   (r["grad_bias"], "bias")):
        want = leaves[k].grad
        rel = ((got.double().cpu() - want).norm() / want.norm()).item()
        assert rel <= 1e-4, (k, rel)  # the fused path's own bound for fp32 gradients


@pytest.mark.parametrize("bits", [8, 32])
def test_steps_of_a_bf16_policy(bits):
    """Three optimizer steps: every tensor moves by the formula's amount from
    the gradients it was given, and the weight's matrix-core copy made again
    after the step gives the plain call's bits."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    d = setup(torch.bfloat16, H=256)
    names = ["w", "b", "W", "bias"]
    grads = {k: torch.empty_like(d[k]) for k in names}
    states = {k: plp.adamw_state(d[k], bits=bits, master=True) for k in names}
    table = plp.adamw_table([d[k] for k in names], [grads[k] for k in names], [states[k] for k in names],
                            weight_decay=[0.0, 0.0, 0.1, 0.0])
    lr, scale = 1e-3, torch.ones(1, device="cuda")
    for step in (1, 2, 3):
        f, s, r, n = loss_and_gradients(d)
        assert ((s["token"] >= 0) & (s["token"] < 700)).all() and torch.isfinite(r["loss"]).all()
        prep = plp.prepare_weight(d["W"])
        again = plp.fused_lmhead_policy_loss_fwd_bwd(f["y"], d["W"], s["token"], d["mask"], d["adv"], B=d["B"],
                                                     T=d["T"], bias=d["bias"], old_logp=s["logp"], temperature=0.9,
                                                     epsilon_low=0.4, epsilon_high=0.4, weight_prepared=prep)
        assert torch.equal(again["grad_weight"], r["grad_weight"])
        for k, gk in (("w", n["grad_weight"]), ("b", n["grad_bias"]), ("W", r["grad_weight"]), ("bias", r["grad_bias"])):
            grads[k].copy_(gk)
        norm = torch.sqrt(sum(g.float().square().sum() for g in grads.values()))
        scale.copy_((1.0 / norm).clamp(max=1.0).reshape(1))  # the usual clipping at 1
        old = {k: states[k]["master"].clone() for k in names}
        plp.adamw_step(table, lr=lr, step=step, grad_scale=scale, betas=(0.9, 0.95))
        for k in names:
            assert torch.equal(d[k], states[k]["master"].bfloat16()), k
            move = (states[k]["master"].double() - old[k].double()).abs()
            # |m hat| <= sqrt(v hat) * sqrt((1 - b1)^2 / (1 - b2)) / ... stays below 1 / sqrt(1 - b2) in
            # any history; plus the decay and the 8-bit states' own steps
            bound = lr * (1 / math.sqrt(1 - 0.95) + 0.1 * old[k].abs().max().item()) * 1.2
            assert move.max().item() <= bound, (k, step, move.max().item())
            if step == 1:
                g1 = grads[k].double() * scale.double()
                first = torch.where(g1.abs() > 1e-5, g1.sign(), torch.zeros_like(g1)) * lr
                sel = g1.abs() > 1e-5  # the first step is lr * sign, up to eps / |g|
                want = old[k].double() * (1 - lr * (0.1 if k == "W" else 0.0)) - first
                assert ((states[k]["master"].double() - want).abs()[sel] <= lr * 1.1e-3 + 1e-6).all(), k


def test_chain_captured_with_other_graphs():
    """The chain without torch's own matrix product, captured twice over
    separate workspaces and replayed alternately."""
    require_gpu()
    import rl_policy_gradient_amd as plp

    def record(seed):
        d = setup(torch.bfloat16, seed=seed)
        N, H = d["x"].shape
        V = d["W"].shape[0]
        logits = (torch.randn(N, V, generator=torch.Generator().manual_seed(seed)) * 2).cuda()
        table = plp.adamw_table([d["w"]], [torch.zeros_like(d["w"])], [plp.adamw_state(d["w"], bits=8, master=True)])
        step = torch.ones(1, dtype=torch.int64, device="cuda")

        def run():
            f = plp.layer_norm_fwd(d["x"], d["w"], d["b"])
            s = plp.sample_tokens(logits, d["u"], top_p=0.9)
            r = plp.fused_lmhead_policy_loss_fwd_bwd(f["y"], d["W"], s["token"], d["mask"], d["adv"], B=d["B"],
                                                     T=d["T"], bias=d["bias"], old_logp=s["logp"])
            n = plp.layer_norm_bwd(r["grad_hidden"], d["x"], d["w"], f["rstd"], f["mean"])
            table.tensors[0][1].copy_(n["grad_weight"])
            plp.adamw_step(table, lr=1e-2, step=step)
            return {"token": s["token"], "loss": r["loss"], "gx": n["grad_x"], "w": d["w"]}

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
