"""The operators around the fused LM-head policy loss, as cases to measure.

A training step of a policy is: sample the completions, run the final norm,
take the fused loss on its output, run the norm backward, step the optimizer.
The cases here are the calls of that loop outside the fused loss: token
sampling (``sample``), the norm's two directions (``norm_fwd``,
``norm_bwd``) and the AdamW step over many tensors (``adamw``).

``run`` computes them in plain torch operations where ``own`` is false and
through ``rl_policy_gradient_amd`` where it is true; ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}
BLOCK = 256  # elements of one scale of the 8-bit states
E4M3_MAX = 448.0


def listed():
    return [
        # one sequence being decoded: the call's latency is what counts
        {"name": "sample_1x151936_bf16_k50_p95", "op": "sample", "N": 1, "V": 151936, "dtype": "bf16", "logits": "peaked",
         "temperature": 0.8, "top_k": 50, "top_p": 0.95, "min_p": 0.0, "per_row": False},
        # a rollout batch for on-policy training: the whole distribution, nothing cut
        {"name": "sample_64x151936_bf16_full", "op": "sample", "N": 64, "V": 151936, "dtype": "bf16", "logits": "peaked",
         "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "per_row": False},
        # a policy early in training: flat rows, so the nucleus holds most of the vocabulary
        {"name": "sample_128x32000_bf16_flat_p90", "op": "sample", "N": 128, "V": 32000, "dtype": "bf16", "logits": "flat",
         "temperature": 1.0, "top_k": 0, "top_p": 0.9, "min_p": 0.0, "per_row": False},
        # a large serving batch, every request with settings of its own
        {"name": "sample_512x151936_f32_mixed", "op": "sample", "N": 512, "V": 151936, "dtype": "f32", "logits": "peaked",
         "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "per_row": True},
        # the final norm of one token being decoded
        {"name": "norm_fwd_1x896_bf16", "op": "norm_fwd", "N": 1, "H": 896, "dtype": "bf16", "rms": False, "bias": True},
        # the final norm of a training batch of 2 x 32768 tokens
        {"name": "norm_fwd_65536x896_bf16_rms", "op": "norm_fwd", "N": 65536, "H": 896, "dtype": "bf16", "rms": True,
         "bias": False},
        # the backward of a short sequence: few rows, the weight's gradient reduced over all of them
        {"name": "norm_bwd_512x896_bf16", "op": "norm_bwd", "N": 512, "H": 896, "dtype": "bf16", "rms": False,
         "bias": True},
        # the backward of a wide fp32 model's batch of 8 x 2048 tokens
        {"name": "norm_bwd_16384x4096_f32_rms", "op": "norm_bwd", "N": 16384, "H": 4096, "dtype": "f32", "rms": True,
         "bias": False},
        # a dozen small tensors: the call's latency is what counts
        {"name": "adamw_small_f32", "op": "adamw", "layers": 2, "H": 64, "V": 0, "param": "f32", "grad": "f32",
         "master": False, "bits": 32},
        # every tensor of a small model at once: 145 tensors, odd lengths among them, 8-bit states
        {"name": "adamw_145_tensors_bf16_8bit", "op": "adamw", "layers": 24, "H": 256, "V": 32001, "param": "bf16",
         "grad": "bf16", "master": True, "bits": 8},
        # the LM head, states in 32 bits beside an fp32 master copy
        {"name": "adamw_head_151936x896_bf16_32bit", "op": "adamw", "layers": 0, "H": 896, "V": 151936, "param": "bf16",
         "grad": "bf16", "master": True, "bits": 32},
        # the same with the states in 8 bits
        {"name": "adamw_head_151936x896_bf16_8bit", "op": "adamw", "layers": 0, "H": 896, "V": 151936, "param": "bf16",
         "grad": "bf16", "master": True, "bits": 8},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "norm_fwd", "norm_bwd", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "sample":
        V = _log_int(rng, 1000, 151936)
        return {"op": op, "N": _log_int(rng, 1, 512), "V": V, "dtype": dtype,
                "logits": rng.choice(["peaked", "peaked", "flat"]),
                "temperature": round(rng.uniform(0.5, 1.5), 2), "top_k": rng.choice([0, 20, 50, 1000]),
                "top_p": rng.choice([1.0, 0.95, 0.8]), "min_p": rng.choice([0.0, 0.0, 0.05]),
                "per_row": rng.random() < 0.5}
    if op in ("norm_fwd", "norm_bwd"):
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            H = (H + 7) // 8 * 8
        return {"op": op, "N": _log_int(rng, 1, min(65536, (1 << 26) // H)), "H": H, "dtype": dtype,
                "rms": rng.random() < 0.5, "bias": rng.random() < 0.5}
    param = dtype
    return {"op": op, "layers": _log_int(rng, 1, 24), "H": _log_int(rng, 64, 512), "V": _log_int(rng, 1000, 65536),
            "param": param, "grad": param if param == "f32" else rng.choice(["bf16", "f32"]),
            "master": param == "bf16" and rng.random() < 0.7, "bits": rng.choice([8, 32])}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


# ---- token sampling --------------------------------------------------------

def _prepare_sample(c, seed):
    g = _gen(seed)
    N, V = c["N"], c["V"]
    # the bulk of a vocabulary, and for a trained policy a few likely tokens
    # that fall off with their rank, at a rate of the row's own
    z = torch.randn(N, V, generator=g, device=DEV) * (1.0 if c["logits"] == "flat" else 2.0)
    if c["logits"] == "peaked":
        k = min(200, V)
        ids = torch.randint(0, V, (N, k), generator=g, device=DEV)
        rate = 0.6 + 2.4 * torch.rand(N, 1, generator=g, device=DEV)
        rank = torch.arange(1, k + 1, device=DEV, dtype=torch.float32)
        top = 18.0 - rate * torch.log(rank) + 0.3 * torch.randn(N, k, generator=g, device=DEV)
        z.scatter_reduce_(1, ids, top, "amax")  # an id drawn twice keeps its larger value, whatever the order
    s = {"logits": z.to(DT[c["dtype"]]), "uniforms": torch.rand(N, generator=g, device=DEV)}
    if c["per_row"]:
        pick = lambda vals, t: torch.tensor(vals, device=DEV, dtype=t)[  # noqa: E731
            torch.randint(0, len(vals), (N,), generator=g, device=DEV)]
        s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.2], torch.float32)
        s["top_k"] = pick([0, 0, 20, 50, 400], torch.int32)
        s["top_p"] = pick([1.0, 0.9, 0.95, 0.99], torch.float32)
        s["min_p"] = pick([0.0, 0.0, 0.02, 0.1], torch.float32)
    else:
        s.update({k: c[k] for k in ("temperature", "top_k", "top_p", "min_p")})
    return s


def _column(v, N, dtype):
    if isinstance(v, torch.Tensor):
        return v.to(dtype).reshape(N, 1)
    # a setting is a 32-bit float: the same value as in a tensor of them
    return torch.full((N, 1), float(np.float32(v)), device=DEV, dtype=dtype)


def _sample_plain(s):
    z = s["logits"].double()
    N, V = z.shape
    tau, p, mp, u = (_column(s[k], N, torch.float64) for k in ("temperature", "top_p", "min_p", "uniforms"))
    k = _column(s["top_k"], N, torch.int64).long()
    k = torch.where((k <= 0) | (k > V), V, k)
    greedy = tau == 0
    m = z.amax(dim=1, keepdim=True)
    w = ((z - m) / torch.where(greedy, 1.0, tau)).exp()
    total = w.sum(dim=1, keepdim=True)
    off = (("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))
    if all(not isinstance(s[key], torch.Tensor) and s[key] == v for key, v in off):
        wk = w  # nothing is cut: the order by value is not needed
        best = ((z == m).cumsum(dim=1) == 0).sum(dim=1, keepdim=True)
    else:
        order = torch.sort(z, dim=1, descending=True, stable=True).indices
        best = order[:, :1]  # the sort is stable: the lowest index of a tie
        ws = w.gather(1, order)
        cum = ws.cumsum(dim=1)
        in_k = torch.arange(V, device=z.device).expand(N, V) < k
        mass_k = cum.gather(1, k - 1)
        keep = in_k & ((cum - ws < p * mass_k) | (p >= 1)) & (ws >= mp)
        keep[:, 0] = True
        kept = torch.zeros_like(keep).scatter_(1, order, keep)
        wk = torch.where(kept, w, 0.0)
    ck = wk.cumsum(dim=1)
    mass = ck[:, -1:]
    token = (ck <= u * mass).sum(dim=1, keepdim=True).clamp_max(V - 1)
    token = torch.where(greedy, best, token)
    lw = (z.gather(1, token) - m) / torch.where(greedy, 1.0, tau)
    logp = torch.where(greedy, 0.0, lw - total.log())
    kept_logp = torch.where(greedy, 0.0, lw - mass.log())
    return {"token": token[:, 0], "logp": logp[:, 0].float(), "kept_logp": kept_logp[:, 0].float()}


def _sample_own(s):
    import rl_policy_gradient_amd as plp
    return plp.sample_tokens(s["logits"], s["uniforms"], temperature=s["temperature"], top_k=s["top_k"],
                             top_p=s["top_p"], min_p=s["min_p"])


def _sample_exact(c, seed):
    s = _prepare_sample(c, seed)
    N, V = c["N"], c["V"]
    host = {k: (v.double().cpu().numpy() if isinstance(v, torch.Tensor) else np.full(N, np.float32(v), np.float64))
            for k, v in s.items()}
    token, logp, kept_logp = np.zeros(N, np.int64), np.zeros(N), np.zeros(N)
    for n in range(N):
        z, tau = host["logits"][n], host["temperature"][n]
        if tau == 0:
            token[n] = int(np.argmax(z))
            continue
        x = (z - z.max()) / tau
        e = np.exp(x)
        order = np.argsort(-z, kind="stable")
        k = int(host["top_k"][n])
        order = order[:k] if 0 < k < V else order
        if host["top_p"][n] < 1:
            run = np.cumsum(e[order])
            order = order[:1 + int(np.searchsorted(run, host["top_p"][n] * run[-1], side="left"))]
        if host["min_p"][n] > 0:
            order = order[:max(1, int((e[order] >= host["min_p"][n]).sum()))]
        ids = np.sort(order)
        run = np.cumsum(e[ids])
        t = int(ids[min(len(ids) - 1, int(np.searchsorted(run, host["uniforms"][n] * run[-1], side="right")))])
        token[n] = t
        logp[n] = x[t] - math.log(e.sum())
        kept_logp[n] = x[t] - math.log(run[-1])
    return {"token": token, "logp": logp, "kept_logp": kept_logp}


# ---- the norm --------------------------------------------------------------

NORM_EPS = 1e-6


def _prepare_norm(c, seed):
    g = _gen(seed)
    N, H, dt = c["N"], c["H"], DT[c["dtype"]]
    # a residual stream: a per-column offset and scale, and rows of unequal size
    x = torch.randn(N, H, generator=g, device=DEV)
    x = x * (0.5 + torch.rand(N, 1, generator=g, device=DEV)) + 0.3 * torch.randn(H, generator=g, device=DEV)
    s = {"x": x.to(dt), "weight": (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(dt),
         "bias": (0.1 * torch.randn(H, generator=g, device=DEV)).to(dt) if c["bias"] else None, "rms": c["rms"]}
    if c["op"] == "norm_bwd":
        # the gradient of a loss averaged over many tokens; the statistics are the forward's
        s["grad_y"] = (1e-3 * torch.randn(N, H, generator=g, device=DEV)).to(dt)
        xd = s["x"].double()
        mean = xd.mean(dim=1, keepdim=True) if not c["rms"] else torch.zeros_like(xd[:, :1])
        s["rstd"] = ((xd - mean).square().mean(dim=1) + NORM_EPS).rsqrt().float()
        s["mean"] = None if c["rms"] else mean[:, 0].float()
    return s


def _norm_fwd_plain(s):
    x, w = s["x"].float(), s["weight"].float()
    out = {}
    if not s["rms"]:
        mean = x.mean(dim=1, keepdim=True)
        x = x - mean
        out["mean"] = mean[:, 0]
    rstd = (x.square().mean(dim=1, keepdim=True) + NORM_EPS).rsqrt()
    y = x * rstd * w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out["y"], out["rstd"] = y.to(s["x"].dtype), rstd[:, 0]
    return out


def _norm_fwd_own(s):
    import rl_policy_gradient_amd as plp
    return plp.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=NORM_EPS, rms=s["rms"])


def _norm_bwd_plain(s):
    x, w, dy, rstd = s["x"].float(), s["weight"].float(), s["grad_y"].float(), s["rstd"][:, None]
    dt = s["x"].dtype
    xh = (x if s["rms"] else x - s["mean"][:, None]) * rstd
    c = dy * w
    t = c - xh * (c * xh).mean(dim=1, keepdim=True)
    if not s["rms"]:
        t = t - c.mean(dim=1, keepdim=True)
    out = {"grad_x": (t * rstd).to(dt), "grad_weight": (dy * xh).sum(dim=0).to(dt)}
    if s["bias"] is not None:
        out["grad_bias"] = dy.sum(dim=0).to(dt)
    return out


def _norm_bwd_own(s):
    import rl_policy_gradient_amd as plp
    return plp.layer_norm_bwd(s["grad_y"], s["x"], s["weight"], s["rstd"], s["mean"], rms=s["rms"],
                              grad_bias=s["bias"] is not None)


def _norm_exact(c, seed):
    s = _prepare_norm(c, seed)
    x, w = s["x"].double(), s["weight"].double()
    H = x.shape[1]
    ones = torch.ones(H, 1, dtype=torch.float64, device=x.device)
    if c["op"] == "norm_fwd":
        mu = torch.zeros_like(x[:, :1]) if c["rms"] else x.mm(ones) / H
        var = ((x - mu) ** 2).mm(ones) / H
        sd = torch.sqrt(var + NORM_EPS)
        y = (x - mu) / sd * w + (s["bias"].double() if c["bias"] else 0.0)
        out = {"y": y, "rstd": (1.0 / sd)[:, 0]}
        if not c["rms"]:
            out["mean"] = mu[:, 0]
        return out
    dy, rstd = s["grad_y"].double(), s["rstd"].double()[:, None]
    xc = x if c["rms"] else x - s["mean"].double()[:, None]
    dxh = dy * w
    # the chain rule through the deviation and the mean, term by term
    dvar = (dxh * xc).mm(ones) * (-0.5) * rstd ** 3
    dx = dxh * rstd + dvar * 2.0 * xc / H
    if not c["rms"]:
        dx = dx - (dxh * rstd).mm(ones) / H
    out = {"grad_x": dx, "grad_weight": (dy * (xc * rstd)).t().mm(torch.ones_like(x[:, :1]))[:, 0]}
    if c["bias"]:
        out["grad_bias"] = dy.t().mm(torch.ones_like(x[:, :1]))[:, 0]
    return out


# ---- AdamW -----------------------------------------------------------------

ADAM = {"lr": 1e-5, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8}
DECAY = 0.1


def _sizes(c):
    """Elements of each tensor and whether it decays: per layer the four
    matrices and two vectors of a decoder block (one of an odd length), then
    the head."""
    H, V = c["H"], c["V"]
    one = [(3 * H * H, True), (H * H, True), (4 * H * H, True), (4 * H * H, True), (H, False), (H + 1, False)]
    return one * c["layers"] + ([(V * H, True)] if V else [])


def _prepare_adamw(c, seed):
    g = _gen(seed)
    sizes = _sizes(c)
    # one flat buffer per kind, every tensor at a multiple of 256 elements of it
    blocks = [-(-n // BLOCK) for n, _ in sizes]
    at = np.concatenate([[0], np.cumsum(blocks)]) * BLOCK
    total = int(at[-1])
    inside = torch.ones(total, dtype=torch.bool, device=DEV)
    for k, (n, _) in enumerate(sizes):
        inside[int(at[k]) + n:int(at[k + 1])] = False
    flat = lambda std: torch.randn(total, generator=g, device=DEV).mul_(std).mul_(inside)  # noqa: E731
    p = flat(0.02)
    s = {"param": p.to(DT[c["param"]]), "master": p if c["master"] else None,
         "grad": flat(1e-3).to(DT[c["grad"]]), "bits": c["bits"], "step": 100,
         "grad_scale": 0.5 + torch.rand(1, generator=g, device=DEV)}
    m, v = flat(3e-4), flat(1e-3).square_().add_(2e-7).mul_(inside)
    if c["bits"] == 8:
        s["exp_avg"], s["exp_avg_scale"] = _to_8bit(m.view(-1, BLOCK), False)
        s["exp_rms"], s["exp_rms_scale"] = _to_8bit(v.sqrt_().view(-1, BLOCK), True)
    else:
        s["exp_avg"], s["exp_avg_sq"] = m, v
    decay = [DECAY if d else 0.0 for _, d in sizes]
    s["decay"] = torch.repeat_interleave(torch.tensor(decay, device=DEV), torch.tensor(blocks, device=DEV))[:, None]
    # each tensor as its own view, as a program holds them
    cut = lambda t: [t[int(at[k]):int(at[k]) + n] for k, (n, _) in enumerate(sizes)]  # noqa: E731
    cutb = lambda t: [t[int(at[k]) // BLOCK:int(at[k + 1]) // BLOCK] for k in range(len(sizes))]  # noqa: E731
    names = [k for k in ("master", "exp_avg", "exp_avg_sq", "exp_rms") if s.get(k) is not None]
    parts = {k: cut(s[k]) for k in names}
    parts.update({k: cutb(s[k]) for k in ("exp_avg_scale", "exp_rms_scale") if k in s})
    states = [{k: v[i] for k, v in parts.items()} for i in range(len(sizes))]
    if own:  # the list of tensors, checked once, as a program keeps it over the steps
        import rl_policy_gradient_amd as plp
        s["table"] = plp.adamw_table(cut(s["param"]), cut(s["grad"]), states, weight_decay=decay)
    return s


def _to_8bit(x, positive):
    """[blocks, 256] fp32 as e4m3 codes (flat) and one scale a block."""
    scale = x.abs().amax(dim=1, keepdim=True) / E4M3_MAX
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    if positive:  # what is above zero stays above zero
        y = torch.where(x > 0, y.clamp_min(2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn).reshape(-1), scale[:, 0]


def _adamw_outputs(s):
    names = ["param", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_rms", "exp_rms_scale"]
    return {k: s[k] for k in names if s.get(k) is not None}


def _adamw_plain(s):
    s["step"] += 1
    b1, b2 = ADAM["beta1"], ADAM["beta2"]
    rows = lambda t: t.view(-1, BLOCK)  # noqa: E731
    g = rows(s["grad"]).float() * s["grad_scale"]
    p = rows(s["param"] if s["master"] is None else s["master"]).float()
    m, lr = rows(s["exp_avg"]).float(), ADAM["lr"]
    if s["bits"] == 8:
        m = m * s["exp_avg_scale"][:, None]
        v = (rows(s["exp_rms"]).float() * s["exp_rms_scale"][:, None]).square()
    else:
        v = rows(s["exp_avg_sq"])
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    root = v.sqrt()
    step_size = lr / (1 - b1 ** s["step"])
    denom = root * (1 / math.sqrt(1 - b2 ** s["step"])) + ADAM["eps"]
    p = p * (1 - lr * s["decay"]) - m / denom * step_size
    s["param"].copy_(p.view(-1))
    if s["master"] is not None:
        s["master"].copy_(p.view(-1))
    if s["bits"] == 8:
        for name, x in (("exp_avg", m), ("exp_rms", root)):
            codes, scale = _to_8bit(x, name == "exp_rms")
            s[name].copy_(codes)
            s[name + "_scale"].copy_(scale)
    else:
        s["exp_avg"].copy_(m.view(-1))
        s["exp_avg_sq"].copy_(v.view(-1))
    return _adamw_outputs(s)


def _adamw_own(s):
    import rl_policy_gradient_amd as plp
    s["step"] += 1
    plp.adamw_step(s["table"], lr=ADAM["lr"], step=s["step"], betas=(ADAM["beta1"], ADAM["beta2"]), eps=ADAM["eps"],
                   grad_scale=s["grad_scale"])
    return _adamw_outputs(s)


def _nearest_e4m3(y):
    """The nearest value with four significant bits, exponent -6 at the least, ties to even."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    unit = torch.exp2(e - 3)
    return torch.round(y / unit) * unit


def _adamw_exact(c, seed):
    s = _prepare_adamw(c, seed)
    t, b1, b2 = s["step"] + 1, ADAM["beta1"], ADAM["beta2"]
    per = lambda k: s[k].double().repeat_interleave(BLOCK)  # noqa: E731
    g = s["grad"].double() * s["grad_scale"].double()
    mom = s["exp_avg"].double() * (per("exp_avg_scale") if c["bits"] == 8 else 1.0)
    sq = (s["exp_rms"].double() * per("exp_rms_scale")) ** 2 if c["bits"] == 8 else s["exp_avg_sq"].double()
    mom = b1 * mom + (1 - b1) * g
    sq = b2 * sq + (1 - b2) * g ** 2
    step = (mom / (1 - b1 ** t)) / (torch.sqrt(sq / (1 - b2 ** t)) + ADAM["eps"])
    w = (s["param"] if s["master"] is None else s["master"]).double()
    w = w - ADAM["lr"] * (step + s["decay"].double().reshape(-1).repeat_interleave(BLOCK) * w)
    out = {"param": w}
    if c["master"]:
        out["master"] = w
    if c["bits"] == 32:
        out.update(exp_avg=mom, exp_avg_sq=sq)
        return out
    for name, x in (("exp_avg", mom), ("exp_rms", sq.sqrt())):
        x = x.view(-1, BLOCK)
        top = x.abs().max(dim=1, keepdim=True).values
        y = x * (E4M3_MAX / top.clamp_min(1e-300))
        q = _nearest_e4m3(y)
        if name == "exp_rms":
            q = torch.where(x > 0, torch.maximum(q, torch.full_like(q, 2.0 ** -9)), q)
        out[name], out[name + "_scale"] = q.reshape(-1), top[:, 0] / E4M3_MAX
    return out


# ---- what the tools call ---------------------------------------------------

def prepare(case, seed):
    return {"sample": _prepare_sample, "norm_fwd": _prepare_norm, "norm_bwd": _prepare_norm,
            "adamw": _prepare_adamw}[case["op"]](case, seed) | {"op": case["op"]}


def run(state):
    if own:
        return {"sample": _sample_own, "norm_fwd": _norm_fwd_own, "norm_bwd": _norm_bwd_own,
                "adamw": _adamw_own}[state["op"]](state)
    return {"sample": _sample_plain, "norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain,
            "adamw": _adamw_plain}[state["op"]](state)


def exact(case, seed):
    return {"sample": _sample_exact, "norm_fwd": _norm_exact, "norm_bwd": _norm_exact,
            "adamw": _adamw_exact}[case["op"]](case, seed)


def work(case):
    op = case["op"]
    if op == "sample":
        n = case["N"] * case["V"]
        return {"bytes": n * ESIZE[case["dtype"]] + 20.0 * case["N"], "flops": 4.0 * n}
    if op in ("norm_fwd", "norm_bwd"):
        N, H, e = case["N"], case["H"], ESIZE[case["dtype"]]
        stats = (4 if case["rms"] else 8) * N
        if op == "norm_fwd":
            return {"bytes": 2.0 * N * H * e + (2 if case["bias"] else 1) * H * e + stats, "flops": 7.0 * N * H}
        return {"bytes": 3.0 * N * H * e + (3 if case["bias"] else 2) * H * e + stats, "flops": 12.0 * N * H}
    n = float(sum(k for k, _ in _sizes(case)))
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    weights = 8 + ESIZE[case["param"]] if case["master"] else 2 * ESIZE[case["param"]]
    return {"bytes": n * (state + weights + ESIZE[case["grad"]]), "flops": 15.0 * n}
