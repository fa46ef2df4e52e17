"""More of the calls around the fused LM-head policy loss, as cases to measure.

Between the rollout and the optimizer a policy's training loop has, beside
sampling, the norm and AdamW: the verification of tokens that a draft proposed
during the rollout (``verify``), the embedding of the tokens and its gradient
(``emb_fwd``, ``emb_bwd``), whose weight is often the head's, and the global
norm of all gradients with the coefficient, or the pass, that clips them
(``gnorm``).

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


def listed():
    return [
        # one sequence being decoded with four drafted tokens: the call's latency is what counts
        {"name": "verify_1x4_151936_bf16_k50_p95", "op": "verify", "B": 1, "K": 4, "V": 151936, "dtype": "bf16",
         "draft": "logits", "temperature": 0.8, "top_k": 50, "top_p": 0.95, "min_p": 0.0, "per_seq": False,
         "ragged": False},
        # an on-policy rollout batch: the whole distribution, nothing cut
        {"name": "verify_64x4_151936_bf16_full", "op": "verify", "B": 64, "K": 4, "V": 151936, "dtype": "bf16",
         "draft": "logits", "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "per_seq": False,
         "ragged": False},
        # a serving batch, every sequence with settings of its own and zero to three drafted tokens
        {"name": "verify_96x3_32000_f32_mixed", "op": "verify", "B": 96, "K": 3, "V": 32000, "dtype": "f32",
         "draft": "logits", "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "per_seq": True,
         "ragged": True},
        # a large batch whose drafts are copied from the prompt: certain tokens, no draft distribution
        {"name": "verify_256x8_32000_bf16_copied", "op": "verify", "B": 256, "K": 8, "V": 32000, "dtype": "bf16",
         "draft": "copied", "temperature": 1.0, "top_k": 0, "top_p": 0.95, "min_p": 0.0, "per_seq": False,
         "ragged": True},
        # the tokens of one decoding step of a serving batch
        {"name": "emb_fwd_64x896_bf16", "op": "emb_fwd", "N": 64, "H": 896, "V": 151936, "dtype": "bf16", "scale": 1.0,
         "pad": 0.0},
        # a training batch of 2 x 32768 tokens, scaled by sqrt(H), an eighth of it padding
        {"name": "emb_fwd_65536x896_bf16_scaled", "op": "emb_fwd", "N": 65536, "H": 896, "V": 151936, "dtype": "bf16",
         "scale": 29.933259, "pad": 0.125},
        # one short sequence, added to the head's gradient (the head and the embedding share their weight)
        {"name": "emb_bwd_512x896_bf16_tied", "op": "emb_bwd", "N": 512, "H": 896, "V": 151936, "dtype": "bf16",
         "grad": "bf16", "scale": 1.0, "pad": 0.0, "accumulate": True},
        # a training batch of 2 x 32768 tokens, an eighth of it padding, the embedding's own gradient
        {"name": "emb_bwd_65536x896_bf16", "op": "emb_bwd", "N": 65536, "H": 896, "V": 151936, "dtype": "bf16",
         "grad": "bf16", "scale": 29.933259, "pad": 0.125, "accumulate": False},
        # a wide fp32 model's batch of 8 x 2048 tokens
        {"name": "emb_bwd_16384x4096_f32", "op": "emb_bwd", "N": 16384, "H": 4096, "V": 32000, "dtype": "f32",
         "grad": "f32", "scale": 1.0, "pad": 0.0, "accumulate": False},
        # a dozen small tensors: the call's latency is what counts
        {"name": "gnorm_small_f32", "op": "gnorm", "layers": 2, "H": 64, "V": 0, "dtype": "f32", "clip": False},
        # every tensor of a small model at once, odd lengths among them, vectors in fp32, clipped where they are
        {"name": "gnorm_145_tensors_mixed_clip", "op": "gnorm", "layers": 24, "H": 256, "V": 32001, "dtype": "mixed",
         "clip": True},
        # every tensor of a model with the 151936 x 896 head, for the step's factor
        {"name": "gnorm_145_tensors_bf16_large", "op": "gnorm", "layers": 24, "H": 896, "V": 151936, "dtype": "bf16",
         "clip": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["verify", "verify", "emb_fwd", "emb_bwd", "emb_bwd", "gnorm"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "verify":
        V, K = _log_int(rng, 1000, 151936), rng.randint(1, 8)
        return {"op": op, "B": _log_int(rng, 1, min(256, 40_000_000 // ((2 * K + 1) * V))), "K": K, "V": V, "dtype": dtype,
                "draft": rng.choice(["logits", "logits", "copied"]),
                "temperature": round(rng.uniform(0.5, 1.5), 2), "top_k": rng.choice([0, 20, 50, 1000]),
                "top_p": rng.choice([1.0, 0.95, 0.8]), "min_p": rng.choice([0.0, 0.0, 0.05]),
                "per_seq": rng.random() < 0.5, "ragged": rng.random() < 0.5}
    if op in ("emb_fwd", "emb_bwd"):
        H = _log_int(rng, 64, 4096)
        if rng.random() < 0.7:
            H = (H + 7) // 8 * 8
        c = {"op": op, "N": _log_int(rng, 1, min(65536, (1 << 25) // H)), "H": H,
             "V": _log_int(rng, 1000, min(151936, (1 << 26) // H)), "dtype": dtype,
             "scale": rng.choice([1.0, round(math.sqrt(H), 4)]), "pad": rng.choice([0.0, 0.1, 0.4])}
        if op == "emb_bwd":
            c["accumulate"] = rng.random() < 0.5
            c["grad"] = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        return c
    return {"op": op, "layers": _log_int(rng, 1, 24), "H": _log_int(rng, 64, 768), "V": _log_int(rng, 1000, 100000),
            "dtype": rng.choice(["bf16", "f32", "mixed"]), "clip": rng.random() < 0.5}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


# ---- verification of drafted tokens ----------------------------------------
# p: the distribution that sampling with the target's settings draws from, q:
# the draft's own (or certain). Draft k is taken if u_k q(d_k) < p(d_k), as long
# as all before it are; the token after the last one taken comes from
# max(0, p - q) where a draft was refused and from p where none was.

SETTINGS = ("temperature", "top_k", "top_p", "min_p")


def _prepare_verify(c, seed):
    g = _gen(seed)
    B, K, V = c["B"], c["K"], c["V"]
    rand = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    # the bulk of a vocabulary and a few likely tokens that fall off with their rank
    z = 2.0 * torch.randn(B, K + 1, V, generator=g, device=DEV)
    n = min(200, V)
    ids = torch.randint(0, V, (B, K + 1, n), generator=g, device=DEV)
    rank = torch.arange(1, n + 1, device=DEV, dtype=torch.float32)
    top = 18.0 - (0.6 + 2.4 * rand(B, K + 1, 1)) * torch.log(rank) + 0.3 * torch.randn(B, K + 1, n, generator=g, device=DEV)
    z.scatter_reduce_(2, ids, top, "amax")  # an id drawn twice keeps its larger value, whatever the order
    s = {"logits": z.to(DT[c["dtype"]]), "uniforms": rand(B, K + 1), "draft_logits": None, "num_drafts": None}
    if c["ragged"]:
        s["num_drafts"] = torch.randint(0, K + 1, (B,), generator=g, device=DEV).int()
    if c["per_seq"]:
        pick = lambda vals, t: torch.tensor(vals, device=DEV, dtype=t)[  # noqa: E731
            torch.randint(0, len(vals), (B,), generator=g, device=DEV)]
        s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.2], torch.float32)
        s["top_k"] = pick([0, 0, 20, 50, 400], torch.int32)
        s["top_p"] = pick([1.0, 0.9, 0.95, 0.99], torch.float32)
        s["min_p"] = pick([0.0, 0.0, 0.02, 0.1], torch.float32)
    else:
        s.update({k: c[k] for k in SETTINGS})
    if c["draft"] == "logits":
        # a smaller model of the same data, sampled with the target's temperature and limits
        s["draft_logits"] = (z[:, :K] + 0.7 * torch.randn(B, K, V, generator=g, device=DEV)).to(DT[c["dtype"]])
        q = _distribution(s["draft_logits"], s)["p"]
        run = q.cumsum(dim=2)
        draft = (run <= rand(B, K, 1).double() * run[:, :, -1:]).sum(dim=2).clamp_max(V - 1)
    else:
        # what followed the same words before: often the likeliest token, sometimes any
        likeliest = z[:, :K].argmax(dim=2)
        draft = torch.where(rand(B, K) < 0.7, likeliest, torch.randint(0, V, (B, K), generator=g, device=DEV))
    s["draft_tokens"] = draft.contiguous()
    return s


def _column(v, B, dtype):
    if isinstance(v, torch.Tensor):
        return v.to(dtype).reshape(B, 1, 1)
    # a setting is a 32-bit float: the same value as in a tensor of them
    return torch.full((B, 1, 1), float(np.float32(v)), device=DEV, dtype=dtype)


def _distribution(logits, s):
    """Of logits [B, R, V] under the settings: the probabilities that sampling
    draws from, and what their log-probs need."""
    z = logits.double()
    B, R, V = z.shape
    tau, p, mp = (_column(s[k], B, torch.float64) for k in ("temperature", "top_p", "min_p"))
    k = _column(s["top_k"], B, torch.int64)
    k = torch.where((k <= 0) | (k > V), V, k)
    greedy = tau == 0
    m = z.amax(dim=2, keepdim=True)
    x = (z - m) / torch.where(greedy, 1.0, tau)
    w = x.exp()
    total = w.sum(dim=2, keepdim=True)
    off = (("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))
    if all(not isinstance(s[key], torch.Tensor) and s[key] == v for key, v in off):
        kept = w  # nothing is cut: the order by value is not needed
    else:
        ws, order = torch.sort(w, dim=2, descending=True, stable=True)
        cum = ws.cumsum(dim=2)
        in_k = torch.arange(V, device=z.device).expand(B, R, V) < k
        mass_k = cum.gather(2, (k - 1).expand(B, R, 1))
        keep = in_k & ((cum - ws < p * mass_k) | (p >= 1)) & (ws >= mp)
        keep[:, :, 0] = True
        kept = torch.where(torch.zeros_like(keep).scatter_(2, order, keep), w, 0.0)
    mass = kept.sum(dim=2, keepdim=True)
    first = (z == m) & ((z == m).cumsum(dim=2) == 1)
    return {"p": torch.where(greedy, first.double(), kept / mass), "x": torch.where(greedy, 0.0, x),
            "log_total": torch.where(greedy, 0.0, total.log()), "log_mass": torch.where(greedy, 0.0, mass.log())}


def _verify_plain(s):
    B, R, V = s["logits"].shape
    K = R - 1
    t, u, draft = _distribution(s["logits"], s), s["uniforms"].double(), s["draft_tokens"]
    n = torch.full((B,), K, device=DEV) if s["num_drafts"] is None else s["num_drafts"].long()
    if s["draft_logits"] is None:
        q = torch.zeros(B, K, V, dtype=torch.float64, device=DEV).scatter_(2, draft[:, :, None], 1.0)
    else:
        q = _distribution(s["draft_logits"], s)["p"]
    at = lambda x, tok: x.gather(2, tok[:, :, None])[:, :, 0]  # noqa: E731
    taken = (u[:, :K] * at(q, draft) < at(t["p"][:, :K], draft)) & (torch.arange(K, device=DEV) < n[:, None])
    count = taken.long().cumprod(dim=1).sum(dim=1)
    rows = torch.arange(B, device=DEV)
    p = t["p"][rows, count]
    rest = p - torch.where((count < n)[:, None], q[rows, count.clamp_max(K - 1)], 0.0)
    rest = rest.clamp_min(0.0)
    rest = torch.where(rest.sum(dim=1, keepdim=True) > 0, rest, p)
    run = rest.cumsum(dim=1)
    last = (run <= u[:, K:] * run[:, -1:]).sum(dim=1).clamp_max(V - 1)
    place = torch.arange(R, device=DEV)
    tokens = torch.where(place < count[:, None], torch.nn.functional.pad(draft, (0, 1)), -1)
    tokens = torch.where(place == count[:, None], last[:, None], tokens)
    used = tokens >= 0
    x = at(t["x"], tokens.clamp_min(0))
    logp = torch.where(used, x - t["log_total"][:, :, 0], 0.0)
    kept_logp = torch.where(used, x - t["log_mass"][:, :, 0], 0.0)
    return {"tokens": tokens, "accepted": count.int(), "logp": logp.float(), "kept_logp": kept_logp.float()}


def _verify_own(s):
    import rl_policy_gradient_amd as plp
    target = {k: s[k] for k in SETTINGS}
    draft = {"draft_" + k: s[k] for k in SETTINGS} if s["draft_logits"] is not None else {}
    return plp.verify_tokens(s["logits"], s["draft_tokens"], s["uniforms"], draft_logits=s["draft_logits"],
                             num_drafts=s["num_drafts"], **target, **draft)


def _verify_exact(c, seed):
    s = _prepare_verify(c, seed)
    B, K = c["B"], c["K"]
    host = {k: (v.double().cpu().numpy() if isinstance(v, torch.Tensor) else v if v is None else
                np.full(B, np.float32(v), np.float64)) for k, v in s.items()}
    draft = s["draft_tokens"].cpu().numpy()
    tokens, accepted = np.full((B, K + 1), -1, np.int64), np.zeros(B, np.int32)
    logp, kept_logp = np.zeros((B, K + 1)), np.zeros((B, K + 1))

    def row(z, b):
        """Probabilities, exponents, and the two masses' logarithms."""
        tau, k, top_p, min_p = (host[key][b] for key in SETTINGS)
        if tau == 0:
            one = np.zeros(len(z))
            one[int(np.argmax(z))] = 1.0
            return one, np.zeros(len(z)), 0.0, 0.0
        x = (z - z.max()) / tau
        e = np.exp(x)
        order = np.argsort(-z, kind="stable")
        order = order[:int(k)] if 0 < k < len(z) else order
        if top_p < 1:
            run = np.cumsum(e[order])
            order = order[:1 + int(np.searchsorted(run, top_p * run[-1], side="left"))]
        if min_p > 0:
            order = order[:max(1, int((e[order] >= min_p).sum()))]
        kept = np.zeros(len(z))
        kept[order] = e[order]
        return kept / kept.sum(), x, math.log(e.sum()), math.log(kept.sum())

    for b in range(B):
        count = K if host["num_drafts"] is None else int(host["num_drafts"][b])
        for k in range(count + 1):
            p, x, log_total, log_mass = row(host["logits"][b, k], b)
            d, q = (int(draft[b, k]), np.zeros(len(p))) if k < count else (-1, np.zeros(len(p)))
            if k < count:
                if host["draft_logits"] is None:
                    q[d] = 1.0
                else:
                    q = row(host["draft_logits"][b, k], b)[0]
            took = k < count and host["uniforms"][b, k] * q[d] < p[d]
            if not took:
                rest = np.maximum(p - q, 0.0)
                run = np.cumsum(rest if rest.sum() > 0 else p)
                d = min(len(p) - 1, int(np.searchsorted(run, host["uniforms"][b, K] * run[-1], side="right")))
            tokens[b, k], logp[b, k], kept_logp[b, k] = d, x[d] - log_total, x[d] - log_mass
            if not took:
                accepted[b] = k
                break
    return {"tokens": tokens, "accepted": accepted, "logp": logp, "kept_logp": kept_logp}


# ---- the embedding ---------------------------------------------------------

def _prepare_emb(c, seed):
    g = _gen(seed)
    N, H, V = c["N"], c["H"], c["V"]
    # words by their rank: the likelier, the lower the index; the commonest is one in log(V)
    tokens = (torch.rand(N, generator=g, device=DEV, dtype=torch.float64) * math.log(V)).exp().long().clamp(1, V) - 1
    if c["pad"] > 0:  # places that hold no token
        tokens = torch.where(torch.rand(N, generator=g, device=DEV) < c["pad"], -1, tokens)
    s = {"tokens": tokens, "scale": c["scale"], "V": V}
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    if c["op"] == "emb_fwd":
        s["weight"] = (0.02 * normal(V, H)).to(DT[c["dtype"]])
        return s
    s["grad_y"] = (1e-3 * normal(N, H)).to(DT[c["dtype"]])
    s["grad_dtype"] = DT[c["grad"]]
    # the head's gradient, to which the embedding's is added where they share the weight
    s["grad_weight"] = (1e-3 * normal(V, H)).to(DT[c["grad"]]) if c["accumulate"] else None
    return s


def _emb_fwd_plain(s):
    t, w = s["tokens"], s["weight"]
    y = w[t.clamp(0, s["V"] - 1)].float() * s["scale"]
    inside = ((t >= 0) & (t < s["V"]))[:, None]
    return {"y": torch.where(inside, y, 0.0).to(w.dtype)}


def _emb_fwd_own(s):
    import rl_policy_gradient_amd as plp
    return plp.embedding_fwd(s["tokens"], s["weight"], scale=s["scale"])


def _emb_bwd_plain(s):
    t, V = s["tokens"], s["V"]
    t = torch.where((t >= 0) & (t < V), t, V)  # one row more, for what is no token
    sums = torch.zeros(V + 1, s["grad_y"].shape[1], device=DEV).index_add_(0, t, s["grad_y"].float())
    gw = sums[:V] * s["scale"]
    if s["grad_weight"] is None:
        return {"grad_weight": gw.to(s["grad_dtype"])}
    s["grad_weight"].copy_(s["grad_weight"].float() + gw)
    return {"grad_weight": s["grad_weight"]}


def _emb_bwd_own(s):
    import rl_policy_gradient_amd as plp
    if s["grad_weight"] is None:
        return plp.embedding_bwd(s["grad_y"], s["tokens"], s["V"], scale=s["scale"], grad_dtype=s["grad_dtype"])
    return plp.embedding_bwd(s["grad_y"], s["tokens"], s["V"], scale=s["scale"], grad_dtype=s["grad_dtype"],
                             accumulate=True, out={"grad_weight": s["grad_weight"]})


def _emb_exact(c, seed):
    s = _prepare_emb(c, seed)
    t, V = s["tokens"], c["V"]
    inside = (t >= 0) & (t < V)
    if c["op"] == "emb_fwd":
        y = torch.zeros(c["N"], c["H"], dtype=torch.float64, device=DEV)
        y[inside] = s["weight"].double().index_select(0, t[inside]) * c["scale"]
        return {"y": y}
    # the rows in their tokens' order: a token's sum is the difference of two running sums
    t, order = torch.sort(t[inside])
    run = torch.nn.functional.pad(s["grad_y"][inside][order].double().cumsum(dim=0), (0, 0, 1, 0))
    ids = torch.arange(V, device=DEV)
    gw = c["scale"] * (run[torch.searchsorted(t, ids, right=True)] - run[torch.searchsorted(t, ids)])
    return {"grad_weight": gw if s["grad_weight"] is None else gw + s["grad_weight"].double()}


# ---- the gradients' norm ---------------------------------------------------

MAX_NORM, NORM_EPS = 1.0, 1e-6
BLOCK = 256


def _sizes(c):
    """Elements of each tensor and whether it is a vector: per layer the four
    matrices and two vectors of a decoder block (one of an odd length), then
    the head."""
    H, V = c["H"], c["V"]
    one = [(4 * H * H, False), (H * H, False), (4 * H * H, False), (3 * H * H, False), (H, True), (H + 1, True)]
    return one * c["layers"] + ([(V * H, False)] if V else [])


def _prepare_gnorm(c, seed):
    g = _gen(seed)
    sizes = _sizes(c)
    kind = ["f32" if c["dtype"] == "f32" or (c["dtype"] == "mixed" and vec) else "bf16" for _, vec in sizes]
    grads, flats = [None] * len(sizes), []
    for dt in sorted(set(kind)):
        # one flat buffer per type, every tensor at a multiple of 256 elements of it
        mine = [i for i, k in enumerate(kind) if k == dt]
        blocks = [-(-sizes[i][0] // BLOCK) for i in mine]
        at = np.concatenate([[0], np.cumsum(blocks)]) * BLOCK
        flat = torch.randn(int(at[-1]), generator=g, device=DEV).mul_(1e-3)
        for j, i in enumerate(mine):
            flat[int(at[j]) + sizes[i][0]:int(at[j + 1])] = 0.0
        flat = flat.to(DT[dt])
        for j, i in enumerate(mine):
            grads[i] = flat[int(at[j]):int(at[j]) + sizes[i][0]]
        flats.append((flat, torch.tensor(mine, device=DEV), torch.from_numpy(at // BLOCK).to(DEV)))
    # sums over five micro-batches of which four held tokens, divided by five
    s = {"grads": grads, "flats": flats, "clip": c["clip"], "grad_scale": torch.full((1,), 1.25, device=DEV)}
    if own:  # the list of tensors, checked once, as a program keeps it over the steps
        import rl_policy_gradient_amd as plp
        s["table"] = plp.grad_table(grads)
    return s


def _gnorm_plain(s):
    squares = torch.zeros(len(s["grads"]), dtype=torch.float64, device=DEV)
    runs = lambda flat: torch.nn.functional.pad(  # noqa: E731
        flat.float().square().view(-1, BLOCK).sum(dim=1, dtype=torch.float64).cumsum(dim=0), (1, 0))
    [squares.index_copy_(0, mine, runs(flat)[at].diff()) for flat, mine, at in s["flats"]]
    factor = s["grad_scale"].double()
    norms = squares.sqrt() * factor
    norm = squares.sum().sqrt() * factor
    scale = (factor * (MAX_NORM / (norm + NORM_EPS)).clamp(max=1.0)).float()
    if s["clip"]:
        [flat.copy_(flat.float() * scale) for flat, _, _ in s["flats"]]
    out = {"norm": norm.float(), "scale": scale, "norms": norms.float()}
    return out | ({"grads": [flat for flat, _, _ in s["flats"]]} if s["clip"] else {})


def _gnorm_own(s):
    import rl_policy_gradient_amd as plp
    out = plp.grad_norm(s["table"], max_norm=MAX_NORM, eps=NORM_EPS, grad_scale=s["grad_scale"], norms=True)
    if s["clip"]:
        plp.clip_grads(s["table"], out["scale"])
        out["grads"] = [flat for flat, _, _ in s["flats"]]
    return out


def _gnorm_exact(c, seed):
    s = _prepare_gnorm(c, seed)
    factor = float(s["grad_scale"])
    dots = [float(torch.dot(x, x)) for x in (g.double() for g in s["grads"])]
    norm = factor * math.sqrt(math.fsum(dots))
    scale = factor * min(1.0, MAX_NORM / (norm + NORM_EPS))
    out = {"norm": np.array([norm]), "scale": np.array([scale]), "norms": factor * np.sqrt(np.array(dots))}
    return out | ({"grads": [flat.double() * scale for flat, _, _ in s["flats"]]} if c["clip"] else {})


# ---- what the tools call ---------------------------------------------------

def prepare(case, seed):
    return {"verify": _prepare_verify, "emb_fwd": _prepare_emb, "emb_bwd": _prepare_emb,
            "gnorm": _prepare_gnorm}[case["op"]](case, seed) | {"op": case["op"]}


def run(state):
    if own:
        return {"verify": _verify_own, "emb_fwd": _emb_fwd_own, "emb_bwd": _emb_bwd_own,
                "gnorm": _gnorm_own}[state["op"]](state)
    return {"verify": _verify_plain, "emb_fwd": _emb_fwd_plain, "emb_bwd": _emb_bwd_plain,
            "gnorm": _gnorm_plain}[state["op"]](state)


def exact(case, seed):
    return {"verify": _verify_exact, "emb_fwd": _emb_exact, "emb_bwd": _emb_exact,
            "gnorm": _gnorm_exact}[case["op"]](case, seed)


def work(case):
    op = case["op"]
    if op == "verify":
        # rows past a sequence's drafts need not be read: half of them where their number varies
        drafts = case["K"] * (0.5 if case["ragged"] else 1.0)
        n = case["B"] * case["V"] * (1 + drafts * (2 if case["draft"] == "logits" else 1))
        return {"bytes": n * ESIZE[case["dtype"]] + case["B"] * (28.0 * case["K"] + 24.0), "flops": 4.0 * n}
    if op in ("emb_fwd", "emb_bwd"):
        N, H, V, e = case["N"] * (1 - case["pad"]), case["H"], case["V"], ESIZE[case["dtype"]]
        # different tokens among N, by their ranks' distribution
        v = np.arange(1, V + 1, dtype=np.float64)
        different = float((1 - np.exp(-N * np.log1p(1 / v) / math.log(V))).sum())
        if op == "emb_fwd":
            return {"bytes": different * H * e + case["N"] * (H * e + 8.0), "flops": 1.0 * N * H}
        w = ESIZE[case["grad"]] * H
        return {"bytes": N * H * e + 8.0 * case["N"] + (2 * different * w if case["accumulate"] else V * w),
                "flops": 1.0 * N * H}
    sizes = _sizes(case)
    byte = sum(n * (4 if case["dtype"] == "f32" or (case["dtype"] == "mixed" and vec) else 2) for n, vec in sizes)
    return {"bytes": byte * (3.0 if case["clip"] else 1.0), "flops": (3.0 if case["clip"] else 2.0) * sum(n for n, _ in sizes)}
