"""The global norm of gradients and their clipping on the GPU against sums in
64 bits: a norm, and a scale, is one rounding to fp32 of a value good to 1e-13."""
import math

import pytest
import torch

from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
MAX32 = 2.0 ** 128 - 2.0 ** 104
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def float32_default():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


def near(got, want):
    """One rounding; below the least normal number half of its spacing."""
    return abs(got - want) <= max(U * abs(want), 2.0 ** -150) * (1 + 1e-6) + 1e-13 * abs(want)


def check(grads, max_norm=None, eps=1e-6, scale=None, **kw):
    import rl_policy_gradient_amd as plp
    s = None if scale is None else torch.tensor([scale], device="cuda")
    out = plp.grad_norm(grads, max_norm=max_norm, eps=eps, grad_scale=s, norms=True, **kw)
    factor = 1.0 if s is None else float(s.double())
    sq = [float(g.double().square().sum()) for g in grads]
    norm = abs(factor) * math.sqrt(math.fsum(sq))
    want = factor * min(1.0, math.inf if max_norm is None else max_norm / (norm + eps) if norm + eps else 1.0)
    if norm > MAX32:  # no longer a value of fp32 (1 + 2^-25 of it would round down to it: no case here is that near)
        assert math.isinf(float(out["norm"])) and math.isnan(float(out["scale"]))
    else:
        assert near(float(out["norm"]), norm), (float(out["norm"]), norm)
        assert near(float(out["scale"]), want), (float(out["scale"]), want)
    for i, q in enumerate(sq):
        n = abs(factor) * math.sqrt(q)
        assert near(float(out["norms"][i]), n) if n <= MAX32 else math.isinf(float(out["norms"][i])), i
    return out


def some(sizes, kinds, seed=0, std=1e-3):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(DT[k]).cuda() for n, k in zip(sizes, kinds)]


SIZES = [[1], [7], [8], [2047], [2048], [2049], [100003], [1 << 20], [3_000_001, 5], [0], [0, 3, 0], [5000, 1, 0, 64, 2048, 9]]


@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_norm(sizes, kind):
    require_gpu()
    grads = some(sizes, [["f32", "bf16"][i % 2] if kind == "mixed" else kind for i in range(len(sizes))], len(sizes))
    check(grads)
    check(grads, max_norm=1e-3)
    check(grads, max_norm=0.5, eps=0.0, scale=0.25)
    check(grads, max_norm=1e-4, scale=-3.0)
    check(grads, max_norm=0.0)


@pytest.mark.parametrize("count", [239, 240, 241, 250, 600])
def test_many_tensors(count):
    """More than one launch holds, some of them empty."""
    require_gpu()
    g = torch.Generator().manual_seed(count)
    sizes = torch.randint(0, 6000, (count,), generator=g).tolist()
    grads = some(sizes, [["f32", "bf16"][i % 2] for i in range(count)], 3)
    import rl_policy_gradient_amd as plp
    out = check(grads, max_norm=0.3)
    before = [x.clone() for x in grads]
    table = plp.grad_table(grads)
    plp.clip_grads(table, out["scale"])
    for a, b in zip(grads, before):
        assert torch.equal(a, (b.float() * out["scale"]).to(b.dtype))


@pytest.mark.parametrize("count,most", [(4096, 5), (5000, 0), (20000, 9), (20000, 700)])
def test_long_lists(count, most):
    """More tensors than a list of few has tiles, most of them of a few elements or
    none: every tensor's norm, the whole one, and the clipping in place."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    g = torch.Generator().manual_seed(count + most)
    sizes = torch.randint(0, most + 1, (count,), generator=g)
    flat = torch.randn(int(sizes.sum()), generator=g).to(DT["bf16" if most == 9 else "f32"])
    grads = list(flat.cuda().split(sizes.tolist()))
    table = plp.grad_table(grads)
    out = plp.grad_norm(table, max_norm=0.25, norms=True)
    own = torch.zeros(count, dtype=torch.float64).index_add_(0, torch.arange(count).repeat_interleave(sizes), flat.double().square())
    assert out["norms"].shape == (count,)
    got, want = out["norms"].cpu().double(), own.sqrt()
    assert ((got - want).abs() <= U * want * (1 + 1e-6) + 1e-13 * want).all()
    norm = math.sqrt(math.fsum(own.tolist()))
    assert near(float(out["norm"]), norm) and near(float(out["scale"]), min(1.0, 0.25 / (norm + 1e-6)))
    plp.clip_grads(table, out["scale"])
    assert torch.equal(torch.cat(grads).cpu(), (flat.float() * out["scale"].cpu()).to(flat.dtype))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_around_what_one_workgroup_takes(more, kind):
    """Lists of about 2^17 elements and 128 tiles, which go in one launch up to there."""
    require_gpu()
    check(some([(1 << 17) - 5000 + more, 4000, 0, 1000], [kind] * 4, 1), max_norm=0.1)
    g = torch.Generator().manual_seed(3)
    check(some(torch.randint(0, 1000, (128 + more,), generator=g).tolist(), ["f32", "bf16"] * 65, 2), max_norm=0.1)
    check(some([2048] * 63 + [1] * (65 + more), [kind] * 130, 4), max_norm=0.1)


def test_sizes_of_the_range():
    """Values whose squares leave fp32 at both ends."""
    require_gpu()
    for v in (1e-45, 1e-38, 1e-30, 1e-20, 1e19, 1e30, 3e38):
        check([torch.full((3,), v, device="cuda"), torch.zeros(9, device="cuda")], max_norm=1.0)
    check([torch.full((5000,), 2.0 ** -126, device="cuda").bfloat16()], max_norm=1.0)
    out = check([torch.tensor([3e38, 1e-30], device="cuda")], max_norm=2.0)
    assert torch.isfinite(out["scale"]).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("at", [0, 2500, 4999])
def test_values_that_are_not_finite(bad, at):
    """The scale is NaN, and neither a clipping nor a step by it changes anything."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    grads = some([5000, 77], ["f32", "bf16"])
    grads[0][at] = bad
    out = plp.grad_norm(grads, max_norm=1.0, norms=True)
    assert not torch.isfinite(out["norm"]).any() and torch.isnan(out["scale"]).all()
    assert not torch.isfinite(out["norms"][0]) and torch.isfinite(out["norms"][1])
    before = [g.clone() for g in grads]
    plp.clip_grads(grads, out["scale"])
    assert all(torch.equal(a.nan_to_num(1, 2, 3), b.nan_to_num(1, 2, 3)) for a, b in zip(grads, before))
    p = torch.ones(5000, device="cuda")
    table = plp.adamw_table([p], [grads[0]], [plp.adamw_state(p)], weight_decay=0.1)
    plp.adamw_step(table, lr=0.1, step=1, grad_scale=out["scale"])
    assert (p == 1).all()
    # a sum that fp32 does not hold; a factor that is none
    big = [torch.full((4,), 3e38, device="cuda")]
    out = plp.grad_norm(big, max_norm=1.0)
    assert torch.isinf(out["norm"]).all() and torch.isnan(out["scale"]).all()
    out = plp.grad_norm([before[1]], max_norm=1.0, grad_scale=torch.tensor([bad], device="cuda"))
    assert torch.isnan(out["scale"]).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 3, 5])
def test_clip_in_place(kind, shift):
    """One product in fp32 and one rounding, whatever the alignment; nothing around it."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    for n in (1, 6, 300, 2048, 70001):
        buf = some([n + 16], [kind], n)[0]
        keep, view = buf.clone(), buf[shift:shift + n]
        for f in (0.3333, 1.0, 0.0, -2.5):
            want = (view.float() * f).to(view.dtype)
            plp.clip_grads([view], torch.tensor([f], device="cuda"))
            assert torch.equal(view, want)
            view.copy_(keep[shift:shift + n])
        assert torch.equal(buf, keep)


def test_clipped_norm_is_the_limit():
    require_gpu()
    import rl_policy_gradient_amd as plp
    grads = some([4000, 333, 20000], ["f32", "f32", "f32"], 5, 1.0)
    table = plp.grad_table(grads)
    first = plp.grad_norm(table, max_norm=2.5)
    plp.clip_grads(table, first["scale"])
    after = float(plp.grad_norm(table)["norm"])
    # each element one rounding, the scale one, eps beside a norm above 100
    assert abs(after - 2.5) <= 2.5 * (3 * U + 1e-6 / 100)


@pytest.mark.parametrize("sizes", [[900, 0, 3000], [70001, 90000, 5] + [33] * 300], ids=len)
def test_what_a_workspace_holds_and_two_streams(sizes):
    """The same results whatever the workspace held, and from two calls at once."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    table = plp.grad_table(some(sizes, ["f32", "bf16", "f32"] * (len(sizes) // 3 + 1)))
    run = lambda **kw: plp.grad_norm(table, max_norm=0.01, norms=True, **kw)  # noqa: E731
    want = run()
    same = lambda r: all(torch.equal(r[k], want[k]) for k in want)  # noqa: E731
    for byte in (0x00, 0x7f, 0xff):
        assert same(run(workspace=torch.full((1 << 20,), byte, dtype=torch.uint8, device="cuda"))), byte
    sides, got = (torch.cuda.Stream(), torch.cuda.Stream()), []
    for side in sides:
        side.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        with torch.cuda.stream(sides[i % 2]):
            got.append(run())
    for side in sides:
        torch.cuda.current_stream().wait_stream(side)
    assert all(map(same, got))


def test_a_tensor_twice_and_overlap():
    require_gpu()
    import rl_policy_gradient_amd as plp
    g = some([500], ["f32"])[0]
    a, b = float(plp.grad_norm([g, g])["norm"]), float(plp.grad_norm([g])["norm"])
    assert abs(a - math.sqrt(2) * b) <= 3 * U * a
    for pair in ([g, g], [g[:300], g[299:]], [g[10:20], g]):
        with pytest.raises(ValueError, match="overlaps"):
            plp.clip_grads(plp.grad_table(pair), torch.ones(1, device="cuda"))
    plp.clip_grads(plp.grad_table([g[:300], g[300:], g[5:5]]), torch.full((1,), 2.0, device="cuda"))


def test_refuses():
    require_gpu()
    import rl_policy_gradient_amd as plp
    g = some([64, 64], ["f32", "bf16"])
    table = plp.grad_table(g)
    with pytest.raises(ValueError, match="grad_scale"):
        plp.grad_norm(table, grad_scale=2.0)
    with pytest.raises(ValueError, match="grad_scale"):
        plp.grad_norm(table, grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="GPU"):
        plp.grad_norm(table, grad_scale=torch.ones(1))
    with pytest.raises(ValueError, match="scale"):
        plp.clip_grads(table, 0.5)
    with pytest.raises(plp.PlpError, match="max_norm"):
        plp.grad_norm(table, max_norm=-1.0)
    with pytest.raises(plp.PlpError, match="eps"):
        plp.grad_norm(table, eps=float("nan"))
    with pytest.raises(plp.PlpError, match="overlap"):
        plp.grad_norm(table, out={"norm": g[0][:1]})
    with pytest.raises(plp.PlpError, match="overlap"):
        plp.clip_grads(table, g[0][3:4])
    with pytest.raises(ValueError, match="contiguous"):
        plp.grad_table([torch.zeros(4, 4, device="cuda").t()])
    with pytest.raises(ValueError, match="dtype"):
        plp.grad_table([torch.zeros(4, dtype=torch.float16, device="cuda")])
    with pytest.raises(ValueError, match="empty list"):
        plp.grad_norm([])
    with pytest.raises(ValueError, match="workspace too small"):
        plp.grad_norm(table, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    g[0].data = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="build it again"):
        plp.grad_norm(table)


def test_a_tensor_past_32_bits():
    require_gpu()
    import rl_policy_gradient_amd as plp
    n = 2 ** 32 + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, 12345, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, n - 2, n - 1]
    for i, k in enumerate(at):
        g[k] = float(i + 1)
    small = torch.tensor([3.0], device="cuda")
    out = plp.grad_norm([g, small], max_norm=1.0, eps=0.0, norms=True)
    assert near(float(out["norm"]), math.sqrt(204 + 9)) and near(float(out["norms"][0]), math.sqrt(204))
    assert float(out["norms"][1]) == 3.0
    plp.clip_grads([g], torch.tensor([0.5], device="cuda"))
    assert [float(g[k]) for k in at] == [0.5 * (i + 1) for i in range(len(at))]


def test_captured_with_the_step():
    """norm -> factor -> AdamW in one graph, replayed with new gradients between
    eager calls; the norm's memory is separate for each."""
    require_gpu()
    import rl_policy_gradient_amd as plp

    def make():
        p = some([3000, 50], ["f32", "f32"], 1, 1.0)
        g = some([3000, 50], ["f32", "f32"], 2, 1.0)
        adam = plp.adamw_table(p, g, [plp.adamw_state(x) for x in p])
        table, step = plp.grad_table(g), torch.ones(1, dtype=torch.int64, device="cuda")

        def run():
            r = plp.grad_norm(table, max_norm=1.0, norms=True)
            plp.adamw_step(adam, lr=1e-2, step=step, grad_scale=r["scale"])
            plp.clip_grads(table, r["scale"])
            return r

        return p, g, step, run

    pe, ge, se, run_e = make()
    pc, gc, sc, run_c = make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_c()
    for i in range(4):
        for a, b in zip(ge, gc):
            a.mul_(3.0 + i)
            b.copy_(a)
        want = run_e()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)
        assert all(torch.equal(a, b) for a, b in zip(pe + ge, pc + gc))
        se += 1
        sc += 1
