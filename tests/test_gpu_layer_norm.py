"""The norm's forward and backward on the GPU against plain 64-bit formulas.

Tolerances count roundings. u = 2^-24 is half a step of fp32, eps_t / 2 half a
step of the output's type. A sum of H terms over 64 lanes takes at most
H / 64 + 6 additions in a row in any of the kernels' orders, so it is off by
at most that many u of the sum of magnitudes; with the handful of products
and the root around it, D = H / 64 + 16 roundings bound every statistic."""
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


def make(N, H, dtype, seed, offset=0.0, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, H, generator=g, dtype=torch.float64) * (0.2 + torch.rand(N, 1, generator=g)) + offset).to(DT[dtype])
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(DT[dtype])
    b = (0.2 * torch.randn(H, generator=g)).to(DT[dtype]) if bias else None
    gy = torch.randn(N, H, generator=g).to(DT[dtype])
    return x, w, b, gy


def ref_fwd(x, w, b, eps, rms):
    x, w = x.double(), w.double()
    mu = torch.zeros(x.shape[:-1] + (1,), dtype=torch.float64) if rms else x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - mu) * rstd * w + (0 if b is None else b.double())
    return y, mu[..., 0], rstd[..., 0]


def check(got, want, tol, what):
    off = (got.double().cpu() - want).abs() - tol
    assert not torch.isnan(got).any(), what
    assert off.max().item() <= 0, (what, off.max().item(), (got.double().cpu() - want).abs().max().item())


def fwd_tols(x, w, b, mu, rstd, y, dtype, rms):
    H = x.shape[-1]
    D = (H / 64 + 16) * U
    xd = x.double().abs()
    ax = xd.mean(-1, keepdim=True)
    tol_mu = D * ax                       # the mean: a sum and a division
    # rstd = (mean (x - mu)^2 + eps)^-1/2: half the relative error of the sum
    # of squares (D, and 2 u of each deviation), and the mean's own error,
    # which moves the mean square by its square only but each deviation by u |mu|
    var = 1 / rstd[..., None] ** 2
    rel = D + 4 * U * (xd + mu.abs()[..., None]).square().mean(-1, keepdim=True).sqrt() / var.sqrt() + tol_mu ** 2 / var
    if rms:
        tol_mu = torch.zeros_like(tol_mu)
        rel = D + 0 * rel
    wd = w.double().abs()
    r = rstd[..., None]
    dev = (x.double() - mu[..., None]).abs()
    ty = wd * r * (tol_mu + dev * (rel + 4 * U)) + 2 * U * y.abs() + (0 if b is None else 2 * U * b.double().abs())
    return ty + torch.finfo(DT[dtype]).eps / 2 * (y.abs() + ty), tol_mu[..., 0], (rel * r)[..., 0]


SIZES = [(1, 1), (1, 896), (3, 2), (5, 7), (2, 64), (4, 63), (7, 65), (33, 128), (257, 896), (19, 897), (6, 1000),
         (9, 2048), (5, 2056), (3, 4096), (2, 4100), (3, 8192), (2, 8200), (2, 16384), (1, 20001), (4099, 32)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H", SIZES)
def test_forward(N, H, dtype, rms):
    require_gpu()
    import rl_policy_gradient_amd as plp
    x, w, b, _ = make(N, H, dtype, 11 * N + H, bias=(N + H) % 3 != 0)
    y, mu, rstd = ref_fwd(x, w, b, 1e-5, rms)
    out = plp.layer_norm_fwd(x.cuda(), w.cuda(), None if b is None else b.cuda(), eps=1e-5, rms=rms)
    assert ("mean" in out) == (not rms)
    ty, tmu, tr = fwd_tols(x, w, b, mu, rstd, y, dtype, rms)
    check(out["y"], y, ty, "y")
    check(out["rstd"], rstd, tr, "rstd")
    if not rms:
        check(out["mean"], mu, tmu, "mean")


@pytest.mark.parametrize("H", [896, 1001, 9000])
def test_forward_large_mean(H):
    """A mean of 1000 beside deviations of 1: taken out before the squares."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    x, w, b, _ = make(6, H, "f32", 3, offset=1000.0)
    y, mu, rstd = ref_fwd(x, w, b, 1e-5, False)
    out = plp.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=1e-5)
    ty, tmu, tr = fwd_tols(x, w, b, mu, rstd, y, "f32", False)
    # the tolerance still says something: D 1000 rstd |w| <= 157 u 1000 * 5 * 2 = 0.1 of y's unit size
    assert ty.max() < 0.1
    check(out["y"], y, ty, "y")
    check(out["mean"], mu, tmu, "mean")
    check(out["rstd"], rstd, tr, "rstd")


def bwd_tols(x, w, gy, mu, rstd, gx, dtype, rms, groups_per):
    H = x.shape[-1]
    D = (H / 64 + 16) * U
    r, m = rstd.double()[:, None], mu.double()[:, None]
    xh = ((x.double() - m) * r).abs()
    c = (gy.double() * w.double()).abs()
    t = r * (c + (0 if rms else c.mean(-1, keepdim=True)) + xh * (c * xh).mean(-1, keepdim=True))
    tx = 2 * D * t
    h = torch.finfo(DT[dtype]).eps / 2
    # a column's sum: groups_per rows one after the other, then the groups
    tw = (groups_per + 4) * U * (gy.double().abs() * xh).sum(0)
    tb = groups_per * U * gy.double().abs().sum(0)
    return tx + h * (gx.abs() + tx), tw, tb, h


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H", SIZES + [(20000, 128), (3000, 896)])
def test_backward(N, H, dtype, rms):
    require_gpu()
    import rl_policy_gradient_amd as plp
    x, w, b, gy = make(N, H, dtype, 7 * N + H)
    _, mu, rstd = ref_fwd(x, w, b, 1e-5, rms)
    mu32, rstd32 = mu.float(), rstd.float()
    # the gradients from the fp32 statistics the call is given
    xd, wd, g = x.double(), w.double(), gy.double()
    r, m = rstd32.double()[:, None], (torch.zeros_like(mu32) if rms else mu32).double()[:, None]
    xh = (xd - m) * r
    c = g * wd
    gx = r * (c - (0 if rms else c.mean(-1, keepdim=True)) - xh * (c * xh).mean(-1, keepdim=True))
    gw, gb = (g * xh).sum(0), g.sum(0)
    out = plp.layer_norm_bwd(gy.cuda(), x.cuda(), w.cuda(), rstd32.cuda(), None if rms else mu32.cuda(), rms=rms)
    # at most 1024 additions in a row within a group, and over the groups
    tx, tw, tb, h = bwd_tols(x, w, gy, m[:, 0], rstd32, gx, dtype, rms, min(N, 1024) + 16)
    check(out["grad_x"], gx, tx, "grad_x")
    check(out["grad_weight"], gw, tw + h * (gw.abs() + tw), "grad_weight")
    check(out["grad_bias"], gb, tb + h * (gb.abs() + tb), "grad_bias")
    again = plp.layer_norm_bwd(gy.cuda(), x.cuda(), w.cuda(), rstd32.cuda(), None if rms else mu32.cuda(), rms=rms)
    for k in out:
        assert torch.equal(out[k], again[k]), k  # fixed order


@pytest.mark.parametrize("rms", [False, True])
def test_gradients_against_autograd_and_differences(rms):
    """The three gradients beside torch's own differentiation of the 64-bit
    forward, and beside central differences of it along random directions."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    N, H, eps = 12, 200, 1e-5
    x, w, b, gy = make(N, H, "f32", 5)
    out = plp.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=eps, rms=rms)
    got = plp.layer_norm_bwd(gy.cuda(), x.cuda(), w.cuda(), out["rstd"], out.get("mean"), rms=rms)
    leaves = [t.double().requires_grad_() for t in (x, w, b)]
    (ref_fwd(*leaves, eps, rms)[0] * gy.double()).sum().backward()
    for k, t in zip(("grad_x", "grad_weight", "grad_bias"), leaves):
        rel = (got[k].double().cpu() - t.grad).norm() / t.grad.norm()
        assert rel <= 40 * U, (k, rel)  # the forward's statistics, rounded, and the sums: under 40 roundings
    g = torch.Generator().manual_seed(1)
    f = lambda x, w, b: (ref_fwd(x, w, b, eps, rms)[0] * gy.double()).sum().item()  # noqa: E731
    base = [t.double() for t in (x, w, b)]
    for i, k in enumerate(("grad_x", "grad_weight", "grad_bias")):
        d = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        hi, lo = [list(base), list(base)]
        h = 1e-4
        hi[i], lo[i] = base[i] + h * d, base[i] - h * d
        num = (f(*hi) - f(*lo)) / (2 * h)
        ana = (got[k].double().cpu() * d).sum().item()
        # h^2 times a third derivative of order one, and the kernel's roundings
        assert abs(num - ana) <= 1e-5 * (got[k].double().cpu().abs() * d.abs()).sum().item(), (k, num, ana)


def test_parts_skipped_and_given_outputs():
    require_gpu()
    import rl_policy_gradient_amd as plp
    x, w, b, gy = (t.cuda() for t in make(40, 896, "bf16", 9))
    f = plp.layer_norm_fwd(x.view(5, 8, 896), w, b)
    assert f["y"].shape == (5, 8, 896) and f["rstd"].shape == (5, 8)
    whole = plp.layer_norm_bwd(gy, x, w, f["rstd"].view(-1), f["mean"].view(-1))
    for part in ("grad_x", "grad_weight", "grad_bias"):
        kw = {k: k == part for k in whole}
        one = plp.layer_norm_bwd(gy, x, w, f["rstd"].view(-1), f["mean"].view(-1), **kw)
        assert list(one) == [part] and torch.equal(one[part], whole[part])
    out = {"y": torch.empty_like(x), "rstd": torch.empty(40, device="cuda"), "mean": torch.empty(40, device="cuda")}
    f2 = plp.layer_norm_fwd(x, w, b, out=out)
    assert f2["y"] is out["y"] and torch.equal(f2["y"], f["y"].view(40, 896))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned_pointers_and_neighbours(dtype):
    """Tensors that start one element into their storage: the same values as
    aligned copies, and nothing outside y and grad_x is written."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    N, H = 21, 896
    x, w, b, gy = (t.cuda() for t in make(N, H, dtype, 4))
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    a = plp.layer_norm_fwd(x, w, b)
    store = torch.full((N * H + 2,), 7.0, dtype=DT[dtype], device="cuda")
    out = {"y": store[1:-1].view(N, H)}
    c = plp.layer_norm_fwd(off(x), off(w), off(b), out=out)
    assert store[0] == 7 and store[-1] == 7
    e = torch.finfo(DT[dtype]).eps  # two roundings of the output, and fp32 sums in another order
    assert ((a["y"].double() - c["y"].double()).abs() <= e * a["y"].double().abs() + 1e-5).all()
    g = plp.layer_norm_bwd(gy, x, w, a["rstd"], a["mean"])
    store.fill_(7.0)
    g2 = plp.layer_norm_bwd(off(gy), off(x), off(w), a["rstd"], a["mean"], out={"grad_x": store[1:-1].view(N, H)})
    assert store[0] == 7 and store[-1] == 7
    for k in g:
        d = (g[k].double() - g2[k].double()).abs()
        assert (d <= e * g[k].double().abs() + 1e-4).all(), k


def test_empty_and_constant_rows():
    require_gpu()
    import rl_policy_gradient_amd as plp
    w = torch.ones(16, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    f = plp.layer_norm_fwd(x, w, w)
    assert f["y"].shape == (0, 16)
    g = plp.layer_norm_bwd(x, x, w, f["rstd"], f["mean"])
    assert (g["grad_weight"] == 0).all() and (g["grad_bias"] == 0).all() and g["grad_x"].shape == (0, 16)
    x = torch.full((3, 16), 5.0, device="cuda")  # no deviation: y is the bias
    f = plp.layer_norm_fwd(x, w, 2 * w, eps=1e-5)
    assert (f["y"] == 2).all() and torch.allclose(f["rstd"], torch.full((3,), 1e-5 ** -0.5, device="cuda"))
    x[1, 3] = float("nan")  # stays in its row
    f = plp.layer_norm_fwd(x, w, 2 * w)
    assert torch.isnan(f["y"][1]).all() and (f["y"][[0, 2]] == 2).all()


def test_captured_and_replayed():
    require_gpu()
    import rl_policy_gradient_amd as plp
    x, w, b, gy = (t.cuda() for t in make(300, 896, "bf16", 2))
    f = plp.layer_norm_fwd(x, w, b)
    g = plp.layer_norm_bwd(gy, x, w, f["rstd"], f["mean"])
    out = {k: torch.empty_like(v) for k, v in {**f, **g}.items()}
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plp.layer_norm_fwd(x, w, b, out=out)
        plp.layer_norm_bwd(gy, x, w, out["rstd"], out["mean"], out=out, workspace=ws)
    for k in range(3):
        x.copy_(torch.randn(x.shape, device="cuda"))
        for v in out.values():
            v.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        f = plp.layer_norm_fwd(x, w, b)
        g = plp.layer_norm_bwd(gy, x, w, f["rstd"], f["mean"])
        for name, v in {**f, **g}.items():
            assert torch.equal(out[name], v), (k, name)


def test_other_stream():
    require_gpu()
    import rl_policy_gradient_amd as plp
    x, w, b, gy = (t.cuda() for t in make(2000, 896, "bf16", 6))
    torch.cuda.synchronize()
    want = plp.layer_norm_fwd(x, w, b)["y"]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = plp.layer_norm_fwd(x, w, b)["y"]
    s.synchronize()
    assert torch.equal(got, want)
    assert np.isfinite(want.float().sum().item())


def test_more_rows_than_one_launch_holds():
    """2^29 + 5 rows: 8 lanes a row, so more threads than a launch can have."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    N = 2 ** 29 + 5
    x = torch.empty(N, 1, dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16).copy_((torch.arange(N, device="cuda", dtype=torch.int32) % 0x0701 + 0x3c00).to(torch.int16)[:, None])
    w = torch.full((1,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = plp.layer_norm_fwd(x, w, eps=1.0, rms=True)
    for i in range(0, N, 2 ** 27):
        v = x[i:i + 2 ** 27, 0].double()
        r = (v * v + 1.0).rsqrt()
        # rstd: the square, the sum, the root and the quotient, half a step each; y: two products and the rounding
        assert ((out["rstd"][i:i + 2 ** 27].double() - r).abs() <= 4 * 2.0 ** -24 * r).all(), i
        y = 3.0 * v * r
        assert ((out["y"][i:i + 2 ** 27, 0].double() - y).abs() <= (2.0 ** -8 + 8 * 2.0 ** -24) * y.abs()).all(), i


def test_offsets_past_32_bits():
    """2.7e9 elements, forward and backward; whole-number gradients, so that
    grad_bias is exact."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    N, H = 3_000_001, 896
    g = torch.Generator().manual_seed(3)
    few = torch.randn(1009, H, generator=g).to(torch.bfloat16).cuda()
    gyf = torch.randint(-1, 2, (1009, H), generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(H, generator=g).to(torch.bfloat16).cuda()
    reps = -(-N // 1009)
    x, gy = few.repeat(reps, 1)[:N], gyf.repeat(reps, 1)[:N]
    out = plp.layer_norm_fwd(x, w)
    gr = plp.layer_norm_bwd(gy, x, w, out["rstd"], out["mean"])
    # the same rows in a small batch give the same bits
    small = plp.layer_norm_fwd(few, w)
    sgx = plp.layer_norm_bwd(gyf, few, w, small["rstd"], small["mean"])["grad_x"]
    for i in range(0, N, 1009 * 500):
        n = min(1009 * 500, N - i)
        at = torch.arange(n, device="cuda") % 1009
        for got, want in ((out["y"], small["y"]), (out["mean"], small["mean"]), (out["rstd"], small["rstd"]),
                          (gr["grad_x"], sgx)):
            assert torch.equal(got[i:i + n], want[at]), i
    last = N - (reps - 1) * 1009
    gb = gyf.double().sum(0) * (reps - 1) + gyf[:last].double().sum(0)
    assert torch.equal(gr["grad_bias"], gb.to(torch.bfloat16))
