"""The norm at every width of its row kernels, and at rows whose statistics
are extreme. Formulas and tolerances are test_gpu_layer_norm.py's."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_layer_norm import DT, float32_default, make  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H", [(1, 16), (5, 32), (9, 64), (300, 64)])
def test_rows_of_one_huge_value(N, H, dtype):
    """A row of one value whose product with rstd is past fp32: it has no
    deviation, so grad_x is rstd (c - mean(c)), and it adds nothing to
    grad_weight. The widths are ones at which some of the lanes that share a
    row have no element of it, and at which the mean is exact."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    x, w, _, gy = make(N, H, dtype, 3)
    x[::2] = 2.0 ** 120
    f = plp.layer_norm_fwd(x.cuda(), w.cuda())
    assert (f["mean"][::2] == 2.0 ** 120).all() and torch.isfinite(f["rstd"]).all() and (f["rstd"][::2] > 256).all()
    out = plp.layer_norm_bwd(gy.cuda(), x.cuda(), w.cuda(), f["rstd"], f["mean"])
    r, m = f["rstd"].double().cpu()[:, None], f["mean"].double().cpu()[:, None]
    xh, c = (x.double() - m) * r, gy.double() * w.double()
    gx = r * (c - c.mean(1, keepdim=True) - xh * (c * xh).mean(1, keepdim=True))
    gw = (gy.double() * xh).sum(0)
    D = (H / 64 + 16) * U
    size = r * (c.abs() + c.abs().mean(1, keepdim=True) + xh.abs() * (c * xh).abs().mean(1, keepdim=True))
    h = torch.finfo(DT[dtype]).eps / 2
    got = out["grad_x"].double().cpu()
    assert ((got - gx).abs() <= 2 * D * size + h * (gx.abs() + 2 * D * size)).all()
    tw = (N + 20) * U * (gy.double() * xh).abs().sum(0)
    assert ((out["grad_weight"].double().cpu() - gw).abs() <= tw + h * (gw.abs() + tw)).all()


LANES = [8, 16, 32, 64, 128, 192, 256, 320, 384, 512, 640, 768, 1024]  # that share a row, 16 elements each
WIDTHS = [h for below, n in zip([0] + LANES, LANES) for h in (16 * below + 1, 16 * n - 8, 16 * n - 1)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", WIDTHS + [128, 256, 300, 512, 5120, 6144, 10240, 16384, 16385, 16392])
def test_both_directions_at_every_width(H, dtype, rms):
    """The shortest and the longest rows of each width, whole numbers of 16
    bytes and not, some that fill it, and the first ones the row kernels do not take: one row,
    an odd number of them, and more than the backward has groups for.

    Additions in a row: a lane's 16, six within a wave and up to 16 waves, or
    H / 256 and eight in the kernels for longer rows; with the products, the
    quotient and the root around them D roundings. A column's sum takes at
    most two rows, then 32 in a workgroup, then 24 and 32 groups."""
    require_gpu()
    import rl_policy_gradient_amd as plp
    slots = max(1, 256 // next((n for n in LANES if 16 * n >= H), 256))
    D = (max(38, H / 256 + 8) + 12) * U
    h = torch.finfo(DT[dtype]).eps / 2
    for N in (1, 2 * slots + 1, (768 * slots if slots > 1 else 512) + 3):
        x, w, b, gy = (t.cuda() for t in make(N, H, dtype, 5 * N + H, offset=0.25))
        xd, wd, g = x.double(), w.double(), gy.double()
        f = plp.layer_norm_fwd(x, w, b, eps=1e-5, rms=rms)
        mu = torch.zeros_like(xd[:, :1]) if rms else xd.mean(1, keepdim=True)
        r = 1 / ((xd - mu).square().mean(1, keepdim=True) + 1e-5).sqrt()
        y = (xd - mu) * r * wd + b.double()
        tm = 0.0 * mu if rms else D * xd.abs().mean(1, keepdim=True)
        # rstd: half the relative error of the squares' sum, each deviation's own, and the square of the mean's
        rel = D + (0.0 if rms else 4 * U * (xd.abs() + mu.abs()).square().mean(1, keepdim=True).sqrt() * r + (tm * r) ** 2)

        def near(got, want, tol, what):
            assert got.shape == want.shape and not torch.isnan(got).any(), (N, what)
            off = ((got.double() - want).abs() - tol).max().item()
            assert off <= 0, (N, what, off)

        near(f["rstd"], r[:, 0], (rel * r)[:, 0], "rstd")
        if not rms:
            near(f["mean"], mu[:, 0], tm[:, 0], "mean")
        ty = wd.abs() * r * (tm + (xd - mu).abs() * (rel + 4 * U)) + 2 * U * (y.abs() + b.double().abs())
        near(f["y"], y, ty + h * (y.abs() + ty), "y")
        out = plp.layer_norm_bwd(gy, x, w, f["rstd"], f.get("mean"), rms=rms)
        r, mu = f["rstd"].double()[:, None], 0.0 if rms else f["mean"].double()[:, None]
        xh, c = (xd - mu) * r, g * wd
        mc = 0.0 if rms else c.mean(1, keepdim=True)
        gx = r * (c - mc - xh * (c * xh).mean(1, keepdim=True))
        size = c.abs() + (0.0 if rms else c.abs().mean(1, keepdim=True)) + xh.abs() * (c * xh).abs().mean(1, keepdim=True)
        tx = 2 * D * r * size
        near(out["grad_x"], gx, tx + h * (gx.abs() + tx), "grad_x")
        tw = (min(N, 90) + 6) * U * (g * xh).abs().sum(0)
        gw, gb = (g * xh).sum(0), g.sum(0)
        near(out["grad_weight"], gw, tw + h * (gw.abs() + tw), "grad_weight")
        tb = min(N, 90) * U * g.abs().sum(0)
        near(out["grad_bias"], gb, tb + h * (gb.abs() + tb), "grad_bias")
