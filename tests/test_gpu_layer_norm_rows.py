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
