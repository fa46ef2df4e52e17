"""A row of logits sampled at every address modulo 16 bytes, in batches of odd
row lengths and alone: the same token. Its log-probs are one rounding to fp32
of values that agree to 1e-13, so two roundings apart at most."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_sampling import DT, LIMITS, U, float32_default, logits  # noqa: F401

pytestmark = pytest.mark.gpu


def same(a, b, what):
    assert torch.equal(a["token"], b["token"]), what
    for k in ("logp", "kept_logp"):
        assert ((a[k].double() - b[k].double()).abs() <= 2 * U * b[k].double().abs() + 2e-13).all(), (what, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau,k,p,mp", LIMITS)
@pytest.mark.parametrize("V,peaked", [(5001, True), (31999, False), (257, False)])
def test_rows_at_any_address(V, peaked, tau, k, p, mp, dtype):
    require_gpu()
    import rl_policy_gradient_amd as plp
    kw = dict(temperature=tau, top_k=k, top_p=p, min_p=mp)
    z, u = (t.cuda() for t in logits(64, V, dtype, 31, peaked))
    batch = plp.sample_tokens(z, u, **kw)  # an odd V: consecutive rows lie at every address modulo 16
    for lead in range(0, 8, 3 if V > 30000 else 1):
        stride = -(-V // 8) * 8
        store = torch.zeros(64 * stride + 8, dtype=DT[dtype], device="cuda")
        moved = store.as_strided((64, V), (stride, 1), lead)
        moved.copy_(z)
        got = plp.sample_tokens(moved, u, **kw)
        same(got, batch, lead)
        one = plp.sample_tokens(moved[5:6], u[5:6], **kw)  # alone at the same address: the same bits
        for n in one:
            assert torch.equal(one[n], got[n][5:6]), (lead, n)
