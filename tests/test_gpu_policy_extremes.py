"""Policy terms whose ratio or divergence is past FP32's range.

The formulas in real numbers: r A = 0 for A = 0 however large r is, so such a
token adds nothing and its gradient is 0; exp(q) - q - 1 grows without bound
with q, so a target of probability 0 under the policy and not under the
reference has an infinite divergence, not an undefined one."""
import math

import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    nsg.build()
    return t


def inputs(torch, T, V):
    gen = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((T, V), generator=gen, device="cuda")
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    return z, y, torch.ones(T, device="cuda")


@pytest.mark.parametrize("T,V", [(4, 100), (400, 5003), (2, 500009)])
@pytest.mark.parametrize("grad", [True, False])
def test_a_ratio_past_the_range_without_an_advantage(torch, T, V, grad):
    z, y, w = inputs(torch, T, V)
    old = nsg.token_logprobs(z, y) - 200
    old[-1] += 200
    adv = torch.zeros(T, device="cuda")
    adv[-1] = 0.5
    got = nsg.policy_loss(z, y, adv, w, old, dlogits=grad)
    want = nsg.policy_loss(z[-1:], y[-1:], adv[-1:], w[-1:], old[-1:])
    assert abs(float(got["stats"][0]) - float(want["stats"][0])) < 1e-5 and float(got["stats"][3]) == 0
    if grad:
        assert int(got["dlogits"][:-1].count_nonzero()) == 0 and bool(torch.isfinite(got["dlogits"]).all())


def test_a_divergence_without_bound(torch):
    z, y, w = inputs(torch, 5, 300)
    z[2, y[2]] = -math.inf
    ref = torch.full((5,), -3.0, device="cuda")
    got = nsg.policy_loss(z, y, w, w, None, ref, kl_coef=0.1)
    assert float(got["stats"][2]) == math.inf and float(got["stats"][0]) == math.inf
    assert float(got["stats"][1]) == -5.0
    rows = [0, 1, 3, 4]
    assert bool(torch.isfinite(got["dlogits"][rows]).all())
    z[0] = math.nan                      # undefined stays undefined
    assert math.isnan(float(nsg.policy_loss(z, y, 0 * w, w)["stats"][0]))
