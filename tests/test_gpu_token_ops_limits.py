"""The loss calls at the end of a vocabulary's range.

Rows of V = 2^31 - 1 zeros: every probability is 1 / V.  The sum of V ones is
exact while it is below 2^24, and rounds at most 16 times on its way to one
block's total: log S, about 21.5, is off by at most 16 u + 4 u 21.5 < 7e-6
(u = 2^-24).  A gradient g (1[v = y] - 1 / V) is then off by parts in 10^5,
which does not move its bf16 rounding from that of the exact value."""
import math

import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu
V = (1 << 31) - 1


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    nsg.build()
    return t


def check_rows(torch, z, y, g):
    """z[t] = g[t] (1[v = y[t]] - 1 / V), element by element."""
    for t in range(len(y)):
        at = float(z[t, y[t]])
        assert at == float(torch.tensor(g[t]).bfloat16())
        other = torch.tensor(-g[t] / V).bfloat16().cuda()
        z[t, y[t]] = other
        step = 1 << 28
        assert all(bool((z[t, a:a + step] == other).all()) for a in range(0, V, step))


def test_losses_of_the_largest_vocabulary(torch):
    """Two rows, the second starting off 16 bytes; targets first and last."""
    z = torch.zeros((2, V), dtype=torch.bfloat16, device="cuda")
    y = [V - 1, 0]
    targets = torch.tensor(y, device="cuda")
    logp = nsg.token_logprobs(z, targets).tolist()
    assert all(abs(x + math.log(V)) <= 7e-6 for x in logp)
    ones = torch.ones(2, device="cuda")
    got = nsg.policy_loss(z, targets, ones, ones, dlogits=z)
    assert got["dlogits"].data_ptr() == z.data_ptr() and float(got["stats"][0]) == -2.0
    check_rows(torch, z, y, [-1.0, -1.0])
    z.zero_()
    got = nsg.preference_loss(z, targets.flip(0), torch.tensor([0, 1, 2], device="cuda"), beta=0.5, dlogits=z)
    assert abs(float(got["margins"][0])) <= 0.5 * 14e-6
    check_rows(torch, z, y[::-1], [-0.25, 0.25])
    z.zero_()
    got = nsg.policy_loss(z, targets, ones, 0 * ones, dlogits=z.fill_(1))   # no row takes part: zeros
    assert all(int(z[t].count_nonzero()) == 0 for t in range(2))
    assert nsg.device_error() == 0
