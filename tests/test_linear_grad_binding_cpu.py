"""Arguments of linear_grad that one gradient alone has no use for, over stand-ins."""
import pytest

import newton_schulz_fp32_gb300 as nsg

torch = pytest.importorskip("torch")
from test_layer_ops_cpu import machine  # noqa: E402,F401

BF16 = torch.bfloat16


@pytest.mark.parametrize("x,weight", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("activation", ["gelu", None])
@pytest.mark.parametrize("dx", [False, True])
def test_pre_is_looked_at_for_the_slope_alone(machine, x, weight, activation, dx):  # noqa: F811
    """A bias's gradient with neither x nor weight beside it takes any pre; so do calls without an activation."""
    if dx and not weight:
        return
    m = machine
    accum, dout = m.tensor(torch.zeros(64)), m.tensor(torch.zeros(5, 4, dtype=BF16))
    pre = m.tensor(torch.zeros(5, 8, dtype=BF16))
    nsg.linear_grad(accum, dout, m.tensor(torch.zeros(5, 8, dtype=BF16)) if x else None,
                    m.tensor(torch.zeros(4, 8, dtype=BF16)) if weight else None, None, (0, 1, 4), dx=dx,
                    activation=activation, pre=pre)
    assert [c[0] for c in m.layer_calls] == ["linear_grad"]
    if dx and activation:
        with pytest.raises(ValueError, match="pre must be"):
            nsg.linear_grad(accum, dout, None, m.tensor(torch.zeros(4, 8, dtype=BF16)), activation=activation,
                            pre=m.tensor(torch.zeros(5, 9, dtype=BF16)))
