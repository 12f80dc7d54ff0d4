"""Norm and rotation of heads where a call is seldom tried: pairs that turn backwards."""
import math

import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layer_forms as forms  # noqa: E402
import test_gpu_layers as base  # noqa: E402

FP32, D64 = torch.float32, torch.float64


@pytest.fixture(autouse=True)
def quiet(cuda_device):
    nsg.build()
    torch.cuda.set_device(0)
    yield
    assert nsg.device_error() == 0


@pytest.mark.parametrize("sign", [1, -1])
def test_far_positions_either_way(sign):
    """Frequencies of either sign lose nothing but their last bits.

    Bound of the angle: the frequency in turns is off by 2^-52 of itself (the turn's own rounding and the quotient's)
    and, in steps of 2^-64, by one step: position * (f 2^-52 + 2 pi 2^-64) radians, on both elements of a pair; the rest as
    in any rotation."""
    freq, axis = nsg.rotary_frequencies(64)
    pos = torch.tensor([0, 1, 1 << 20, (1 << 31) - 1, 1 << 35, (1 << 40) + 12345], dtype=torch.int64, device="cuda")
    x = base.normal(1, (6, 2, 64), 1.0, FP32)
    y = nsg.norm_rotary(x, None, pos, sign * freq, axis, norm=False)[0]
    cos, sin = (torch.from_numpy(v).cuda() for v in base._exact_rotation(pos.cpu().tolist(), sign * freq))
    want = forms.turned(x.to(D64), cos, sin, False)
    off = pos.double()[:, None] * (torch.from_numpy(freq).cuda() * 2.0 ** -52 + 2 * math.pi * 2.0 ** -64)
    bound = (math.pi + 3) * 2.0 ** -22 + 2 * torch.cat([off, off], 1)[:, None]
    base.close(y, want, bound * x.abs().amax(2, keepdim=True).double())
    back = nsg.norm_rotary_grad(x, None, None, None, pos, -sign * freq, axis, norm=False)[0]   # the gradient turns back
    base.close(back, want, bound * x.abs().amax(2, keepdim=True).double())
