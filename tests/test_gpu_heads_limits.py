"""Norm and rotation of heads where a call is seldom tried: pairs that turn backwards,
and tokens that are none in calls without a rotation."""
import math

import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layer_forms as forms  # noqa: E402
import test_gpu_layers as base  # noqa: E402

BF16, FP32, D64 = torch.bfloat16, torch.float32, torch.float64


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


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dim,axes", [(64, 1), (67, 1), (128, 3), (256, 2)])
def test_tokens_that_are_none_without_a_rotation(dim, axes, dtype):
    """A padded batch's norms: zeros, no part in the weight's gradient, whatever lies there."""
    T = 45
    x, d = base.normal(1, (T, 3, dim), 1.0, dtype), base.normal(2, (T, 3, dim), 0.1, dtype)
    w = (1 + base.normal(3, (dim,), 0.2, FP32)).to(dtype)
    pos = base.positions_of(4, T, axes, dtype=torch.int64 if axes > 1 else torch.int32)
    gone = torch.zeros(T, dtype=torch.bool, device="cuda")
    gone[[0, 9, 44]] = True
    pos[gone, axes - 1] = -3
    bad, bad_d = x.clone(), d.clone()
    bad[gone], bad_d[gone] = math.nan, math.inf
    want = nsg.norm_rotary(x, None, q_weight=w)[0].masked_fill(gone[:, None, None], 0.0)
    got, other = nsg.norm_rotary(bad, bad[:, :1], pos, q_weight=w, k_weight=w)
    assert torch.equal(got, want) and torch.equal(other, want[:, :1])
    assert torch.equal(nsg.norm_rotary(bad, None, pos, norm=False)[0], x.masked_fill(gone[:, None, None], 0.0))
    still = d.masked_fill(gone[:, None, None], 0.0)   # tokens whose gradient is 0 add 0 to the weight's
    one, two = torch.zeros(dim, device="cuda"), torch.zeros(dim, device="cuda")
    a = nsg.norm_rotary_grad(still, x, q_weight=w, accum=one, q_param=(0, 1, dim))[0]
    b = nsg.norm_rotary_grad(bad_d, bad, positions=pos, q_weight=w, accum=two, q_param=(0, 1, dim))[0]
    assert torch.equal(a, b) and torch.equal(one, two) and not bool(b[gone].any())
    assert torch.equal(nsg.norm_rotary_grad(bad_d, None, positions=pos, norm=False)[0], still)
