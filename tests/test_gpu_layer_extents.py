"""The layer operators at the far ends of their extents: parameters behind element 2^31
of accum, very many tokens, features or heads.  Bounds as in test_gpu_linear and
test_gpu_layers."""
import math

import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layer_forms as forms  # noqa: E402
import test_gpu_layers as heads  # noqa: E402
import test_gpu_linear as base  # noqa: E402

BF16, FP32, D64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(autouse=True)
def quiet(cuda_device):
    nsg.build()
    torch.cuda.set_device(0)
    yield
    assert nsg.device_error() == 0
    torch.cuda.empty_cache()


def test_parameters_behind_element_2_to_the_31():
    T, K, N, first = 130, 72, 40, (1 << 31) + 12
    elements = first + N * K + N + 64
    accum = torch.empty(elements, device="cuda")
    tail = accum[first - 8:]
    tail.copy_(base.normal(1, (len(tail),), 0.1, FP32))
    old = tail.clone()
    x, dout = base.normal(2, (T, K)), base.normal(3, (T, N), 0.1)
    nsg.linear_grad(accum, dout, x, None, (first, N, K), (first + N * K, 1, N), dx=False)
    _, _, dw, ew, db, eb = base.grad_form(dout, x, base.normal(4, (N, K)), None, None)
    g, e = torch.cat([dw.reshape(-1), db]), torch.cat([ew.reshape(-1), eb])
    want = old.to(D64)
    want[8:8 + len(g)] += g
    bound = torch.zeros_like(want)
    bound[8:8 + len(g)] = e * 1.01 + 2.0 ** -23 * (want.abs() + old.abs())[8:8 + len(g)]
    base.close(tail, want, bound)
    q, d = heads.normal(5, (9, 3, 64), 1.0, FP32), heads.normal(6, (9, 3, 64), 0.1, FP32)
    near = torch.zeros(64, device="cuda")
    args = dict(scale=0.5, overwrite=True)
    nsg.norm_rotary_grad(d, q, accum=near, q_param=(0, 1, 64), **args)
    nsg.norm_rotary_grad(d, q, accum=accum, q_param=(first, 1, 64), **args)
    assert torch.equal(accum[first:first + 64], near)


@pytest.mark.parametrize("T,K,N", [(1, 1 << 22, 3), (3, 1 << 20, 5), (5, 8, 1 << 20), (1 << 20, 8, 8), ((1 << 20) + 3, 9, 1)])
def test_long_and_narrow_layers(T, K, N):
    x, w = base.normal(1, (T, K)), base.normal(2, (N, K), 1 / math.sqrt(K))
    bias = base.normal(3, (N,), 0.5)
    want, bound, *_ = base.forward_form(x, w, bias, "silu", None, 0.0, None, 0, FP32)
    base.close(nsg.linear(x, w, bias, "silu", out_dtype=FP32), want, bound)
    dout = base.normal(4, (T, N), 0.1)
    accum = torch.zeros(N * K + N, device="cuda")
    dx = nsg.linear_grad(accum, dout, x, w, (0, N, K), (N * K, 1, N))
    want, bound, dw, ew, db, eb = base.grad_form(dout, x, w, None, None)
    base.close(dx, want, bound, "dx")
    v = torch.cat([dw.reshape(-1), db])
    base.close(accum, v, torch.cat([ew.reshape(-1), eb]) * 1.01 + 2.0 ** -23 * v.abs(), "accum")


@pytest.mark.parametrize("T,H,D", [(1, 1 << 18, 8), (1 << 18, 1, 8), (2, 70000, 20)])
def test_many_heads_and_many_tokens(T, H, D):
    freq, axis = nsg.rotary_frequencies(D)
    pos = heads.positions_of(1, T, 1)
    x = heads.normal(2, (T, H, D), 1.0, FP32)
    cos, sin = forms.rotation(pos, freq, axis)
    want = forms.heads_forward(x, None, True, 1e-6, cos, sin, False)
    heads.close(nsg.norm_rotary(x, None, pos, freq, axis)[0], want, heads.forward_bound(x, None, True, 1e-6, cos, want, FP32))
    d = heads.normal(3, (T, H, D), 0.1, FP32)
    accum = torch.zeros(D, device="cuda")
    dx = nsg.norm_rotary_grad(d, x, positions=pos, inv_freq=freq, axis=axis, accum=accum, q_param=(0, 1, D))[0]
    want, dw = forms.heads_backward(d, x, None, True, 1e-6, cos, sin, False)
    size = forms.turned(d.to(D64), cos, -sin, False).abs()
    r = 1 / torch.sqrt((x.to(D64) ** 2).mean(2, keepdim=True) + 1e-6)
    e = (math.pi + 3) * 2.0 ** -22 * size.amax(2, keepdim=True)
    n = x.to(D64).abs() * r
    mean, en = (size * n).mean(2, keepdim=True), (D + 12) * 2.0 ** -24
    bound = r * (e + n * (e * n).mean(2, keepdim=True) + 2 * en * (size + n * mean))
    heads.close(dx, want, bound * 1.01 + 1.01 * 2.0 ** -24 * (want.abs() + bound))
    e_dw = (en * size * n + e * n).sum((0, 1)) + 2800 * 2.0 ** -24 * (size * n).sum((0, 1))
    heads.close(accum, dw, e_dw * 1.01 + 2.0 ** -23 * dw.abs())
