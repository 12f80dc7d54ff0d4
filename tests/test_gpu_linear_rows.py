"""Tokens that hold infinities or the ends of the type, and large products called one
behind the other.  Bounds as in test_gpu_linear."""
import math

import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import test_gpu_linear as base  # noqa: E402

BF16, FP32, D64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(autouse=True)
def quiet(cuda_device):
    nsg.build()
    torch.cuda.set_device(0)
    yield
    assert nsg.device_error() == 0


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("T,K,N", [(1, 520, 264), (2, 520, 264), (4, 520, 264), (5, 520, 264), (40, 520, 264), (300, 520, 264),
                                   (300, 521, 263), (2304, 2112, 2568)])
def test_infinities_and_the_ends_of_the_type(T, K, N, out):
    """A token with an infinity, with two, and one of the type's highest and lowest values: what the formula says of its
    row.  (Weights so small that no sum of the last leaves FP32.)"""
    x, w = base.normal(1, (T, K)), base.normal(2, (N, K), 1e-4)
    top = torch.finfo(BF16).max
    rows = {}
    for r, kind in ((0, "inf"), (T // 2, "both"), (T - 1, "end")):
        rows[r] = kind   # the last of them, where they are one
        x[r] = base.normal(3 + r, (K,))
        if kind == "end":
            x[r] = torch.where(x[r] < 0, -top, top)
        else:
            x[r, K // 3] = math.inf
            if kind == "both":
                x[r, K - 1] = -math.inf
    y = nsg.linear(x, w, out_dtype=out)
    want, bound, *_ = base.forward_form(x, w, None, None, None, 0.0, None, 0, out)
    for r, kind in rows.items():
        if kind == "end":
            base.close(y[r], want[r], bound[r])
        else:
            assert torch.equal(y[r].to(D64).nan_to_num(nan=7.0), want[r].nan_to_num(nan=7.0)) and not bool(y[r].isfinite().any())
    clean = [r for r in range(T) if r not in rows]
    if clean:
        base.close(y[clean], want[clean], bound[clean])


@pytest.mark.parametrize("T,K,N", [(2304, 2112, 2568), (4100, 1096, 4352), (8192, 2048, 2048)])
def test_large_products_repeat_themselves(T, K, N):
    """The same bits each time, one call behind the other, among other work."""
    x, w, dout = base.normal(1, (T, K)), base.normal(2, (N, K), 0.03), base.normal(3, (T, N), 0.1)
    pre = base.normal(4, (T, K))
    seen = None
    for i in range(6):
        accum = torch.zeros(N * K + N, device="cuda")
        y, u = nsg.linear(x, w, activation="silu", pre=True)
        dx = nsg.linear_grad(accum, dout, x, w, (0, N, K), (N * K, 1, N), activation="silu", pre=pre)
        got = (y, u, dx, accum)
        if i % 2:
            torch.cuda.synchronize()
        seen = seen or got
        assert all(torch.equal(a, b) for a, b in zip(got, seen))
