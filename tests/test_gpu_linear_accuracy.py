"""How exactly the dense layer's sums are formed, seen on operands of one sign.

Bounds.  Tensor memory adds 16 terms at a time and cuts off.  A product of two bf16
has 16 bits; while the sum is no more than 2^8 times a term, all of them lie in its 24,
and a step loses less than a unit of 2^-23 of what has been summed so far, on average
half of the whole: a pass of d terms at most d / 32 * 2^-23 of its sum S.  Behind that
bits of the products are cut off too, so that long passes lose more (measured 1.7 times
that bound at 65536 terms); no result is formed in passes of more than 4096.  A result
in FP32 and the sums into accum are formed in passes of d = 1024 terms on pairs of SMs
(256 for gradients of up to 2048 tokens), 256 on single SMs, what is rounded to bf16 in
passes of 4096.  The sums of p passes are FP32 additions, each off by 2^-24 of what has
been summed, half of S on average: p / 2 * 2^-24.  Joining the blocks of a cluster,
scale and result are at most 6 roundings of 2^-24 more.  One pass of all the terms of
these cases is past the bound: at least k / 45 * 2^-23, measured, against
(d / 32 + p / 4 + 3) * 2^-23.  What FP32 multiply-adds sum (one token) is at most 32 terms a
lane, 5 steps over the lanes and 8 warps: (32 + 5 + 8) * 2^-24.

A result's rounding to bf16, at most half a step, is without a sign: the mean over n
elements is off by no more than six standard deviations, 6 * 2^-8 / sqrt(3 n), beyond
what the passes lose."""
import math

import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import test_gpu_linear as base  # noqa: E402

BF16, FP32, D64 = torch.bfloat16, torch.float32, torch.float64
UNIT = 2.0 ** -23


@pytest.fixture(autouse=True)
def quiet(cuda_device):
    nsg.build()
    torch.cuda.set_device(0)
    yield
    assert nsg.device_error() == 0


def positive(seed, shape):
    return base.normal(seed, shape).abs()


def passes(k, depth, blocks=1):
    """The bound above, of sums of k terms in passes of `depth`, shared out to `blocks` blocks."""
    each = math.ceil(k / blocks)
    return (min(each, depth) / 32 + math.ceil(each / depth) / 4 + 3) * UNIT


def within(got, want, bound):
    off = ((got.to(D64) - want).abs() / want).max()
    assert float(off) <= bound, (float(off), bound)


# tokens, out_features: tiles of 256 x 256 and 256 x 128 on pairs of SMs, 128 x 128 on single ones, whose blocks share the
# terms out, few tokens
@pytest.mark.parametrize("T,N,depth,blocks", [(2048, 2048, 1024, 1), (2048, 1024, 1024, 1), (1024, 1024, 256, 2),
                                              (512, 1024, 256, 4), (40, 4096, 256, 4)])
@pytest.mark.parametrize("K", [1024, 8192, 16384])
def test_results_in_fp32(T, N, K, depth, blocks):
    x, w = positive(1, (T, K)), positive(2, (N, K))
    if K <= 1024:   # whichever kernel takes so few terms
        depth, blocks = 1024, 1
    within(nsg.linear(x, w, out_dtype=FP32), x.to(D64) @ w.to(D64).T, passes(K, depth, blocks))


def test_one_token_in_fp32():
    x, w = positive(1, (1, 8192)), positive(2, (1000, 8192))
    within(nsg.linear(x, w, out_dtype=FP32), x.to(D64) @ w.to(D64).T, 46 / 2 * UNIT)


@pytest.mark.parametrize("N,K,depth,blocks", [(2048, 2048, 1024, 1), (2048, 1024, 1024, 1), (1024, 1024, 256, 2)])
@pytest.mark.parametrize("T", [2048, 8192, 16384])
def test_sums_into_accum(N, K, T, depth, blocks):
    x, dout = positive(1, (T, K)), positive(2, (T, N))
    accum = torch.empty(N * K, device="cuda")
    nsg.linear_grad(accum, dout, x, None, (0, N, K), overwrite=True, dx=False)
    if T <= 2048:
        depth, blocks = 256, 1
    within(accum.view(N, K), dout.to(D64).T @ x.to(D64), passes(T, depth, blocks))


@pytest.mark.parametrize("T,N,K", [(2048, 2048, 4096), (2048, 2048, 16384), (300, 9000, 66000)])
def test_results_in_bf16_have_no_more_of_a_bias(T, N, K):
    """The sums' accuracy, which the results' own rounding hides element by element."""
    spread = 1 + torch.rand((T, 1), generator=torch.Generator().manual_seed(3)).cuda()
    x, w = (positive(1, (T, K)).float() * spread).to(BF16), positive(2, (N, K))
    want = x.to(D64) @ w.to(D64).T
    bound = passes(K, 4096) + 6 * 2.0 ** -8 / math.sqrt(3 * want.numel())
    for y in (nsg.linear(x, w), nsg.linear_grad(None, x, None, w.T.contiguous())):   # dx of the layer turned round
        assert abs(float(((y.to(D64) - want) / want).mean())) <= bound
