"""The losses over more rows than SMs can hold at once: rows that are streamed
(304 and more of over 8 KiB without a gradient, and rows too long to be held),
by blocks of every width, odd lengths, strides and starts, masked rows.

The formulas in 64 bits and their bounds are those of test_gpu_losses: a
streaming block of W threads adds a row in 4 W sums, W >= 64, so V / 256 terms
one after the other at most, and joins them in at most 2 + 5 + W / 32 steps;
its reference m lies below the maximum by up to 8 / s, which adds no more than
40 u to log S (3 u 8 for the exponents, 16 u for log S and s (z_y - m)
themselves): within tol(V), whose terms are V / 128 + 64 and 4 log V + 16 u.  Calls
with and without the gradient take different kernels here, so each is held
against the formulas and not against the other."""
import math

import numpy as np
import pytest

import newton_schulz_fp32_gb300 as nsg
import test_gpu_losses as one

pytestmark = pytest.mark.gpu
U = one.U

MANY = [  # tokens, vocabulary, extra stride, first element
    (304, 4097, 0, 0), (305, 5003, 1, 3), (2047, 5003, 0, 0), (303, 8193, 0, 0), (305, 16391, 0, 5),
    (2047, 16391, 1, 0), (305, 50001, 0, 0), (2047, 50001, 3, 1), (305, 131072, 0, 0), (2047, 131072, 8, 0)]


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    nsg.build()
    return t


def inputs(torch, T, V, pad, off, dtype, s):
    """Logits, targets (some none) and a policy's inputs; what takes no part is NaN."""
    z, y = one.make_logits(torch, T, V, dtype, 7 * T + V, V + pad, off)
    adv, w, old, ref = one.policy_inputs(torch, T, z, y, s, T + V)
    y[::11] = -100
    out = (y < 0) | (w == 0)
    for t in (adv, old, ref):
        t[out] = math.nan
    z[out] = math.nan
    return z, y, adv, w, old, ref, out


@pytest.mark.parametrize("shape", MANY)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_of_many_rows(torch, shape, dtype):
    T, V, pad, off = shape
    for s, index in ((1.0, torch.int64), (0.8, torch.int32)):
        z, y = one.make_logits(torch, T, V, dtype, T + V, V + pad, off)
        y[::5] = -1
        z[::5] = math.nan
        y = y.to(index)
        got = nsg.token_logprobs(z, y, s)
        want, bound = one.logp64(torch, torch.where((y >= 0)[:, None], z, 0.0), y, float(np.float32(s)))
        assert bool(((got.double() - want).abs() <= bound).all()) and bool((got[y < 0] == 0).all())
        assert torch.equal(got, nsg.token_logprobs(z, y, s))
    assert nsg.device_error() == 0


def check_policy(torch, got, want, out, T, grad):
    logp, err, d, bound, stats, serr = want
    assert bool(((got["logp"].double() - logp).abs() <= err).all()) and bool((got["logp"][out] == 0).all())
    assert bool(((got["stats"].double() - stats).abs() <= serr + 2 * U * stats.abs()).all())
    if grad:
        assert bool(((got["dlogits"].double() - d).abs() <= bound).all()) and bool((got["dlogits"][out] == 0).all())
    else:
        assert got["dlogits"] is None


@pytest.mark.parametrize("shape", MANY)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_policy_loss_of_many_rows(torch, shape, dtype):
    T, V, pad, off = shape
    s = 1.25 if T % 2 else 1.0
    z, y, adv, w, old, ref, out = inputs(torch, T, V, pad, off, dtype, s)
    want = one.policy_reference(torch, z, y, adv, w, old, ref, 0.2, 0.3, 0.1, s)
    for grad in (True, False):
        got = nsg.policy_loss(z, y, adv, w, old, ref, 0.2, 0.3, 0.1, s, dlogits=grad)
        check_policy(torch, got, want, out, T, grad)
        again = nsg.policy_loss(z, y, adv, w, old, ref, 0.2, 0.3, 0.1, s, dlogits=grad)
        assert all(torch.equal(got[k], again[k]) for k in got if got[k] is not None)
    own = z.clone(memory_format=torch.contiguous_format)
    check_policy(torch, nsg.policy_loss(own, y, adv, w, old, ref, 0.2, 0.3, 0.1, s, dlogits=own), want, out, T, True)
    assert nsg.device_error() == 0


@pytest.mark.parametrize("shape", MANY)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_preference_loss_of_many_rows(torch, shape, dtype):
    T, V, pad, off = shape
    B = 5
    s = 0.8 if T % 2 else 1.0
    z, y, _, _, _, ref, out = inputs(torch, T, V, pad, off, dtype, s)
    y[out] = -100
    y = y.to(torch.int32 if T % 2 else torch.int64)
    offs, offsets = one.make_offsets(torch, T, B, T, "int64" if T % 2 else "int32")
    pw = torch.rand(B, device="cuda")
    pw[3] = 0
    want = one.preference_reference(torch, z, y, offs, ref, 0.1, 0.1, pw, s)
    logp, err, h, herr, d, bound, stats, staterr = want
    sure = bool((h.abs() > herr).logical_or(h == 0).all())
    for grad in (True, False):
        got = nsg.preference_loss(z, y, offsets, ref, 0.1, 0.1, pw, s, dlogits=grad)
        assert bool(((got["logp"].double() - logp).abs() <= err).all()) and bool((got["logp"][out] == 0).all())
        assert bool(((got["margins"].double() - h).abs() <= herr).all())
        near = (got["stats"].double() - stats).abs() <= staterr + 4 * U * stats.abs()
        assert bool(near[[0, 1, 3]].all()) and (not sure or bool(near[2]))
        if grad:
            assert bool(((got["dlogits"].double() - d).abs() <= bound).all()) and bool((got["dlogits"][out] == 0).all())
        again = nsg.preference_loss(z, y, offsets, ref, 0.1, 0.1, pw, s, dlogits=grad)
        assert all(torch.equal(got[k], again[k]) for k in got if got[k] is not None)
    own = z.clone(memory_format=torch.contiguous_format)
    mine = nsg.preference_loss(own, y, offsets, ref, 0.1, 0.1, pw, s, dlogits=own)["dlogits"]
    assert bool(((mine.double() - d).abs() <= bound).all())
    assert nsg.device_error() == 0


@pytest.mark.parametrize("shape,dtype", [((310, 500009, 0, 1), "fp32"), ((310, 900001, 1, 0), "bf16")])
def test_gradient_of_many_rows_too_long_to_be_held(torch, shape, dtype):
    """Two passes over each row by one block; also in place."""
    T, V, pad, off = shape
    z, y, adv, w, old, ref, out = inputs(torch, T, V, pad, off, dtype, 1.0)
    want = one.policy_reference(torch, z, y, adv, w, old, ref, 0.2, 0.3, 0.1, 1.0)
    check_policy(torch, nsg.policy_loss(z, y, adv, w, old, ref, 0.2, 0.3, 0.1), want, out, T, True)
    check_policy(torch, nsg.policy_loss(z, y, adv, w, old, ref, 0.2, 0.3, 0.1, dlogits=z), want, out, T, True)
    assert nsg.device_error() == 0
