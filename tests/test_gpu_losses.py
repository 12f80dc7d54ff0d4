"""Target log-probabilities, the clipped policy loss and the preference loss
against the formulas in 64 bits on the same inputs.

Tolerances, derived from the arithmetic (u = 2^-24; s the logit scale, m the
row's maximum, x = s (z - m) <= 0):
* each e = 2^(x log2 e) carries the roundings of z - m, of the scale and of
  the product (3 u |x|) and the exponential's own error (2^-22 relative);
* S sums at most V / 128 terms one after the other and joins them by trees
  of at most 64 further steps: (V / 128 + 64) u;
* so log S, and logp = x_y - log S, are off by at most
      tol(V) = u (V / 128 + 64) + 2^-22 (log V + 4)   and 4 u (|x_y| + |log S|)
  (the terms' 3 u |x| weigh e / S, which keeps their sum below 3 u log V);
* the gradient g (1[y] - p): p is off by p (2 tol + 4 u |x|), g by
  d g / d logp times logp's error plus a few roundings, the output by one
  rounding of its type;
* sums over tokens are FP64, so the statistics carry the tokens' errors."""
import math

import numpy as np
import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    nsg.build()
    return t


def tol(V):
    return U * (V / 128 + 64) + 2.0 ** -22 * (math.log(V) + 4)


def kinds(torch):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}


def make_logits(torch, T, V, dtype, seed, stride=None, offset=0, spread=2.0):
    """T x V logits with the given row stride and first element, and targets;
    what lies between the rows is NaN."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    stride = stride or V
    store = torch.full((offset + T * stride + 16,), float("nan"), device="cuda").to(kinds(torch)[dtype])
    z = store[offset:offset + T * stride].view(T, stride)[:, :V]
    z.copy_(spread * torch.randn((T, V), generator=gen, device="cuda"))
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    if V > 8:
        z[:, V // 3] = -math.inf          # a forbidden word
        y = torch.where(y == V // 3, V // 2, y)
    z.scatter_add_(1, y[:, None], torch.full((T, 1), 4.0, device="cuda").to(z.dtype))
    return z, y


def softmax64(torch, z, s):
    """(log-probabilities, x = s (z - max)) in 64 bits."""
    x = z.double() * s
    x = x - x.max(1, keepdim=True).values
    return x - x.exp().sum(1, keepdim=True).log(), x


def logp64(torch, z, y, s):
    lp, x = softmax64(torch, z, s)
    at = y.long().clamp(min=0)[:, None]
    got, xy = lp.gather(1, at)[:, 0], x.gather(1, at)[:, 0]
    bound = tol(z.shape[1]) + 4 * U * (xy.abs() + (xy - got).abs())
    return torch.where(y >= 0, got, 0.0), bound


SHAPES = [  # tokens, vocabulary, extra stride, first element
    (1, 1, 0, 0), (3, 2, 0, 0), (5, 7, 0, 1), (4, 8, 0, 0), (9, 9, 2, 3), (33, 1000, 0, 0), (2, 1025, 0, 0),
    (65, 4096, 0, 0), (17, 5003, 0, 0), (3, 16384, 0, 0), (2, 16391, 0, 5), (40, 32768, 32, 0), (7, 50001, 0, 0),
    (1, 65537, 0, 0), (2, 70000, 1, 2), (1, 131072, 0, 0), (5, 131072, 0, 0), (200, 131072, 0, 0),
    (3, 200003, 0, 0), (2, 300007, 0, 1), (1, 600000, 0, 0)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_token_logprobs(torch, shape, dtype):
    T, V, pad, off = shape
    z, y = make_logits(torch, T, V, dtype, 3 * T + V, V + pad, off)
    for s, index in ((1.0, torch.int64), (0.7, torch.int32)):
        t = y.to(index)
        if T > 2:
            t[1] = -100
        got = nsg.token_logprobs(z, t, s)
        want, bound = logp64(torch, z, t, float(np.float32(s)))
        assert bool(((got.double() - want).abs() <= bound).all())
        assert T <= 2 or float(got[1]) == 0.0
        assert torch.equal(got, nsg.token_logprobs(z, t, s))
    assert nsg.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [5, 700, 40000, 300000])
def test_token_logprobs_of_special_rows(torch, dtype, V):
    z, y = make_logits(torch, 9, V, dtype, V)
    low = torch.finfo(z.dtype).min
    z[0] = -math.inf                       # nothing allowed
    z[1] = low                             # all at the type's lowest value: uniform
    z[2] = low
    z[2, V - 1] = 1.0                      # one word left
    y[2] = V - 1
    z[3, 2] = float("nan")
    z[4, 1] = math.inf
    z[5] = -math.inf
    z[5, V - 1] = -5.0                     # one word left, the last
    y[5] = V - 1
    y[6] = 0
    z[6, 0] = -math.inf                    # the target is forbidden
    z[7] = float("nan")
    y[7] = -1                              # not read
    z[8] = 3e38                            # large and equal: uniform
    got = nsg.token_logprobs(z, y).double().cpu()
    assert math.isnan(got[0]) and math.isnan(got[3]) and math.isnan(got[4])
    for k in (1, 8):
        assert abs(float(got[k]) + math.log(V)) <= tol(V) + 4 * U * math.log(V)
    assert float(got[2]) == 0.0 and float(got[5]) == 0.0
    assert float(got[6]) == -math.inf and float(got[7]) == 0.0


def policy_reference(torch, z, y, adv, w, old, ref, lo, hi, beta, s):
    """The formulas in 64 bits, and bounds."""
    on = (y >= 0) & (w != 0)
    lp, x = softmax64(torch, torch.where(on[:, None], z.double(), 0.0), s)
    at = y.long().clamp(min=0)[:, None]
    logp = torch.where(on, lp.gather(1, at)[:, 0], 0.0)
    xy = x.gather(1, at)[:, 0]
    err = tol(z.shape[1]) + 4 * U * (xy.abs() + (xy - logp).abs())
    w = torch.where(on, w.double(), 0.0)
    a = torch.where(on, adv.double(), 0.0)
    r = torch.ones_like(logp) if old is None else (logp - torch.where(on, old.double(), 0.0)).exp()
    free, held = r * a, r.clamp(1 - lo, 1 + hi) * a
    cut = free > held
    term = torch.where(cut, -held, -free)
    c = torch.where(cut, 0.0, -free)
    slope = r * a.abs()                       # d c / d logp, for the bound
    kl = torch.zeros_like(logp)
    if ref is not None:
        q = torch.where(on, ref.double(), 0.0) - logp
        kl = torch.expm1(q) - q
        c = c - beta * torch.expm1(q)
        slope = slope + beta * q.exp()
    c = w * c
    g = s * c
    p = lp.exp()
    hot = torch.zeros_like(p).scatter_(1, at, 1.0)
    d = torch.where(on[:, None], g[:, None] * (hot - p), 0.0)
    gerr = s * w.abs() * (slope * (err + 8 * U) + 4 * U * c.abs() / w.abs().clamp(min=1e-30))
    bound = gerr[:, None] * (hot + p) + g.abs()[:, None] * (p * (2 * tol(z.shape[1]) + 4 * U * x.abs().nan_to_num(posinf=0)) + 2 * U * hot)
    bound = bound + d.abs() * (2.0 ** -8 if z.dtype == torch.bfloat16 else 2 * U) + 1e-37
    stats = torch.stack([(w * (term + beta * kl)).sum(), (w * term).sum(), (w * kl).sum(), (w * cut).sum()])
    werr = (w.abs() * (slope + (0 if ref is None else 1) * ((torch.expm1(q) if ref is not None else a).abs() + 1)) * (err + 8 * U)).sum()
    tiny = 4 * U * (w.abs() * (term.abs() + kl.abs() * (1 + beta) + 1)).sum() + 1e-30
    return logp, err, d, bound, stats, werr + tiny


def policy_inputs(torch, T, z, y, s, seed, mask=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logp, _ = logp64(torch, z, y, s)
    moved = 0.3 * torch.randn(T, generator=gen, device="cuda")
    for edge in (math.log(0.8), math.log(1.3)):   # rounding would decide the branch on the edge
        moved = torch.where((moved - edge).abs() < 1e-2, moved + 4e-2, moved)
    old = (logp - moved.double()).float()
    ref = (logp + 0.3 * torch.randn(T, generator=gen, device="cuda").double()).float()
    adv = torch.randn(T, generator=gen, device="cuda")
    w = (torch.rand(T, generator=gen, device="cuda") >= mask).float() / max(1, T)
    return adv, w, old, ref


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_policy_loss(torch, shape, dtype):
    T, V, pad, off = shape
    s = 1.25 if T % 2 else 1.0
    z, y = make_logits(torch, T, V, dtype, 5 * T + V, V + pad, off)
    adv, w, old, ref = policy_inputs(torch, T, z, y, s, T + V)
    y = y.to(torch.int32 if T % 2 else torch.int64)
    if T > 4:
        y[3] = -100
    out = (y < 0) | (w == 0)
    for t in (adv, old, ref):
        t[out] = float("nan")              # what takes no part may hold anything
    z[out] = float("nan")
    for beta, o, r in ((0.1, old, ref), (0.0, old, None), (0.05, None, ref)):
        got = nsg.policy_loss(z, y, adv, w, o, r, 0.2, 0.3, beta, s)
        logp, err, d, bound, stats, serr = policy_reference(torch, z, y, adv, w, o, r, 0.2, 0.3, beta, s)
        assert bool(((got["logp"].double() - logp).abs() <= err).all())
        assert got["dlogits"].shape == z.shape and got["dlogits"].dtype == z.dtype
        assert bool(((got["dlogits"].double() - d).abs() <= bound).all())
        assert bool((got["dlogits"][out] == 0).all())
        assert bool(((got["stats"].double() - stats).abs() <= serr + 2 * U * stats.abs()).all())
        again = nsg.policy_loss(z, y, adv, w, o, r, 0.2, 0.3, beta, s)
        loss = nsg.policy_loss(z, y, adv, w, o, r, 0.2, 0.3, beta, s, dlogits=False)
        assert loss["dlogits"] is None
        for k in ("stats", "logp"):
            assert torch.equal(got[k], again[k]) and torch.equal(got[k], loss[k])
        assert torch.equal(got["dlogits"], again["dlogits"])
        if V <= 50001:
            own = z.clone(memory_format=torch.contiguous_format)
            mine = nsg.policy_loss(own, y, adv, w, o, r, 0.2, 0.3, beta, s, dlogits=own)["dlogits"]
            assert mine.data_ptr() == own.data_ptr()
            if z.is_contiguous() and z.data_ptr() % 16 == own.data_ptr() % 16:
                assert torch.equal(mine, got["dlogits"])
            else:   # another alignment sums in another order
                assert bool(((mine.double() - d).abs() <= bound).all())
    assert nsg.device_error() == 0


@pytest.mark.parametrize("pad_in,pad_out,off_in,off_out", [(0, 3, 0, 0), (8, 0, 0, 1), (1, 2, 3, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_rows_of_another_alignment(torch, pad_in, pad_out, off_in, off_out, dtype):
    T, V = 6, 4099
    z, y = make_logits(torch, T, V, dtype, 2, V + pad_in, off_in)
    adv, w, old, ref = policy_inputs(torch, T, z, y, 1.0, 3, 0.0)
    store = torch.full((off_out + T * (V + pad_out),), 7.0, device="cuda").to(z.dtype)
    d = store[off_out:].view(T, V + pad_out)
    got = nsg.policy_loss(z, y, adv, w, old, ref, 0.2, 0.3, 0.1, dlogits=d[:, :V])
    want = nsg.policy_loss(z, y, adv, w, old, ref, 0.2, 0.3, 0.1)
    assert torch.equal(got["dlogits"], want["dlogits"]) and bool((d[:, V:] == 7).all())
    assert bool((store[:off_out] == 7).all())


def test_policy_loss_of_extremes(torch):
    """Ratios and divergences that overflow stay with their tokens; rows of one
    word, forbidden targets."""
    V = 1000
    z, y = make_logits(torch, 6, V, "fp32", 3)
    z[4] = -math.inf
    z[4, 7] = 2.0
    y[4] = 7
    y[5] = 0
    z[5, 0] = -math.inf
    logp, _ = logp64(torch, z, y, 1.0)
    old = logp.float()
    ref = logp.float()
    old[0] -= 200.0                       # the ratio overflows: clipped for A > 0
    adv = torch.tensor([1.0, 0.0, -1.0, 2.0, 1.0, 1.0], device="cuda")
    old[5], ref[5] = -3.0, 0.0
    w = torch.ones(6, device="cuda")
    got = nsg.policy_loss(z, y, adv, w, old, None, 0.2, 0.2)
    assert abs(float(got["stats"][0]) - (-1.2 + 0 + 1 - 2 - 1 - 0)) < 1e-4
    d = got["dlogits"]
    assert bool(torch.isfinite(d).all()) and bool((d[0] == 0).all()) and bool((d[1] == 0).all())
    assert bool((d[4] == 0).all())        # p = 1 at the only word: g (1 - 1)
    assert float(got["stats"][3]) == 1.0 and float(got["logp"][5]) == -math.inf
    bad = y.clone()
    bad[2], bad[3] = V, 1 << 40
    got = nsg.policy_loss(z, bad, adv, w, old, None, 0.2, 0.2)
    assert nsg.device_error() == 17 and nsg.device_error() == 0
    assert bool((got["dlogits"][2:4] == 0).all()) and bool((got["logp"][2:4] == 0).all())


def preference_reference(torch, z, y, offsets, ref, beta, ls, pw, s):
    B = (len(offsets) - 1) // 2
    on = y >= 0
    lp, x = softmax64(torch, torch.where(on[:, None], z.double(), 0.0), s)
    at = y.long().clamp(min=0)[:, None]
    logp = torch.where(on, lp.gather(1, at)[:, 0], 0.0)
    xy = x.gather(1, at)[:, 0]
    err = torch.where(on, tol(z.shape[1]) + 4 * U * (xy.abs() + (xy - logp).abs()), 0.0)
    q = logp - (0.0 if ref is None else torch.where(on, ref.double(), 0.0))
    sums = torch.stack([q[a:b].sum() for a, b in zip(offsets[:-1], offsets[1:])])
    serr = torch.stack([err[a:b].sum() for a, b in zip(offsets[:-1], offsets[1:])])
    h = beta * (sums[:B] - sums[B:])
    herr = abs(beta) * (serr[:B] + serr[B:]) + 4 * U * h.abs()
    w = torch.full((B,), 1.0 / B, dtype=torch.float64, device=z.device) if pw is None else pw.double()
    F = torch.nn.functional
    loss = -(1 - ls) * F.logsigmoid(h) - ls * F.logsigmoid(-h)
    dh = torch.where(w == 0, 0.0, w * beta * (ls * torch.sigmoid(h) - (1 - ls) * torch.sigmoid(-h)))
    dherr = w.abs() * abs(beta) * (herr + 8 * U)
    c, cerr = torch.zeros_like(logp), torch.zeros_like(logp)
    for i in range(2 * B):
        k = slice(offsets[i], offsets[i + 1])
        c[k] = dh[i % B] * (1 if i < B else -1)
        cerr[k] = dherr[i % B]
    g = s * torch.where(on, c, 0.0)
    p = lp.exp()
    hot = torch.zeros_like(p).scatter_(1, at, 1.0)
    d = g[:, None] * (hot - p)
    bound = (s * cerr)[:, None] * (hot + p) + g.abs()[:, None] * (p * (2 * tol(z.shape[1]) + 4 * U * x.abs().nan_to_num(posinf=0)) + 4 * U * hot)
    bound = bound + d.abs() * (2.0 ** -8 if z.dtype == torch.bfloat16 else 2 * U) + 1e-37
    stats = torch.stack([(w * loss).sum(), (w * h).sum(), (w * (h > 0)).sum(), w.sum()])
    staterr = (w.abs() * (herr + 8 * U * (1 + loss))).sum()
    return logp, err, h, herr, d, bound, stats, staterr


def make_offsets(torch, T, B, seed, index):
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(0, T + 1, 2 * B + 1))
    if B > 1:
        cuts[2] = cuts[1]                  # an empty sequence
    return cuts.tolist(), torch.from_numpy(cuts.astype(np.int64 if index == "int64" else np.int32)).cuda()


@pytest.mark.parametrize("case", [  # tokens, pairs, vocabulary, extra stride, first element
    (2, 1, 3, 0, 0), (40, 2, 1000, 0, 0), (61, 5, 4099, 0, 1), (33, 1, 16384, 0, 0), (90, 8, 32768, 0, 0),
    (24, 3, 50001, 1, 0), (50, 2, 131072, 0, 0), (9, 2, 300007, 0, 0), (700, 300, 64, 0, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_preference_loss(torch, case, dtype):
    T, B, V, pad, off = case
    s = 0.8 if B % 2 else 1.0
    z, y = make_logits(torch, T, V, dtype, T + V, V + pad, off)
    offs, offsets = make_offsets(torch, T, B, T, "int64" if B % 2 else "int32")
    gen = torch.Generator(device="cuda").manual_seed(B)
    y = torch.where(torch.rand(T, generator=gen, device="cuda") < 0.25, -100, y)
    logp, _ = logp64(torch, z, y, s)
    ref = (logp + 0.5 * torch.randn(T, generator=gen, device="cuda").double()).float()
    ref[y < 0] = float("nan")
    z[y < 0] = float("nan")
    pw = torch.rand(B, generator=gen, device="cuda")
    if B > 1:
        pw[1] = 0
    for beta, ls, r, weights in ((0.1, 0.0, ref, None), (0.5, 0.1, ref, pw), (0.01, 0.5, None, pw)):
        got = nsg.preference_loss(z, y, offsets, r, beta, ls, weights, s)
        want = preference_reference(torch, z, y, offs, r, beta, ls, weights, s)
        logp, err, h, herr, d, bound, stats, staterr = want
        assert bool(((got["logp"].double() - logp).abs() <= err).all())
        assert bool(((got["margins"].double() - h).abs() <= herr).all())
        assert bool(((got["dlogits"].double() - d).abs() <= bound).all())
        assert bool((got["dlogits"][y < 0] == 0).all())
        sure = bool((h.abs() > herr).logical_or(h == 0).all())
        near = (got["stats"].double() - stats).abs() <= staterr + 4 * U * stats.abs()
        assert bool(near[[0, 1, 3]].all()) and (not sure or bool(near[2]))
        again = nsg.preference_loss(z, y, offsets, r, beta, ls, weights, s)
        loss = nsg.preference_loss(z, y, offsets, r, beta, ls, weights, s, dlogits=False)
        for k in ("stats", "logp", "margins"):
            assert torch.equal(got[k], again[k]) and torch.equal(got[k], loss[k])
        assert torch.equal(got["dlogits"], again["dlogits"])
        own = z.clone(memory_format=torch.contiguous_format)
        mine = nsg.preference_loss(own, y, offsets, r, beta, ls, weights, s, dlogits=own)["dlogits"]
        assert bool(((mine.double() - d).abs() <= bound).all())
    assert nsg.device_error() == 0


def test_preference_loss_far_margins_and_bad_offsets(torch):
    z, y = make_logits(torch, 8, 500, "fp32", 1)
    logp, _ = logp64(torch, z, y, 1.0)
    ref = logp.float()
    offsets = torch.tensor([0, 1, 2, 3, 4, 5, 6], device="cuda")
    ref[0] -= 5e4                          # margins of 5000, -5000 and 0: no overflow
    ref[1] += 5e4
    got = nsg.preference_loss(z, y, offsets, ref, 0.1, 0.1)
    h = got["margins"].double()
    assert abs(float(h[0]) - 5000) < 1e-2 and abs(float(h[1]) + 5000) < 1e-2 and abs(float(h[2])) < 1e-5
    want = (0.1 * 5000 + 0.9 * 5000 + math.log(2)) / 3
    assert abs(float(got["stats"][0]) - want) < 1e-2 and bool(torch.isfinite(got["dlogits"]).all())
    assert bool((got["dlogits"][6:] == 0).all())      # tokens of no sequence
    bad = torch.tensor([0, 3, 2, 9, 8], device="cuda")
    nsg.preference_loss(z, y, bad, ref, 0.1)
    assert nsg.device_error() == 18 and nsg.device_error() == 0


def test_gradients_against_differences(torch):
    """Both losses' gradients along random directions against central
    differences of the 64-bit losses."""
    T, V, B = 24, 65, 2
    z, y = make_logits(torch, T, V, "fp32", 8)
    z[:, V // 3] = -3.0
    y[5] = -1
    gen = torch.Generator(device="cuda").manual_seed(2)
    adv, w, old, ref = policy_inputs(torch, T, z, y, 1.1, 4)
    offs, offsets = make_offsets(torch, T, B, 3, "int64")
    d1 = nsg.policy_loss(z, y, adv, w, old, ref, 0.2, 0.3, 0.1, 1.1)["dlogits"].double()
    d2 = nsg.preference_loss(z, y, offsets, ref, 0.3, 0.1, None, 1.1)["dlogits"].double()
    f1 = lambda x: float(policy_reference(torch, x, y, adv, w, old, ref, 0.2, 0.3, 0.1, 1.1)[4][0])  # noqa: E731
    f2 = lambda x: float(preference_reference(torch, x, y, offs, ref, 0.3, 0.1, None, 1.1)[6][0])    # noqa: E731
    for _ in range(6):
        u = torch.randn((T, V), generator=gen, device="cuda").double()
        step = 1e-5
        for f, d in ((f1, d1), (f2, d2)):
            want = (f(z.double() + step * u) - f(z.double() - step * u)) / (2 * step)
            got = float((d * u).sum())
            assert abs(got - want) <= 1e-5 * float((d * u).abs().sum() + 1e-3)


def test_streams_graph_and_zero_tokens(torch):
    T, V = 30, 20000
    z, y = make_logits(torch, T, V, "bf16", 8)
    adv, w, old, ref = policy_inputs(torch, T, z, y, 1.0, 4)
    offsets = torch.tensor([0, 10, 15, 22, 30], device="cuda", dtype=torch.int32)
    calls = [lambda st: nsg.policy_loss(z, y, adv, w, old, ref, kl_coef=0.1, stream=st),
             lambda st: nsg.preference_loss(z, y, offsets, ref, stream=st),
             lambda st: {"logp": nsg.token_logprobs(z, y, stream=st)}]
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for st in (side, side.cuda_stream):
            got = call(st)
            side.synchronize()
            assert all(torch.equal(got[k], want[k]) for k in want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = call(None)
        for _ in range(2):
            for v in got.values():
                v.fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(got[k], want[k]) for k in want)
    e = torch.empty(0, device="cuda")
    got = nsg.policy_loss(z[:0], y[:0], e, e)
    assert bool((got["stats"] == 0).all()) and got["dlogits"].shape == (0, V)
    got = nsg.preference_loss(z[:0], y[:0], offsets[:1] * 0)
    assert bool((got["stats"] == 0).all()) and got["margins"].numel() == 0
    got = nsg.preference_loss(z, y, offsets[:1] * 0)          # tokens, but no pairs
    assert bool((got["stats"] == 0).all()) and bool((got["dlogits"] == 0).all())
    assert nsg.token_logprobs(z[:0], y[:0]).numel() == 0


def test_offsets_past_32_bits(torch):
    """Logits of more than 2^31 elements: the last rows are the right ones."""
    T, V = 16500, 131072
    z = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    z[T - 1, V - 1] = 10.0
    y = torch.full((T,), -1, device="cuda")
    y[T - 1], y[T - 2] = V - 1, 5
    got = nsg.token_logprobs(z, y).double()
    want = 10 - math.log(math.exp(10) + V - 1)
    assert abs(float(got[T - 1]) - want) <= tol(V) * 20 and abs(float(got[T - 2]) + math.log(V)) <= tol(V) * 20
    w = torch.ones(T, device="cuda")
    out = nsg.policy_loss(z, y, w, w, None, None, dlogits=z)["dlogits"]
    p = math.exp(want)
    assert abs(float(out[T - 1, V - 1]) + (1 - p)) <= 2.0 ** -8
    assert float(out[T - 3].abs().max()) == 0.0
