"""Dropout and the norm and rotation of heads on a GPU, against the formulas in
64 bits.

Bounds.  Dropout: whole draws, so the mask is exact; a kept value is one FP32
product, one FP32 sum and one rounding to the type.  Norm: the sum of squares
of d <= 256 terms is off by d * 2^-24 relative at most, half that for its root,
the root and two products 4 units more: (d / 2 + 6) * 2^-24 of |n|.  Rotation:
cos and sin are off by 2^-23 each (their argument, a fraction of a turn in
FP32, by 2^-25 of up to half a turn: 2^-24 * pi), so a turned value by
(pi + 3) * 2^-23 * (|a| + |b|), and by the 2^-53 of the frequency times the
position, which is nothing here.  Gradients: the mean of g w n is a sum of d
terms: d * 2^-24 * sum |g w n| / d.  The weight's gradient sums tokens x heads
terms in FP32, in pieces of at most c terms that are then added in pairs of
few levels: with c <= 2048 terms in a row, (2048 + 700) * 2^-24 * S bounds it."""
import math

import numpy as np
import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layer_forms as forms  # noqa: E402

BF16, FP32, D64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(autouse=True)
def quiet(cuda_device):
    nsg.build()
    torch.cuda.set_device(0)
    yield
    assert nsg.device_error() == 0


def normal(seed, shape, spread=1.0, dtype=BF16):
    gen = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(shape, generator=gen)).to(dtype).cuda()


def generator(seed=77, step=2):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def close(got, want, bound, what=""):
    off = (got.to(D64) - want).abs() - bound
    bad = ~(off <= 1e-30)
    assert not bool(bad.any()), (what, int(bad.sum()), tuple(bad.nonzero()[0].tolist()), float(off.max()))


# ------------------------------------------------------------------ dropout

def dropout_form(x, res, rate, rng, site):
    y = x.to(D64) * forms.keep(*x.shape, rate, rng, site, "cuda") if rate else x.to(D64)
    s = y if res is None else y + res.to(D64)
    return s, 2.0 ** -23 * (y.abs() + s.abs()) + 1.01 * forms.HALF_STEP[x.dtype] * s.abs()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (2, 9), (5, 64), (33, 100), (7, 768), (300, 1001),
                                       (2, 4104), (1, 70000), (1025, 16)])
@pytest.mark.parametrize("rate,residual", [(0.1, False), (0.5, True), (0.0, True), (65535 / 65536, False)])
def test_dropout(rows, cols, dtype, rate, residual):
    x, rng = normal(rows + cols, (rows, cols), 1.0, dtype), generator(rows * 7 - 1000, cols)
    res = normal(3, (rows, cols), 1.0, dtype) if residual else None
    y = nsg.dropout(x, rate, rng, 6, res)
    assert y.dtype == dtype
    close(y, *dropout_form(x, res, rate, rng, 6))
    assert torch.equal(y, nsg.dropout(x, rate, rng, 6, res))


def test_known_draws():
    """The first words that the paper's authors publish for Philox4x32-10: counter and key all zeros, all ones."""
    for seed, step, site, row, group, words in (
            (0, 0, 0, 0, 0, (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),):
        bits = forms.draws(row + 1, 8 * (group + 1), seed, step, site)[row, 8 * group:]
        assert [int(bits[2 * i]) | int(bits[2 * i + 1]) << 16 for i in range(4)] == list(words)
    x = torch.ones((1, 8), device="cuda")
    rng = generator(0, 0)
    for j, w in enumerate((0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)):
        for half in range(2):
            bit = w >> 16 * half & 0xFFFF
            at = 2 * j + half
            assert float(nsg.dropout(x, bit / 65536, rng)[0, at]) > 0
            assert float(nsg.dropout(x, (bit + 1) / 65536, rng)[0, at]) == 0


def test_seeds_steps_and_sites_differ():
    x = torch.ones((64, 512), device="cuda")
    base = nsg.dropout(x, 0.5, generator(1, 1), 1)
    seen = [base]
    for rng, site in ((generator(2, 1), 1), (generator(1, 2), 1), (generator(1, 1), 2), (generator(1 + (1 << 40), 1), 1),
                      (generator(-1, 1), 1), (generator(1, 1), 0xFFFFFFFF)):
        y = nsg.dropout(x, 0.5, rng, site)
        for other in seen:   # 32768 fair draws agree in half of them, +- 6 standard deviations
            assert abs(float((y == other).float().mean()) - 0.5) < 6 * 0.5 / math.sqrt(x.numel())
        seen.append(y)
    assert torch.equal(base, nsg.dropout(x, 0.5, generator(1, 1 + (1 << 32)), 1))   # the step's low 32 bits


def test_dropout_in_place_strides_and_values_left_out():
    for dtype in (BF16, FP32):
        for shift in (0, 1, 8):
            whole, rng = normal(1, (50, 140), 1.0, dtype), generator()
            keep, x = whole.clone(), whole[:, shift:shift + 100]
            res = normal(2, (50, 113), 1.0, dtype)[:, shift:shift + 100]
            want = nsg.dropout(x.contiguous(), 0.3, rng, 1, res.contiguous())
            assert torch.equal(nsg.dropout(x, 0.3, rng, 1, res), want)
            assert nsg.dropout(x, 0.3, rng, 1, res, out=x) is x
            assert torch.equal(x, want) and torch.equal(whole[:, :shift], keep[:, :shift])
            assert torch.equal(whole[:, shift + 100:], keep[:, shift + 100:])
            mine = res.contiguous()
            assert torch.equal(nsg.dropout(keep[:, shift:shift + 100], 0.3, rng, 1, mine, out=mine), want)
    x = torch.full((8, 64), float("nan"), device="cuda")
    y = nsg.dropout(x, 0.5, generator(), 1)
    assert torch.equal(torch.isnan(y), forms.keep(8, 64, 0.5, generator(), 1, "cuda") != 0)
    assert bool((y[~torch.isnan(y)] == 0).all())
    assert nsg.dropout(torch.empty((0, 8), device="cuda"), 0.5, generator()).shape == (0, 8)
    z = normal(3, (4, 6, 32))
    assert torch.equal(nsg.dropout(z, 0.5, generator()), nsg.dropout(z.view(24, 32), 0.5, generator()).view(4, 6, 32))


def test_dropout_offsets_past_32_bits():
    far = (1 << 31) + 16
    room = torch.zeros(far * 2 + 64, dtype=BF16, device="cuda")
    x = room.as_strided((3, 40), (far, 1))
    x.copy_(normal(1, (3, 40)))
    close(nsg.dropout(x, 0.2, generator()), *dropout_form(x, None, 0.2, generator(), 0))


# ------------------------------------------------------------------ norm and rotation

def turns(dim, rot, axes, interleaved=False, own=False):
    if rot == 0:
        return None, None
    pairs = rot // 2
    sections = [pairs * (i + 1) // axes - pairs * i // axes for i in range(axes)]
    return nsg.rotary_frequencies(rot, 10000.0, sections, own)


def positions_of(seed, T, axes, far=1 << 14, gone=0.0, dtype=torch.int64):
    gen = torch.Generator().manual_seed(seed)
    p = torch.randint(0, far, (T, axes), generator=gen)
    if gone:
        drop = torch.rand(T, generator=gen) < gone
        p[drop, torch.randint(0, axes, (int(drop.sum()),), generator=gen)] = -1 - torch.randint(0, 5, (int(drop.sum()),))
    return p.to(dtype).cuda()


def forward_bound(x, w, norm, eps, cos, want, dtype):
    d = x.shape[2]
    n = forms.heads_forward(x, w, norm, eps, None, None, False).abs()
    e = (d / 2 + 6) * 2.0 ** -24 * n if norm else 0 * n
    if cos is not None:   # what a pair shares, wherever its partner is
        e = e + (e.amax(2, keepdim=True) + (math.pi + 3) * 2.0 ** -22 * n.amax(2, keepdim=True))
    return e * 1.01 + 1.01 * forms.HALF_STEP[dtype] * (want.abs() + e)


HEADS = [(1, 1, 1, 1, 0, 1), (1, 1, 1, 2, 2, 1), (5, 3, 1, 7, 4, 1), (9, 4, 2, 40, 40, 2), (33, 12, 12, 64, 64, 1),
         (17, 8, 2, 80, 60, 3), (130, 6, 3, 96, 48, 1), (1, 32, 8, 128, 128, 1), (257, 32, 8, 128, 128, 3),
         (70, 5, 1, 128, 64, 2), (40, 3, 2, 255, 254, 4), (64, 2, 1, 256, 256, 8), (3000, 4, 1, 64, 64, 1)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,H,G,D,rot,axes", HEADS)
def test_norm_rotary(T, H, G, D, rot, axes, norm, interleaved, dtype):
    packed = normal(T + D, (T, H + 2 * G, D), 1.5, dtype)
    q, k = packed[:, :H], packed[:, H:H + G]
    qw = (1 + normal(2, (D,), 0.3, FP32)).to(dtype) if norm else None
    freq, axis = turns(D, rot, axes)
    pos = positions_of(5, T, axes, gone=0.2 if T > 3 else 0.0, dtype=torch.int32 if D % 3 else torch.int64)
    kept = packed.clone()
    a, b = nsg.norm_rotary(q, k, pos if rot else None, freq, axis, interleaved, norm, qw, None, 1e-5)
    assert torch.equal(packed, kept)
    cos, sin = forms.rotation(pos, freq, axis) if rot else (None, None)
    off = ((pos < 0).any(1) if rot else torch.zeros(T, dtype=torch.bool, device="cuda"))[:, None, None]
    for got, x, w in ((a, q, qw), (b, k, None)):
        want = forms.heads_forward(x, w, norm, 1e-5, cos, sin, interleaved)
        bound = forward_bound(x, w, norm, 1e-5, cos, want, dtype)
        close(got, torch.where(off, 0.0, want), bound)
        assert not bool(got[off[:, 0, 0]].any())
    # in place, and one group alone, have the same bits
    nsg.norm_rotary(q, k, pos if rot else None, freq, axis, interleaved, norm, qw, None, 1e-5, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(packed[:, H + G:], kept[:, H + G:])
    only = nsg.norm_rotary(kept[:, H:H + G], None, pos if rot else None, freq, axis, interleaved, norm, None, eps=1e-5)
    assert only[1] is None and torch.equal(only[0], b)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,H,G,D,rot,axes", HEADS)
def test_norm_rotary_grad(T, H, G, D, rot, axes, norm, interleaved, dtype):
    packed, douts = normal(T + D, (T, H + 2 * G, D), 1.5, dtype), normal(T + D + 1, (T, H + G, D), 0.1, dtype)
    q, k, dq, dk = packed[:, :H], packed[:, H:H + G], douts[:, :H], douts[:, H:]
    qw = (1 + normal(2, (D,), 0.3, FP32)).to(dtype) if norm else None
    kw = (1 + normal(3, (D,), 0.3, FP32)).to(dtype) if norm and D % 2 else None
    freq, axis = turns(D, rot, axes)
    pos = positions_of(5, T, axes, gone=0.2 if T > 3 else 0.0)
    accum = normal(4, (4 * D + 3,), 1.0, FP32)
    old = accum.clone()
    table = np.array([(0, D + D // 2, 2), (D + D // 2, 3 * D, 2 + D + D // 2 + D // 3)], dtype=nsg.PART_DTYPE)
    params = dict(accum=accum, q_param=(0, 1, D), k_param=(2 * D, D, 1), parts=table, scale=0.5) if norm else {}
    args = (pos if rot else None, freq, axis, interleaved, norm, qw, kw, 1e-5)
    a, b = nsg.norm_rotary_grad(dq, q if norm else None, dk, k if norm else None, *args, **params)
    cos, sin = forms.rotation(pos, freq, axis) if rot else (None, None)
    on = ~((pos < 0).any(1) if rot else torch.zeros(T, dtype=torch.bool, device="cuda"))[:, None, None]
    sums = []
    for got, d, x, w in ((a, dq, q, qw), (b, dk, k, kw)):
        d, x = torch.where(on, d.to(D64), 0.0), torch.where(on, x.to(D64), 1.0)
        want, dw = forms.heads_backward(d, x, w, norm, 1e-5, cos, sin, interleaved)
        g = (d if cos is None else forms.turned(d, cos, -sin, interleaved)).abs()
        e = (math.pi + 3) * 2.0 ** -22 * g.amax(2, keepdim=True) * (cos is not None)
        if norm:
            r = 1 / torch.sqrt((x * x).mean(2, keepdim=True) + 1e-5)
            n, top = x.abs() * r, 1.0 if w is None else float(w.abs().max())
            mean = (g * n).mean(2, keepdim=True) * top
            en = (D + 12) * 2.0 ** -24
            # each term's own relative error and what the turned gradient's adds
            e_dw = (en * g * n + e * n).sum((0, 1)) + 2800 * 2.0 ** -24 * (g * n).sum((0, 1))
            e = r * (top * e + n * top * (e * n).mean(2, keepdim=True) + 2 * en * (top * g + n * mean))
            sums.append((dw, e_dw))
        close(got, want, e * 1.01 + 1.01 * forms.HALF_STEP[dtype] * (want.abs() + e))
    if norm:
        def flat(t):
            return torch.cat([t[s:s + e - b] for b, e, s in table.tolist()])
        new, before = flat(accum).to(D64), flat(old).to(D64)
        for off, (dw, e) in ((0, sums[0]), (2 * D, sums[1])):
            v = before[off:off + D] + 0.5 * dw
            close(new[off:off + D], v, 0.5 * e * 1.01 + 2.0 ** -23 * (v.abs() + before[off:off + D].abs()), "weight")
        assert torch.equal(flat(accum)[D:2 * D], flat(old)[D:2 * D])
        again = old.clone()
        nsg.norm_rotary_grad(dq, q, dk, k, *args, **dict(params, accum=again))
        assert torch.equal(again, accum)
        nsg.norm_rotary_grad(dq, q, dk, k, *args, **dict(params, accum=again, overwrite=True))
        v = 0.5 * torch.cat([sums[0][0], sums[1][0]])
        e = 0.5 * torch.cat([sums[0][1], sums[1][1]])
        close(torch.cat([flat(again)[:D], flat(again)[2 * D:]]), v, e * 1.01 + 2.0 ** -23 * v.abs())
    # in place of dout, and of x, the same bits
    x2, d2 = packed.clone(), douts.clone()
    r = nsg.norm_rotary_grad(d2[:, :H], q if norm else None, d2[:, H:], k if norm else None, *args, dq_out=d2[:, :H],
                             dk_out=d2[:, H:])
    assert torch.equal(r[0], a) and torch.equal(r[1], b) and torch.equal(d2[:, :H], a)
    if norm:
        nsg.norm_rotary_grad(dq, x2[:, :H], dk, x2[:, H:H + G], *args, dq_out=x2[:, :H], dk_out=x2[:, H:H + G])
        assert torch.equal(x2[:, :H], a) and torch.equal(x2[:, H:H + G], b)


def test_far_positions():
    """Positions up to 2^31 and past it: the angle's error stays that of the frequency's last bit."""
    freq, axis = nsg.rotary_frequencies(64)
    pos = torch.tensor([0, 1, 1 << 20, (1 << 20) + 1, (1 << 31) - 1, 1 << 35], dtype=torch.int64, device="cuda")
    x = normal(1, (6, 2, 64), 1.0, FP32)
    y = nsg.norm_rotary(x, None, pos, freq, axis, norm=False)[0]
    cos, sin = (torch.from_numpy(v).cuda() for v in _exact_rotation(pos.cpu().tolist(), freq))
    want = forms.turned(x.to(D64), cos, sin, False)
    far = pos.double()[:, None, None] * 2.0 ** -52
    close(y, want, ((math.pi + 3) * 2.0 ** -22 + 2 * far) * x.abs().amax(2, keepdim=True).double())


def _exact_rotation(positions, freq):
    """In rational arithmetic modulo a turn (pi to 60 digits)."""
    from fractions import Fraction
    turn = 2 * Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)
    a = [[float((Fraction(p) * Fraction(float(f))) % turn) for f in freq] for p in positions]
    return np.cos(np.array(a)), np.sin(np.array(a))


def test_layouts_of_heads():
    """Heads before tokens, batches, rows that do not start on 16 bytes, an expanded tensor."""
    freq, axis = nsg.rotary_frequencies(64)
    x = normal(1, (3, 20, 64))                      # heads x tokens x dim
    pos = positions_of(2, 20, 1)
    want = nsg.norm_rotary(x.transpose(0, 1).contiguous(), None, pos, freq, axis)[0]
    assert torch.equal(nsg.norm_rotary(x.transpose(0, 1), None, pos, freq, axis)[0], want)
    out = torch.empty_like(x).transpose(0, 1)
    assert nsg.norm_rotary(x.transpose(0, 1), None, pos, freq, axis, q_out=out)[0] is out and torch.equal(out, want)
    batch = normal(3, (4, 5, 3, 64))
    y = nsg.norm_rotary(batch, batch[:, :, :1], pos.view(4, 5), freq, axis)
    assert y[0].shape == (4, 5, 3, 64) and y[1].shape == (4, 5, 1, 64) and torch.equal(y[0][:, :, :1], y[1])
    odd = normal(4, (20, 3, 67))[:, :, 1:65]
    got = nsg.norm_rotary(odd, None, pos, freq, axis)[0]
    same = nsg.norm_rotary(odd.contiguous(), None, pos, freq, axis)[0]
    assert float((got.float() - same.float()).abs().max()) <= 2.0 ** -7 * float(same.float().abs().max())
    one = normal(5, (1, 1, 64))
    y = nsg.norm_rotary(one.expand(20, 3, 64), None, pos, freq, axis)[0]
    assert torch.equal(y[:, 0], y[:, 2])
    nothing = torch.empty((0, 3, 64), dtype=BF16, device="cuda")
    assert nsg.norm_rotary(nothing, None, pos[:0], freq, axis)[0].shape == (0, 3, 64)
    accum = torch.ones(64, device="cuda")
    nsg.norm_rotary_grad(nothing, nothing, None, None, pos[:0], freq, axis, accum=accum, q_param=(0, 1, 64),
                         overwrite=True)
    assert not bool(accum.any())


def test_no_tokens_on_several_axes():
    freq, axis = nsg.rotary_frequencies(64, sections=[8, 12, 12])
    nothing, pos = (torch.empty((0, *n), dtype=t, device="cuda") for n, t in (((3, 64), BF16), ((3,), torch.int64)))
    accum = torch.ones(64, device="cuda")
    assert nsg.norm_rotary(nothing, None, pos, freq, axis)[0].shape == (0, 3, 64)
    assert nsg.norm_rotary_grad(nothing, nothing, None, None, pos, freq, axis, accum=accum,
                                q_param=(0, 1, 64))[0].shape == (0, 3, 64)
    assert bool((accum == 1).all())


def test_tokens_that_are_none_may_hold_anything():
    freq, axis = nsg.rotary_frequencies(128)
    T = 40
    pos = positions_of(1, T, 1)
    gone = torch.zeros(T, dtype=torch.bool, device="cuda")
    gone[[0, 7, 39]] = True
    pos[gone] = -100
    x, d = normal(2, (T, 4, 128)), normal(3, (T, 4, 128), 0.1)
    bad, bad_d = x.clone(), d.clone()
    bad[gone], bad_d[gone] = float("nan"), float("inf")
    w = (1 + normal(4, (128,), 0.1, FP32)).to(BF16)
    y, z = (nsg.norm_rotary(v, None, pos, freq, axis, q_weight=w)[0] for v in (x, bad))
    assert torch.equal(y, z) and not bool(z[gone].any())
    one, two = torch.zeros(128, device="cuda"), torch.zeros(128, device="cuda")
    a = nsg.norm_rotary_grad(d, x, None, None, pos, freq, axis, q_weight=w, accum=one, q_param=(0, 1, 128))[0]
    b = nsg.norm_rotary_grad(bad_d, bad, None, None, pos, freq, axis, q_weight=w, accum=two, q_param=(0, 1, 128))[0]
    assert torch.equal(a, b) and torch.equal(one, two) and not bool(b[gone].any())
    pos[:] = -1
    two.fill_(5.0)
    b = nsg.norm_rotary_grad(bad_d, bad, None, None, pos, freq, axis, q_weight=w, accum=two, q_param=(0, 1, 128),
                             overwrite=True)[0]
    assert not bool(b.any()) and not bool(two.any())


def test_elements_behind_the_pairs_stay_apart():
    """An infinite or NaN element that is not turned changes no other."""
    freq, axis = nsg.rotary_frequencies(64)
    for dtype, dim in ((BF16, 96), (FP32, 80), (BF16, 67)):
        pos = positions_of(1, 6, 1)
        x = normal(2, (6, 3, dim), 1.0, dtype)
        clean = nsg.norm_rotary(x, None, pos, freq, axis, norm=False)[0]
        back = nsg.norm_rotary_grad(x, None, None, None, pos, freq, axis, norm=False)[0]
        bad = x.clone()
        bad[:, :, 65] = float("inf")
        bad[:, :, dim - 1] = float("nan")
        keep = [i for i in range(dim) if i not in (65, dim - 1)]
        for got, want in ((nsg.norm_rotary(bad, None, pos, freq, axis, norm=False)[0], clean),
                          (nsg.norm_rotary_grad(bad, None, None, None, pos, freq, axis, norm=False)[0], back)):
            assert torch.equal(got[..., keep], want[..., keep]) and bool(torch.isnan(got[..., dim - 1]).all())
            assert bool(torch.isinf(got[..., 65]).all())


def test_streams_and_graphs():
    freq, axis = nsg.rotary_frequencies(64)
    x, d, pos = normal(1, (50, 4, 64)), normal(2, (50, 4, 64), 0.1), positions_of(3, 50, 1)
    accum, rng = torch.zeros(64, device="cuda"), generator()

    def calls():
        a = nsg.norm_rotary(x, None, pos, freq, axis)[0]
        b = nsg.norm_rotary_grad(d, x, None, None, pos, freq, axis, accum=accum, q_param=(0, 1, 64), overwrite=True)[0]
        return a, b, accum.clone(), nsg.dropout(x.view(50, 256), 0.5, rng)

    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = calls()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    pos0 = pos.clone()
    pos.add_(1)
    graph.replay()
    assert not torch.equal(held[0], want[0])
    pos.copy_(pos0)
    accum.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    r = nsg.norm_rotary(x, None, pos, freq, axis, stream=side)[0]
    side.synchronize()
    assert torch.equal(r, want[0])


def test_head_offsets_past_32_bits():
    far = (1 << 31) + 16
    room = torch.zeros(far * 2 + 256, dtype=BF16, device="cuda")
    x = room.as_strided((3, 2, 64), (far, 64, 1))
    x.copy_(normal(1, (3, 2, 64)))
    freq, axis = nsg.rotary_frequencies(64)
    pos = positions_of(3, 3, 1)
    want = nsg.norm_rotary(x.contiguous(), None, pos, freq, axis)[0]
    assert torch.equal(nsg.norm_rotary(x, None, pos, freq, axis)[0], want)
    nsg.norm_rotary(x, None, pos, freq, axis, q_out=x)
    assert torch.equal(x, want)
