"""The dense layer and its gradients on a GPU, against the formulas in 64 bits.

Bounds.  A product's FP32 sum of k terms is formed 16 terms at a time, each
step losing at most an FP32 unit of the partial sum (the tensor cores cut off,
which is twice a rounding), so it is off by at most (k / 16 + 16) * 2^-23 * S
with S = sum |a b|.  A sum by FP32 additions one by one stays inside that too
but for sums of a few terms, which the 16 covers.  The epilogue: an activation
changes that error by at most its slope (1.13 for gelu, 1.1 for silu, 2 |u| for
relu2), and has its own: the exponential of h is off by (4 + |h|) units of
2^-23 at most, the division by 2, so the value by |y| (4 + |h|) 2^-22.
Bias, residual, dropout's factor and scale are one FP32 rounding each, the
result one half step of its type.  A slope is off by less than 2^-17 (its terms
are below 1.2, with the same errors, times at most |h| exp(-|h|) < 0.4)."""
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


def product_error(a, b):
    """Bound of the error of a @ b (64-bit values of bf16 tensors)."""
    return (a.shape[1] / 16 + 16) * 2.0 ** -23 * (a.abs() @ b.abs())


def sigmoid_argument(u, kind):
    return (1.6 * u * (1 + 0.0448 * u * u)).abs() if kind == "gelu" else u.abs()


def forward_form(x, w, bias, kind, residual, rate, rng, site, dtype):
    """(out, its bound, pre, its bound)."""
    a, b = x.to(D64), w.to(D64).T
    u, e = a @ b, product_error(a, b)
    if bias is not None:
        u = u + bias.to(D64)
        e = e + 2.0 ** -24 * u.abs()
    y, slope = forms.act(u, kind)
    top = {"relu2": 2 * (u.abs() + e), "gelu": 1.13, "silu": 1.1}.get(kind, 1.0)
    ey = e * top
    if kind not in (None, "none", "relu"):
        ey = ey + y.abs() * (4 + sigmoid_argument(u, kind)) * 2.0 ** -22
    if rate:
        k = forms.keep(*u.shape, rate, rng, site, u.device)
        y, ey = y * k, ey * k + 2.0 ** -23 * (y * k).abs()
    if residual is not None:
        y = y + residual.to(D64)
        ey = ey + 2.0 ** -24 * y.abs()
    half = forms.HALF_STEP
    return y, ey * 1.01 + half[dtype] * y.abs() * 1.01, u, e * 1.01 + half[BF16] * u.abs() * 1.01


def close(got, want, bound, what=""):
    off = (got.to(D64) - want).abs() - bound
    bad = ~(off <= 1e-30)
    assert not bool(bad.any()), (what, int(bad.sum()), tuple(bad.nonzero()[0].tolist()), float(off.max()))


SIZES = [(1, 1, 1), (1, 64, 64), (3, 7, 5), (2, 4096, 768), (16, 64, 512), (17, 1001, 763), (33, 200, 136),
         (64, 768, 1024), (100, 520, 72), (128, 64, 256), (129, 65, 257), (256, 1024, 640), (300, 2056, 512),
         (513, 136, 1000), (1, 14336, 260), (1030, 2064, 776), (2, 100, 14336)]
WAYS = [dict(), dict(bias=BF16, act="gelu", pre=True), dict(bias=FP32, act="silu", residual=True, rate=0.1),
        dict(act="relu", residual=True, out=FP32), dict(bias=BF16, act="relu2", pre=True, rate=0.5, out=FP32),
        dict(bias=BF16, act="gelu", pre=True, residual=True, rate=0.25)]


def forward_case(T, K, N, way, seed):
    x, w = normal(seed, (T, K)), normal(seed + 1, (N, K), 1 / math.sqrt(K))
    bias = normal(seed + 2, (N,), 0.5, way["bias"]) if "bias" in way else None
    out = way.get("out", BF16)
    residual = normal(seed + 3, (T, N), 1.0, out) if way.get("residual") else None
    return x, w, bias, residual, out


@pytest.mark.parametrize("way", range(len(WAYS)))
@pytest.mark.parametrize("T,K,N", SIZES)
def test_forward(T, K, N, way):
    way = WAYS[way]
    x, w, bias, residual, out = forward_case(T, K, N, way, 10 * T + K + N)
    rng, rate, kind = generator(), way.get("rate", 0.0), way.get("act")
    r = nsg.linear(x, w, bias, kind, residual, rate, rng, 9, out_dtype=out, pre=way.get("pre", False))
    y, u = r if way.get("pre") else (r, None)
    want, bound, pre, pre_bound = forward_form(x, w, bias, kind, residual, rate, rng, 9, out)
    assert y.dtype == out and y.shape == (T, N)
    close(y, want, bound, "out")
    if u is not None:
        assert u.dtype == BF16
        close(u, pre, pre_bound, "pre")


LARGE = [(2304, 2112, 2568), (4100, 1096, 4352), (70, 5000, 9000), (1500, 4608, 1160), (12000, 136, 520)]


@pytest.mark.parametrize("way", [0, 3, 5])
@pytest.mark.parametrize("T,K,N", LARGE)
def test_forward_of_many_tiles(T, K, N, way):
    """More tiles than pairs of SMs, sums in several pieces, results held while the next tile is formed."""
    way = WAYS[way]
    x, w, bias, residual, out = forward_case(T, K, N, way, T + K + N)
    rng, rate, kind = generator(), way.get("rate", 0.0), way.get("act")
    r = nsg.linear(x, w, bias, kind, residual, rate, rng, 9, out_dtype=out, pre=way.get("pre", False))
    y, u = r if way.get("pre") else (r, None)
    want, bound, pre, pre_bound = forward_form(x, w, bias, kind, residual, rate, rng, 9, out)
    close(y, want, bound, "out")
    if u is not None:
        close(u, pre, pre_bound, "pre")


def test_very_many_terms():
    """More terms of a bf16 result than are summed in one pass."""
    T, K, N = 300, 66000, 9000
    x, w, bias, _, _ = forward_case(T, K, N, WAYS[1], 1)
    want, bound, *_ = forward_form(x, w, bias, "gelu", None, 0.0, None, 0, BF16)
    close(nsg.linear(x, w, bias, "gelu"), want, bound, "out")


@pytest.mark.parametrize("parts,overwrite", [(0, False), (8, True)])
@pytest.mark.parametrize("T,K,N", LARGE + [(40, 2568, 4352), (1, 1032, 2056), (2048, 768, 768), (4096, 512, 512),
                                            (16384, 256, 256), (2047, 1001, 763)])
def test_gradients_of_many_tiles(T, K, N, parts, overwrite):
    x, dout, w = normal(1, (T, K)), normal(2, (T, N), 0.1), normal(3, (N, K), 1 / math.sqrt(K))
    pre = normal(4, (T, K))
    accum, table = buffer(N * K + N, parts) if parts else (normal(9, (N * K + N,), 0.1, FP32), None)
    flat = (lambda t: t) if table is None else (lambda t: gather(t, table))
    old = flat(accum).to(D64)
    dx = nsg.linear_grad(accum, dout, x, w, (0, N, K), (N * K, 1, N), table, 0.5, overwrite, "gelu", pre)
    want, bound, dw, ew, db, eb = grad_form(dout, x, w, "gelu", pre)
    close(dx, want, bound, "dx")
    v = old * (0 if overwrite else 1) + 0.5 * torch.cat([dw.reshape(-1), db])
    close(flat(accum), v, 0.505 * torch.cat([ew.reshape(-1), eb]) + 2.0 ** -23 * (v.abs() + old.abs()), "accum")


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 9, 33, 64, 65])
@pytest.mark.parametrize("K,N", [(256, 8), (2048, 9), (2056, 1031), (4104, 2048)])
def test_few_tokens(T, K, N):
    """Every way a few tokens may go, with all that a result may have."""
    for way in (WAYS[5], dict(bias=FP32, act="silu", residual=True, pre=True, out=FP32)):
        x, w, bias, residual, out = forward_case(T, K, N, way, T + K + N)
        args = (bias, way["act"], residual, way.get("rate", 0.0), generator(), 9)
        y, u = nsg.linear(x, w, *args, out_dtype=out, pre=True)
        want, bound, pre, pre_bound = forward_form(x, w, *args, out)
        close(y, want, bound, "out")
        close(u, pre, pre_bound, "pre")
        wide = torch.zeros((T, K + 8), dtype=BF16, device="cuda")   # rows with a stride
        wide[:, :K] = x
        assert torch.equal(nsg.linear(wide[:, :K], w, *args, out_dtype=out), y)


def test_calls_at_the_same_time():
    """Two streams at once, each with products, gradients and copies of operands of its own."""
    T, K, N = 700, 1001, 520
    x, w, dout = normal(1, (T, K)), normal(2, (N, K), 0.03), normal(3, (T, N), 0.1)

    def calls():
        accum = torch.zeros(N * K + N, device="cuda")
        y = nsg.linear(x, w, activation="gelu")
        dx = nsg.linear_grad(accum, dout, x, w, (0, N, K), (N * K, 1, N))
        return y, dx, accum

    want = calls()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(5):
        for stream in streams:
            with torch.cuda.stream(stream):
                got.append(calls())
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_what_follows_sees_all_of_a_call():
    """A gradient call's kernels run beside one another; whatever comes next in the stream waits for all of them."""
    T, K, N = 3000, 1288, 1032
    x, w, dout = normal(1, (T, K)), normal(2, (N, K), 0.03), normal(3, (T, N), 0.1)
    accum = torch.zeros(N * K + N, device="cuda")
    want_dx = nsg.linear_grad(accum, dout, x, w, (0, N, K), (N * K, 1, N), overwrite=True)
    want = accum.clone()
    for _ in range(20):
        dx = torch.full((T, K), 7.0, dtype=BF16, device="cuda")
        accum.fill_(3.0)
        nsg.linear_grad(accum, dout, x, w, (0, N, K), (N * K, 1, N), overwrite=True, dx=dx)
        a, b = dx.clone(), accum.clone()        # torch's kernels
        y = nsg.linear(dx, w)                   # and the library's, which start early
        dx.zero_()
        assert torch.equal(a, want_dx) and torch.equal(b, want)
        assert torch.equal(y, nsg.linear(want_dx, w))


def test_the_same_call_gives_the_same_bits():
    for T, K, N in ((1, 4096, 512), (40, 1000, 768), (700, 4096, 776)):
        x, w, bias, residual, _ = forward_case(T, K, N, WAYS[2], 5)
        a, b = (nsg.linear(x, w, bias, "silu", residual, 0.1, generator(), 3) for _ in range(2))
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,K,N", [(1, 40, 24), (5, 136, 64), (130, 129, 200), (300, 520, 264), (64, 512, 511)])
@pytest.mark.parametrize("shift", [0, 1, 3, 8])
def test_strides_and_starts(T, K, N, shift):
    """Operands and results as parts of larger tensors; what lies between the rows stays."""
    x = normal(1, (T, K + 24))[:, shift:shift + K]
    w = normal(2, (N, K + 13), 1 / math.sqrt(K))[:, shift:shift + K]
    whole = normal(3, (T, N + 37))
    out, before = whole[:, shift:shift + N], whole.clone()
    res = normal(4, (T, N + 11))[:, shift:shift + N]
    pre_whole = torch.full((T, N + 17), 7.0, device="cuda", dtype=BF16)
    pre = pre_whole[:, shift:shift + N]
    rng = generator()
    r = nsg.linear(x, w, None, "gelu", res, 0.2, rng, 1, out=out, pre=pre)
    assert r[0] is out and r[1] is pre
    want, bound, u, ub = forward_form(x, w, None, "gelu", res, 0.2, rng, 1, BF16)
    close(out, want, bound)
    close(pre, u, ub)
    for t, n in ((whole, before), (pre_whole, torch.full_like(pre_whole, 7.0))):
        assert torch.equal(t[:, :shift], n[:, :shift]) and torch.equal(t[:, shift + N:], n[:, shift + N:])


def test_joined_dimensions():
    """Batches; a slice of a batch that needs a copy; one row repeated by an expanded tensor (no stride) is refused."""
    row, w = normal(1, (1, 264)), normal(2, (96, 264), 0.06)
    with pytest.raises(nsg.MuonError, match="x_stride"):
        nsg.linear(row.expand(50, 264), w)
    x = normal(3, (4, 9, 264))
    for part in (x, x[:, :-1], x[:, :, :256]):
        y, u = nsg.linear(part, w[:, :part.shape[2]], pre=True, residual=None)
        assert y.shape == (*part.shape[:2], 96) and u.shape == y.shape
        want, bound, _, _ = forward_form(part.reshape(-1, part.shape[2]), w[:, :part.shape[2]], None, None, None, 0.0,
                                         None, 0, BF16)
        close(y.reshape(-1, 96), want, bound)


def test_residual_in_place():
    for T, N in ((1, 512), (33, 257), (400, 768)):
        x, w = normal(1, (T, 768)), normal(2, (N, 768), 0.03)
        res = normal(3, (T, N), 1.0, FP32)
        want = nsg.linear(x, w, residual=res, out_dtype=FP32)
        mine = res.clone()
        assert nsg.linear(x, w, residual=mine, out=mine) is mine
        assert torch.equal(mine, want)


def test_no_tokens():
    w = normal(1, (24, 16))
    y, u = nsg.linear(torch.empty((0, 16), dtype=BF16, device="cuda"), w, pre=True)
    assert y.shape == u.shape == (0, 24)


def test_rows_do_not_meet():
    """A token of NaN, infinities or the type's ends changes its own row alone."""
    for T in (5, 40, 300):
        x, w = normal(1, (T, 520)), normal(2, (264, 520), 0.04)
        clean = nsg.linear(x, w, activation="gelu")
        bad = x.clone()
        bad[2, 5], bad[4, 7] = float("nan"), float("inf")
        bad[3] = torch.finfo(BF16).max
        y = nsg.linear(bad, w, activation="gelu")
        rest = [t for t in range(T) if t not in (2, 3, 4)]
        assert torch.equal(y[rest], clean[rest])
        assert bool(torch.isnan(y[2]).all()) and not bool(torch.isfinite(bad[4].float()).all())


def test_dropped_values_may_be_anything():
    """0 where an infinite value is left out, and the residual comes through."""
    x = torch.full((40, 64), 3e38, device="cuda", dtype=BF16)
    w = torch.full((96, 64), 3e38, device="cuda", dtype=BF16)
    res = normal(1, (40, 96), 1.0, FP32)
    rng = generator()
    y = nsg.linear(x, w, residual=res, dropout=0.5, rng=rng, site=4, out_dtype=FP32)
    gone = forms.keep(40, 96, 0.5, rng, 4, "cuda") == 0
    assert torch.equal(y[gone], res[gone]) and bool(torch.isinf(y[~gone]).all())


def test_activations_at_the_ends():
    """u from the lowest to the highest value of the type: slopes and values stay what the formulas say."""
    u = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 30.0, -30.0, 1e4, -1e4, 1e19, -1e19, 3e38, -3e38, float("nan")])
    x = u.to(BF16).cuda()[:, None].contiguous()
    one = torch.ones((1, 1), dtype=BF16, device="cuda")
    for kind in ("relu", "relu2", "gelu", "silu"):
        y = nsg.linear(x, one, activation=kind, out_dtype=FP32)[:, 0].double().cpu()
        v = x[:, 0].double().cpu()
        pos = v.clamp(min=0)
        far = v.abs() >= 30
        want = pos * pos if kind == "relu2" else pos
        assert torch.equal(y[far].nan_to_num(), want[far].float().double().nan_to_num()) or \
            torch.allclose(y[far], want[far].float().double(), rtol=1e-6, atol=1e-10)
        assert bool(torch.isnan(y[-1]))
        d = nsg.linear_grad(None, torch.ones_like(x), None, one, activation=kind, pre=x)[:, 0].double().cpu()
        w = {"relu2": 2 * pos}.get(kind, (v > 0).double())
        assert torch.allclose(d[far], w[far].to(BF16).double(), rtol=2.0 ** -7, atol=1e-10), (kind, d, w)
        assert bool(torch.isnan(d[-1]))
        assert float(d[0]) == (0.0 if kind.startswith("relu") else 0.5)


# ------------------------------------------------------------------ gradients

def buffer(elements, parts, seed=9, gap=5):
    """A flat buffer cut into uneven partitions with gaps between them in storage, and its table."""
    cuts = [0] + sorted({elements * (2 * i + 1) // (2 * parts) for i in range(1, parts)}) + [elements]
    table, at = np.zeros(len(cuts) - 1, dtype=nsg.PART_DTYPE), 3
    for i in range(len(cuts) - 1):
        table[i] = (cuts[i], cuts[i + 1], at)
        at += cuts[i + 1] - cuts[i] + gap
    return normal(seed, (at + 7,), 0.1, FP32), table


def gather(accum, table):
    return torch.cat([accum[s:s + e - b] for b, e, s in table.tolist()])


def grad_form(dout, x, w, kind, pre):
    d, a, b = dout.to(D64), x.to(D64), w.to(D64)
    dx, ex = d @ b, product_error(d, b)
    if kind not in (None, "none"):
        s = forms.act(pre.to(D64), kind)[1]
        top = s.abs() if kind == "relu2" else 1.2
        ex = ex * top + 2.0 ** -17 * dx.abs() * (s.abs() if kind == "relu2" else 1)
        dx = dx * s
    return (dx, ex * 1.01 + 1.01 * 2.0 ** -8 * dx.abs(), d.T @ a, product_error(d.T, a), d.sum(0),
            (len(d) / 16 + 16) * 2.0 ** -23 * d.abs().sum(0))


GRAD_SIZES = [(1, 1, 1), (1, 64, 64), (3, 7, 5), (2, 768, 512), (17, 1001, 763), (64, 264, 136), (100, 72, 520),
              (128, 256, 64), (130, 257, 65), (513, 136, 1000), (1030, 768, 776), (2500, 520, 264), (4097, 64, 72)]


@pytest.mark.parametrize("parts,overwrite,kind", [(0, True, None), (3, False, "gelu"), (8, True, "silu"),
                                                  (1, False, "relu2")])
@pytest.mark.parametrize("T,K,N", GRAD_SIZES)
def test_gradients(T, K, N, parts, overwrite, kind):
    pre = normal(1, (T, K))
    x = forms.act(pre.to(D64), kind)[0].to(BF16)
    dout, w = normal(2, (T, N), 0.1), normal(3, (N, K), 1 / math.sqrt(K))
    first = 11
    elements = first + N * K + 3 + N + 2
    if parts:
        accum, table = buffer(elements, parts)
    else:
        accum, table = normal(9, (elements,), 0.1, FP32), None
    old = accum.clone()
    param, bias = (first, N, K), (first + N * K + 3, 1, N)
    dx = nsg.linear_grad(accum, dout, x, w, param, bias, table, 0.25, overwrite, kind, pre if kind else None)
    want, bound, dw, ew, db, eb = grad_form(dout, x, w, kind, pre)
    assert dx.dtype == BF16
    close(dx, want, bound, "dx")
    flat = (lambda t: t) if table is None else (lambda t: gather(t, table))
    new, before = flat(accum).to(D64), flat(old).to(D64)
    for off, n, g, e in ((first, N * K, dw.reshape(-1), ew.reshape(-1)), (bias[0], N, db, eb)):
        v = before[off:off + n] * (0 if overwrite else 1) + 0.25 * g
        close(new[off:off + n], v, 0.25 * e * 1.01 + 2.0 ** -23 * (v.abs() + before[off:off + n].abs()), "accum")
    # nothing else of the buffer has changed
    mask = torch.ones(elements, dtype=torch.bool, device="cuda")
    mask[first:first + N * K] = mask[bias[0]:bias[0] + N] = False
    assert torch.equal(flat(accum)[mask], flat(old)[mask])
    if table is not None:
        inside = torch.zeros(len(accum), dtype=torch.bool, device="cuda")
        for b, e, s in table.tolist():
            inside[s:s + e - b] = True
        assert torch.equal(accum[~inside], old[~inside])


def test_gradients_are_reproducible_and_apart():
    """The same call gives the same bits; each gradient asked for alone is right too (its sum may run in another order)."""
    T, K, N = 700, 776, 520
    x, dout, w = normal(1, (T, K)), normal(2, (T, N), 0.1), normal(3, (N, K), 0.04)
    param, bias = (0, N, K), (N * K, N, 1)
    one, two, three, four = (torch.zeros(N * K + N, device="cuda") for _ in range(4))
    a = nsg.linear_grad(one, dout, x, w, param, bias)
    b = nsg.linear_grad(two, dout, x, w, param, bias)
    assert torch.equal(a, b) and torch.equal(one, two)
    want, bound, dw, ew, db, eb = grad_form(dout, x, w, None, None)
    for t in (three, four):
        assert nsg.linear_grad(t, dout, x, None, param, dx=False) is None
        close(t[:N * K].view(N, K), dw, ew * 1.01 + 2.0 ** -23 * dw.abs())
        assert not bool(t[N * K:].any())
        nsg.linear_grad(t, dout, None, None, None, bias, dx=False)
        close(t[N * K:], db, eb * 1.01 + 2.0 ** -23 * db.abs())
        close(nsg.linear_grad(None, dout, None, w), want, bound)
    assert torch.equal(three, four)
    mine = torch.empty((T, K + 3), dtype=BF16, device="cuda")[:, 1:K + 1]
    assert nsg.linear_grad(None, dout, None, w, dx=mine) is mine
    assert torch.equal(mine, nsg.linear_grad(None, dout, None, w))


def test_no_tokens_zero_the_gradients():
    accum = torch.ones(40, device="cuda")
    none = torch.empty((0, 4), dtype=BF16, device="cuda")
    args = (accum, none, torch.empty((0, 8), dtype=BF16, device="cuda"), normal(1, (4, 8)), (1, 4, 8), (35, 1, 4))
    assert nsg.linear_grad(*args).shape == (0, 8) and bool((accum == 1).all())
    nsg.linear_grad(*args, overwrite=True)
    assert not bool(accum[1:33].any()) and not bool(accum[35:39].any()) and accum[0] == accum[33] == accum[39] == 1


@pytest.mark.parametrize("shift", [1, 8])
def test_gradient_operands_of_any_layout(shift):
    T, K, N = 260, 200, 136
    dout = normal(1, (T, N + 9), 0.1)[:, shift:shift + N]
    x = normal(2, (T, K + 24))[:, shift:shift + K]
    w = normal(3, (N, K + 11), 0.07)[:, shift:shift + K]
    pre = normal(4, (T, K + 9))[:, shift:shift + K]
    accum = torch.zeros(N * K + N, device="cuda")
    dx = nsg.linear_grad(accum, dout, x, w, (0, N, K), (N * K, 1, N), activation="gelu", pre=pre)
    want, bound, dw, ew, db, eb = grad_form(dout, x, w, "gelu", pre)
    close(dx, want, bound)
    close(accum[:N * K].view(N, K), dw, ew * 1.01 + 2.0 ** -23 * dw.abs())
    close(accum[N * K:], db, eb * 1.01 + 2.0 ** -23 * db.abs())


def test_streams_and_graphs():
    T, K, N = 200, 264, 136
    x, w, dout = normal(1, (T, K)), normal(2, (N, K), 0.06), normal(3, (T, N), 0.1)
    odd, oddw = normal(4, (T, 33)), normal(5, (N, 33), 0.2)
    rng = generator()
    accum = torch.zeros(N * K, device="cuda")

    def calls():
        accum.zero_()
        y = nsg.linear(x, w, None, "silu", dropout=0.3, rng=rng, site=1)
        z = nsg.linear(odd, oddw)
        return y, z, nsg.linear_grad(accum, dout, x, w, (0, N, K)), accum.clone()

    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = calls()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = nsg.linear(x, w, None, "silu", dropout=0.3, rng=rng, site=1, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for step in (2, 3, 2):
        rng[1] = step
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], want[0]) == (step == 2)
        assert all(torch.equal(a, b) for a, b in zip(held[1:], want[1:]))


def test_offsets_past_32_bits():
    """Rows 2^31 + 24 elements apart: byte offsets past 2^32, element offsets past 2^31."""
    K, N, far = 72, 40, (1 << 31) + 24
    room = torch.empty(far * 2 + 200, dtype=BF16, device="cuda")
    x = room.as_strided((3, K), (far, 1))
    x.copy_(normal(1, (3, K)))
    w = normal(2, (N, K), 0.1)
    out = room.as_strided((3, N), (far, 1), 96)
    close(nsg.linear(x, w), *forward_form(x, w, None, None, None, 0.0, None, 0, BF16)[:2])
    y = nsg.linear(normal(3, (3, K)), w, out=out)
    close(y, *forward_form(normal(3, (3, K)), w, None, None, None, 0.0, None, 0, BF16)[:2])
