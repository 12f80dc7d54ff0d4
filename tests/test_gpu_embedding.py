"""Embedding lookup and its gradient against plain torch on the same inputs.

Tolerances, derived from the arithmetic:
* lookup: one FP32 product, rounded once to the output type -- bit for bit
  torch's ``(table.float() * scale).to(out)``;
* gradient: accum + scale * sum in FP32.  A sum of n terms in any order is
  off by at most (n - 1) u sum|x| (u = 2^-24), the scaling and the last sum
  add one rounding each, so |error| <= u ((n + 1) scale sum|x| + |result|),
  taken twice over; rows of no token keep their bits (or are exactly 0 with
  overwrite)."""
import numpy as np
import pytest

import newton_schulz_fp32_gb300 as nsg
import workloads as wl
from harness import bits, to_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    nsg.build()
    return t


def make_ids(torch, kind, n, rows, seed, dtype):
    rng = np.random.default_rng(seed)
    if kind == "zipf":
        ids = np.minimum((rows + 1.0) ** rng.random(n) - 1, rows - 1).astype(np.int64)
    elif kind == "uniform":
        ids = rng.integers(0, rows, n)
    elif kind == "one":
        ids = np.full(n, rows // 2)
    elif kind == "padded":
        ids = np.where(rng.random(n) < 0.4, -1 - rng.integers(0, 100, n), rng.integers(0, rows, n))
    elif kind == "none":
        ids = np.full(n, -1)
    elif kind == "runs":   # runs that end on and around the borders of blocks of 32
        ids = np.repeat(np.arange(n), 32)[:n] % rows
        ids[:33] = rows - 1
        ids = rng.permutation(ids)
    return torch.from_numpy(ids.astype(np.int64 if dtype == "int64" else np.int32)).cuda()


def reference_grad(torch, accum, dout, ids, scale, overwrite):
    """(result, bound) in 64 bits; accum rows x cols."""
    first = torch.zeros_like(accum, dtype=torch.float64) if overwrite else accum.double()
    size = torch.zeros_like(first)
    keep = (ids >= 0) & (ids < accum.shape[0])
    d = dout[keep].double() * scale
    rows = ids[keep].long()
    first.index_add_(0, rows, d)
    size.index_add_(0, rows, d.abs())
    n = torch.zeros(accum.shape[0], dtype=torch.float64, device=accum.device)
    n.index_add_(0, rows, torch.ones_like(rows, dtype=torch.float64))
    bound = 2 * U * ((n[:, None] + 1) * size + first.abs())
    return first, bound, n


LOOKUP = [  # tokens, rows, cols, extra table stride, extra out stride, base offset
    (1, 1, 1, 0, 0, 0), (1, 100, 768, 0, 0, 0), (7, 50, 8, 0, 0, 0), (33, 1000, 7, 0, 0, 0),
    (1000, 513, 1001, 0, 0, 0), (257, 300, 4096, 0, 0, 0), (100, 300, 1000, 24, 8, 0),
    (100, 300, 1000, 3, 5, 1), (4099, 70, 96, 0, 0, 0), (3, 11, 20000, 0, 0, 3)]


@pytest.mark.parametrize("shape", LOOKUP)
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_lookup(torch, shape, types):
    T, V, D, ps, po, off = shape
    kinds = {"bf16": torch.bfloat16, "fp32": torch.float32}
    gen = torch.Generator(device="cuda").manual_seed(T + V)
    table = torch.randn(V * (D + ps) + off, generator=gen, device="cuda").to(kinds[types[0]])
    table = table[off:].view(V, D + ps)[:, :D]
    for index, kind in (("int64", "zipf"), ("int32", "padded")):
        ids = make_ids(torch, kind, T, V, T, index)
        store = torch.full((T * (D + po) + off,), 7.0, device="cuda").to(kinds[types[1]])
        out = store[off:].view(T, D + po)
        nsg.embedding(table, ids, scale=1.7, out=out[:, :D])
        want = (table.float()[ids.long().clamp(min=0)] * 1.7).to(kinds[types[1]])
        want[ids < 0] = 0
        assert torch.equal(out[:, :D], want)
        assert bool((out[:, D:] == 7).all())   # between the rows nothing is written
        got = nsg.embedding(table, ids, scale=1.7, out_dtype=kinds[types[1]])
        assert got.shape == (T, D) and torch.equal(got, want)
    assert nsg.device_error() == 0


def test_lookup_shapes_and_special_values(torch):
    table = torch.tensor([[1.0, float("inf")], [float("nan"), -0.0], [2.0, 3e38]], device="cuda")
    ids = torch.tensor([[0, 1, -5], [2, 2, 0]], device="cuda")
    out = nsg.embedding(table, ids, scale=2.0)
    assert out.shape == (2, 3, 2)
    want = (table * 2.0)[ids.clamp(min=0)]
    want[ids < 0] = 0
    assert torch.equal(out.nan_to_num(nan=5.5), want.nan_to_num(nan=5.5))
    assert nsg.embedding(table, ids[:0]).shape == (0, 3, 2)
    bad = torch.tensor([0, 3, 1 << 40], device="cuda")
    out = nsg.embedding(table, bad)
    assert torch.equal(out[1:], torch.zeros_like(out[1:])) and torch.equal(out[0], table[0])
    assert nsg.device_error() == 17 and nsg.device_error() == 0


GRAD = [  # tokens, rows, cols, ids
    (0, 5, 3, "zipf"), (1, 1, 1, "uniform"), (1, 9, 768, "uniform"), (31, 100, 64, "zipf"),
    (32, 100, 8, "one"), (33, 7, 1000, "one"), (64, 40, 129, "runs"), (999, 50, 24, "zipf"),
    (1024, 3000, 768, "zipf"), (2049, 64, 40, "runs"), (5003, 501, 1001, "padded"),
    (4096, 70000, 16, "uniform"), (3000, 10, 4096, "zipf"), (300, 20, 2056, "none"),
    (20000, 513, 12, "one"), (70001, 300000, 8, "zipf")]


@pytest.mark.parametrize("shape", GRAD)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("overwrite", [False, True])
def test_gradient_dense(torch, shape, dtype, overwrite):
    T, V, D, kind = shape
    gen = torch.Generator(device="cuda").manual_seed(T * 31 + D)
    ids = make_ids(torch, kind, T, V, T + D, "int64" if T % 2 else "int32")
    dout = torch.randn((T, D), generator=gen, device="cuda")
    dout = dout.to(torch.bfloat16) if dtype == "bf16" else dout
    off = (T * 3) % 8
    accum = torch.randn(off + V * D + 5, generator=gen, device="cuda")
    before = accum.clone()
    again = accum.clone()
    nsg.embedding_grad(accum, dout, ids, (off, V, D), scale=0.3, overwrite=overwrite)
    scale = float(np.float32(0.3))
    want, bound, n = reference_grad(torch, before[off:off + V * D].view(V, D), dout, ids, scale, overwrite)
    got = accum[off:off + V * D].view(V, D)
    assert bool(((got.double() - want).abs() <= bound).all())
    idle = n == 0
    if overwrite:
        assert bool((got[idle] == 0).all())
    else:
        assert torch.equal(got[idle], before[off:off + V * D].view(V, D)[idle])
    assert torch.equal(accum[:off], before[:off]) and torch.equal(accum[off + V * D:], before[off + V * D:])
    nsg.embedding_grad(again, dout, ids, (off, V, D), scale=0.3, overwrite=overwrite)
    assert torch.equal(again, accum)   # one order of sums, whatever the timing
    assert nsg.device_error() == 0


@pytest.mark.parametrize("storage,nparts", [("identity", 1), ("identity", 8), ("rank_major", 4),
                                            ("shuffled", 3), ("shuffled", 40)])
@pytest.mark.parametrize("cols", [37, 64])
@pytest.mark.parametrize("T", [900, 3001])
def test_gradient_in_partitions(torch, storage, nparts, cols, T):
    """The parameter between others of a partitioned buffer: cut anywhere,
    also inside a row; padding and the other parameters untouched."""
    rows = 211
    lay = wl.build_layout([[wl.ParamSpec("w", 17, 13)],
                           [wl.ParamSpec("ln", 1, 33, use_muon=False),
                            wl.ParamSpec("table", rows, cols, use_muon=False),
                            wl.ParamSpec("odd", 7, 5, use_muon=False)]], 16, nparts, storage, 3)
    mats = wl.gaussian_grads(lay, 11, 0, None, bf16=False)
    start = wl.storage_with_sentinels(lay, mats)
    ids = make_ids(torch, "zipf", T, rows, 5, "int64")
    gen = torch.Generator(device="cuda").manual_seed(8)
    dout = torch.randn((T, cols), generator=gen, device="cuda").to(torch.bfloat16)
    dense = None
    for overwrite in (False, True):
        accum = to_dev(start, torch)
        nsg.embedding_grad(accum, dout, ids, lay.params[2], parts=lay.parts, scale=0.25, overwrite=overwrite)
        got = accum.cpu().numpy()
        pad = wl.padding_mask(lay)
        assert (bits(got)[pad] == wl.NAN_SENTINEL_BITS).all()
        out = wl.unpack(lay, got)
        for k in (0, 1, 3):
            np.testing.assert_array_equal(bits(out[k]), bits(mats[k]))
        dense = torch.from_numpy(mats[2].copy()).cuda().reshape(-1)
        nsg.embedding_grad(dense, dout, ids, (0, rows, cols), scale=0.25, overwrite=overwrite)
        np.testing.assert_array_equal(bits(out[2]), bits(dense.cpu().numpy().reshape(rows, cols)))
    assert nsg.device_error() == 0


@pytest.mark.parametrize("T", [700, 5000])
@pytest.mark.parametrize("cols", [64, 72])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_of_rows_cut_on_16_bytes(torch, T, cols, dtype):
    """Rows that start on 16 bytes, some of them cut between partitions: the
    same bits as without partitions, for few and for many tokens."""
    rows = 301
    lay = wl.build_layout([[wl.ParamSpec("table", rows, cols, use_muon=False)]], 16, 7, "rank_major", 3)
    gen = torch.Generator(device="cuda").manual_seed(T)
    ids = make_ids(torch, "zipf", T, rows, 5, "int32")
    dout = torch.randn((T, cols), generator=gen, device="cuda")
    dout = dout.to(torch.bfloat16) if dtype == "bf16" else dout
    first = torch.randn(lay.storage_size, generator=gen, device="cuda")
    for overwrite in (False, True):
        accum, dense = first.clone(), first.clone()
        nsg.embedding_grad(accum, dout, ids, lay.params[0], parts=lay.parts, scale=0.5, overwrite=overwrite)
        nsg.embedding_grad(dense, dout, ids, (0, rows, cols), scale=0.5, overwrite=overwrite)
        n = rows * cols
        assert torch.equal(accum[:n], dense[:n]) and torch.equal(accum[n:], first[n:])
        want, bound, _ = reference_grad(torch, first[:n].view(rows, cols), dout, ids, 0.5, overwrite)
        assert bool(((accum[:n].view(rows, cols).double() - want).abs() <= bound).all())


def test_gradient_of_special_values_and_strides(torch):
    V, D, T = 20, 72, 400
    gen = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn((T, D + 9), generator=gen, device="cuda").to(torch.bfloat16)
    ids = make_ids(torch, "padded", T, V, 2, "int64")
    wide[ids < 0] = float("nan")                 # tokens that take no part may hold anything
    inf_row, nan_row = int(ids[ids >= 0][0]), int(ids[ids >= 0][1])
    at = int((ids == inf_row).nonzero()[0])
    wide[at, 3] = float("inf")
    wide[int((ids == nan_row).nonzero()[0]), 5] = float("nan")
    for off in (0, 1, 8):
        dout = wide[:, off:off + D]
        accum = torch.zeros(V * D, device="cuda")
        nsg.embedding_grad(accum, dout, ids, (0, V, D))
        got = accum.view(V, D)
        keep = ids >= 0
        want = torch.zeros((V, D), dtype=torch.float64, device="cuda")
        want.index_add_(0, ids[keep], dout[keep].double())
        fine = torch.isfinite(want)
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
        assert bool(((got.double() - want).abs()[fine] <= 1e-3).all())
    bad = ids.clone()
    bad[7], bad[11] = V, 1 << 33
    accum, other = torch.zeros(V * D, device="cuda"), torch.zeros(V * D, device="cuda")
    nsg.embedding_grad(accum, dout.contiguous(), bad, (0, V, D))
    assert nsg.device_error() == 17
    bad[7], bad[11] = -1, -1
    nsg.embedding_grad(other, dout.contiguous(), bad, (0, V, D))
    assert torch.equal(accum.nan_to_num(nan=9.0), other.nan_to_num(nan=9.0)) and nsg.device_error() == 0


def test_gradient_is_the_lookups(torch):
    """<grad(dout), dE> = <dout, lookup(dE)> for any dE: the gradient against
    differences of the (linear) lookup."""
    V, D, T = 301, 96, 777
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids = make_ids(torch, "zipf", T, V, 6, "int64")
    dout = torch.randn((T, D), generator=gen, device="cuda")
    e0, de = (torch.randn((V, D), generator=gen, device="cuda") for _ in range(2))
    accum = torch.empty(V * D, device="cuda")
    nsg.embedding_grad(accum, dout, ids, (0, V, D), scale=3.0, overwrite=True)
    step = 0.5
    diff = (nsg.embedding(e0 + step * de, ids, 3.0).double() - nsg.embedding(e0 - step * de, ids, 3.0).double())
    want = float((dout.double() * diff).sum() / (2 * step))
    got = float((accum.view(V, D).double() * de.double()).sum())
    # T * D products of unit size, each off by a few FP32 roundings of values up to ~10
    assert abs(got - want) <= 32 * U * 10 * (T * D) ** 0.5 * 10


def test_streams_and_graph(torch):
    """On another stream than torch's current one, and captured."""
    V, D, T = 500, 256, 3000
    gen = torch.Generator(device="cuda").manual_seed(9)
    table = torch.randn((V, D), generator=gen, device="cuda").to(torch.bfloat16)
    ids = make_ids(torch, "zipf", T, V, 6, "int64")
    dout = torch.randn((T, D), generator=gen, device="cuda").to(torch.bfloat16)
    want = nsg.embedding(table, ids, 2.0)
    acc = torch.zeros(V * D, device="cuda")
    nsg.embedding_grad(acc, dout, ids, (0, V, D))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.zeros(V * D, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    got = nsg.embedding(table, ids, 2.0, stream=side)
    nsg.embedding_grad(other, dout, ids, (0, V, D), stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(other, acc)
    third = torch.zeros(V * D, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = nsg.embedding(table, ids, 2.0)
        nsg.embedding_grad(third, dout, ids, (0, V, D), overwrite=True)
    for _ in range(2):
        third.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(third, acc)


def test_offsets_past_32_bits(torch):
    """A table and an accumulation buffer of more than 2^32 elements."""
    D, V = 4096, (1 << 20) + 4096
    table = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, 1 << 20, V - 1, 5], device="cuda")
    rows = torch.randn((5, D), device="cuda").to(torch.bfloat16)
    rows[3] = rows[0]
    table[ids] = rows
    assert torch.equal(nsg.embedding(table, ids), rows)
    del table
    accum = torch.zeros(V * D, device="cuda")
    nsg.embedding_grad(accum, rows, ids, (0, V, D))
    got = accum.view(V, D)
    assert torch.equal(got[V - 1], rows[0].float() * 2) and torch.equal(got[1 << 20], rows[2].float())
    assert torch.equal(got[5], rows[4].float()) and torch.equal(got[0], rows[1].float())
    assert int((got.sum(1, dtype=torch.float64) != 0).sum()) == 4
