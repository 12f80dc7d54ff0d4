"""What the layer entry points refuse, on the host before any CUDA call, their
workspace sizes, and the formulas their GPU tests compare with (slopes against
differences).  The addresses are made up: tests of the library run only where
no GPU could be handed them."""
import ctypes
import glob
import math

import numpy as np
import pytest

import newton_schulz_fp32_gb300 as nsg

torch = pytest.importorskip("torch")
import layer_forms as forms  # noqa: E402
import standin  # noqa: E402

no_gpu = pytest.mark.skipif(bool(glob.glob("/dev/nvidia[0-9]*")) or torch.cuda.is_available(),
                            reason="made-up addresses stay away from a GPU")
FAKE = 1 << 30   # a non-NULL, aligned address that is never dereferenced
STEP = 1 << 24   # between tensors
KEEP = []


@pytest.fixture(scope="module")
def lib():
    nsg.build()
    return nsg.lib()


def refused(lib, rc, word, code=nsg.MUON_ERR_INVALID):
    assert rc == code, (rc, lib.muon_last_error())
    assert word in lib.muon_last_error().decode(), (word, lib.muon_last_error())


def fill(struct, values):
    a = struct()
    for k, v in values.items():
        setattr(a, k, v)
    return a


LINEAR = dict(struct_size=ctypes.sizeof(nsg.LinearArgs), activation=3, n_tokens=50, in_features=64, out_features=40,
              x=FAKE, x_stride=64, weight=FAKE + STEP, weight_stride=64, bias=FAKE + 2 * STEP, pre=FAKE + 3 * STEP,
              pre_stride=40, residual=FAKE + 4 * STEP, residual_stride=40, out=FAKE + 5 * STEP, out_stride=40,
              rng=FAKE + 6 * STEP, bias_dtype=0, out_dtype=0, dropout=0.1, site=0)


@no_gpu
@pytest.mark.parametrize("change,word", [
    (dict(struct_size=8), "struct_size"), (dict(activation=5), "activation"), (dict(activation=-1), "activation"),
    (dict(n_tokens=-1), "n_tokens"), (dict(n_tokens=(1 << 30) + 1), "n_tokens"), (dict(in_features=0), "features"),
    (dict(out_features=(1 << 24) + 1), "features"), (dict(x=None), "x is NULL"), (dict(x=FAKE + 1), "x is NULL or mis"),
    (dict(x_stride=63), "x_stride"), (dict(weight=None), "weight"), (dict(weight_stride=10), "weight_stride"),
    (dict(x_stride=1 << 62), "x_stride"), (dict(out=None), "out"), (dict(out_stride=39), "out_stride"),
    (dict(pre=FAKE + 1), "pre"), (dict(pre_stride=0), "pre_stride"), (dict(residual_stride=1), "residual_stride"),
    (dict(out_dtype=2), "out_dtype"), (dict(bias_dtype=3), "bias"), (dict(bias=FAKE + 1), "bias"),
    (dict(dropout=-0.1), "rate"), (dict(dropout=1.0), "rate"), (dict(dropout=math.nan), "rate"),
    (dict(dropout=1 - 2.0 ** -18), "1 - 2^-17"), (dict(rng=None), "rng"), (dict(rng=FAKE + 4), "rng"),
    (dict(out=FAKE + 64), "overlap"), (dict(out=FAKE + STEP), "overlap"), (dict(out=FAKE + 2 * STEP), "overlap"),
    (dict(pre=FAKE + 5 * STEP + 16), "overlap"), (dict(pre=FAKE + 4 * STEP), "overlap"),
    (dict(residual=FAKE + 5 * STEP, residual_stride=41), "overlap"), (dict(out=FAKE + 6 * STEP), "overlap"),
    (dict(residual=FAKE + 5 * STEP + 2), "overlap")])
def test_linear_refuses(lib, change, word):
    a, n = fill(nsg.LinearArgs, dict(LINEAR, **change)), ctypes.c_size_t()
    refused(lib, lib.muon_linear(ctypes.byref(a), None, 0, None), word)
    refused(lib, lib.muon_linear_workspace(ctypes.byref(a), ctypes.byref(n)), word)


@no_gpu
def test_linear_refuses_no_arguments_and_too_many_tiles(lib):
    refused(lib, lib.muon_linear(None, None, 0, None), "args")
    a = fill(nsg.LinearArgs, dict(LINEAR, n_tokens=1 << 30, in_features=8, out_features=1 << 24, x_stride=8,
                                  weight_stride=8))
    refused(lib, lib.muon_linear(ctypes.byref(a), None, 0, None), "too many", nsg.MUON_ERR_UNSUPPORTED)


def param(offset=0, rows=40, cols=64):
    KEEP.append(np.array([(offset, rows, cols, 0, 0)], dtype=nsg.PARAM_DTYPE))
    return KEEP[-1].ctypes.data


def table(*rows):
    KEEP.append(np.array(list(rows), dtype=nsg.PART_DTYPE))
    return dict(parts=KEEP[-1].ctypes.data, nparts=len(rows))


GRAD = dict(struct_size=ctypes.sizeof(nsg.LinearGradArgs), activation=3, n_tokens=50, in_features=64, out_features=40,
            dout=FAKE, dout_stride=40, x=FAKE + STEP, x_stride=64, weight=FAKE + 2 * STEP, weight_stride=64,
            pre=FAKE + 3 * STEP, pre_stride=64, dx=FAKE + 4 * STEP, dx_stride=64, accum=FAKE + 5 * STEP,
            accum_elems=4000, parts=None, nparts=0, overwrite=0, scale=1.0, reserved=0)


@no_gpu
@pytest.mark.parametrize("change,word", [
    (dict(struct_size=0), "struct_size"), (dict(reserved=1), "reserved"), (dict(activation=9), "activation"),
    (dict(n_tokens=-1), "n_tokens"), (dict(out_features=0), "features"), (dict(overwrite=2), "overwrite"),
    (dict(scale=math.inf), "scale"), (dict(dout=None), "dout"), (dict(dout_stride=39), "dout_stride"),
    (dict(x=None), "x is NULL"), (dict(x_stride=1), "x_stride"), (dict(weight=None), "weight"),
    (dict(pre=None), "pre"), (dict(pre_stride=63), "pre_stride"), (dict(dx=FAKE + 4 * STEP + 1), "dx"),
    (dict(dx_stride=63), "dx_stride"), (dict(accum=None), "accum"), (dict(accum=FAKE + 4), "accum"),
    (dict(accum_elems=2599), "accum_elems"), (dict(nparts=1), "parts"), (dict(nparts=-1), "parts"),
    (dict(dx=FAKE), "overlap"), (dict(dx=FAKE + STEP), "overlap"), (dict(dx=FAKE + 2 * STEP), "overlap"),
    (dict(dx=FAKE + 3 * STEP), "overlap"), (dict(dx=FAKE + 5 * STEP), "overlap"),
    (dict(x=FAKE + 5 * STEP), "overlap"), (dict(dout=FAKE + 5 * STEP + 32), "overlap"),
    (("param", dict(rows=41)), "out_features x in"), (("param", dict(offset=-1)), "offset"),
    (("bias", dict(rows=1, cols=39)), "out_features"), (("bias", dict(offset=2559, rows=1, cols=40)), "overlap"),
    (table((0, 2000, 0), (2000, 3000, 1500)), "storage"), (table((0, 2599, 0)), "covered"),
    (table((0, 3000, 2000)), "accum_elems")])
def test_linear_grad_refuses(lib, change, word):
    values = dict(GRAD, param=param(), bias=param(2560, 1, 40))
    if isinstance(change, tuple):
        values[change[0]] = param(**dict(dict(offset=0) if change[0] == "param" else dict(offset=2560), **change[1]))
    else:
        values.update(change)
    a, n = fill(nsg.LinearGradArgs, values), ctypes.c_size_t()
    refused(lib, lib.muon_linear_grad(ctypes.byref(a), None, 0, None), word)
    refused(lib, lib.muon_linear_grad_workspace(ctypes.byref(a), ctypes.byref(n)), word)


DROP = dict(x=FAKE, xs=64, res=FAKE + STEP, rs=64, out=FAKE + 2 * STEP, os=64, dtype=0, rows=50, cols=64, rate=0.1,
            rng=FAKE + 3 * STEP, site=0, stream=None)


@no_gpu
@pytest.mark.parametrize("change,word", [
    (dict(x=None), "NULL"), (dict(out=None), "NULL"), (dict(x=FAKE + 1), "aligned"), (dict(res=FAKE + 1), "aligned"),
    (dict(xs=63), "strides"), (dict(rs=63), "strides"), (dict(os=63), "strides"), (dict(xs=1 << 62), "strides"),
    (dict(dtype=2), "dtype"), (dict(rows=-1), "rows"), (dict(rows=(1 << 30) + 1), "rows"), (dict(cols=0), "cols"),
    (dict(rate=1.0), "rate"), (dict(rate=math.nan), "rate"), (dict(rng=None), "rng"), (dict(rng=FAKE + 4), "rng"),
    (dict(out=FAKE + 128), "overlap"), (dict(out=FAKE, os=65), "overlap"), (dict(out=FAKE + STEP + 2), "overlap"),
    (dict(out=FAKE + 3 * STEP), "overlap")])
def test_dropout_refuses(lib, change, word):
    refused(lib, lib.muon_dropout(*dict(DROP, **change).values()), word)


def heads(kind, **change):
    base = dict(x=FAKE, x_stride=512, x_head_stride=64, weight=FAKE + STEP, out=FAKE + 2 * STEP, out_stride=256,
                out_head_stride=64, heads=4, reserved=0) if kind is nsg.Heads else \
        dict(dout=FAKE, dout_stride=512, dout_head_stride=64, x=FAKE + STEP, x_stride=512, x_head_stride=64,
             weight=FAKE + 2 * STEP, dx=FAKE + 3 * STEP, dx_stride=256, dx_head_stride=64, param=None, heads=4,
             reserved=0)
    return fill(kind, dict(base, **change))


FREQ = np.ones(32)
AXIS = np.zeros(32, dtype=np.int32)


def rotary(lib, groups, **change):
    arr = (type(groups[0]) * len(groups))(*groups)
    a = dict(groups=arr, n_groups=len(groups), dtype=0, n=50, dim=64, norm=1, eps=1e-6, pos=FAKE + 8 * STEP, pt=1,
             axes=1, freq=FREQ.ctypes.data, axis=AXIS.ctypes.data, pairs=32, inter=0)
    tail = {}
    if isinstance(groups[0], nsg.HeadsGrad):
        tail = dict(accum=FAKE + 9 * STEP, elems=200, parts=None, nparts=0, scale=1.0, overwrite=0,
                    ws=FAKE + 10 * STEP, wb=1 << 20)
    a.update(tail)
    a["stream"] = None
    a.update(change)
    return (lib.muon_norm_rotary_grad if tail else lib.muon_norm_rotary)(*a.values())


BOTH = [(dict(n_groups=0), "n_groups"), (dict(n_groups=3), "n_groups"), (dict(dtype=2), "dtype"), (dict(n=-1), "n_tokens"),
        (dict(dim=0), "head_dim"), (dict(dim=257), "head_dim"), (dict(norm=2), "norm"), (dict(eps=-1.0), "eps"),
        (dict(eps=math.nan), "eps"), (dict(pos=None), "positions"), (dict(pos=FAKE + 4), "positions"),
        (dict(pt=2), "positions_type"), (dict(axes=0), "axes"), (dict(axes=9), "axes"), (dict(freq=None), "inv_freq"),
        (dict(pairs=33), "pairs"), (dict(pairs=-1), "pairs"), (dict(inter=2), "interleaved")]


@no_gpu
@pytest.mark.parametrize("kind", [nsg.Heads, nsg.HeadsGrad])
@pytest.mark.parametrize("change,word", BOTH)
def test_norm_rotary_refuses(lib, change, word, kind):
    refused(lib, rotary(lib, [heads(kind)], **change), word)


@no_gpu
def test_norm_rotary_refuses_bad_turns(lib):
    for kind in (nsg.Heads, nsg.HeadsGrad):
        bad = FREQ.copy()
        bad[3] = math.inf
        refused(lib, rotary(lib, [heads(kind)], freq=bad.ctypes.data), "finite")
        for v in (-1, 1):
            off = AXIS.copy()
            off[5] = v
            refused(lib, rotary(lib, [heads(kind)], axis=off.ctypes.data), "axis")


@no_gpu
@pytest.mark.parametrize("first,second,word", [
    (dict(x=None), None, "x is NULL"), (dict(x=FAKE + 1), None, "x is NULL or mis"), (dict(out=None), None, "out"),
    (dict(x_stride=-1), None, "strides"), (dict(heads=0), None, "heads"), (dict(reserved=1), None, "reserved"),
    (dict(weight=FAKE + STEP + 1), None, "weight"), (dict(out_stride=255), None, "overlap one another"),
    (dict(out_head_stride=63), None, "overlap one another"), (dict(out=FAKE + 2), None, "overlaps"),
    (dict(out=FAKE, out_stride=512, out_head_stride=65), None, "overlaps"), (dict(out=FAKE + STEP), None, "weight"),
    (dict(out=FAKE + 8 * STEP), None, "positions"), (dict(), dict(), "overlaps"),
    (dict(), dict(out=FAKE + 2 * STEP + 64), "overlaps"), (dict(out=FAKE, out_stride=512), dict(), "overlaps"),
    (dict(out=FAKE + 128, out_stride=512), None, "overlaps")])
def test_heads_refuse(lib, first, second, word):
    groups = [heads(nsg.Heads, **first)] + ([] if second is None else [heads(nsg.Heads, **second)])
    refused(lib, rotary(lib, groups), word)


@no_gpu
@pytest.mark.parametrize("first,change,word", [
    (dict(dout=None), {}, "dout"), (dict(x=None), {}, "x is NULL"), (dict(dx=None), {}, "dx"),
    (dict(dx_stride=100), {}, "overlap one another"), (dict(dx=FAKE + 2), {}, "overlaps"),
    (dict(dx=FAKE + STEP + 2), {}, "overlaps"), (dict(dx=FAKE + 2 * STEP), {}, "weight"),
    (dict(dx=FAKE + 8 * STEP), {}, "positions"), (dict(dx=FAKE + 9 * STEP), {}, "accum"),
    (dict(dx=FAKE + 10 * STEP), {}, "workspace"), (dict(param=param(0, 1, 63)), {}, "head_dim"),
    (dict(param=param(0, 1, 64)), dict(norm=0), "without norm"), (dict(param=param(0, 1, 64)), dict(ws=None), "workspace"),
    (dict(param=param(0, 1, 64)), dict(wb=64), "workspace"), (dict(param=param(0, 1, 64)), dict(accum=None), "accum"),
    (dict(param=param(137, 1, 64)), {}, "accum_elems"), (dict(param=param(-1, 1, 64)), {}, "offset"),
    (dict(), dict(scale=math.nan), "scale"), (dict(), dict(overwrite=3), "overwrite")])
def test_heads_grad_refuse(lib, first, change, word):
    base = dict(param=param(0, 1, 64)) if "param" not in first else {}
    refused(lib, rotary(lib, [heads(nsg.HeadsGrad, **dict(base, **first))], **change), word)


@no_gpu
def test_two_params_may_not_meet(lib):
    a = heads(nsg.HeadsGrad, param=param(0, 1, 64))
    b = heads(nsg.HeadsGrad, param=param(63, 1, 64), dout=FAKE + 4 * STEP, x=FAKE + 5 * STEP, dx=FAKE + 6 * STEP)
    refused(lib, rotary(lib, [a, b]), "params overlap")


def test_workspaces(lib):
    n = nsg.norm_rotary_grad_workspace
    assert n(0, 64) == 0 and 0 < n(1, 64) <= n(100, 64) <= n(1 << 30, 64) <= 1 << 24
    for bad in ((-1, 64), (1, 0), (1, 257)):
        with pytest.raises(nsg.MuonError):
            n(*bad)


# ------------------------------------------------------------------ the binding

def test_python_refuses_before_the_library():
    m = torch.zeros
    bf = lambda *s: m(s, dtype=torch.bfloat16)  # noqa: E731
    for call, word in (
            (lambda: nsg.linear(m(2, 8), bf(4, 8)), "x must be bfloat16"),
            (lambda: nsg.linear(bf(2, 8), bf(4, 7)), "out_features x in_features"),
            (lambda: nsg.linear(bf(2, 8), bf(4, 8), activation="tanh"), "unknown activation"),
            (lambda: nsg.linear(bf(2, 8), bf(4, 8), bias=m(5)), "bias must have"),
            (lambda: nsg.linear(bf(2, 8), bf(4, 8), residual=m(2, 5)), "residual must be 2 x 4"),
            (lambda: nsg.linear(bf(2, 8), bf(4, 8), rng=m(2)), "rng must be"),
            (lambda: nsg.linear(bf(2, 8), bf(4, 8), site=-1), "site must be"),
            (lambda: nsg.linear(bf(2, 8), bf(4, 8), out=bf(2, 4), out_dtype=torch.float32), "out_dtype"),
            (lambda: nsg.linear(bf(2, 8), bf(4, 8)), "CUDA device"),
            (lambda: nsg.linear_grad(None, bf(2, 4), bf(2, 8), bf(4, 8), (0, 4, 8)), "accum is needed"),
            (lambda: nsg.linear_grad(None, bf(2, 4), None, None), "weight is needed"),
            (lambda: nsg.linear_grad(m(32), bf(2, 4), None, bf(4, 8), (0, 4, 8)), "x is needed"),
            (lambda: nsg.linear_grad(None, bf(2, 4), None, bf(4, 8), activation="relu"), "pre is needed"),
            (lambda: nsg.dropout(m(2, 8), 0.5, m(3, dtype=torch.int64)), "rng must be"),
            (lambda: nsg.dropout(m(2, 8), 0.5, None, residual=bf(2, 8)), "residual must be 2 x 8"),
            (lambda: nsg.norm_rotary(bf(2, 3, 8), bf(2, 3, 6)), "k must have"),
            (lambda: nsg.norm_rotary(bf(2, 3, 8), inv_freq=np.ones(4)), "positions are needed"),
            (lambda: nsg.norm_rotary(bf(2, 3, 8), positions=m(2, dtype=torch.int64), inv_freq=np.ones(4, "f4")),
             "inv_freq must be"),
            (lambda: nsg.norm_rotary(bf(2, 3, 8), positions=m(3, dtype=torch.int64), inv_freq=np.ones(4)),
             "positions must be"),
            (lambda: nsg.norm_rotary(bf(2, 3, 8), positions=m(2, dtype=torch.int64), inv_freq=np.ones(4),
                                     axis=np.zeros(3, np.int32)), "axis must be"),
            (lambda: nsg.norm_rotary(bf(2, 8, 3).transpose(1, 2)), "heads must be contiguous"),
            (lambda: nsg.norm_rotary(bf(2, 3, 8), q_weight=m(8)), "q_weight must have"),
            (lambda: nsg.norm_rotary_grad(bf(2, 3, 8), bf(2, 3, 8), q_param=(0, 1, 8)), "accum is needed"),
            (lambda: nsg.rotary_frequencies(7), "even"), (lambda: nsg.rotary_frequencies(8, sections=[1, 2]), "add up")):
        with pytest.raises(ValueError, match=word):
            call()


@pytest.fixture
def machine(monkeypatch):
    """The binding over stand-ins, with the layers' functions too."""
    calls = []
    with standin.machine(monkeypatch) as m:
        keep, P = [], ctypes.c_void_p

        def recorder(name, *types):
            def call(*args):
                calls.append((name, args))
                return 0
            keep.append(ctypes.CFUNCTYPE(ctypes.c_int, *types)(call))
            return ctypes.cast(keep[-1], P).value
        I, I64, F, Z, U, D = (ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint32, P)
        table = {n: ctypes.cast(getattr(nsg.lib(), n), P).value for n in nsg.EXPORTED
                 if n.startswith(("muon_linear", "muon_dropout", "muon_norm_rotary"))}
        table.update(muon_linear=recorder("linear", P, P, Z, P), muon_linear_grad=recorder("linear_grad", P, P, Z, P),
                     muon_dropout=recorder("dropout", P, I64, P, I64, P, I64, I, I64, I, F, P, U, P),
                     muon_norm_rotary=recorder("rotary", D, I, I, I64, I, I, F, P, I, I, P, P, I, I, P))
        nsg._native().init_layers(table)
        m.layer_calls = calls
        yield m


def test_copies_and_calls_are_on_the_stream_of_the_call(machine):
    m = machine
    x = torch.zeros(2, 5, 8, dtype=torch.bfloat16)
    w = m.tensor(torch.zeros(4, 8, dtype=torch.bfloat16))
    for stream, handle in ((m.on_stream(7), 7), (9, 9), (None, 0)):
        m.copies.clear()
        m.layer_calls.clear()
        y = nsg.linear(m.tensor(x[:, :-1]), w, stream=stream)
        assert m.copies == [handle] and tuple(y.shape) == (2, 4, 4)
        nsg.dropout(m.tensor(x), 0.0, None, stream=stream)
        assert m.copies == [handle]   # the batch is a matrix in memory
        assert [(c[1][-1] or 0) for c in m.layer_calls] == [handle, handle]
    with pytest.raises(ValueError, match="another device"):
        nsg.linear(m.tensor(x), w, stream=m.on_stream(7, 1))


def test_tensors_on_another_device_make_it_current(machine):
    m = machine
    x, w = m.tensor(torch.zeros(3, 8, dtype=torch.bfloat16), 1), m.tensor(torch.zeros(4, 8, dtype=torch.bfloat16), 1)
    nsg.linear(x, w)
    nsg.norm_rotary(m.tensor(torch.zeros(3, 2, 8), 1), norm=True)
    nsg.dropout(m.tensor(torch.zeros(3, 8), 1), 0.0, None)
    assert [c[0] for c in m.layer_calls] == ["linear", "rotary", "dropout"] and m.device == 0
    with pytest.raises(ValueError, match="one device"):
        nsg.linear(x, m.tensor(torch.zeros(4, 8, dtype=torch.bfloat16), 0))


@pytest.mark.parametrize("shape", [(0, 3), (2, 0, 3), (0,)])
def test_no_tokens_on_several_axes(machine, shape):
    """Positions of an empty batch say nothing about their axes: the pairs' do."""
    freq, axis = nsg.rotary_frequencies(8, sections=[1, 1, 2])
    x = machine.tensor(torch.zeros(*shape[:-1], 2, 8) if len(shape) > 1 else torch.zeros(0, 2, 8))
    nsg.norm_rotary(x, None, machine.tensor(torch.zeros(shape, dtype=torch.int64)), freq, axis)
    args = machine.layer_calls[-1][1]
    assert args[3] == 0 and args[9] == 3


# ------------------------------------------------------------------ the forms

@pytest.mark.parametrize("kind", ["relu", "relu2", "gelu", "silu"])
def test_slopes_against_differences(kind):
    u = torch.linspace(-9, 9, 400, dtype=torch.float64) + 1e-3
    h = 1e-6
    diff = (forms.act(u + h, kind)[0] - forms.act(u - h, kind)[0]) / (2 * h)
    assert torch.allclose(forms.act(u, kind)[1], diff, atol=1e-8)


@pytest.mark.parametrize("norm,interleaved", [(True, False), (True, True), (False, False)])
def test_head_gradients_against_differences(norm, interleaved):
    gen = torch.Generator().manual_seed(1)
    x, d = (torch.randn((3, 2, 10), generator=gen, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.1 * torch.randn(10, generator=gen, dtype=torch.float64)
    freq, axis = nsg.rotary_frequencies(8, 100.0, [1, 3])
    cos, sin = forms.rotation(torch.tensor([[1, 2], [0, 5], [9, 1]]), freq, axis)
    f = lambda x, w: (d * forms.heads_forward(x, w, norm, 1e-3, cos, sin, interleaved)).sum()  # noqa: E731
    dx, dw = forms.heads_backward(d, x, w, norm, 1e-3, cos, sin, interleaved)
    h = 1e-6
    for t, grad, other in ((x, dx, lambda v: f(v, w)), (w, dw, lambda v: f(x, v))):
        if grad is None:
            continue
        for i in range(t.numel()):
            e = torch.zeros_like(t).view(-1)
            e[i] = h
            diff = (other(t + e.view(t.shape)) - other(t - e.view(t.shape))) / (2 * h)
            assert abs(float(diff - grad.reshape(-1)[i])) < 1e-7


def test_philox_words():
    """The words that the method's authors publish for a counter and key of zeros."""
    bits = forms.draws(1, 8, 0, 0, 0)[0]
    words = [int(bits[2 * i]) | int(bits[2 * i + 1]) << 16 for i in range(4)]
    assert words == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def test_frequencies():
    freq, axis = nsg.rotary_frequencies(8, 100.0)
    assert np.allclose(freq, 100.0 ** (-np.arange(4) / 4)) and not axis.any() and axis.dtype == np.int32
    freq, axis = nsg.rotary_frequencies(12, 100.0, [2, 1, 3])
    assert axis.tolist() == [0, 0, 1, 2, 2, 2] and np.allclose(freq, 100.0 ** (-np.arange(6) / 6))
    freq, _ = nsg.rotary_frequencies(12, 100.0, [2, 1, 3], own_ladder=True)
    assert np.allclose(freq, 100.0 ** -np.array([0, 0.5, 0, 0, 1 / 3, 2 / 3]))
