"""Arguments of heads that are seldom seen, on the host: positions without a rotation are looked at, checked and
passed on; arrays of another byte order are refused."""

import numpy as np
import pytest

import newton_schulz_fp32_gb300 as nsg

torch = pytest.importorskip("torch")
from test_layer_ops_cpu import FAKE, STEP, heads, lib, machine, no_gpu, refused, rotary  # noqa: E402,F401


@no_gpu
@pytest.mark.parametrize("kind", [nsg.Heads, nsg.HeadsGrad])
@pytest.mark.parametrize("change,word", [
    (dict(pos=FAKE + 4), "positions"), (dict(pt=2), "positions_type"), (dict(axes=0), "axes"), (dict(axes=9), "axes"),
    (dict(pos=None), "overlaps")])
def test_positions_without_a_rotation_are_checked(lib, change, word, kind):  # noqa: F811
    if word == "overlaps":
        change = dict(pos=FAKE + (2 if kind is nsg.Heads else 3) * STEP)   # where the result lies
    refused(lib, rotary(lib, [heads(kind)], pairs=0, freq=None, axis=None, **change), word)


@pytest.mark.parametrize("shape,type_,axes", [((5,), torch.int32, 1), ((5, 3), torch.int64, 3)])
@pytest.mark.parametrize("freq", [None, np.empty(0)])
def test_positions_reach_the_library(machine, shape, type_, axes, freq):  # noqa: F811
    pos = torch.zeros(shape, dtype=type_)
    nsg.norm_rotary(machine.tensor(torch.zeros(5, 2, 8)), None, machine.tensor(pos), freq)
    args = machine.layer_calls[-1][1]
    assert args[7] == pos.data_ptr() and args[8] == (type_ is torch.int64) and args[9] == axes and args[12] == 0
    nsg.norm_rotary(machine.tensor(torch.zeros(5, 2, 8)), None, None, freq)
    assert not machine.layer_calls[-1][1][7]
    for bad in (torch.zeros(4, dtype=type_), torch.zeros(5), torch.zeros((5, 2), dtype=type_)[:, 0]):
        with pytest.raises(ValueError, match="positions"):
            nsg.norm_rotary(machine.tensor(torch.zeros(5, 2, 8)), None, machine.tensor(bad), freq)


def test_arrays_of_another_byte_order_are_refused(machine):  # noqa: F811
    """Their bytes would be read the wrong way round."""
    q, pos = machine.tensor(torch.zeros(5, 2, 8)), machine.tensor(torch.zeros(5, dtype=torch.int64))
    freq, axis = np.ones(4), np.zeros(4, dtype=np.int32)
    for f, a, word in ((freq.astype(">f8"), axis, "inv_freq must be"), (freq, axis.astype(">i4"), "axis must be")):
        with pytest.raises(ValueError, match=word):
            nsg.norm_rotary(q, None, pos, f, a)
    for f, a in ((freq, axis), (freq.astype("<f8"), axis.astype("<i4"))):
        nsg.norm_rotary(q, None, pos, f, a)
    assert len(machine.layer_calls) == 2
