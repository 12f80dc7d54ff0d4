"""The builder where the Python binding's C half cannot be compiled, or was
compiled for another interpreter; and which tests run beside a GPU."""
import os
import pathlib
import sys
import sysconfig
import types

import pytest

import newton_schulz_fp32_gb300 as nsg
from newton_schulz_fp32_gb300 import builder


def test_the_library_is_built_without_pythons_headers(monkeypatch, tmp_path):
    """The Muon step goes through ctypes and needs none of them."""
    nsg.build()
    monkeypatch.setattr(builder, "HERE", str(tmp_path))   # where the binding is looked for
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a: {"include": str(tmp_path)})
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert builder.build() == builder.LIB
    assert os.listdir(tmp_path) == []


def test_the_binding_is_this_interpreters(monkeypatch, tmp_path):
    """Its name says for which interpreter it is, so that another one does not
    load it."""
    nsg.build()
    monkeypatch.setattr(builder, "HERE", str(tmp_path))
    builder.build()
    assert os.listdir(tmp_path) == ["_binding" + sysconfig.get_config_var("EXT_SUFFIX")]
    built = os.path.getmtime(tmp_path / os.listdir(tmp_path)[0])
    builder.build()
    assert os.path.getmtime(tmp_path / os.listdir(tmp_path)[0]) == built


def test_made_up_addresses_stay_away_from_a_gpu(monkeypatch):
    """Beside a GPU's device node the refusal tests are skipped, torch or not."""
    import conftest
    marks = []
    items = [types.SimpleNamespace(path=pathlib.Path("tests") / name, add_marker=lambda m, n=name: marks.append((n, m.name)))
             for name in (conftest.MADE_UP_ADDRESSES, "test_library_cpu.py")]
    assert (pathlib.Path(conftest.__file__).parent / conftest.MADE_UP_ADDRESSES).exists()
    monkeypatch.setattr(conftest, "gpu_nodes", lambda: [])
    conftest.pytest_collection_modifyitems(items)
    assert marks == []
    monkeypatch.setattr(conftest, "gpu_nodes", lambda: ["/dev/nvidia0"])
    conftest.pytest_collection_modifyitems(items)
    assert marks == [(conftest.MADE_UP_ADDRESSES, "skip")]


def test_calls_without_the_binding_say_so(monkeypatch):
    torch = pytest.importorskip("torch")
    nsg.build()
    monkeypatch.setattr(nsg, "_bound", None)
    monkeypatch.delattr(nsg, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "newton_schulz_fp32_gb300._binding", None)
    with pytest.raises(nsg.MuonError, match="build it"):
        nsg.token_logprobs(torch.zeros(1, 2), torch.zeros(1, dtype=torch.int64))
