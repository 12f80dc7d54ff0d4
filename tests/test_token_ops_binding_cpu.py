"""What the Python entry points of the embedding and loss operators do around
the library's calls: streams, devices, copies, scratch and outputs, over
stand-ins for CUDA tensors."""
import numpy as np
import pytest

import newton_schulz_fp32_gb300 as nsg
import standin

torch = pytest.importorskip("torch")


@pytest.fixture
def m(monkeypatch):
    with standin.machine(monkeypatch) as machine:
        yield machine


def grad_inputs(m, dout):
    n = dout.numel() // dout.shape[-1]
    return (m.tensor(torch.zeros(10 * dout.shape[-1])), m.tensor(dout), m.tensor(torch.zeros(n, dtype=torch.int64)),
            (0, 10, dout.shape[-1]))


def test_a_gradient_that_has_to_be_copied_is_copied_on_the_calls_stream(m):
    """dx[:, :-1] is no matrix: its copy has to follow what `stream` waited
    for, and to be finished before the kernels on `stream`."""
    dx = torch.arange(2.0 * 5 * 8).view(2, 5, 8)
    args = grad_inputs(m, dx[:, :-1])
    for stream, handle in ((m.on_stream(7), 7), (9, 9), (None, 0)):
        m.copies.clear()
        m.calls.clear()
        nsg.embedding_grad(*args, stream=stream)
        assert m.copies == [handle]
        (_, call), = m.calls
        assert (call[-1] or 0) == handle and call[2] != dx.data_ptr() and call[4] == 8 and call[7] == 8


def test_a_gradient_that_is_a_matrix_in_memory_is_not_copied(m):
    dx = torch.zeros(2, 4, 8)
    nsg.embedding_grad(*grad_inputs(m, dx), stream=5)
    (_, call), = m.calls
    assert m.copies == [] and call[2] == dx.data_ptr() and call[-1] == 5
