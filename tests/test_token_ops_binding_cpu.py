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


def test_a_stream_of_another_device_is_refused(m):
    """Nothing may be skipped in silence: the call computes, or it raises."""
    args = grad_inputs(m, torch.zeros(4, 8))
    z, y = m.tensor(torch.zeros(4, 8)), m.tensor(torch.zeros(4, dtype=torch.int64))
    a = m.tensor(torch.zeros(4))
    offsets = m.tensor(torch.zeros(3, dtype=torch.int64))
    away = m.on_stream(7, 1)
    for call in (lambda: nsg.embedding_grad(*args, stream=away), lambda: nsg.embedding(z, y, stream=away),
                 lambda: nsg.token_logprobs(z, y, stream=away), lambda: nsg.policy_loss(z, y, a, a, stream=away),
                 lambda: nsg.preference_loss(z, y, offsets, stream=away)):
        with pytest.raises(ValueError, match="another device"):
            call()
        assert (m.device, m.stream) == (0, 0)
    assert m.calls == []


def test_tensors_of_another_device_than_the_current_one(m):
    """The call makes their device current, with its stream or the given one."""
    accum, dout, ids, param = grad_inputs(m, torch.zeros(4, 8))
    for t in (accum, dout, ids):
        t.index, t.device.index = 1, 1
    assert nsg.embedding_grad(accum, dout, ids, param) is accum
    assert nsg.embedding_grad(accum, dout, ids, param, stream=m.on_stream(7, 1)) is accum
    assert nsg.embedding_grad(accum, dout, ids, param, stream=9) is accum
    assert [c[1][-1] or 0 for c in m.calls] == [0, 7, 9] and m.device == 0


def test_a_workspace_has_to_be_contiguous(m):
    """An expanded tensor has less memory than elements; between the elements
    of a slice lies what is somebody else's."""
    args = grad_inputs(m, torch.zeros(2000, 8))
    z, y = m.tensor(torch.zeros(4, 8)), m.tensor(torch.zeros(4, dtype=torch.int64))
    offsets = m.tensor(torch.zeros(3, dtype=torch.int64))
    need = max(nsg.embedding_grad_workspace(2000, 8), nsg.preference_loss_workspace(4))
    whole = torch.empty(2 * need, dtype=torch.uint8)
    for bad in (torch.empty(1, dtype=torch.uint8).expand(need), whole[::2]):
        work = m.tensor(bad)
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            nsg.embedding_grad(*args, workspace=work)
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            nsg.preference_loss(z, y, offsets, workspace=work)
    assert m.calls == []
    work = m.tensor(whole[:need].view(torch.int32) if need % 4 == 0 else whole[:need])
    nsg.embedding_grad(*args, workspace=work)
    nsg.preference_loss(z, y, offsets, workspace=work)
    (_, g), (_, p) = m.calls
    assert g[-3] == p[-3] == whole.data_ptr() and g[-2] == p[-2] == need


@pytest.mark.parametrize("dtype,per", [(torch.bfloat16, 8), (torch.float32, 4)])
@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_a_new_gradient_is_no_larger_than_its_rows(m, dtype, per, loss):
    """logits[:, -1] of a batch of sequences: the new gradient's rows lie as the
    logits' do against 16 bytes, without the sequences between them."""
    for rows, vocab, stride in ((3, 1000, 40 * 1000), (1, 1000, 40 * 1000), (3, 1001, 40 * 1001), (1, 7, 7 * 9),
                                (3, 1000, 1000), (3, 1000, 1024), (3, 1001, 1002), (5, 1001, 1001), (2, 1, 1), (3, 1, 77)):
        z = m.tensor(torch.zeros(rows * stride, dtype=dtype).view(rows, stride)[:, :vocab])
        y = m.tensor(torch.zeros(rows, dtype=torch.int64))
        a = m.tensor(torch.zeros(rows))
        m.calls.clear()
        m.made.clear()
        if loss == "policy":
            d = nsg.policy_loss(z, y, a, a)["dlogits"]
        else:
            d = nsg.preference_loss(z, y, m.tensor(torch.zeros(3, dtype=torch.int64)))["dlogits"]
        made = m.made[0]   # the buffer behind it
        (_, call), = m.calls
        given = call[2], call[-2 if loss == "policy" else -4]
        assert d.shape == (rows, vocab) and d.dtype == dtype and d.data_ptr() == made.data_ptr()
        assert given[1] == made.shape[1] and vocab <= given[1] < vocab + per
        assert rows == 1 or (given[0] == stride and given[1] % per == stride % per and d.stride()[0] == given[1])
        if stride == vocab:
            assert d.is_contiguous() and made.shape == (rows, vocab)
