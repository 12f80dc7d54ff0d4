"""Error codes of several operators, pending at once."""
import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu


def test_no_code_is_lost_beside_another():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nsg.build()
    table = torch.zeros((4, 8), device="cuda")
    z, y = torch.zeros((6, 9), device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda")
    assert nsg.device_error() == 0
    nsg.embedding(table, torch.tensor([0, 4], device="cuda"))                         # an id past the table
    nsg.preference_loss(z, y, torch.tensor([0, 3, 2], device="cuda"))                # offsets that decrease
    assert sorted(nsg.device_error() for _ in range(2)) == [17, 18]
    assert nsg.device_error() == 0
    nsg.token_logprobs(z, y + 9)                                                     # targets past the vocabulary
    nsg.embedding_grad(torch.zeros(32, device="cuda"), torch.zeros((1, 8), device="cuda"), y[:1] + 4, (0, 4, 8))
    assert [nsg.device_error() for _ in range(3)] == [17, 17, 0]
