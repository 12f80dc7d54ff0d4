"""Embedding and loss calls on tensors as programs have them: batches of
sequences, slices of them, a workspace of the caller's, other streams."""
import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    nsg.build()
    return t


def batch(torch, B, S, D, V, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, V, (B, S), generator=gen, device="cuda")
    return ids, torch.randn((B, S + 1, D), generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("shape", [(3, 5, 8), (4, 300, 33), (2, 2000, 64)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_gradient_of_batches_and_slices(torch, shape, dtype):
    """dout of three dimensions: as it is, without its last step (no matrix in
    memory), and in the order sequence, batch; the same bits as the matrix."""
    B, S, D = shape
    V = 50
    ids, dx = batch(torch, B, S, D, V, getattr(torch, dtype), S)
    for part, index in ((dx[:, :-1].contiguous(), ids), (dx[:, :-1], ids),
                        (dx[:, :-1].transpose(0, 1), ids.t().contiguous())):
        want, got = torch.zeros(V * D, device="cuda"), torch.zeros(V * D, device="cuda")
        nsg.embedding_grad(want, part.reshape(-1, D).clone(), index.reshape(-1), (0, V, D))
        nsg.embedding_grad(got, part, index, (0, V, D))
        assert torch.equal(got, want)
    assert nsg.device_error() == 0


@pytest.mark.parametrize("S", [300, 2000])
def test_copied_gradient_on_another_stream(torch, S):
    """The current stream is kept busy after the side stream has what it needs:
    a copy made on the current one would be read before it is there."""
    B, D, V = 2, 64, 50
    ids, dx = batch(torch, B, S, D, V, torch.float32, S)
    want = torch.zeros(V * D, device="cuda")
    nsg.embedding_grad(want, dx[:, :-1].reshape(-1, D).clone(), ids, (0, V, D))
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = torch.zeros(V * D, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        busy = torch.randn((4096, 4096), device="cuda")
        for _ in range(20):
            busy = busy @ busy * 1e-2
        nsg.embedding_grad(got, dx[:, :-1], ids, (0, V, D), stream=stream)
        side.synchronize()
        assert torch.equal(got, want)
        torch.cuda.synchronize()


def test_logits_of_batches(torch):
    """Logits and targets of three and two dimensions: the same bits as matrices."""
    B, S, V = 3, 7, 1001
    gen = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn((B, S, V), generator=gen, device="cuda").to(torch.bfloat16)
    y = torch.randint(0, V, (B, S), generator=gen, device="cuda")
    adv, w, old = (torch.rand((B, S), generator=gen, device="cuda") for _ in range(3))
    flat = z.view(-1, V)
    lp = nsg.token_logprobs(z, y)
    assert lp.shape == (B, S) and torch.equal(lp.view(-1), nsg.token_logprobs(flat, y.view(-1)))
    a = nsg.policy_loss(z, y, adv, w, old - 7)
    b = nsg.policy_loss(flat, y.view(-1), adv.view(-1), w.view(-1), old.view(-1) - 7)
    assert a["dlogits"].shape == (B * S, V) and torch.equal(a["dlogits"], b["dlogits"])
    assert torch.equal(a["stats"], b["stats"])
    offsets = torch.tensor([0, 7, 21], device="cuda")
    c, d = nsg.preference_loss(z, y, offsets), nsg.preference_loss(flat, y.view(-1), offsets)
    assert torch.equal(c["dlogits"], d["dlogits"]) and torch.equal(c["margins"], d["margins"])
    with pytest.raises(RuntimeError):
        nsg.token_logprobs(z[:, :-1], y[:, :-1].contiguous())   # no matrix in memory: refused
    own = z.clone()
    nsg.policy_loss(own, y, adv, w, old - 7, dlogits=own)
    assert torch.equal(own.view(-1, V), a["dlogits"])


@pytest.mark.parametrize("V", [131072, 50001, 33000])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [1, 64, 700])
def test_policy_gradient_in_place_of_rows_over_several_blocks(torch, V, dtype, T):
    """The target anywhere in a row that several blocks hold, the gradient in
    place of the logits: the same bits as beside them."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    z = torch.randn((T, V), generator=gen, device="cuda").to(getattr(torch, dtype))
    borders = [0, 1, 7, 8, V - 1, V - 2, V - 9] + [k * V // 8 + d for k in range(1, 8) for d in (-9, -1, 0, 1, 8)]
    y = torch.tensor([borders[t % len(borders)] for t in range(T)], device="cuda")
    adv, w = torch.randn(T, generator=gen, device="cuda"), torch.rand(T, generator=gen, device="cuda")
    w[T // 3] = 0 if T > 1 else 1
    lp = nsg.token_logprobs(z, y)
    old = lp - 0.1 * torch.randn(T, generator=gen, device="cuda")
    want = nsg.policy_loss(z, y, adv, w, old, lp, kl_coef=0.1)
    for _ in range(3):
        own = z.clone()
        got = nsg.policy_loss(own, y, adv, w, old, lp, kl_coef=0.1, dlogits=own)
        assert torch.equal(own, want["dlogits"])
        assert torch.equal(got["logp"], want["logp"]) and torch.equal(got["stats"], want["stats"])
    assert nsg.device_error() == 0


@pytest.mark.parametrize("T", [1025, 5000, 40000])
def test_workspace_of_the_callers(torch, T):
    """A workspace of exactly the bytes asked for: the same bits as with a new
    one, and nothing written past it; a byte less is refused."""
    D, V = 24, 700
    gen = torch.Generator(device="cuda").manual_seed(T)
    ids = (700 ** torch.rand(T, generator=gen, device="cuda") - 1).long()
    dout = torch.randn((T, D), generator=gen, device="cuda")
    z = torch.randn((T, 65), generator=gen, device="cuda")
    offsets = torch.tensor([0, T // 3, T // 2, T - 5, T], device="cuda")
    y = torch.randint(-9, 65, (T,), generator=gen, device="cuda")
    want = torch.zeros(V * D, device="cuda")
    nsg.embedding_grad(want, dout, ids, (0, V, D))
    loss = nsg.preference_loss(z, y, offsets)
    for need, call in ((nsg.embedding_grad_workspace(T, D), "grad"), (nsg.preference_loss_workspace(T), "loss")):
        whole = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        got = torch.zeros(V * D, device="cuda")
        if call == "grad":
            nsg.embedding_grad(got, dout, ids, (0, V, D), workspace=whole[:need])
            assert torch.equal(got, want)
            with pytest.raises(nsg.MuonError, match="workspace"):
                nsg.embedding_grad(got, dout, ids, (0, V, D), workspace=whole[:need - 1])
        else:
            again = nsg.preference_loss(z, y, offsets, workspace=whole[:need])
            assert all(torch.equal(again[k], loss[k]) for k in loss)
            with pytest.raises(nsg.MuonError, match="workspace"):
                nsg.preference_loss(z, y, offsets, workspace=whole[:need - 1])
        assert bool((whole[need:] == 0xA5).all())
    assert nsg.device_error() == 0


@pytest.mark.parametrize("V", [1000, 1001, 40003])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_logits_of_the_last_step(torch, V, dtype):
    """logits[:, -1] of a batch of sequences: the new gradient takes its own
    rows' memory, and has the bits of a contiguous copy's."""
    B, S = 5, 9
    gen = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((B, S, V), generator=gen, device="cuda").to(getattr(torch, dtype))[:, -1]
    y = torch.randint(0, V, (B,), generator=gen, device="cuda")
    adv, w = (torch.rand(B, generator=gen, device="cuda") for _ in range(2))
    offsets = torch.tensor([0, 2, 5], device="cuda")
    for call in (lambda x: nsg.policy_loss(x, y, adv, w), lambda x: nsg.preference_loss(x, y, offsets)):
        got = call(z)["dlogits"]
        assert got.untyped_storage().nbytes() < B * (V + 8) * got.element_size()
        laid = torch.empty_strided((B, V), got.stride(), dtype=z.dtype, device="cuda").copy_(z)
        if z.data_ptr() % 16 == 0:
            assert torch.equal(got, call(laid)["dlogits"])
    assert nsg.device_error() == 0
