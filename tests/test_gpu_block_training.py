"""The layer operators together, as the block-training example runs them: that it
runs, the same way twice, and that its gradients are those of the model.

The gradients' bound: the reference is the model in 64 bits over the same bf16
weights and masks.  Between the loss and a parameter lie at most 20 roundings to
bf16 on the way there and back (12 activations, 8 gradients), each at most 2^-8 of
the value rounded; to first order their effects add, each as large relative to
the gradient as the rounding to its value, up to how much a layer's
condition enlarges it, for which a factor of 2 is allowed: 40 * 2^-8 = 0.16 in
norm (their signs are random, so what is seen is several times less)."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layer_forms as forms  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D64 = torch.float64


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import block_training
    block_training.nsg.build()
    return block_training


def reference_loss(ex, model, w, tokens, targets, weights):
    """The model's loss in 64 bits, differentiable in w."""
    rows, length = tokens.shape
    x0 = w["embed"][tokens].view(-1, ex.DIM)
    q, k, v = model.heads(x0 @ w["qkv"].T)
    cos, sin = forms.rotation(model.positions(tokens), *model.turns)

    def head(x, weight):
        n = x / torch.sqrt((x * x).mean(2, keepdim=True) + 1e-6) * weight
        a, b, c, s = n[..., :ex.HEAD // 2], n[..., ex.HEAD // 2:], cos[:, None], sin[:, None]
        return torch.cat([a * c - b * s, b * c + a * s], 2).view(rows, length, -1, ex.HEAD)

    mixed = ex.attention(head(q, w["q_norm"][0]), head(k, w["k_norm"][0]), v.reshape(rows, length, -1, ex.HEAD))
    keep = [forms.keep(rows * length, ex.DIM, ex.RATE, model.rng, site, "cuda") for site in (0, 1)]
    x1 = x0 + keep[0] * (mixed.reshape(-1, ex.HEADS * ex.HEAD) @ w["out"].T)
    h = forms.act(x1 @ w["up"].T + w["up_bias"][0], "gelu")[0]
    x2 = x1 + keep[1] * (h @ w["down"].T)
    logp = torch.log_softmax(x2 @ w["head"].T, 1)
    y = targets.reshape(-1)
    return -(weights.double() * torch.where(y >= 0, logp.gather(1, y.clamp(min=0)[:, None])[:, 0], 0.0)).sum()


def test_gradients_are_the_models(example):
    model = example.Model(5)
    data = example.batch(torch.Generator(device="cuda").manual_seed(2), rows=6, length=29)
    model.accum.fill_(float("nan"))   # every parameter's gradient is put there, none added to what was
    loss = model.gradients(*data)
    w = {n: v.to(D64).requires_grad_() for n, v in model.w.items()}
    want = reference_loss(example, model, w, *data)
    grads = dict(zip(w, torch.autograd.grad(want, list(w.values()))))
    assert abs(float(loss) - float(want.detach())) < 0.16 * abs(float(want.detach()))
    for name, got in model.views(model.accum).items():
        off = float((got.double() - grads[name]).norm() / grads[name].norm())
        assert off < 0.16, (name, off)
    assert example.nsg.device_error() == 0


def test_a_step_of_the_gradient_changes_the_loss_by_its_square(example):
    """The 64-bit loss along the kernels' gradient: its difference over 2 h against <gradient, direction>.
    The direction is the kernels' own gradient g, so the two agree up to its relative error, 0.16 of |g|^2."""
    model = example.Model(6)
    data = example.batch(torch.Generator(device="cuda").manual_seed(3), rows=4, length=16)
    model.gradients(*data)
    g = {n: v.to(D64) for n, v in model.views(model.accum).items()}
    size = sum(float((v * v).sum()) for v in g.values())
    h = 1e-4 / size ** 0.5
    at = lambda t: float(reference_loss(example, model, {n: v.to(D64) + t * g[n] for n, v in model.w.items()}, *data))  # noqa: E731
    assert abs((at(h) - at(-h)) / (2 * h) - size) < 0.16 * size


def test_training_runs_and_is_reproducible(example):
    masters = []
    for _ in range(2):
        model, gen = example.Model(3), torch.Generator(device="cuda").manual_seed(4)
        losses = [model.train(*example.batch(gen, rows=8)) for _ in range(3)]
        assert all(bool(torch.isfinite(v)) for v in losses) and bool(torch.isfinite(model.master).all())
        masters.append(model.master.clone())
    assert torch.equal(masters[0], masters[1])
    assert example.nsg.device_error() == 0


def test_a_captured_step_draws_anew(example):
    """Forward and backward captured once and replayed: the same bits as eager calls at the same dropout step."""
    model = example.Model(7)
    data = example.batch(torch.Generator(device="cuda").manual_seed(5), rows=4)
    want = []
    for step in (0, 1):
        model.rng[1] = step
        model.gradients(*data)
        want.append(model.accum.clone())
    assert not torch.equal(*want)
    model.rng[1] = 0
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.gradients(*data)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        model.gradients(*data)
    for step in (1, 0, 1):
        model.rng[1] = step
        model.accum.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(model.accum, want[step])
