"""The block-training example's loss and gradients against the model in 64 bits on
the host, as near as roundings without a sign leave them.

Bounds.  A rounding to bf16 is off by 2^-8 / sqrt(3) of the value in root mean square
at most.  Between the loss and a parameter lie at most 20 of them (12 activations, 8
gradients), whose errors have no common sign and add as their squares:
sqrt(20) * 2^-8 / sqrt(3) = 0.0101 of the gradient, up to how much the model's
condition enlarges it, for which a factor of 2 is allowed, and 2 again as a margin:
0.04.  The logits have 12 roundings behind them: 0.0156 of their size with the factor
of 2; a token's log-probability is off by sqrt(2) times that at most in root mean
square, and the weighted mean over the tokens by no more; with the margin 0.045 of the
logits' root mean square.

A factor that is missing on the way back is seen: with dropout at 0.1 the kept
elements' 65536 / (65536 - 6554) is 1.11, so that what passes one dropout without it is
0.1 off."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layer_forms as forms  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D64 = torch.float64
GRADIENT, LOGITS = 0.04, 0.045


@pytest.fixture(scope="module")
def example(cuda_device):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import block_training
    block_training.nsg.build()
    return block_training


class Drop(torch.autograd.Function):
    """x * there on the way there, times `back` on the way back."""

    @staticmethod
    def forward(ctx, x, there, back):
        ctx.back = back
        return x * there

    @staticmethod
    def backward(ctx, g):
        return g * ctx.back, None, None


def reference(ex, model, w, tokens, targets, weights, forget=False):
    """The model's loss and logits in 64 bits on the host; forget: dropout's factor is left out on the way back."""
    rows, length = tokens.shape
    x0 = w["embed"][tokens].view(-1, ex.DIM)
    q, k, v = model.heads(x0 @ w["qkv"].T)
    cos, sin = forms.rotation(torch.arange(length).expand(rows, length).reshape(-1, 1), *model.turns)

    def head(x, weight):
        n = x / torch.sqrt((x * x).mean(2, keepdim=True) + 1e-6) * weight
        return forms.turned(n, cos, sin, False).view(rows, length, -1, ex.HEAD)

    def drop(x, site):
        keep = forms.keep(rows * length, ex.DIM, ex.RATE, model.rng, site)
        return Drop.apply(x, keep, (keep > 0).to(D64) if forget else keep)

    mixed = ex.attention(head(q, w["q_norm"][0]), head(k, w["k_norm"][0]), v.reshape(rows, length, -1, ex.HEAD))
    x1 = x0 + drop(mixed.reshape(-1, ex.HEADS * ex.HEAD) @ w["out"].T, 0)
    h = forms.act(x1 @ w["up"].T + w["up_bias"][0], "gelu")[0]
    logits = (x1 + drop(h @ w["down"].T, 1)) @ w["head"].T
    y = targets.reshape(-1)
    logp = torch.log_softmax(logits, 1).gather(1, y.clamp(min=0)[:, None])[:, 0]
    return -(weights.to(D64) * torch.where(y >= 0, logp, 0.0)).sum(), logits.detach()


def host(w):
    return {n: v.to("cpu", D64) for n, v in w.items()}


@pytest.mark.parametrize("seed,rows,length", [(5, 6, 29), (11, 3, 64)])
def test_loss_and_gradients(example, seed, rows, length):
    model = example.Model(seed)
    data = example.batch(torch.Generator(device="cuda").manual_seed(seed), rows, length)
    on_host = [t.cpu() for t in data]
    loss = float(model.gradients(*data))
    got = host(model.views(model.accum))
    w = {n: v.requires_grad_() for n, v in host(model.w).items()}
    want, logits = reference(example, model, w, *on_host)
    assert abs(loss - float(want.detach())) <= LOGITS * float(logits.square().mean().sqrt())
    grads = dict(zip(w, torch.autograd.grad(want, list(w.values()))))
    far = {n: float((got[n] - g).norm() / g.norm()) for n, g in grads.items()}
    assert max(far.values()) <= GRADIENT, far
    # the same bound tells a missing factor
    forgotten, _ = reference(example, model, w, *on_host, forget=True)
    grads = dict(zip(w, torch.autograd.grad(forgotten, list(w.values()))))
    for n in ("down", "up", "up_bias", "out"):   # all of their gradients passes through a dropout
        assert float((got[n] - grads[n]).norm() / grads[n].norm()) > GRADIENT, n


def test_along_the_gradient(example):
    """The 64-bit loss's difference along the kernels' gradient g against |g|^2."""
    model = example.Model(6)
    data = example.batch(torch.Generator(device="cuda").manual_seed(3), rows=4, length=16)
    model.gradients(*data)
    on_host, g, w = [t.cpu() for t in data], host(model.views(model.accum)), host(model.w)
    size = sum(float((v * v).sum()) for v in g.values())
    h = 1e-4 / size ** 0.5
    at = lambda t: float(reference(example, model, {n: v + t * g[n] for n, v in w.items()}, *on_host)[0])  # noqa: E731
    assert abs((at(h) - at(-h)) / (2 * h) - size) <= GRADIENT * size
