"""Post-training a small language model with the Muon step: a policy loss on
sampled tokens, then a preference loss on pairs of answers.

The model predicts the next token from the current one: an embedding, one
hidden matrix (trained by Muon) and an output head.  Embedding and head are
auxiliary parameters of the same flat FP32 buffers and get the fused Adam
step.  Per training step:

    embedding       tokens -> activations
    token_logprobs  the frozen reference's scores of the sampled tokens
    policy_loss /   loss and the gradient of the logits, which replaces them
    preference_loss
    accumulate      the dense gradients (hidden matrix, head) into accum
    embedding_grad  the embedding's rows, straight into accum
    step_ex         Muon on the hidden matrix, Adam on embedding and head

Run:  python examples/post_training.py
"""
import math
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_fp32_gb300 as nsg  # noqa: E402

VOCAB, DIM = 64, 128


class Model:
    """Flat FP32 buffers of [embedding | hidden | head] and bf16 weights."""

    def __init__(self, seed=0):
        import torch
        self.torch = torch
        rows = [(VOCAB, DIM, 0), (DIM, DIM, 1), (VOCAB, DIM, 0)]
        self.params = np.zeros(3, dtype=nsg.PARAM_DTYPE)
        offset = 0
        for i, (r, c, muon) in enumerate(rows):
            self.params[i] = (offset, r, c, 0, muon)
            offset += r * c
        half = -(-offset // 256) * 128   # two partitions, as two ranks' slices laid side by side
        self.parts = np.array([(0, half, 0), (half, 2 * half, half)], dtype=nsg.PART_DTYPE)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        flat = lambda: torch.zeros(2 * half, device="cuda")  # noqa: E731
        self.accum, self.momentum, self.master, self.m, self.v = (flat() for _ in range(5))
        self.master.copy_(torch.randn(2 * half, generator=gen, device="cuda") / math.sqrt(DIM))
        self.dense = torch.zeros(2 * half, device="cuda", dtype=torch.bfloat16)
        self.steps = 0
        self.refresh()

    def views(self, flat):
        return [flat[int(p["offset"]):int(p["offset"]) + int(p["rows"]) * int(p["cols"])].view(int(p["rows"]), int(p["cols"]))
                for p in self.params]

    def refresh(self):
        self.table, self.hidden, self.head = (w.to(self.torch.bfloat16) for w in self.views(self.master))

    def forward(self, tokens):
        x = nsg.embedding(self.table, tokens, scale=math.sqrt(DIM))
        h = self.torch.tanh(x @ self.hidden.T)
        return x, h, h @ self.head.T

    def train(self, tokens, loss, lr):
        """One step on `loss(logits)`, which replaces the logits by their
        gradient and returns its statistics."""
        x, h, logits = self.forward(tokens)
        stats = loss(logits)
        d = logits                                              # now d loss / d logits
        da = (d @ self.head).float() * (1 - h.float() ** 2)
        da = da.to(self.torch.bfloat16)
        _, g_hidden, g_head = self.views(self.dense)
        g_hidden.copy_(da.T @ x)
        g_head.copy_(d.T @ h)
        nsg.accumulate(self.accum, self.dense, 1.0, overwrite=True, params=self.params[1:], parts=self.parts)
        nsg.embedding_grad(self.accum, da @ self.hidden, tokens, self.params[0], parts=self.parts,
                           scale=math.sqrt(DIM), overwrite=True)
        self.steps += 1
        nsg.step_ex(self.accum, self.momentum, self.master, self.params, self.parts, beta=0.9, lr=lr,
                    ns_method="standard", clip=1.0, operand_mode="bf16",
                    adam=dict(lr=lr, beta1=0.9, beta2=0.99, eps=1e-8, step=self.steps, exp_avg=self.m,
                              exp_avg_sq=self.v))
        self.refresh()
        return stats


def wanted(tokens):
    """The next token the task rewards."""
    return (5 * tokens + 3) % VOCAB


def policy_tuning(model, steps=60, tokens=4096, epochs=2, seed=1):
    """Samples from the policy, rewards the wanted token, and takes `epochs`
    clipped steps per sample, held near the starting model by the KL term.
    Returns the mean reward before each step."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ref = [w.clone() for w in (model.table, model.hidden, model.head)]
    rewards = []
    for _ in range(steps):
        ask = torch.randint(0, VOCAB, (tokens,), generator=gen, device="cuda")
        logits = model.forward(ask)[2]
        answer = torch.multinomial(torch.softmax(logits.float(), 1), 1, generator=gen)[:, 0]
        reward = (answer == wanted(ask)).float()
        rewards.append(float(reward.mean()))
        adv = (reward - reward.mean()) / (reward.std() + 1e-6)
        old = nsg.token_logprobs(logits, answer)
        h = torch.tanh(nsg.embedding(ref[0], ask, scale=math.sqrt(DIM)) @ ref[1].T)
        ref_logp = nsg.token_logprobs(h @ ref[2].T, answer)
        weights = torch.full((tokens,), 1.0 / tokens, device="cuda")
        for _ in range(epochs):
            model.train(ask, lambda z: nsg.policy_loss(z, answer, adv, weights, old, ref_logp, kl_coef=1e-3,
                                                       dlogits=z)["stats"], lr=0.02)
    return rewards


def preference_tuning(model, steps=20, pairs=64, length=16, seed=2):
    """Pairs of answers of which the first follows another rule more often.
    Returns the loss at every step."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ref = [w.clone() for w in (model.table, model.hidden, model.head)]
    losses = []
    offsets = torch.arange(2 * pairs + 1, device="cuda") * length
    for _ in range(steps):
        ask = torch.randint(0, VOCAB, (2 * pairs * length,), generator=gen, device="cuda")
        follows = torch.rand(ask.shape, generator=gen, device="cuda")
        follows = follows < torch.where(torch.arange(len(ask), device="cuda") < pairs * length, 0.8, 0.2)
        noise = torch.randint(0, VOCAB, ask.shape, generator=gen, device="cuda")
        answer = torch.where(follows, (ask + 1) % VOCAB, noise)
        answer[::length] = -100                                 # the first token of each is the prompt's
        h = torch.tanh(nsg.embedding(ref[0], ask, scale=math.sqrt(DIM)) @ ref[1].T)
        ref_logp = nsg.token_logprobs(h @ ref[2].T, answer)
        stats = model.train(ask, lambda z: nsg.preference_loss(z, answer, offsets, ref_logp, beta=0.1,
                                                               dlogits=z)["stats"], lr=0.01)
        losses.append(float(stats[0]))
    return losses


def main():
    nsg.build()
    model = Model()
    rewards = policy_tuning(model)
    print(f"policy tuning: mean reward {rewards[0]:.3f} -> {rewards[-1]:.3f}")
    losses = preference_tuning(model)
    print(f"preference tuning: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    assert nsg.device_error() == 0
    return rewards, losses


if __name__ == "__main__":
    main()
