"""Training a small attention block with the Muon step: every product, dropout,
norm and rotation of a training step through the library, gradients of all
parameters straight into the flat accumulation buffer.

The task is to name the token before the current one, which takes attention.
The matrices inside the block are trained by Muon, the rest (embedding, head, norm
weights, bias) by the fused Adam step.  Attention itself, small here, is torch's.
Per training step:

    embedding            tokens -> activations
    linear               queries, keys and values in one projection
    norm_rotary          queries and keys normalised and turned by position
    linear               output projection, dropout, added to the stream
    linear, linear       the feed-forward layer; its argument is kept
    linear, policy_loss  logits and the weighted cross entropy's gradient
    linear_grad,
    dropout,
    norm_rotary_grad     the way back, each parameter's gradient into accum
    embedding_grad       the embedding's rows, into accum
    step_ex              Muon on the matrices, Adam on the rest

Run:  python examples/block_training.py
"""
import math
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_fp32_gb300 as nsg  # noqa: E402

VOCAB, DIM, HEADS, KV, HEAD, WIDE, RATE = 64, 128, 4, 2, 32, 320, 0.1
PACKED = HEADS + 2 * KV

# name, rows, cols, trained by Muon
PARAMS = [("embed", VOCAB, DIM, 0), ("qkv", PACKED * HEAD, DIM, 1), ("q_norm", 1, HEAD, 0), ("k_norm", 1, HEAD, 0),
          ("out", DIM, HEADS * HEAD, 1), ("up", WIDE, DIM, 1), ("up_bias", 1, WIDE, 0), ("down", DIM, WIDE, 1),
          ("head", VOCAB, DIM, 0)]


def attention(q, k, v):
    """Causal attention of a batch (batch x time x heads x head), keys and values shared by groups of heads."""
    import torch
    k, v = (t.repeat_interleave(HEADS // KV, 2) for t in (k, v))
    s = torch.einsum("bthd,bshd->bhts", q, k) / math.sqrt(HEAD)
    past = torch.ones(s.shape[-2:], dtype=torch.bool, device=s.device).tril()
    return torch.einsum("bhts,bshd->bthd", torch.softmax(s.masked_fill(~past, -math.inf), -1), v)


class Model:
    """Flat FP32 buffers of the parameters above in two partitions, and bf16 weights."""

    def __init__(self, seed=0):
        import torch
        self.torch = torch
        self.params = np.zeros(len(PARAMS), dtype=nsg.PARAM_DTYPE)
        self.at, offset = {}, 0
        for i, (name, rows, cols, muon) in enumerate(PARAMS):
            self.params[i] = (offset, rows, cols, 0, muon)
            self.at[name] = self.params[i]
            offset += rows * cols
        half = -(-offset // 256) * 128
        self.parts = np.array([(0, half, 0), (half, 2 * half, half)], dtype=nsg.PART_DTYPE)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        flat = lambda: torch.zeros(2 * half, device="cuda")  # noqa: E731
        self.accum, self.momentum, self.master, self.m, self.v = (flat() for _ in range(5))
        for name, w in self.views(self.master).items():
            if name.endswith("norm"):
                w.fill_(1.0)
            elif name != "up_bias":
                w.copy_(torch.randn(w.shape, generator=gen, device="cuda") / math.sqrt(w.shape[1]))
        self.rng = torch.tensor([seed, 0], device="cuda")   # of dropout: seed, step
        self.turns = nsg.rotary_frequencies(HEAD)
        self.steps = 0
        self.refresh()

    def views(self, flat):
        return {name: flat[int(p["offset"]):int(p["offset"]) + int(p["rows"]) * int(p["cols"])].view(int(p["rows"]), int(p["cols"]))
                for name, p in self.at.items()}

    def refresh(self):
        self.w = {name: w.to(self.torch.bfloat16) for name, w in self.views(self.master).items()}

    def positions(self, tokens):
        b, t = tokens.shape
        return self.torch.arange(t, device="cuda").expand(b, t).reshape(b * t, 1).contiguous()

    def heads(self, qkv):
        """Queries, keys and values of a packed projection."""
        h = qkv.view(-1, PACKED, HEAD)
        return h[:, :HEADS], h[:, HEADS:HEADS + KV], h[:, HEADS + KV:]

    def forward(self, tokens):
        w, s = self.w, {}
        s["x0"] = nsg.embedding(w["embed"], tokens).view(-1, DIM)
        s["qkv"] = nsg.linear(s["x0"], w["qkv"])
        q, k, v = self.heads(s["qkv"])
        s["pos"] = self.positions(tokens)
        q, k = nsg.norm_rotary(q, k, s["pos"], *self.turns, q_weight=w["q_norm"][0], k_weight=w["k_norm"][0])
        shape = (*tokens.shape, -1, HEAD)
        s["leaves"] = [t.float().reshape(shape).requires_grad_() for t in (q, k, v)]
        s["mixed"] = attention(*s["leaves"])
        s["a"] = s["mixed"].detach().to(self.torch.bfloat16).reshape(-1, HEADS * HEAD)
        drop = dict(dropout=RATE, rng=self.rng)
        s["x1"] = nsg.linear(s["a"], w["out"], residual=s["x0"], site=0, **drop)
        s["h"], s["u"] = nsg.linear(s["x1"], w["up"], bias=w["up_bias"][0], activation="gelu", pre=True)
        s["x2"] = nsg.linear(s["h"], w["down"], residual=s["x1"], site=1, **drop)
        s["logits"] = nsg.linear(s["x2"], w["head"])
        return s

    def gradients(self, tokens, targets, weights):
        """The weighted cross entropy's gradients into accum; returns the loss."""
        torch, w, at = self.torch, self.w, self.at
        s = self.forward(tokens)
        ones = torch.ones(targets.numel(), device="cuda")
        r = nsg.policy_loss(s["logits"], targets.reshape(-1), ones, weights, dlogits=s["logits"])
        loss = -(weights * r["logp"]).sum()
        into = dict(parts=self.parts, overwrite=True)
        grad = lambda d, x, name, **kw: nsg.linear_grad(self.accum, d, x, w[name], at[name], **into, **kw)  # noqa: E731
        dx2 = grad(r["dlogits"], s["x2"], "head")
        du = grad(nsg.dropout(dx2, RATE, self.rng, 1), s["h"], "down", activation="gelu", pre=s["u"])
        dx1 = grad(du, s["x1"], "up", bias_param=at["up_bias"])
        dx1 = nsg.dropout(dx1, 0.0, None, residual=dx2)                   # both ways into x1
        da = grad(nsg.dropout(dx1, RATE, self.rng, 0), s["a"], "out")
        dq, dk, dv = torch.autograd.grad(s["mixed"], s["leaves"], da.float().reshape(s["mixed"].shape))
        dqkv = torch.empty_like(s["qkv"])
        q, k, _ = self.heads(s["qkv"])
        dq_out, dk_out, dv_out = self.heads(dqkv)
        bf16 = lambda t: t.to(torch.bfloat16).reshape(-1, t.shape[2], HEAD)  # noqa: E731
        nsg.norm_rotary_grad(bf16(dq), q, bf16(dk), k, s["pos"], *self.turns, q_weight=w["q_norm"][0],
                             k_weight=w["k_norm"][0], accum=self.accum, q_param=at["q_norm"], k_param=at["k_norm"],
                             dq_out=dq_out, dk_out=dk_out, **into)
        dv_out.copy_(bf16(dv))
        dx0 = nsg.dropout(grad(dqkv, s["x0"], "qkv"), 0.0, None, residual=dx1)
        nsg.embedding_grad(self.accum, dx0, tokens, at["embed"], **into)
        return loss

    def train(self, tokens, targets, weights, lr=0.02):
        loss = self.gradients(tokens, targets, weights)
        self.steps += 1
        nsg.step_ex(self.accum, self.momentum, self.master, self.params, self.parts, beta=0.9, lr=lr,
                    ns_method="standard", clip=1.0, operand_mode="bf16",
                    adam=dict(lr=lr / 4, beta1=0.9, beta2=0.99, eps=1e-8, step=self.steps, exp_avg=self.m,
                              exp_avg_sq=self.v))
        self.rng[1] += 1   # the next step draws anew
        self.refresh()
        return loss


def batch(gen, rows=32, length=32):
    """Tokens, and the token before each; the first has none."""
    import torch
    tokens = torch.randint(0, VOCAB, (rows, length), generator=gen, device="cuda")
    targets = torch.cat([torch.full_like(tokens[:, :1], -1), tokens[:, :-1]], 1)
    weights = (targets.reshape(-1) >= 0).float()
    return tokens, targets, weights / weights.sum()


def main(steps=100):
    import torch
    nsg.build()
    model, gen = Model(), torch.Generator(device="cuda").manual_seed(1)
    losses = [model.train(*batch(gen)) for _ in range(steps)]
    print(f"loss {float(losses[0]):.3f} -> {float(losses[-1]):.3f}")
    assert nsg.device_error() == 0
    return [float(v) for v in losses]


if __name__ == "__main__":
    main()
