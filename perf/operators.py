"""The operators at the two ends of a language model -- embedding lookup, its
gradient into the flat accumulation buffer, log-probabilities of target
tokens, the clipped policy loss with a KL term and the preference loss of
paired log ratios, both with the gradient of the logits -- as cases to be
measured.

Each case is one call as a training or scoring program makes it.  ``run``
computes it in elementary torch operations in 32 bits, or, where ``own`` is
true, through ``newton_schulz_fp32_gb300``; ``exact`` computes it in 64 bits.
Sizes: the widths (768, 4096) and partition counts of this repository's
configurations, generic vocabularies, odd sizes of all of them."""
import math

import numpy as np
import torch

own = False

KINDS = {"bf16": torch.bfloat16, "fp32": torch.float32}
ROWS_AT_ONCE = 1 << 25   # elements of logits that prepare() and exact() take at a time


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the next token of one sequence: a latency-bound call
        dict(name="lookup_token", op="lookup", tokens=1, vocab=32768, dim=768, dtype="bf16", index="int64"),
        # the tokens of one training micro-batch, rows of 8 KiB scaled by sqrt(dim)
        dict(name="lookup_batch", op="lookup", tokens=32768, vocab=131072, dim=4096, dtype="bf16", index="int64"),
        # a short micro-batch added to a small table's accumulated gradient
        dict(name="embgrad_small", op="embgrad", tokens=512, vocab=32768, dim=768, dtype="bf16", index="int64",
             overwrite=False, padding=0.0, offset=0, parts=1),
        # the first micro-batch of a step (the old sum is overwritten), padded sequences, a table packed
        # behind an odd-sized parameter, odd sizes, FP32 activations
        dict(name="embgrad_odd", op="embgrad", tokens=5003, vocab=50001, dim=1001, dtype="fp32", index="int32",
             overwrite=True, padding=0.2, offset=35, parts=8),
        # a later micro-batch of a large model's step, the table cut over eight ranks' partitions
        dict(name="embgrad_large", op="embgrad", tokens=32768, vocab=131072, dim=4096, dtype="bf16", index="int64",
             overwrite=False, padding=0.0, offset=0, parts=8),
        # scoring one token (a reference model beside a sampler)
        dict(name="logprob_token", op="logprob", tokens=1, vocab=131072, dtype="bf16", index="int64",
             scale=1.0, ignored=0.0),
        # scoring a batch of sequences with the reference model
        dict(name="logprob_batch", op="logprob", tokens=8192, vocab=131072, dtype="bf16", index="int64",
             scale=1.0, ignored=0.1),
        # one short answer
        dict(name="policy_small", op="policy", tokens=48, vocab=32768, dtype="bf16", index="int64",
             scale=1.0, masked=0.0, kl=0.05),
        # FP32 logits at a sampling temperature, odd sizes, prompts masked out
        dict(name="policy_odd", op="policy", tokens=2047, vocab=50001, dtype="fp32", index="int32",
             scale=1.25, masked=0.3, kl=0.0),
        # a micro-batch of long answers of a large vocabulary
        dict(name="policy_large", op="policy", tokens=8192, vocab=131072, dtype="bf16", index="int64",
             scale=1.0, masked=0.05, kl=0.02),
        # two pairs of short answers
        dict(name="preference_small", op="preference", tokens=96, pairs=2, vocab=32768, dtype="bf16",
             index="int64", scale=1.0, prompt=0.2, smoothing=0.0),
        # eight pairs of long answers, prompts without targets
        dict(name="preference_large", op="preference", tokens=8192, pairs=8, vocab=131072, dtype="bf16",
             index="int64", scale=1.0, prompt=0.25, smoothing=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "embgrad", "logprob", "policy", "preference"])
    dtype, index = rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["int64", "int32"])
    vocab = _log_int(rng, 2000, 131072)
    if op in ("lookup", "embgrad"):
        dim = _log_int(rng, 64, 4096)
        dim = rng.choice([dim, dim // 8 * 8, dim // 128 * 128 or 64])
        c = dict(op=op, tokens=_log_int(rng, 1, 32768 if dtype == "bf16" else 16384), vocab=vocab, dim=dim,
                 dtype=dtype, index=index)
        if op == "embgrad":
            c.update(overwrite=rng.random() < 0.5, padding=rng.choice([0.0, 0.1, 0.5]),
                     offset=rng.choice([0, 128, 35]), parts=rng.choice([1, 2, 8, 64]))
        return c
    most = (1 << 30) // (1 if dtype == "bf16" else 2) // vocab
    c = dict(op=op, tokens=_log_int(rng, 1, min(most, 32768)), vocab=vocab, dtype=dtype, index=index,
             scale=rng.choice([1.0, 1.0, 0.8, 1.25]))
    if op == "logprob":
        c.update(ignored=rng.choice([0.0, 0.1, 0.5]))
    elif op == "policy":
        c.update(masked=rng.choice([0.0, 0.1, 0.5]), kl=rng.choice([0.0, 0.02, 0.1]))
    else:
        c.update(pairs=min(_log_int(rng, 1, 64), max(1, c["tokens"] // 4)), prompt=rng.choice([0.0, 0.25, 0.5]),
                 smoothing=rng.choice([0.0, 0.1]))
    return c


# ------------------------------------------------------------------ inputs

def _zipf(n, vocab, gen):
    """Token ids whose frequency falls as 1 / (id + 1), as text's do."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    return torch.clamp((float(vocab + 1) ** u).long() - 1, 0, vocab - 1)


def _chunks(tokens, vocab):
    rows = max(1, ROWS_AT_ONCE // vocab)
    return [(a, min(tokens, a + rows)) for a in range(0, tokens, rows)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c, T = case, case["tokens"]
    index = torch.int64 if c["index"] == "int64" else torch.int32
    if c["op"] == "lookup":
        table = torch.randn((c["vocab"], c["dim"]), generator=gen, device="cuda", dtype=torch.float32)
        return dict(case=c, table=table.mul_(0.02).to(KINDS[c["dtype"]]), ids=_zipf(T, c["vocab"], gen).to(index),
                    scale=math.sqrt(c["dim"]))
    if c["op"] == "embgrad":
        V, D, P = c["vocab"], c["dim"], c["parts"]
        ids = _zipf(T, V, gen)
        if c["padding"]:
            ids = torch.where(torch.rand(T, generator=gen, device="cuda") < c["padding"], -1, ids)
        dout = (1e-2 * torch.randn((T, D), generator=gen, device="cuda")).to(KINDS[c["dtype"]])
        each = -(-(c["offset"] + V * D) // (128 * P)) * 128
        accum = 1e-2 * torch.randn(each * P, generator=gen, device="cuda")
        parts = np.array([(p * each, (p + 1) * each, p * each) for p in range(P)],
                         dtype=[("flat_begin", "<i8"), ("flat_end", "<i8"), ("storage_offset", "<i8")])
        return dict(case=c, ids=ids.to(index), dout=dout, accum=accum, parts=parts,
                    param=(c["offset"], V, D), scale=0.25)

    def make_logits():
        """Logits of spread 2, some words forbidden (minus infinity), the target's lifted, and the targets."""
        V = c["vocab"]
        y = _zipf(T, V, gen)
        z = torch.empty((T, V), dtype=KINDS[c["dtype"]], device="cuda")
        lift = 4.0 + 3.0 * torch.randn(T, generator=gen, device="cuda")
        forbidden = torch.randint(0, V, (max(1, V // 1000),), generator=gen, device="cuda")
        for a, b in _chunks(T, V):
            x = torch.randn((b - a, V), generator=gen, device="cuda").mul_(2.0)
            x[:, forbidden] = -math.inf
            z[a:b] = x.scatter_(1, y[a:b, None], lift[a:b, None])
        return z, y

    def score(z, y):
        """The targets' log-probabilities, as a program that sampled them has them."""
        out = torch.empty(T, device="cuda")
        for a, b in _chunks(*z.shape):
            x = z[a:b].float() * c["scale"]
            out[a:b] = x.gather(1, y[a:b, None])[:, 0] - torch.logsumexp(x, 1)
        return out

    z, targets = make_logits()
    s = dict(case=c, logits=z, scale=c["scale"])
    if c["op"] == "logprob":
        if c["ignored"]:
            targets = torch.where(torch.rand(T, generator=gen, device="cuda") < c["ignored"], -100, targets)
        return dict(s, targets=targets.to(index))
    logp = score(z, targets)
    ref = logp + 0.2 * torch.randn(T, generator=gen, device="cuda")
    if c["op"] == "policy":
        moved = 0.15 * torch.randn(T, generator=gen, device="cuda")
        for edge in (math.log(0.8), math.log(1.25)):   # on the edge itself rounding would decide the branch
            moved = torch.where((moved - edge).abs() < 1e-3, moved + 4e-3, moved)
        mask = (torch.rand(T, generator=gen, device="cuda") >= c["masked"]).float()
        adv = torch.randn(T, generator=gen, device="cuda")
        return dict(s, targets=targets.to(index), old=logp - moved, ref=ref if c["kl"] else None, adv=adv,
                    weights=mask / mask.sum().clamp(min=1.0), clip=(0.2, 0.25), kl=c["kl"])
    B = c["pairs"]
    cuts = torch.sort(torch.randint(0, T + 1, (2 * B - 1,), generator=gen, device="cuda")).values
    even = torch.arange(1, 2 * B, device="cuda") * T // (2 * B)
    cuts = (cuts + 3 * even) // 4   # lengths that differ, as answers' do
    ends = torch.tensor([T], device="cuda")
    offsets = torch.cat([ends * 0, cuts, ends])
    place = torch.arange(T, device="cuda")
    seq = torch.clamp(torch.searchsorted(offsets, place, right=True) - 1, 0, 2 * B - 1)
    share = (place - offsets[seq]).float() / (offsets[seq + 1] - offsets[seq]).clamp(min=1).float()
    targets = torch.where(share < c["prompt"], -100, targets)
    return dict(s, targets=targets.to(index), ref=ref, offsets=offsets.to(index), beta=0.1,
                smoothing=c["smoothing"])


# ------------------------------------------------------------------ plain form

def _plain_rows(z, targets, scale, active):
    """exp(z - max), their sums and the targets' log-probabilities (0 where not active)."""
    x = z.float() * scale
    m = x.max(1, keepdim=True).values
    zt = (x.gather(1, targets[:, None]) - m)[:, 0]
    e = x.sub_(m).exp_()
    total = e.sum(1)
    return e, total, torch.where(active, zt - total.log(), 0.0)


def _plain_dlogits(e, total, coef, targets, scale, active, dtype):
    """coef * scale * (1[v = target] - e / total), 0 in rows that are not active."""
    d = e.mul_((-coef * scale / total)[:, None])
    d.scatter_add_(1, targets[:, None], (coef * scale)[:, None])
    return torch.where(active[:, None], d, 0.0).to(dtype)


def _plain(s):
    c = s["case"]
    if c["op"] == "lookup":
        return (s["table"][s["ids"].long()].float() * s["scale"]).to(s["table"].dtype)
    if c["op"] == "embgrad":
        off, V, D = s["param"]
        g = s["accum"][off:off + V * D].view(V, D)
        if c["overwrite"]:
            g.zero_()
        ids = s["ids"].long()
        d = torch.where((ids >= 0)[:, None], s["dout"].float() * s["scale"], 0.0)
        return g.index_add_(0, ids.clamp(min=0), d)
    z, targets = s["logits"], s["targets"].long()
    valid = targets >= 0
    targets = targets.clamp(min=0)
    if c["op"] == "logprob":
        return _plain_rows(z, targets, s["scale"], valid)[2]
    if c["op"] == "policy":
        w, adv = s["weights"], s["adv"]
        active = valid & (w != 0)
        e, total, logp = _plain_rows(z, targets, s["scale"], active)
        r = (logp - s["old"]).exp()
        free, held = r * adv, r.clamp(1 - s["clip"][0], 1 + s["clip"][1]) * adv
        term, cut = -torch.minimum(free, held), free > held
        dlogp = torch.where(cut, 0.0, -free)
        kl = torch.zeros_like(logp)
        if s["ref"] is not None:
            q = s["ref"] - logp
            kl = q.exp() - q - 1
            dlogp = dlogp + s["kl"] * (1 - q.exp())
        ww = torch.where(active, w, 0.0)
        stats = torch.stack([(ww * (term + s["kl"] * kl)).sum(), (ww * term).sum(), (ww * kl).sum(),
                             (ww * cut).sum()])
        return dict(stats=stats, logp=logp,
                    dlogits=_plain_dlogits(e, total, ww * dlogp, targets, s["scale"], active, z.dtype))
    e, total, logp = _plain_rows(z, targets, s["scale"], valid)
    T, B = z.shape[0], c["pairs"]
    off = s["offsets"].long()
    seq = (torch.arange(T, device=z.device)[:, None] >= off[None, 1:-1]).sum(1)
    ratio = torch.zeros(2 * B, device=z.device).index_add_(0, seq, torch.where(valid, logp - s["ref"], 0.0))
    h = s["beta"] * (ratio[:B] - ratio[B:])
    ls = s["smoothing"]
    soft = lambda x: torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))  # noqa: E731
    loss = (1 - ls) * soft(-h) + ls * soft(h)
    dh = (ls - 1) / (1 + h.exp()) + ls / (1 + (-h).exp())
    g = torch.cat([dh, -dh]) * (s["beta"] / B)
    stats = torch.stack([loss.mean(), h.mean(), (h > 0).float().mean()])
    return dict(stats=stats, margins=h, logp=logp,
                dlogits=_plain_dlogits(e, total, g[seq], targets, s["scale"], valid, z.dtype))


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import newton_schulz_fp32_gb300 as nsg
    c = s["case"]
    if c["op"] == "lookup":
        return nsg.embedding(s["table"], s["ids"], scale=s["scale"])
    if c["op"] == "embgrad":
        off, V, D = s["param"]
        nsg.embedding_grad(s["accum"], s["dout"], s["ids"], s["param"], parts=s["parts"], scale=s["scale"],
                           overwrite=c["overwrite"])
        return s["accum"][off:off + V * D].view(V, D)
    if c["op"] == "logprob":
        return nsg.token_logprobs(s["logits"], s["targets"], logit_scale=s["scale"])
    if c["op"] == "policy":
        r = nsg.policy_loss(s["logits"], s["targets"], s["adv"], s["weights"], old_logp=s["old"],
                            ref_logp=s["ref"], clip_low=s["clip"][0], clip_high=s["clip"][1], kl_coef=s["kl"],
                            logit_scale=s["scale"])
        return dict(stats=r["stats"], logp=r["logp"], dlogits=r["dlogits"])
    r = nsg.preference_loss(s["logits"], s["targets"], s["offsets"], ref_logp=s["ref"], beta=s["beta"],
                            label_smoothing=s["smoothing"], logit_scale=s["scale"])
    return dict(stats=r["stats"][:3], margins=r["margins"], logp=r["logp"], dlogits=r["dlogits"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c, D64 = case, torch.float64
    if c["op"] == "lookup":
        out = torch.empty((c["tokens"], c["dim"]), dtype=D64, device="cuda")
        for t in range(0, c["tokens"], 4096):
            out[t:t + 4096] = s["scale"] * s["table"].index_select(0, s["ids"][t:t + 4096].long()).to(D64)
        return out
    if c["op"] == "embgrad":
        off, V, D = s["param"]
        first = s["accum"][off:off + V * D].to(D64).view(V, D)
        if c["overwrite"]:
            first.zero_()
        kept = s["ids"] >= 0
        order = torch.argsort(s["ids"][kept].long(), stable=True)
        rows = s["ids"][kept].long()[order]
        part = s["dout"][kept][order].to(D64)
        ids, counts = torch.unique_consecutive(rows, return_counts=True)
        ends = counts.cumsum(0).cpu().tolist()
        begin = 0
        single = (counts == 1).cpu().tolist()
        if len(ends):   # rows of one token at once, the others one by one
            at = counts.cumsum(0) - 1
            one = counts == 1
            first[ids[one]] += s["scale"] * part[at[one]]
        for k, end in enumerate(ends):
            if not single[k]:
                first[ids[k]] += s["scale"] * part[begin:end].sum(0)
            begin = end
        return first
    z, scale, T = s["logits"], float(s["scale"]), c["tokens"]
    y = s["targets"].long()
    on = y >= 0
    if c["op"] == "policy":
        on = on & (s["weights"] != 0)
    lse, logp = torch.zeros(T, dtype=D64, device="cuda"), torch.zeros(T, dtype=D64, device="cuda")
    for a, b in _chunks(*z.shape):
        x = z[a:b].to(D64) * scale
        lse[a:b] = torch.logsumexp(x, 1)
        logp[a:b] = x.gather(1, y[a:b, None].clamp(min=0))[:, 0] - lse[a:b]
    logp = torch.where(on, logp, 0.0)
    if c["op"] == "logprob":
        return logp
    if c["op"] == "policy":
        w, adv, old = (s[k].to(D64) for k in ("weights", "adv", "old"))
        w = torch.where(on, w, 0.0)
        lo, hi = 1 - s["clip"][0], 1 + s["clip"][1]
        r = torch.exp(logp - old)
        cut = ((adv > 0) & (r > hi)) | ((adv < 0) & (r < lo))
        term = -torch.where(cut, torch.where(adv > 0, hi, lo), r) * adv
        dl = torch.where(cut, 0.0, -adv * r)
        kl = torch.zeros_like(logp)
        if s["ref"] is not None:
            q = s["ref"].to(D64) - logp
            kl = torch.expm1(q) - q
            dl = dl - s["kl"] * torch.expm1(q)
        coef = w * dl
        out = dict(stats=torch.stack([torch.dot(w, term) + s["kl"] * torch.dot(w, kl), torch.dot(w, term),
                                      torch.dot(w, kl), w[cut].sum()]), logp=logp)
    else:
        B, off = c["pairs"], s["offsets"].long().tolist()
        ratio = torch.where(on, logp - s["ref"].to(D64), 0.0)
        sums = torch.stack([ratio[a:b].sum() for a, b in zip(off[:-1], off[1:])])
        h = s["beta"] * (sums[:B] - sums[B:])
        ls = s["smoothing"]
        loss = -(1 - ls) * torch.nn.functional.logsigmoid(h) - ls * torch.nn.functional.logsigmoid(-h)
        dh = s["beta"] / B * (torch.sigmoid(h) - (1 - ls))
        coef = torch.zeros(T, dtype=D64, device="cuda")
        for k in range(2 * B):
            coef[off[k]:off[k + 1]] = dh[k % B] if k < B else -dh[k % B]
        out = dict(stats=torch.stack([loss.mean(), h.mean(), (h > 0).to(D64).mean()]), margins=h, logp=logp)
    coef = torch.where(on, coef, 0.0) * scale
    d = torch.empty(z.shape, dtype=D64, device="cuda")
    for a, b in _chunks(*z.shape):
        p = torch.exp(z[a:b].to(D64) * scale - lse[a:b, None])
        p.scatter_add_(1, y[a:b, None].clamp(min=0), torch.full((b - a, 1), -1.0, dtype=D64, device="cuda"))
        d[a:b] = torch.where(on[a:b, None], -coef[a:b, None] * p, 0.0)
    out["dlogits"] = d
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def _distinct(tokens, vocab):
    """The expected number of distinct ids among so many of _zipf's."""
    k = torch.arange(1, vocab + 1, dtype=torch.float64)
    p = torch.log1p(1 / k) / math.log(vocab + 1)
    return float((1 - (1 - p) ** tokens).sum())


def work(case):
    c, T, V = case, case["tokens"], case["vocab"]
    es = 2 if c["dtype"] == "bf16" else 4
    ix = 8 if c["index"] == "int64" else 4
    if c["op"] == "lookup":
        return {"bytes": T * ix + (_distinct(T, V) + T) * c["dim"] * es, "flops": T * c["dim"]}
    if c["op"] == "embgrad":
        used = T * (1 - c["padding"])
        rows = V * 4 if c["overwrite"] else _distinct(used, V) * 8
        return {"bytes": T * ix + (used * es + rows) * c["dim"], "flops": used * c["dim"] + T}
    off = c.get("ignored", c.get("masked", c.get("prompt", 0.0)))
    read, flops = (1 - off) * T * V * es, 4.0 * (1 - off) * T * V
    if c["op"] == "logprob":
        return {"bytes": read + T * (ix + 4), "flops": flops}
    return {"bytes": read + T * V * es + T * (ix + 20), "flops": 2 * flops}
