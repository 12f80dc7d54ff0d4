"""The operators of a model's layers -- the matrix product with bias,
activation, dropout and residual, its gradients into the flat accumulation
buffer, dropout from a counter, the norm and rotation of query and key heads
and its gradients -- as cases to be measured.

Each case is one call as a training or sampling program makes it.  ``run``
computes it in elementary torch operations in 32 bits (angles in 64), or, where
``own`` is true, through ``newton_schulz_fp32_gb300``; ``exact`` computes it in
64 bits.  Sizes: the widths (768, 4096, 14336), head counts and partition
counts of this repository's configurations, and odd sizes."""
import math

import numpy as np
import torch

own = False

KINDS = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # sampling: one token through an output projection, added to the residual stream
        dict(name="linear_token", op="linear", tokens=1, fin=4096, fout=4096, out="bf16", bias=False, act="none",
             pre=False, residual=True, rate=0.0),
        # odd sizes, everything in the epilogue, a residual stream held in FP32
        dict(name="linear_odd", op="linear", tokens=1001, fin=1001, fout=763, out="fp32", bias=True, act="gelu",
             pre=True, residual=True, rate=0.1),
        # the wide half of a training micro-batch's feed-forward layer; its argument is kept for the way back
        dict(name="linear_large", op="linear", tokens=8192, fin=4096, fout=14336, out="bf16", bias=False, act="silu",
             pre=True, residual=False, rate=0.0),
        # a short micro-batch through a small model's attention output, added to what others left
        dict(name="lingrad_small", op="lingrad", tokens=1024, fin=768, fout=768, bias=True, act="none",
             overwrite=False, offset=0, parts=8),
        # odd sizes, behind an odd-sized parameter, cut by partitions, through the activation before the layer
        dict(name="lingrad_odd", op="lingrad", tokens=2047, fin=1001, fout=763, bias=True, act="gelu",
             overwrite=True, offset=35, parts=8),
        # the narrow half of a feed-forward layer, first micro-batch of a step
        dict(name="lingrad_large", op="lingrad", tokens=8192, fin=14336, fout=4096, bias=False, act="silu",
             overwrite=True, offset=128, parts=64),
        # a small layer's activations, without a residual
        dict(name="dropout_small", op="dropout", rows=255, cols=768, dtype="bf16", residual=False, rate=0.1),
        # the residual stream of a large micro-batch
        dict(name="dropout_large", op="dropout", rows=16384, cols=4096, dtype="bf16", residual=True, rate=0.1),
        # sampling: one token far into a text
        dict(name="rotary_token", op="rotary", tokens=1, heads=32, kv=8, dim=128, rot=128, axes=1, norm=True,
             interleaved=False, dtype="bf16", far=1 << 20),
        # a training micro-batch of images among text: time, height and width, heads cut out of a packed projection
        dict(name="rotary_large", op="rotary", tokens=16384, heads=32, kv=8, dim=128, rot=128, axes=3, norm=True,
             interleaved=False, dtype="bf16", far=1 << 14),
        # a small model in FP32, neighbours turned as pairs, a part of each head alone
        dict(name="rotgrad_small", op="rotgrad", tokens=777, heads=12, kv=12, dim=80, rot=60, axes=1, norm=True,
             interleaved=True, dtype="fp32", far=1 << 12, overwrite=False, parts=2),
        # the way back of the large micro-batch
        dict(name="rotgrad_large", op="rotgrad", tokens=16384, heads=32, kv=8, dim=128, rot=128, axes=3, norm=True,
             interleaved=False, dtype="bf16", far=1 << 14, overwrite=True, parts=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    n = _log_int(rng, lo, hi)
    return rng.choice([n, max(lo, n // 8 * 8), max(lo, n // 128 * 128)])


def draw(rng):
    op = rng.choice(["linear", "lingrad", "dropout", "rotary", "rotgrad"])
    if op in ("linear", "lingrad"):
        fin, fout = _size(rng, 64, 14336), _size(rng, 64, 14336)
        most = 8192 * 4096 * 14336 // (fin * fout)
        c = dict(op=op, tokens=_log_int(rng, 1, min(16384, most)), fin=fin, fout=fout, bias=rng.random() < 0.5,
                 act=rng.choice(["none", "relu", "relu2", "gelu", "silu"]))
        if op == "lingrad":
            c.update(overwrite=rng.random() < 0.5, offset=rng.choice([0, 128, 35]), parts=rng.choice([1, 2, 8, 64]))
        else:
            c.update(out=rng.choice(["bf16", "bf16", "fp32"]), pre=rng.random() < 0.5, residual=rng.random() < 0.5,
                     rate=rng.choice([0.0, 0.0, 0.1]))
        return c
    if op == "dropout":
        cols = _size(rng, 64, 8192)
        return dict(op=op, rows=_log_int(rng, 1, (1 << 25) // cols), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), residual=rng.random() < 0.5,
                    rate=rng.choice([0.05, 0.1, 0.5]))
    dim = rng.choice([40, 64, 80, 96, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4])
    axes = rng.choice([1, 1, 2, 3])
    most = (1 << 25) // (dim * (heads + kv))
    c = dict(op=op, tokens=_log_int(rng, 1, min(most, 65536)), heads=heads, kv=kv, dim=dim,
             rot=rng.choice([dim, dim, dim // 8 * 4]), axes=axes, norm=rng.random() < 0.8,
             interleaved=rng.random() < 0.3, dtype=rng.choice(["bf16", "bf16", "fp32"]),
             far=_log_int(rng, 1 << 10, 1 << 20))
    if op == "rotgrad":
        c.update(overwrite=rng.random() < 0.5, parts=rng.choice([1, 2, 8]))
    return c


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, spread, dtype):
    """Normal values, made in pieces so that no FP32 copy of a large one is needed."""
    out = torch.empty(shape, device="cuda", dtype=dtype)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 26):
        part = flat[a:a + (1 << 26)]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(spread))
    return out


def _buffer(gen, elements, parts):
    """An accumulation buffer of so many elements in equal partitions, and its table."""
    each = -(-elements // (128 * parts)) * 128
    table = np.array([(p * each, (p + 1) * each, p * each) for p in range(parts)],
                     dtype=[("flat_begin", "<i8"), ("flat_end", "<i8"), ("storage_offset", "<i8")])
    return _normal(gen, (each * parts,), 1e-2, torch.float32), table


def _frequencies(c):
    """Radians a position turns each pair by, and the axis that turns it: contiguous shares of the pairs."""
    pairs = c["rot"] // 2
    freq = 10000.0 ** (-np.arange(pairs, dtype=np.float64) / pairs)
    axis = (np.arange(pairs) * c["axes"] // pairs).astype(np.int32)
    return freq, axis


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c, bf16 = case, torch.bfloat16
    rng = torch.tensor([int(seed) * 7919 + 12345, 3], device="cuda", dtype=torch.int64)   # seed, step
    if c["op"] == "linear":
        T, K, N = c["tokens"], c["fin"], c["fout"]
        return dict(case=c, x=_normal(gen, (T, K), 1.0, bf16), weight=_normal(gen, (N, K), 1 / math.sqrt(K), bf16),
                    bias=_normal(gen, (N,), 0.5, bf16) if c["bias"] else None, rng=rng,
                    residual=_normal(gen, (T, N), 1.0, KINDS[c["out"]]) if c["residual"] else None)
    if c["op"] == "lingrad":
        T, K, N = c["tokens"], c["fin"], c["fout"]
        pre = _normal(gen, (T, K), 1.0, bf16)
        x = pre
        if c["act"] != "none":   # the layer's input is what the activation made of it
            x = torch.empty_like(pre)
            for a in range(0, T, 1024):
                x[a:a + 1024] = _act(pre[a:a + 1024].float(), c["act"]).to(bf16)
        accum, parts = _buffer(gen, c["offset"] + N * K + N, c["parts"])
        return dict(case=c, dout=_normal(gen, (T, N), 1e-2, bf16), x=x, pre=pre if c["act"] != "none" else None,
                    weight=_normal(gen, (N, K), 1 / math.sqrt(K), bf16), accum=accum, parts=parts,
                    param=(c["offset"], N, K), bias=(c["offset"] + N * K, 1, N) if c["bias"] else None, scale=0.25)
    if c["op"] == "dropout":
        shape, kind = (c["rows"], c["cols"]), KINDS[c["dtype"]]
        return dict(case=c, x=_normal(gen, shape, 1.0, kind), rng=rng,
                    residual=_normal(gen, shape, 1.0, kind) if c["residual"] else None)
    T, H, G, D, kind = c["tokens"], c["heads"], c["kv"], c["dim"], KINDS[c["dtype"]]
    packed = _normal(gen, (T, H + 2 * G, D), 1.0, kind)   # queries, keys and values of one projection
    positions = torch.randint(0, c["far"], (T, c["axes"]), generator=gen, device="cuda")
    freq, axis = _frequencies(c)
    s = dict(case=c, q=packed[:, :H], k=packed[:, H:H + G], positions=positions, freq=freq, axis=axis,
             qw=_normal(gen, (D,), 0.1, torch.float32).add_(1.0).to(kind) if c["norm"] else None,
             kw=_normal(gen, (D,), 0.1, torch.float32).add_(1.0).to(kind) if c["norm"] else None)
    if c["op"] == "rotgrad":
        accum, parts = _buffer(gen, 2 * D, c["parts"])
        s.update(dq=_normal(gen, (T, H, D), 1e-2, kind), dk=_normal(gen, (T, G, D), 1e-2, kind), accum=accum,
                 parts=parts, qp=(0, 1, D) if c["norm"] else None, kp=(D, 1, D) if c["norm"] else None, scale=0.25)
    return s


# ------------------------------------------------------------------ plain form

def _act(u, kind):
    if kind == "relu":
        return u.clamp(min=0)
    if kind == "relu2":
        return u.clamp(min=0) ** 2
    if kind == "gelu":
        return 0.5 * u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
    if kind == "silu":
        return u / (1 + torch.exp(-u))
    return u


def _act_slope(u, kind):
    if kind == "relu":
        return (u > 0).to(u.dtype)
    if kind == "relu2":
        return 2 * u.clamp(min=0)
    if kind == "gelu":
        t = torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3))
        return 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * u * u)
    s = 1 / (1 + torch.exp(-u))
    return s * (1 + u * (1 - s))


MULTIPLIERS, STEPS, LOW = (0xD2511F53, 0xCD9E8D57), (0x9E3779B9, 0xBB67AE85), 0xFFFFFFFF


def _wide(a, m):
    """High and low 32 bits of a * m (both below 2^32) in 64-bit integers."""
    p, q = a * (m & 0xFFFF), a * (m >> 16)
    return (q + (p >> 16)) >> 16, (p + ((q & 0xFFFF) << 16)) & LOW


def _draws(rows, cols, rng, site):
    """16 random bits for each element: Philox4x32-10 of (column / 8, row, site, step) under the seed."""
    groups = -(-cols // 8)
    k0, k1 = rng[0] & LOW, (rng[0] >> 32) & LOW
    c0 = torch.arange(groups, device="cuda")[None, :].expand(rows, groups)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, groups)
    c2 = torch.full_like(c0, site)
    c3 = (rng[1] & LOW).expand(rows, groups)
    for _ in range(10):
        h0, l0 = _wide(c0, MULTIPLIERS[0])
        h1, l1 = _wide(c2, MULTIPLIERS[1])
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + STEPS[0]) & LOW, (k1 + STEPS[1]) & LOW
    words = torch.stack([c0, c1, c2, c3], 2)
    return torch.stack([words & 0xFFFF, words >> 16], 3).view(rows, groups * 8)[:, :cols]


def _dropped(x, rate, rng, site):
    """x (FP32) with elements left out, the others scaled up: the rate in steps of 2^-16."""
    least = int(rate * 65536 + 0.5)
    return torch.where(_draws(*x.shape, rng, site) >= least, x * (65536 / (65536 - least)), 0.0)


def _turned(x, s, back=False):
    """The heads' pairs turned by their angles (`back`: the other way)."""
    c = s["case"]
    half = c["rot"] // 2
    at = s["positions"][:, torch.from_numpy(s["axis"]).to("cuda").long()].double()
    angle = at * torch.from_numpy(s["freq"]).to("cuda")
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    sin = -sin if back else sin
    out = x.clone()
    if c["interleaved"]:
        a, b = x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]
        out[..., 0:c["rot"]:2], out[..., 1:c["rot"]:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:c["rot"]]
        out[..., :half], out[..., half:c["rot"]] = a * cos - b * sin, b * cos + a * sin
    return out


def _turned_gradient(s, dout, x, w):
    """Gradients of the heads and of the norm's weight."""
    g = _turned(dout.float(), s, back=True)
    if w is None:
        return g.to(dout.dtype), None
    r = torch.rsqrt((x.float() ** 2).mean(2, keepdim=True) + EPS)
    n = x.float() * r
    gw = g * w.float()
    return (r * (gw - n * (gw * n).mean(2, keepdim=True))).to(dout.dtype), (g * n).sum((0, 1))


def _collect(s, param, value):
    """A parameter's gradient in the accumulation buffer."""
    off, n = param[0], param[1] * param[2]
    g = s["accum"][off:off + n].view(param[1:])
    if s["case"]["overwrite"]:
        g.copy_(s["scale"] * value.view(param[1:]))
    else:
        g.add_(value.view(param[1:]), alpha=s["scale"])
    return g


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        u = s["x"].float() @ s["weight"].float().T
        if s["bias"] is not None:
            u = u + s["bias"].float()
        y = _act(u, c["act"])
        if c["rate"]:
            y = _dropped(y, c["rate"], s["rng"], 5)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = dict(out=y.to(KINDS[c["out"]]))
        if c["pre"]:
            out["pre"] = u.to(torch.bfloat16)
        return out
    if c["op"] == "lingrad":
        d = s["dout"].float()
        dx = d @ s["weight"].float()
        if s["pre"] is not None:
            dx = dx * _act_slope(s["pre"].float(), c["act"])
        out = dict(dx=dx.to(torch.bfloat16), dw=_collect(s, s["param"], d.T @ s["x"].float()))
        if s["bias"] is not None:
            out["db"] = _collect(s, s["bias"], d.sum(0))
        return out
    if c["op"] == "dropout":
        y = _dropped(s["x"].float(), c["rate"], s["rng"], 5)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(s["x"].dtype)
    if c["op"] == "rotary":
        out = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            n = x.float()
            if w is not None:
                n = n * torch.rsqrt((n ** 2).mean(2, keepdim=True) + EPS) * w.float()
            out.append(_turned(n, s).to(x.dtype))
        return out
    dq, wq = _turned_gradient(s, s["dq"], s["q"], s["qw"])
    dk, wk = _turned_gradient(s, s["dk"], s["k"], s["kw"])
    if wq is None:
        return [dq, dk]
    return [dq, dk, _collect(s, s["qp"], wq), _collect(s, s["kp"], wk)]


# ------------------------------------------------------------------ the framework's calls

def _view(s, param):
    return s["accum"][param[0]:param[0] + param[1] * param[2]].view(param[1:])


def _own(s):
    import newton_schulz_fp32_gb300 as nsg
    c = s["case"]
    if c["op"] == "linear":
        r = nsg.linear(s["x"], s["weight"], bias=s["bias"], activation=c["act"], residual=s["residual"],
                       dropout=c["rate"], rng=s["rng"], site=5, out_dtype=KINDS[c["out"]], pre=c["pre"])
        return dict(out=r[0], pre=r[1]) if c["pre"] else dict(out=r)
    if c["op"] == "lingrad":
        dx = nsg.linear_grad(s["accum"], s["dout"], s["x"], s["weight"], s["param"], bias_param=s["bias"],
                             parts=s["parts"], scale=s["scale"], overwrite=c["overwrite"], activation=c["act"],
                             pre=s["pre"])
        out = dict(dx=dx, dw=_view(s, s["param"]))
        if s["bias"] is not None:
            out["db"] = _view(s, s["bias"])
        return out
    if c["op"] == "dropout":
        return nsg.dropout(s["x"], c["rate"], s["rng"], site=5, residual=s["residual"])
    if c["op"] == "rotary":
        return list(nsg.norm_rotary(s["q"], s["k"], positions=s["positions"], inv_freq=s["freq"], axis=s["axis"],
                                    interleaved=c["interleaved"], norm=c["norm"], q_weight=s["qw"],
                                    k_weight=s["kw"], eps=EPS))
    dq, dk = nsg.norm_rotary_grad(s["dq"], s["q"], s["dk"], s["k"], positions=s["positions"], inv_freq=s["freq"],
                                  axis=s["axis"], interleaved=c["interleaved"], norm=c["norm"], q_weight=s["qw"],
                                  k_weight=s["kw"], eps=EPS, accum=s["accum"], q_param=s["qp"], k_param=s["kp"],
                                  parts=s["parts"], scale=s["scale"], overwrite=c["overwrite"])
    return [dq, dk, _view(s, s["qp"]), _view(s, s["kp"])] if c["norm"] else [dq, dk]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits

def _keep64(rows, cols, rng, site, rate):
    """What each element is multiplied by: 0, or what makes up for the others (unsigned 64-bit words on the host)."""
    seed, step = (int(v) & (2 ** 64 - 1) for v in rng.cpu())
    u = lambda v: np.uint64(v)  # noqa: E731
    low, half = u(LOW), u(32)
    least = int(rate * 65536 + 0.5)
    gain = 65536 / (65536 - least)
    groups = (cols + 7) // 8
    out = np.empty((rows, groups, 8), dtype=np.float64)
    for r0 in range(0, rows, 2048):
        r = np.arange(r0, min(rows, r0 + 2048), dtype=np.uint64)
        word = [np.tile(np.arange(groups, dtype=np.uint64), (len(r), 1)), np.repeat(r[:, None], groups, 1),
                np.full((len(r), groups), site, np.uint64), np.full((len(r), groups), step & LOW, np.uint64)]
        key = [seed & LOW, seed >> 32]
        for _ in range(10):
            p, q = word[0] * u(0xD2511F53), word[2] * u(0xCD9E8D57)   # 32 x 32 bits: no more than 64
            word = [(q >> half) ^ word[1] ^ u(key[0]), q & low, (p >> half) ^ word[3] ^ u(key[1]), p & low]
            key = [(key[0] + 0x9E3779B9) & LOW, (key[1] + 0xBB67AE85) & LOW]
        for j in range(8):
            bits = (word[j // 2] >> u(16 * (j % 2))) & u(0xFFFF)
            out[r0:r0 + len(r), :, j] = np.where(bits >= u(least), gain, 0.0)
    return torch.from_numpy(out.reshape(rows, groups * 8)[:, :cols]).to("cuda")


def _rotation64(s):
    """Each token's rotation as complex numbers, pairs last."""
    p = s["positions"].to(torch.float64)
    angles = torch.stack([p[:, int(a)] * float(f) for a, f in zip(s["axis"], s["freq"])], 1)
    return torch.polar(torch.ones_like(angles), angles)


def _turn64(x, z, c):
    pairs = c["rot"] // 2
    first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else \
        (slice(0, pairs), slice(pairs, c["rot"]))
    y = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z[:, None]
    out = x.clone()
    out[..., first], out[..., second] = y.real, y.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c, D64 = case, torch.float64
    if c["op"] == "linear":
        w = s["weight"].to(D64)
        u = torch.empty((c["tokens"], c["fout"]), dtype=D64, device="cuda")
        for a in range(0, c["tokens"], 2048):
            u[a:a + 2048] = torch.mm(s["x"][a:a + 2048].to(D64), w.t())
        if s["bias"] is not None:
            u += s["bias"].to(D64)
        kind = c["act"]
        if kind == "gelu":
            y = u * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * u * (1 + 0.044715 * u * u))
        elif kind == "silu":
            y = u * torch.sigmoid(u)
        elif kind == "none":
            y = u
        else:
            y = torch.where(u > 0, u * u if kind == "relu2" else u, 0.0)
        if c["rate"]:
            y = y * _keep64(*y.shape, s["rng"], 5, c["rate"])
        if s["residual"] is not None:
            y = y + s["residual"].to(D64)
        return dict(out=y, pre=u) if c["pre"] else dict(out=y)
    if c["op"] == "lingrad":
        T, K, N = c["tokens"], c["fin"], c["fout"]
        w = s["weight"].to(D64)
        dx = torch.empty((T, K), dtype=D64, device="cuda")
        dw, db = torch.zeros((N, K), dtype=D64, device="cuda"), torch.zeros(N, dtype=D64, device="cuda")
        for a in range(0, T, 2048):
            d = s["dout"][a:a + 2048].to(D64)
            dw.addmm_(d.t(), s["x"][a:a + 2048].to(D64))
            db += d.sum(0)
            part = d @ w
            if s["pre"] is not None:
                with torch.enable_grad():   # the slope, from the value's definition
                    v = s["pre"][a:a + 2048].to(D64).requires_grad_()
                    kind = c["act"]
                    if kind == "gelu":
                        y = v * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * v * (1 + 0.044715 * v * v))
                    elif kind == "silu":
                        y = v * torch.sigmoid(v)
                    else:
                        y = torch.relu(v) ** (2 if kind == "relu2" else 1)
                    part = part * torch.autograd.grad(y.sum(), v)[0]
            dx[a:a + 2048] = part
        at = c["offset"]
        old = s["accum"].to(D64)
        keep = 0.0 if c["overwrite"] else 1.0
        out = dict(dx=dx, dw=keep * old[at:at + N * K].view(N, K) + s["scale"] * dw)
        if s["bias"] is not None:
            out["db"] = (keep * old[at + N * K:at + N * K + N] + s["scale"] * db).view(1, N)
        return out
    if c["op"] == "dropout":
        y = s["x"].to(D64) * _keep64(c["rows"], c["cols"], s["rng"], 5, c["rate"])
        return y if s["residual"] is None else y + s["residual"].to(D64)
    z = _rotation64(s)
    if c["op"] == "rotary":
        out = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.to(D64)
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(D64)
            out.append(_turn64(x, z, c))
        return out
    out, sums = [], []
    for d, x, w in ((s["dq"], s["q"], s["qw"]), (s["dk"], s["k"], s["kw"])):
        g = _turn64(d.to(D64), z.conj(), c)
        if w is not None:
            x = x.to(D64)
            rms = torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
            sums.append(torch.einsum("thd,thd->d", g, x / rms))
            g = g * w.to(D64)
            g = g / rms - x * (g * x).mean(-1, keepdim=True) / rms ** 3
        out.append(g)
    for i, v in enumerate(sums):
        old = 0.0 if c["overwrite"] else s["accum"][i * c["dim"]:(i + 1) * c["dim"]].to(D64)
        out.append((old + s["scale"] * v).view(1, -1))
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] in ("linear", "lingrad"):
        T, K, N = c["tokens"], c["fin"], c["fout"]
        if c["op"] == "linear":
            es = 2 if c["out"] == "bf16" else 4
            return {"bytes": 2 * (T * K + N * K + N * c["bias"]) + T * N * (es * (1 + c["residual"]) + 2 * c["pre"]),
                    "flops": 2 * T * K * N}
        sums = (N * K + N * c["bias"]) * (4 if c["overwrite"] else 8)
        return {"bytes": 2 * (T * N + T * K * (3 if c["act"] != "none" else 2) + N * K) + sums,
                "flops": 4 * T * K * N}
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        return {"bytes": n * es * (2 + c["residual"]), "flops": 2 * n}
    n = c["tokens"] * (c["heads"] + c["kv"]) * c["dim"]
    if c["op"] == "rotary":
        return {"bytes": 2 * n * es + c["tokens"] * c["axes"] * 8, "flops": 8 * n}
    return {"bytes": (3 if c["norm"] else 2) * n * es + c["tokens"] * c["axes"] * 8, "flops": 16 * n}
