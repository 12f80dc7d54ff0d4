"""Plain 64-bit forms of the layer operators, shared by their tests: numpy and
torch on the CPU or the GPU, written from the formulas."""
import math

import numpy as np
import torch

D64 = torch.float64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # largest relative error of a rounding


def act(u, kind):
    """The activation and its slope."""
    one = torch.ones_like(u)
    if kind in (None, "none"):
        return u, one
    if kind in ("relu", "relu2"):
        r = torch.where(u > 0, u, torch.zeros_like(u))
        return (r, (u > 0).to(u.dtype)) if kind == "relu" else (r * r, 2 * r)
    if kind == "silu":
        s = torch.sigmoid(u)
        return u * s, s + u * s * (1 - s)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (u + 0.044715 * u ** 3))
    return 0.5 * u * (1 + t), 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * c * (1 + 3 * 0.044715 * u * u)


def least(rate):
    return math.floor(rate * 65536 + 0.5)


def draws(rows, cols, seed, step, site):
    """16 bits per element: Philox4x32-10, in Python's unbounded integers over numpy objects' 64-bit words."""
    m = np.uint64(0xFFFFFFFF)
    groups = (cols + 7) // 8
    g, r = np.meshgrid(np.arange(groups, dtype=np.uint64), np.arange(rows, dtype=np.uint64))
    c = [g, r, np.full_like(g, site), np.full_like(g, step & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & m, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    bits = np.stack([(c[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF) for j in range(8)], 2)
    return torch.from_numpy(bits.reshape(rows, groups * 8)[:, :cols].astype(np.int64))


def keep(rows, cols, rate, rng, site, device="cpu"):
    """What each element is multiplied by."""
    seed, step = (int(v) % (1 << 64) for v in rng.cpu())
    n = least(rate)
    return torch.where(draws(rows, cols, seed, step, site) >= n, 65536 / (65536 - n), 0.0).to(D64).to(device)


def rotation(positions, inv_freq, axis):
    """cos and sin, tokens x pairs."""
    p = positions.to(D64)
    p = p.view(p.shape[0], -1)
    axis = torch.zeros(len(inv_freq), dtype=torch.int64) if axis is None else torch.from_numpy(axis).long()
    angle = p[:, axis.to(p.device)] * torch.from_numpy(inv_freq).to(p.device)
    return torch.cos(angle), torch.sin(angle)


def turned(x, cos, sin, interleaved):
    pairs = cos.shape[1]
    a = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    b = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    out = x.clone()
    c, s = cos[:, None], sin[:, None]
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def heads_forward(x, w, norm, eps, cos, sin, interleaved):
    x = x.to(D64)
    if norm:
        x = x / torch.sqrt((x * x).mean(2, keepdim=True) + eps)
        if w is not None:
            x = x * w.to(D64)
    return x if cos is None else turned(x, cos, sin, interleaved)


def heads_backward(dout, x, w, norm, eps, cos, sin, interleaved):
    """dx and the weight's gradient (None without norm)."""
    g = dout.to(D64)
    if cos is not None:
        g = turned(g, cos, -sin, interleaved)
    if not norm:
        return g, None
    x = x.to(D64)
    r = 1 / torch.sqrt((x * x).mean(2, keepdim=True) + eps)
    n = x * r
    dw = (g * n).sum((0, 1))
    if w is not None:
        g = g * w.to(D64)
    return r * (g - n * (g * n).mean(2, keepdim=True)), dw
