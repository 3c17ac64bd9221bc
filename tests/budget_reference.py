"""Rotary positions, the weight that keys receive, and eviction from their definitions, in 64 bits.
Shares nothing with the package."""
import math

import numpy as np
import torch

from tests import kv_reference as kv

PAGE = 64


def angles(turns, pos):
    """Angles in radians of 64-bit turn fractions at whole positions: [len(pos), len(turns)], f64."""
    out = np.empty((len(pos), len(turns)))
    for i, p in enumerate(pos):
        for j, t in enumerate(turns):
            f = (int(t) * int(p)) % (1 << 64)
            out[i, j] = (f - (1 << 64) if f >> 63 else f) * (2.0 * math.pi / 2.0 ** 64)
    return out


def turn(x, angle, rot, interleaved, magnitude):
    """f64 rows x [n, heads, dim] turned by angle [n, rot / 2]; and the sum of each value's |products|."""
    c, s = (torch.from_numpy(f(angle)).to(x.device)[:, None] * magnitude for f in (np.cos, np.sin))
    pair = torch.arange(rot // 2, device=x.device)
    i, j = (2 * pair, 2 * pair + 1) if interleaved else (pair, pair + rot // 2)
    a, b = x[..., i], x[..., j]
    out, size = x.clone(), torch.zeros_like(x)
    out[..., i], out[..., j] = a * c - b * s, a * s + b * c
    size[..., i], size[..., j] = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    return out, size


def received(q, k, pos, scale, window=0, sinks=0):
    """What keys k [keys, kv heads, D] receive from rows q [n, heads, D] at positions pos: (weights [kv heads,
    keys], the same sums with each row's weight times 1 + S, S the row's largest scale * sum |q| |k|)."""
    n, heads, D = q.shape
    keys, hk = k.shape[:2]
    qg = q.reshape(n, hk, heads // hk, D)
    p, j = pos[:, None], torch.arange(keys, device=q.device)[None]
    ok = j <= p
    if window:
        ok &= (j > p - window) | (j < sinks)
    ok = ok[:, None, None, :]
    x = torch.where(ok, torch.einsum("nhgd,jhd->nhgj", qg, k) * scale, float("-inf"))
    w = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e300))
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    S = torch.where(ok, torch.einsum("nhgd,jhd->nhgj", qg.abs(), k.abs()) * scale, 0.0).amax(-1, keepdim=True)
    return w.sum((0, 2)), (w * (1.0 + S)).sum((0, 2))


def stays(w, keep, first, last):
    """Places, in order, of the tokens that stay of weights w [n] (numpy f32)."""
    n = len(w)
    if n <= keep:
        return list(range(n))
    middle = range(first, n - last)
    rank = sorted(middle, key=lambda i: (math.isnan(w[i]), 0.0 if math.isnan(w[i]) else -float(w[i])))   # stable: ties in order
    return sorted([*range(first), *rank[:keep - first - last], *range(n - last, n)])


def move(pages, to, new, old, D):
    """Codes and scales of slot old of piece `pages` (uint8 [72 D]) into slot new of piece `to`."""
    for kind in "kv":
        for d in range(D):
            byte, shift = kv.code_place(kind, old, d, D)
            n = int(pages[byte]) >> shift & 15
            byte, shift = kv.code_place(kind, new, d, D)
            to[byte] = (int(to[byte]) & (0xF0 >> shift)) | n << shift
        for g in range(D // 32):
            a, b = kv.scale_place(kind, old, g, D), kv.scale_place(kind, new, g, D)
            to[b:b + 2] = pages[a:a + 2]
