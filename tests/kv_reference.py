"""The 4-bit key/value cache and the attention over it from their definitions, in 64 bits and
one value at a time where the layout is concerned.  Shares nothing with the package."""
import numpy as np

PAGE = 64


def quantise(x):
    """f64 rows [..., D] -> codes 0..15 [..., D], scales f64 [..., D/32]."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = np.where(np.isnan(g), 0.0, np.abs(g)).max(-1)
    t = np.minimum(amax, 1e30) / 7.5
    m, e = np.frexp(np.maximum(t, 2.0 ** -40))          # m in [1/2, 1)
    s = np.clip(np.ldexp(np.ceil(m * 128.0), e - 7), 2.0 ** -14, 896.0)
    y = np.clip(np.nan_to_num(g, nan=0.0, posinf=1e30, neginf=-1e30) / s[..., None], -8.0, 7.0)
    return (np.rint(y) + 8).astype(np.int64).reshape(x.shape), s


def values(x):
    n, s = quantise(x)
    return (n - 8) * np.repeat(s, 32, axis=-1)


def code_place(kind, t, d, D):
    """(byte, shift) of value d of slot t in a piece of head size D."""
    if kind == "k":
        g, r = d // 32, d % 32
        u, p, h = r // 8, r % 8 // 2, r % 2
        turn = (t >> 1) & 3 if D == 128 else (t >> 2) & 1
        bit = 4 * p + 16 * h
        return t * (D // 2) + 16 * (g ^ turn) + 4 * u + bit // 8, bit % 8
    p, e, a = t // 2, t % 2, d // 16
    turn = ((p >> 2) ^ (2 * p & 6)) & 7 if D == 128 else ((p >> 2) ^ (p & 2)) & 3
    bit = 4 * (d % 4) + 16 * e
    return 36 * D + p * D + 16 * (a ^ turn) + 4 * (d % 16 // 4) + bit // 8, bit % 8


def scale_place(kind, t, g, D):
    if kind == "k":
        return 32 * D + 2 * (t * (D // 32) + g)
    return 68 * D + 2 * ((t // 2 * (D // 32) + g) * 2 + t % 2)


def put(pages, page, slot, k, v):
    """One token's k and v [heads, D] (f64) into uint8 pages [n, heads, 72 D]."""
    D = k.shape[1]
    for kind, x in (("k", k), ("v", v)):
        n, s = quantise(x)
        for h in range(k.shape[0]):
            piece = pages[page, h]
            for d in range(D):
                byte, shift = code_place(kind, slot, d, D)
                piece[byte] = (int(piece[byte]) & (0xF0 >> shift)) | int(n[h, d]) << shift
            for g in range(D // 32):
                at = scale_place(kind, slot, g, D)
                piece[at:at + 2] = np.frombuffer(np.float16(s[h, g]).tobytes(), np.uint8)


def attend(q, k, v, pos, scale, window=0, sinks=0):
    """q [n, heads, D] at positions pos [n] over k, v [keys, kv heads, D], all f64 (torch).
    Returns (out, S): S [n, heads] bounds scale * sum |q| |k| over the visible keys, for tolerances."""
    import torch
    n, heads, D = q.shape
    keys, hk = k.shape[:2]
    group = heads // hk
    p = pos[:, None]
    j = torch.arange(keys, device=q.device)[None]
    ok = j <= p
    if window:
        ok &= (j > p - window) | (j < sinks)
    ok = ok[:, None, None, :]
    qg = q.reshape(n, hk, group, D)
    if keys == 0:
        return torch.zeros_like(q), torch.zeros(n, heads, device=q.device, dtype=q.dtype)
    x = torch.where(ok, torch.einsum("nhgd,jhd->nhgj", qg, k) * scale, float("-inf"))
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m.isinf(), 0.0, m))
    total = w.sum(-1, keepdim=True)
    o = torch.einsum("nhgj,jhd->nhgd", w, v) / torch.where(total == 0, 1.0, total)
    S = torch.where(ok, torch.einsum("nhgd,jhd->nhgj", qg.abs(), k.abs()) * scale, 0.0).amax(-1)
    return o.reshape(n, heads, D), S.reshape(n, heads)
