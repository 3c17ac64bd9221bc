"""Timing cases of rotary positions and of a 4-bit key/value cache that is held to a budget: rotating
rows, writing rotated keys into the cache, attention that also adds up the weight each key received,
and moving the tokens with the most weight to fewer pages.

Each case is a dict of plain values.  ``run`` with ``own`` false computes it with elementary torch
operations in 32 bits (angles in 64), with ``own`` true through the package's entry points ``rope``,
``kv_write_rope``, ``kv_attend_weights`` and ``kv_evict``.

Rotary positions: with f_i the angle per position of pair i, values (a, b) of a pair at position p become
(a c - b s, a s + b c), c = m cos(p f_i), s = m sin(p f_i).  Pair i is values (i, i + rot/2) of a head, or
(2i, 2i + 1) interleaved; values from rot on stay.

The cache is that of ``kv_write``: pages of 64 tokens, per (page, kv head) 72 * dim bytes,

    K codes   64 tokens x dim/2 bytes     16 bytes per group of 32 values
    K scales  64 x dim/32 f16             [token][group]
    V codes   32 token pairs x dim bytes  16 bytes per 16 values of two tokens
    V scales  32 x dim/32 x 2 f16         [token pair][group][token]

with value = scale * (code - 8), scale of 7 significant bits.  The weights are f32 [page][kv head][64].
"""
import math

import torch

own = False

PAGE = 64
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------- cases
def _rope(name, dtype, rows, heads, dim, rot, interleaved, scaling, far):
    """Positions below far; scaling stretches a context of 4096."""
    return {"name": name, "op": "rope", "dtype": dtype, "rows": rows, "heads": heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "scaling": scaling, "far": far}


def _enter(name, dtype, batch, new, length, heads, kv_heads, dim, rot, interleaved, scaling):
    """new and length are (shortest, longest) over the sequences of the batch."""
    return {"name": name, "op": "enter", "dtype": dtype, "batch": batch, "new_lo": new[0], "new_hi": new[1],
            "len_lo": length[0], "len_hi": length[1], "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "scaling": scaling}


def _weigh(name, dtype, batch, new, length, heads, kv_heads, dim, window=0, sinks=0, decay=1.0):
    return {"name": name, "op": "weigh", "dtype": dtype, "batch": batch, "new_lo": new[0], "new_hi": new[1],
            "len_lo": length[0], "len_hi": length[1], "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "window": window, "sinks": sinks, "decay": decay}


def _evict(name, batch, length, kv_heads, dim, keep, first, last):
    return {"name": name, "op": "evict", "batch": batch, "new_lo": 1, "new_hi": 1, "len_lo": length[0],
            "len_hi": length[1], "kv_heads": kv_heads, "dim": dim, "keep": keep, "first": first, "last": last}


def listed():
    return [
        # the queries of a decoding step, far into a stretched context: latency
        _rope("rope_step", "bf16", 64, 32, 128, 128, False, "yarn", 131072),
        # the queries of a prompt of the 7B shape, in the 32 bits that the linear layers give
        _rope("rope_prompt", "f32", 3314, 32, 128, 128, True, "none", 3314),
        # heads of an odd size of which only a part turns
        _rope("rope_part", "f16", 8191, 16, 80, 32, False, "linear", 8191),
        # one decoding step of a small batch: rows turned, keys and values into the cache, and read back
        _enter("enter_step", "f32", 8, (1, 1), (130, 3314), 32, 8, 128, 128, False, "bands"),
        # prompts of a ragged batch enter the cache, and are read back
        _enter("enter_prompt", "f32", 3, (700, 3314), (700, 3314), 32, 8, 128, 128, False, "none"),
        # a single token over one long document, and what each key received
        _weigh("weigh_step_long", "f32", 1, (1, 1), (131071, 131071), 32, 8, 128),
        # a decoding step of a ragged batch with shared heads, old weight fading
        _weigh("weigh_step_batch", "bf16", 64, (1, 1), (95, 8192), 32, 8, 128, 0, 0, 0.98),
        # the last tokens of each prompt tell which of its keys matter
        _weigh("weigh_last_rows", "f16", 6, (16, 32), (3000, 30000), 32, 8, 128),
        # a whole prompt of the 7B shape
        _weigh("weigh_prompt", "f32", 1, (3314, 3314), (3314, 3314), 32, 32, 128),
        # a few short sequences have outgrown their budget
        _evict("evict_short", 4, (1101, 1280), 8, 128, 1024, 4, 128),
        # a batch of conversations cut to half of the longest
        _evict("evict_batch", 64, (2000, 8192), 8, 128, 4096, 4, 512),
        # one long document cut to an eighth
        _evict("evict_long", 1, (131071, 131071), 8, 128, 16383, 65, 1000),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["rope", "rope", "enter", "enter", "step", "step", "prompt", "prompt", "evict", "evict"])
    dtype = rng.choice(sorted(DTYPES))
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    interleaved = rng.random() < 0.5
    if kind == "rope":
        dim = rng.choice([64, 80, 96, 112, 128, 128, 160, 192, 256])
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        heads = _log(rng, 1, 64)
        rows = _log(rng, 1, max(2, min(16384, (1 << 25) // (heads * dim))))
        case = _rope("", dtype, rows, heads, dim, rot, interleaved, scaling, _log(rng, max(rows, 2), 1 << 20))
        del case["name"]
        return case
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if g * kv_heads <= 64])
    heads = group * kv_heads
    if kind == "enter":
        batch = _log(rng, 1, 64)
        top = max(1, (1 << 24) // ((heads + 2 * kv_heads) * dim * batch))
        new = _log(rng, 1, min(top + 1, 4096))
        more = _log(rng, 1, 8192)
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        case = _enter("", dtype, batch, (max(1, new // 2), new), (new, new + more), heads, kv_heads, dim, rot,
                      interleaved, scaling)
    elif kind == "evict":
        batch = _log(rng, 1, 64)
        top = min(131072, (1 << 22) * 64 // (kv_heads * batch * dim))
        length = _log(rng, 40, max(80, top))
        keep = max(2, int(length * rng.uniform(0.1, 0.95)))
        first = rng.choice([0, 1, 4, min(65, keep // 2)])
        first = min(first, keep // 2)
        case = _evict("", batch, (max(1, length // 3), length), kv_heads, dim, keep, first,
                      rng.randint(0, keep - first))
    else:
        batch = _log(rng, 1, 64) if kind == "step" else _log(rng, 1, 8)
        window = rng.choice([0, 0, _log(rng, 16, 4096)])
        sinks = rng.choice([0, 1, 4, 65]) if window else 0
        if kind == "step":
            new = rng.choice([1, 1, 1, 2, 4, 7])
            top = min(131072, 131072 * 8 * 128 // (kv_heads * batch * dim), (1 << 28) // (heads * batch * new))
            length = new + _log(rng, 1, max(2, top))
        else:
            length = _log(rng, 33, 16384)
            room = (1 << 29) // (heads * batch * length)
            new = max(1, min(length, room, _log(rng, 17, 4096)))
        case = _weigh("", dtype, batch, (max(1, new // 2), new), (max(new, length // 3), length), heads, kv_heads,
                      dim, window, sinks, rng.choice([1.0, 1.0, 0.9]))
    del case["name"]
    return case


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, uneven, the longest first."""
    return [hi] + [lo + int((hi - lo) * ((i * 0.6180339887) % 1.0)) for i in range(1, n)]


def _batch(case):
    """(new tokens, length) of each sequence."""
    new = _spread(case["new_lo"], case["new_hi"], case["batch"])
    length = _spread(case["len_lo"], case["len_hi"], case["batch"])
    return new, [max(n, m) for n, m in zip(new, length)]


def _visible(p, window, sinks):
    """Keys that a query at position p sees."""
    return p + 1 if window == 0 else min(p + 1, window + max(0, min(sinks, p + 1 - window)))


def work(case):
    if case["op"] == "rope":        # rows in and out; two products and a sum a value, its share of an angle
        n = case["rows"] * case["heads"] * case["dim"]
        return {"bytes": 2 * n * (4 if case["dtype"] == "f32" else 2) + 4 * case["rows"],
                "flops": 3 * case["rows"] * case["heads"] * case["rot"]}
    new, length = _batch(case)
    dim, hk = case["dim"], case["kv_heads"]
    values = 2 * hk * dim
    if case["op"] == "evict":       # a weight of each token, 4.5 bits a value of those that stay, in and out
        stay = sum(min(m, case["keep"]) for m in length)
        return {"bytes": 4 * hk * sum(length) + stay * (2 * values * 0.5625 + 8 * hk), "flops": 2 * hk * sum(length)}
    wide = 4 if case["dtype"] == "f32" else 2
    rows = sum(new) * case["heads"] * dim
    if case["op"] == "enter":       # rows in, turned queries out, 4.5 bits a value out and in again, values out
        n = sum(new) * values
        return {"bytes": 2 * rows * wide + n * (wide + 2 + 2 * 0.5625) + 4 * sum(new),
                "flops": 3 * rows // dim * case["rot"] + 6 * n}
    pairs = keys = 0
    for n, m in zip(new, length):
        first = m - n
        pairs += sum(_visible(p, case["window"], case["sinks"]) for p in range(first, m))
        seen = m if case["window"] == 0 else min(m, case["window"] + n - 1 + min(case["sinks"], m))
        keys += min(m, seen)
    return {"bytes": 2 * rows * wide + keys * values * 0.5625 + 8 * hk * sum(length),
            "flops": (4 * dim + 1) * case["heads"] * pairs}


# ------------------------------------------------------------------------------------- plain form
def _frequencies(rot, scaling, factor=32.0, original=4096.0, base=10000.0):
    """Angle per position of each pair (f64) and the factor on cosine and sine."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":            # a larger base, by which the slowest pair turns factor times slower
        base = base * factor ** (rot / max(rot - 2.0, 1.0)) if rot > 2 else base
    f = base ** (-2.0 * i / rot)
    m = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":         # fast pairs stay, slow ones are stretched, a ramp between
        def at(turns):
            return rot * math.log(original / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo = min(max(math.floor(at(32.0)), 0), rot - 1)
        hi = min(max(math.ceil(at(1.0)), 0), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f = f / factor * ramp + f * (1.0 - ramp)
        m = 0.1 * math.log(factor) + 1.0
    elif scaling == "bands":        # by wavelength: below original / 4 as they are, above original stretched
        smooth = ((original * f / (2.0 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
        f = (1.0 - smooth) * f / factor + smooth * f
    return f, m


def _turn(x, pos, s):
    """Rows x [n, heads, dim] at positions pos [n], in 32 bits."""
    angle = pos.double()[:, None] * s["freq"]
    c, d = ((y.float() * s["magnitude"])[:, None] for y in (angle.cos(), angle.sin()))
    x, rot = x.float(), s["rot"]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = a * c - b * d, a * d + b * c
    turned = torch.stack([p, q], -1).flatten(-2) if s["interleaved"] else torch.cat([p, q], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _maps(dim, device):
    """Byte and shift of the code, and byte of the scale, of each (token, value) of a piece."""
    t = torch.arange(PAGE, device=device)[:, None]
    d = torch.arange(dim, device=device)[None, :]
    ng, g, r = dim // 32, d // 32, d % 32
    place = g ^ ((t >> (1 if dim == 128 else 2)) & (ng - 1))
    maps = {"k_byte": t * (dim // 2) + place * 16 + (r // 8) * 4 + (r % 2) * 2 + (r % 8) // 4,
            "k_shift": 4 * (((r % 8) // 2) % 2) + 0 * t,
            "k_scale": 32 * dim + (t * ng + g) * 2}
    pair, block = t // 2, d // 16
    place = block ^ (((pair >> 2) ^ (pair << 1 & 6 if dim == 128 else pair & 2)) & (dim // 16 - 1))
    maps["v_byte"] = 36 * dim + pair * dim + place * 16 + (d % 16) // 4 * 4 + (t % 2) * 2 + (d % 4) // 2
    maps["v_shift"] = 4 * (d % 2) + 0 * t
    maps["v_scale"] = 68 * dim + ((pair * ng + g) * 2 + t % 2) * 2
    for x in ("k", "v"):    # the values of each byte, low one first, and the bytes
        maps[x + "_order"] = torch.argsort(maps[x + "_byte"] * 8 + maps[x + "_shift"], dim=-1)
        maps[x + "_bytes"] = maps[x + "_byte"].gather(-1, maps[x + "_order"])[:, ::2]
    return maps


def _quantise(x):
    """f32 [..., dim] -> codes 0..15 and scales [..., dim/32]."""
    x = x.float()
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = g.abs().amax(-1)
    s = amax / torch.full_like(amax, 7.5)
    s = ((s.view(torch.int32) + 0x1FFFF) & ~0x1FFFF).view(torch.float32).clamp(2.0 ** -14, 896.0)
    c = (g / s[..., None]).round().clamp(-8, 7) + 8
    return c.to(torch.uint8).reshape(x.shape), s.half()


def _put(pages, page, head, slot, codes, scales, name, maps):
    """Codes [..., dim] and scales [..., dim/32] into slot of (page, head), three tensors of [...]."""
    dim = codes.shape[-1]
    order = maps[name + "_order"][slot].expand(codes.shape)
    both = codes.gather(-1, order).reshape(*codes.shape[:-1], dim // 2, 2)
    page, head = page[..., None], head[..., None]
    pages[page, head, maps[name + "_bytes"][slot]] = both[..., 0] | (both[..., 1] << 4)
    at = maps[name + "_scale"][slot][..., ::32]
    raw = scales.contiguous().view(torch.uint8).reshape(*scales.shape, 2)
    pages[page, head, at] = raw[..., 0]
    pages[page, head, at + 1] = raw[..., 1]


def _get(pages, page, head, slot, name, maps):
    """The reverse."""
    page, head = page[..., None], head[..., None]
    codes = (pages[page, head, maps[name + "_byte"][slot]] >> maps[name + "_shift"][slot].to(torch.uint8)) & 15
    return codes, pages.view(torch.float16)[page, head, maps[name + "_scale"][slot][..., ::32] // 2]


def _store(pages, page, slot, k, v, maps):
    """Rows k, v [n, kv heads, dim] into slot[n] of page[n]."""
    head = torch.arange(k.shape[1], device=k.device)[None]
    for x, name in ((k, "k"), (v, "v")):
        _put(pages, page[:, None], head, slot[:, None], *_quantise(x), name, maps)


def _load(pieces, name, maps):
    """uint8 pieces [..., 72 * dim] -> f32 values [..., 64, dim]."""
    by, sh, at = maps[name + "_byte"], maps[name + "_shift"].to(torch.uint8), maps[name + "_scale"]
    codes = ((pieces[..., by] >> sh) & 15).float() - 8.0
    scales = pieces.view(torch.float16)[..., at[:, ::32] // 2].float()
    return codes * scales.repeat_interleave(32, -1)


def _places(s):
    """(sequence, position, page, slot) of each packed row."""
    row = torch.arange(s["rows"], device=s["start"].device, dtype=torch.int32)
    b = torch.searchsorted(s["start"][1:], row, right=True)
    pos = (s["length"][b] - s["start"][b + 1] + row).long()
    return b, pos, s["table"][b, pos // PAGE].long(), pos % PAGE


def _plain_rope(s):
    return _turn(s["x"], s["pos"], s).to(s["x"].dtype)


def _plain_enter(s):
    _, _, page, slot = _places(s)
    maps, pages = s["maps"], s["pages"]
    _store(pages, page, slot, _turn(s["k"], s["pos"], s), s["v"], maps)
    out = [_turn(s["q"], s["pos"], s).to(s["q"].dtype)]
    head = torch.arange(s["kv_heads"], device=page.device)[None]
    for name in ("k", "v"):
        codes, scales = _get(pages, page[:, None], head, slot[:, None], name, maps)
        out.append(((codes.float() - 8.0) * scales.float().repeat_interleave(32, -1)).half())
    return out


def _plain_weigh(s):
    q, hk, dim = s["q"], s["kv_heads"], s["dim"]
    n, heads = q.shape[:2]
    batch, group, dev = s["table"].shape[0], heads // hk, q.device
    # the whole cache of the batch in 32 bits: [batch, kv heads, keys, dim]
    pieces = s["pages"][s["table"].clamp(min=0).long()].transpose(1, 2)
    keys = s["table"].shape[1] * PAGE
    j = torch.arange(keys, device=dev)
    held = j[None] < s["length"][:, None]
    k, v = (torch.where(held[:, None, :, None], _load(pieces, x, s["maps"]).reshape(batch, hk, keys, dim), 0.0)
            for x in ("k", "v"))
    # the rows of the batch, padded to the longest: [batch, kv heads, rows * group, dim]
    b, pos, _, _ = _places(s)
    i = torch.arange(n, device=dev) - s["start"][b]
    rows = s["max_q"]
    wide = torch.zeros(batch, rows, hk, group, dim, device=dev)
    wide[b, i] = q.reshape(n, hk, group, dim).float()
    at = torch.full((batch, rows), -1, device=dev, dtype=torch.long)
    at[b, i] = pos
    wide = wide.permute(0, 2, 1, 3, 4).reshape(batch, hk, rows * group, dim)
    x = wide @ k.transpose(-1, -2)
    x *= s["scale"]
    seen = j[None, None] <= at[..., None]
    if s["window"]:
        seen &= (j[None, None] > at[..., None] - s["window"]) | (j < s["sinks"])
    seen = seen[:, None, :, None]
    x = x.reshape(batch, hk, rows, group, keys).masked_fill_(~seen, float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(m).exp_()
    p /= p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = p.reshape(batch, hk, rows * group, keys) @ v
    o = o.reshape(batch, hk, rows, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, rows, heads, dim)[b, i]
    # what each key received, added to what it had; new keys had nothing
    got = p.sum((2, 3))
    page = s["table"].clamp(min=0).long()
    old = s["weights"][page].transpose(1, 2).reshape(batch, hk, keys)
    new = (s["start"][1:] - s["start"][:-1])[:, None, None]
    got += torch.where(j < s["length"][:, None, None] - new, old * s["decay"], 0.0)
    where = held.nonzero(as_tuple=True)
    s["into"][page[where[0], where[1] // PAGE], :, where[1] % PAGE] = got.transpose(1, 2)[where]
    return [o.to(q.dtype), s["into"]]


def _plain_evict(s):
    table, length, keep, hk, maps = s["table"], s["length"].long(), s["keep"], s["kv_heads"], s["maps"]
    batch, dev = table.shape[0], table.device
    j = torch.arange(table.shape[1] * PAGE, device=dev)
    w = s["weights"][table.clamp(min=0).long()].transpose(1, 2).reshape(batch, hk, -1)
    m = length[:, None, None]
    w = torch.where((j < s["first"]) | (j >= m - s["last"]), float("inf"), w)
    w = torch.where(j < m, w, float("-inf"))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    stay = torch.minimum(length, torch.full_like(length, keep))
    order = torch.where(torch.arange(order.shape[-1], device=dev) < stay[:, None, None], order, j.numel())
    order = order.sort(-1).values
    kept = torch.full((batch, hk, keep), -1, device=dev, dtype=torch.int32)
    kept[..., :order.shape[-1]] = torch.where(order < j.numel(), order, -1).int()
    # (sequence, head, place) of what stays
    b, h, i = (kept >= 0).nonzero(as_tuple=True)
    old = kept[b, h, i].long()
    page, slot = table[b, old // PAGE].long(), old % PAGE
    page_to, slot_to = s["new_table"][b, i // PAGE].long(), i % PAGE
    for name in ("k", "v"):
        _put(s["pages"], page_to, h, slot_to, *_get(s["pages"], page, h, slot, name, maps), name, maps)
    s["weights"][page_to, h, slot_to] = s["weights"][page, h, slot]
    return [s["pages"], s["weights"], stay.int(), kept]


# ------------------------------------------------------------------------------------------ state
def _plan(s, case, dev):
    freq, s["magnitude"] = _frequencies(case["rot"], case["scaling"])
    s["freq"], s["rot"], s["interleaved"] = freq.to(dev), case["rot"], case["interleaved"]
    if own:         # a program keeps this beside its weights
        import quant_int8_mmq_gb300 as mmq
        s["plan"] = mmq.rope_plan(case["rot"], interleaved=case["interleaved"], scaling=case["scaling"], factor=32.0,
                                  original=4096, device=dev)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "rope":
        _plan(s, case, dev)
        # part of a wider row, as a product of several projections leaves it
        n, heads, dim = case["rows"], case["heads"], case["dim"]
        wide = torch.randn(n, heads * dim + 2 * dim, device=dev, generator=gen).to(DTYPES[case["dtype"]])
        s["x"] = wide[:, :heads * dim].view(n, heads, dim)
        s["pos"] = torch.arange(n, device=dev, dtype=torch.int32) + int(seed) % 7
        if n < case["far"] // 4:    # tokens of several sequences
            s["pos"] = torch.randint(0, case["far"], (n,), device=dev, dtype=torch.int32, generator=gen)
        return s
    new, length = _batch(case)
    batch, hk, dim = case["batch"], case["kv_heads"], case["dim"]
    maps = _maps(dim, dev)
    need = [-(-m // PAGE) for m in length]
    stay = [-(-min(m, case.get("keep", 0)) // PAGE) for m in length]
    num = sum(need) + sum(stay) + 3
    # pages in no order; entries past a sequence's last page are no pages
    perm = torch.randperm(num, device=dev, generator=gen).to(torch.int32)

    def take(counts, at):
        first = torch.tensor([at] + counts, device=dev).cumsum(0)
        col = torch.arange(max(max(counts), 1), device=dev)
        used = col[None] < torch.tensor(counts, device=dev)[:, None]
        return torch.where(used, perm[(first[:-1, None] + col[None]).clamp(max=num - 1)], -1).contiguous()

    table = take(need, 0)
    start = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    rows = sum(new)
    s.update(maps=maps, table=table, start=start, rows=rows, kv_heads=hk, dim=dim, max_q=max(new), max_kv=max(length),
             length=torch.tensor(length, device=dev, dtype=torch.int32))
    # slots that no token has been written to hold whatever the memory held
    pages = torch.randint(0, 256, (num, hk, 72 * dim), device=dev, dtype=torch.uint8, generator=gen)
    s["pages"] = pages
    if case["op"] == "evict":
        # what the bytes stand for does not matter to a move.  A few keys have most of the weight, many
        # the same little or none
        w = torch.randn(num, hk, PAGE, device=dev, generator=gen).mul_(3.0).exp_()
        s["weights"] = torch.where(w < 0.05, torch.where(w < 0.01, 0.0, 0.03125), w)
        s["new_table"] = take(stay, sum(need))
        s["keep"], s["first"], s["last"] = case["keep"], case["first"], case["last"]
        return s
    dtype = DTYPES[case["dtype"]]
    # keys have a few strong channels, values a few strong tokens
    loud = 1.0 + 4.0 * (torch.rand(hk, dim, device=dev, generator=gen) < 0.05)

    def kv(n):
        k = torch.randn(n, hk, dim, device=dev, generator=gen)
        k *= loud
        v = torch.randn(n, hk, dim, device=dev, generator=gen)
        v *= torch.rand(n, 1, 1, device=dev, generator=gen) + 0.5
        return k, v

    if case["op"] == "enter":
        _plan(s, case, dev)
        s["k"], s["v"] = (x.to(dtype) for x in kv(rows))
        s["pos"] = _places(s)[1].int()
    else:
        # every token of every sequence, a page of each sequence at a time
        tail = torch.tensor(length, device=dev)
        seq = torch.repeat_interleave(torch.arange(batch, device=dev), tail)
        pos = torch.arange(sum(length), device=dev) - torch.repeat_interleave(tail.cumsum(0) - tail, tail)
        for lo in range(0, sum(length), 1 << 16):
            b, p = seq[lo:lo + (1 << 16)], pos[lo:lo + (1 << 16)]
            k, v = kv(b.numel())
            _store(pages, table[b, p // PAGE].long(), p % PAGE, k, v, maps)
        s["scale"] = dim ** -0.5
        s["window"], s["sinks"], s["decay"] = case["window"], case["sinks"], case["decay"]
        # what earlier steps have added up, and where the sums with this step's go
        s["weights"] = torch.randn(num, hk, PAGE, device=dev, generator=gen).exp_()
        s["into"] = torch.zeros(num, hk, PAGE, device=dev)
    s["q"] = (1.5 * torch.randn(rows, case["heads"], dim, device=dev, generator=gen)).to(dtype)
    return s


def run(s):
    if not own:
        return {"rope": _plain_rope, "enter": _plain_enter, "weigh": _plain_weigh, "evict": _plain_evict}[s["op"]](s)
    import quant_int8_mmq_gb300 as mmq
    if s["op"] == "rope":
        return mmq.rope(s["x"], s["pos"], s["plan"])
    cache = (s["pages"], s["table"], s["start"], s["length"])
    if s["op"] == "enter":
        q = mmq.kv_write_rope(s["q"], s["k"], s["v"], s["pos"], s["plan"], *cache)
        return [q, *mmq.kv_read(*cache, s["rows"])]
    if s["op"] == "weigh":
        return list(mmq.kv_attend_weights(s["q"], s["weights"], *cache, max_q=s["max_q"], max_kv=s["max_kv"],
                                          scale=s["scale"], window=s["window"], sinks=s["sinks"], decay=s["decay"],
                                          into=s["into"]))
    length, kept = mmq.kv_evict(s["weights"], *cache, s["new_table"], s["keep"], first=s["first"], last=s["last"],
                                max_kv=s["max_kv"])
    return [s["pages"], s["weights"], length, kept]


# ------------------------------------------------------------------------------- the definition, 64 bits
def _values64(x):
    """What the cache holds for f64 rows: groups of 32, 4-bit codes, a scale of 7 significant bits."""
    g = x.unflatten(-1, (-1, 32))
    t = (g.abs().amax(-1, keepdim=True) / 7.5).clamp(min=2.0 ** -14)
    # the unit in the seventh significant place: t's power of two, 6 places down
    unit = (((t.view(torch.int64) >> 52) - 6) << 52).view(torch.float64)
    s = (torch.ceil(t / unit) * unit).clamp(2.0 ** -14, 896.0)
    return (s * torch.clamp(torch.round(g / s), -8, 7)).flatten(-2)


def _turn64(x, pos, s):
    """Rows as complex numbers times m e^(i p f)."""
    z, rot = x.double(), s["rot"]
    order = torch.arange(rot, device=z.device)
    order = order if s["interleaved"] else order.view(2, -1).T.flatten()
    pairs = torch.view_as_complex(z[..., order].unflatten(-1, (-1, 2)).contiguous())
    angle = torch.outer(pos.double(), s["freq"])
    pairs = pairs * torch.polar(torch.full_like(angle, s["magnitude"]), angle)[:, None]
    out = z.clone()
    out[..., order] = torch.view_as_real(pairs).flatten(-2)
    return out


def _decode64(piece, dim):
    """Pieces [n, kv heads, 72 * dim] -> K and V [kv heads, n * 64, dim] in 64 bits, value by value."""
    piece = piece.transpose(0, 1).contiguous()
    n = piece.shape[:2]
    ng = dim // 32
    words = piece.view(torch.int32)
    k = torch.empty(*n, PAGE, dim, dtype=torch.float64, device=piece.device)
    v = torch.empty_like(k)
    half = piece.view(torch.float16).double()
    for t in range(PAGE):
        for g in range(ng):
            at = t * (dim // 8) + (g ^ ((t >> (1 if dim == 128 else 2)) & (ng - 1))) * 4
            for u in range(4):
                for p in range(4):
                    for h in range(2):
                        code = (words[..., at + u] >> (4 * p + 16 * h)) & 15
                        k[..., t, 32 * g + 8 * u + 2 * p + h] = (code - 8) * half[..., 16 * dim + t * ng + g]
        for block in range(dim // 16):
            turn = (t // 8) ^ (t // 2 % 4 * 2) if dim == 128 else (t // 8 % 4) ^ (t // 4 % 2 * 2)
            at = 9 * dim + (t // 2) * (dim // 4) + (block ^ (turn & 7)) * 4
            for d in range(16):
                code = (words[..., at + d // 4] >> (4 * (d % 4) + 16 * (t % 2))) & 15
                v[..., t, 16 * block + d] = (code - 8) * half[..., 34 * dim + (t // 2 * ng + block // 2) * 2 + t % 2]
    return k.flatten(1, 2), v.flatten(1, 2)


def _moved64(s):
    """The weights after a move, a sequence and head at a time."""
    out = s["weights"].double()
    for b, m in enumerate(s["length"].tolist()):
        j = torch.arange(m, device=out.device)
        page = s["table"][b, j // PAGE].long()
        free = slice(min(s["first"], m), max(min(s["first"], m), m - s["last"]))
        for h in range(s["kv_heads"]):
            w = s["weights"][page, h, j % PAGE].double()
            n = max(min(m, s["keep"]) - (m - (free.stop - free.start)), 0)
            # the n-th largest, all above it, and the first of those that equal it
            stays = torch.ones(m, dtype=torch.bool, device=out.device)
            if free.stop - free.start > n:
                c = w[free]
                least = c.topk(n).values[-1] if n else float("inf")
                over, same = c > least, c == least
                stays[free] = over | (same & (same.cumsum(0) <= n - over.sum()))
            i = torch.arange(int(stays.sum()), device=out.device)
            out[s["new_table"][b, i // PAGE].long(), h, i % PAGE] = w[stays]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turn64(s["x"], s["pos"], s)
    if case["op"] == "enter":
        return [_turn64(s["q"], s["pos"], s), _values64(_turn64(s["k"], s["pos"], s)), _values64(s["v"].double())]
    if case["op"] == "evict":
        return [None, _moved64(s), None, None]      # the others are bytes and whole numbers
    table, length, start = s["table"].cpu(), s["length"].tolist(), s["start"].tolist()
    hk, dim = s["kv_heads"], s["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    into = s["into"].double()
    # the pages of all sequences, one after another
    pages = [table[b, :-(-m // PAGE)].long() for b, m in enumerate(length)]
    k, v = _decode64(s["pages"][torch.cat(pages).cuda()], dim)
    for h in range(hk):
        lo = 0
        for b, m in enumerate(length):
            kb, vb = k[h, lo:lo + m], v[h, lo:lo + m]
            lo += pages[b].numel() * PAGE
            group = case["heads"] // hk
            n = start[b + 1] - start[b]
            at = pages[b].cuda()
            had = s["weights"][at, h].double().flatten()[:m] * s["decay"]
            had[m - n:] = 0.0
            for i in range(0, n, 1024):
                c = min(1024, n - i)
                rows = slice(start[b] + i, start[b] + i + c)
                q = s["q"][rows, h * group:(h + 1) * group].double()
                x = torch.einsum("igd,jd->igj", q, kb) * s["scale"]
                p = torch.arange(m - n + i, m - n + i + c, device="cuda")[:, None]
                j = torch.arange(m, device="cuda")[None]
                ok = j <= p
                if s["window"]:
                    ok &= (p - j < s["window"]) | (j < s["sinks"])
                w = torch.softmax(torch.where(ok[:, None], x, float("-inf")), -1)
                out[rows, h * group:(h + 1) * group] = torch.einsum("igj,jd->igd", w, vb)
                had += w.sum((0, 1))
            mine = into[at, h].flatten()
            mine[:m] = had
            into[at, h] = mine.view(-1, PAGE)
    return [out, into]
