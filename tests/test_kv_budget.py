"""Refusals, size queries and host arithmetic of rotary positions, weighed attention and eviction (no
GPU needed)."""
import math
from fractions import Fraction

import pytest

import quant_int8_mmq_gb300 as mmq
from tests.test_kv import ALIGN, ARG, OK, P16, SHAPE, UNSUPPORTED, cache, rows


def plan(**kw):
    f = dict(turns=P16, rot_dim=128, interleaved=0, magnitude=1.0)
    f.update(kw)
    return mmq.RopePlan(*(f[n] for n, _ in mmq.RopePlan._fields_))


def rope(p=None, x=None, out=None, pos=P16, heads=2, dim=128, n=4):
    return mmq.load().mmq_rope(p or plan(), x or rows(), out or rows(), pos, heads, dim, n, None)


def enter(c=None, p=None, q=None, q_out=None, heads=2, k=None, v=None, pos=P16, n=4):
    return mmq.load().mmq_kv_write_rope(c or cache(), p or plan(), q or rows(), q_out or rows(), heads, k or rows(),
                                        v or rows(), pos, n, None)


def weigh(c=None, q=None, out=None, heads=2, n=4, max_q=4, max_kv=256, scale=0.1, window=0, sinks=0, w=P16, to=P16,
          decay=1.0, ws=P16, size=1 << 40):
    return mmq.load().mmq_kv_attend_weights(c or cache(), q or rows(), out or rows(), heads, n, max_q, max_kv, scale,
                                            window, sinks, w, to, decay, ws, size, None)


def evict(c=None, w=P16, table=P16, pages=4, keep=200, first=4, last=64, max_kv=1000, length=P16, kept=P16):
    return mmq.load().mmq_kv_evict(c or cache(), w, table, pages, keep, first, last, max_kv, length, kept, None)


@pytest.mark.parametrize("call", [enter, weigh, evict])
def test_cache_is_checked_by_every_call(mmq_lib, call):
    for kw, st in ((dict(head_dim=80), SHAPE), (dict(kv_heads=0), SHAPE), (dict(num_pages=0), SHAPE), (dict(batch=0), SHAPE),
                   (dict(max_pages=0), SHAPE), (dict(max_pages=(1 << 24) + 1), SHAPE), (dict(pages=None), ARG),
                   (dict(table=None), ARG), (dict(length=None), ARG), (dict(pages=P16 + 8), ALIGN),
                   (dict(table=P16 + 2), ALIGN), (dict(length=P16 + 2), ALIGN)):
        assert call(c=cache(**kw)) == st, kw


@pytest.mark.parametrize("call,names", [(rope, ("x", "out")), (enter, ("q", "q_out", "k", "v")), (weigh, ("q", "out"))])
def test_rows_are_checked_by_every_call(mmq_lib, call, names):
    for name in names:
        for kw, st in ((dict(data=None), ARG), (dict(dtype=3), ARG), (dict(token_stride=-256), ARG),
                       (dict(head_stride=-128), ARG), (dict(token_stride=1 << 41), SHAPE), (dict(data=P16 + 2), ALIGN)):
            assert call(**{name: rows(**kw)}) == st, (name, kw)
        assert call(**{name: rows(dtype=1)}) == ARG          # one type for all
    written = {"x": "out", "q": "q_out"}.get(names[0]) if names[0] == "x" or len(names) > 2 else "out"
    for kw in (dict(token_stride=0), dict(head_stride=0), dict(token_stride=200)):
        assert call(**{written: rows(**kw)}) == ARG, kw


@pytest.mark.parametrize("call", [rope, enter])
def test_plans_and_positions_are_checked(mmq_lib, call):
    for kw, st in ((dict(turns=None), ARG), (dict(turns=P16 + 4), ALIGN), (dict(rot_dim=0), SHAPE), (dict(rot_dim=63), SHAPE),
                   (dict(rot_dim=130), SHAPE), (dict(interleaved=2), ARG), (dict(interleaved=-1), ARG),
                   (dict(magnitude=float("nan")), ARG), (dict(magnitude=float("inf")), ARG)):
        assert call(p=plan(**kw)) == st, kw
    assert call(pos=None) == ARG and call(pos=P16 + 2) == ALIGN
    for kw in (dict(heads=0), dict(heads=1025), dict(n=-1), dict(n=(1 << 22) + 1)):
        assert call(**kw) == SHAPE, kw


def test_heads_of_any_size_turn(mmq_lib):
    assert mmq.load().mmq_rope(None, rows(), rows(), P16, 2, 128, 4, None) == ARG
    assert rope(dim=1025, p=plan(rot_dim=64)) == SHAPE
    assert rope(dim=64, p=plan(rot_dim=66)) == SHAPE


def test_weights_and_decay_are_checked(mmq_lib):
    for kw, st in ((dict(w=None), ARG), (dict(to=None), ARG), (dict(w=P16 + 8), ALIGN), (dict(to=P16 + 4), ALIGN),
                   (dict(decay=-0.1), ARG), (dict(decay=1.5), ARG), (dict(decay=float("nan")), ARG), (dict(heads=3), SHAPE),
                   (dict(scale=0.0), ARG), (dict(window=-1), ARG), (dict(max_q=-1), ARG), (dict(n=-1), SHAPE)):
        assert weigh(**kw) == st, kw
    need = mmq.mmq_kv_attend_weights_workspace_bytes(cache(), 0, 2, 4, 4, 256)
    assert need >= 4 * 2 * 8 and need % 16 == 0
    assert weigh(ws=None) == ARG and weigh(size=need - 1) == ARG and weigh(ws=P16 + 8) == ALIGN
    many = cache(max_pages=4096)
    assert (mmq.mmq_kv_attend_weights_workspace_bytes(many, 0, 2, 1, 1, 4096 * 64)
            > mmq.mmq_kv_attend_workspace_bytes(many, 0, 2, 1, 1, 4096 * 64))
    assert mmq.load().mmq_kv_attend_weights_workspace_bytes(cache(), 0, 2, 4, 4, 256, 0, 0, None) == ARG


def test_evictions_numbers_are_checked(mmq_lib):
    for kw, st in ((dict(w=None), ARG), (dict(table=None), ARG), (dict(length=None), ARG), (dict(kept=None), ARG),
                   (dict(w=P16 + 4), ALIGN), (dict(table=P16 + 2), ALIGN), (dict(length=P16 + 1), ALIGN),
                   (dict(kept=P16 + 2), ALIGN), (dict(first=-1), ARG), (dict(last=-1), ARG), (dict(max_kv=-1), ARG),
                   (dict(keep=0), SHAPE), (dict(pages=0), SHAPE), (dict(keep=257), SHAPE), (dict(first=137), SHAPE),
                   (dict(first=(1 << 31) - 1, last=(1 << 31) - 1), SHAPE), (dict(pages=(1 << 24) + 1), SHAPE)):
        assert evict(**kw) == st, kw
    assert evict(c=cache(batch=1 << 20, kv_heads=1024)) == SHAPE


def test_no_rows_is_no_work(mmq_lib):
    before = mmq.mmq_launch_count()
    none = rows(data=None)
    assert rope(x=none, out=none, pos=None, n=0) == OK and enter(q=none, q_out=none, k=none, v=none, pos=None, n=0) == OK
    assert weigh(q=none, out=none, n=0, ws=None, size=0) == OK
    assert mmq.mmq_kv_attend_weights_workspace_bytes(cache(), 0, 2, 0, 1, 64) == 0
    assert mmq.mmq_launch_count() == before


def test_without_a_gpu_calls_are_unsupported(mmq_lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert rope() == enter() == weigh() == evict() == UNSUPPORTED


def test_turns_are_the_fraction(mmq_lib):
    """1 / (2 pi) to 60 digits; the turns are off by less than one unit of 2^-64, f64 frequencies being exact."""
    inv = Fraction(159154943091895335768883763372514362034459645740456448747667, 10 ** 60)
    freq = [1.0, 0.5, 1e-4, 10000.0 ** (-2 / 128), 6.283185307179586, 123456.789, -0.75, 1e6, -1e6, 0.0, 5e-324, 2.0 ** -60]
    for f, t in zip(freq, mmq.mmq_rope_turns(freq)):
        want = Fraction(f) * inv * 2 ** 64
        off = (t - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) < 1, f
    for bad in ([math.nan], [math.inf], [1.1e6], [1.0, -math.inf]):
        with pytest.raises(mmq.MMQError):
            mmq.mmq_rope_turns(bad)
    for n in (0, 513):
        with pytest.raises(mmq.MMQError):
            mmq.mmq_rope_turns([1.0] * n)


def test_frequencies_of_each_scaling(mmq_lib):
    rot, base, s, L = 64, 10000.0, 8.0, 2048.0
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
    close = lambda a, b: all(abs(x - y) <= 1e-13 * abs(y) for x, y in zip(a, b)) and len(a) == len(b)   # noqa: E731
    assert close(mmq.mmq_rope_frequencies("none", rot, base)[0], plain)
    assert close(mmq.mmq_rope_frequencies("linear", rot, base, s)[0], [f / s for f in plain])
    ntk = mmq.mmq_rope_frequencies("ntk", rot, base, s)[0]
    assert ntk[0] == 1.0 and abs(ntk[-1] * s / plain[-1] - 1) < 1e-12
    assert mmq.mmq_rope_frequencies("ntk", 2, base, s) == ([1.0], 1.0)
    yarn, m = mmq.mmq_rope_frequencies("yarn", rot, base, s, L)
    assert abs(m - (0.1 * math.log(s) + 1)) < 1e-6
    turns = [L * f / (2 * math.pi) for f in plain]
    inner = [i for i in range(rot // 2) if 1 < turns[i] < 32]
    for i in range(rot // 2):
        if i < inner[0] - 1:
            assert abs(yarn[i] / plain[i] - 1) < 1e-13
        if i > inner[-1] + 1:
            assert abs(yarn[i] * s / plain[i] - 1) < 1e-13
        assert plain[i] / s * (1 - 1e-13) <= yarn[i] <= plain[i] * (1 + 1e-13)
    # the ramp is even in the pair's number
    ramp = [(1 - yarn[i] / plain[i]) / (1 - 1 / s) for i in inner[1:-1]]
    steps = [b - a for a, b in zip(ramp, ramp[1:])]
    assert max(steps) - min(steps) < 1e-12 and min(steps) > 0
    bands, m = mmq.mmq_rope_frequencies("bands", rot, base, s, L)
    assert m == 1.0
    for f, t, b in zip(plain, turns, bands):
        near = min(max((t - 1) / 3, 0), 1)
        assert abs(b - (near * f + (1 - near) * f / s)) <= 1e-13 * f
    assert mmq.mmq_rope_frequencies("yarn", rot, base, 1.0, L)[1] == 1.0
    for bad in (("none", 63, base), ("none", 0, base), ("none", 1026, base), ("none", rot, 1.0), ("none", rot, math.inf),
                ("linear", rot, base, 0.5), ("linear", rot, base, math.nan), ("yarn", rot, base, s, 0.0), ("bands", rot, base, s),
                (5, rot, base, s, L), (-1, rot, base), ("ntk", rot, 1e300, 1e300)):
        with pytest.raises(mmq.MMQError):
            mmq.mmq_rope_frequencies(*bad)


def test_tensor_helpers_refuse(mmq_lib):
    import torch
    p = mmq.rope_plan(64, device="cpu")
    x, pos = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    table, start, length = (torch.zeros(s, dtype=torch.int32) for s in ((1, 4), (2,), (1,)))
    pages, w = mmq.kv_pages(4, 2, 64, device="cpu"), mmq.kv_weights(4, 2, device="cpu")
    assert w.shape == (4, 2, 64) and w.dtype == torch.float32
    for call in (lambda: mmq.rope(x, pos, p), lambda: mmq.kv_write_rope(x, x, x, pos, p, pages, table, start, length),
                 lambda: mmq.kv_attend_weights(x, w, pages, table, start, length, 3),
                 lambda: mmq.kv_evict(w, pages, table, start, length, table, 8)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="scaling"):
        mmq.rope_plan(64, scaling="other", device="cpu")
    with pytest.raises(ValueError, match="freq"):
        mmq.rope_plan(64, freq=[1.0], device="cpu")
    assert mmq.rope_plan(4, freq=[0.5, 0.25], magnitude=2.0, device="cpu").magnitude == 2.0


def test_helpers_check_shapes_types_and_devices(mmq_lib, monkeypatch):
    """Host memory that claims to be on a device, and no library behind it."""
    import torch

    class OnZero(torch.Tensor):
        def get_device(self):
            return 0

    class OnOne(torch.Tensor):
        def get_device(self):
            return 1

    def at(*shape, dtype=torch.int32, cls=OnZero):
        return torch.zeros(*shape, dtype=dtype).as_subclass(cls)

    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    p = mmq.rope_plan(64, device="cpu")
    p.held = p.held.as_subclass(OnZero)
    far = mmq.rope_plan(64, device="cpu")
    far.held = far.held.as_subclass(OnOne)
    monkeypatch.setattr(mmq, "_lib", Library())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    x = at(3, 2, 64, dtype=torch.float32)
    pos = at(3)
    cache = at(4, 2, 72 * 64, dtype=torch.uint8), at(1, 4), at(2), at(1)
    w, ws = at(4, 2, 64, dtype=torch.float32), at(4096, dtype=torch.uint8)
    new, kept = at(1, 1), at(1, 2, 8)

    def weigh(**kw):
        a = dict(q=x, weights=w, out=x, workspace=ws)
        a.update(kw)
        return mmq.kv_attend_weights(a.pop("q"), a.pop("weights"), *cache, 3, **a)

    def evict(**kw):
        a = dict(weights=w, new_table=new, keep=8, first=1, last=2, new_length=at(1), kept=kept)
        a.update(kw)
        return mmq.kv_evict(a.pop("weights"), *cache, a.pop("new_table"), a.pop("keep"), **a)

    mmq.rope(x, pos, p, out=x)
    mmq.kv_write_rope(x, x, x, pos, p, *cache, out=x)
    weigh()
    evict()
    assert [c for c in calls if not c.endswith("bytes")] == ["mmq_rope", "mmq_kv_write_rope", "mmq_kv_attend_weights",
                                                             "mmq_kv_evict"]
    calls.clear()
    one = at(3, 2, 64, dtype=torch.float32, cls=OnOne)
    for what, call in (
            ("pos", lambda: mmq.rope(x, pos.long(), p, out=x)), ("pos", lambda: mmq.rope(x, at(4), p, out=x)),
            ("pos", lambda: mmq.rope(x, at(3, cls=OnOne), p, out=x)), ("plan", lambda: mmq.rope(x, pos, far, out=x)),
            ("current device", lambda: mmq.rope(one, pos, p, out=x)), ("out", lambda: mmq.rope(x, pos, p, out=one)),
            ("x must", lambda: mmq.rope(x[0], pos, p)), ("out", lambda: mmq.rope(x, pos, p, out=x[:2])),
            ("pos", lambda: mmq.kv_write_rope(x, x, x, at(6)[::2], p, *cache, out=x)),
            ("k must", lambda: mmq.kv_write_rope(x, x[:, :1], x, pos, p, *cache, out=x)),
            ("q must", lambda: mmq.kv_write_rope(x[0], x, x, pos, p, *cache, out=x)),
            ("weights", lambda: weigh(weights=w.double())), ("weights", lambda: weigh(weights=w[:3])),
            ("into", lambda: weigh(into=at(4, 2, 64, dtype=torch.float32, cls=OnOne))), ("q must", lambda: weigh(q=x[0])),
            ("workspace", lambda: weigh(workspace=ws[:8])), ("out", lambda: weigh(out=x[:2])),
            ("weights", lambda: evict(weights=w[:, :1])), ("new_table", lambda: evict(new_table=at(2, 1))),
            ("new_table", lambda: evict(new_table=new.long())), ("new_table", lambda: evict(new_table=at(1, 1, cls=OnOne))),
            ("keep", lambda: evict(keep=65)), ("keep", lambda: evict(keep=0)), ("first", lambda: evict(first=-1)),
            ("keep", lambda: evict(first=8)), ("last", lambda: evict(last=1 << 40)), ("new_length", lambda: evict(new_length=at(2))),
            ("kept", lambda: evict(kept=kept[..., :4]))):
        if what == "workspace":
            monkeypatch.setattr(mmq, "mmq_kv_attend_weights_workspace_bytes", lambda *a: 64)
        with pytest.raises(ValueError, match=what):
            call()
    assert [c for c in calls if not c.endswith("bytes")] == []


def test_numbers_past_32_bits_are_not_cut(mmq_lib):
    for rot in (2 ** 32 + 64, 2 ** 40, -2 ** 40):
        with pytest.raises(mmq.MMQError):
            mmq.mmq_rope_frequencies("none", rot)


def test_every_cta_waits_for_the_kernel_before_it(mmq_lib):
    """Kernels of the cache start while the one ahead of them runs, and what that one wrote is only visible to a CTA
    that has waited itself: the wait stands in no branch, and nothing that may have been written is touched before it."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(mmq.__file__), "csrc")
    seen = []
    for path in sorted(glob.glob(os.path.join(csrc, "kv_*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for found in re.finditer(r"__global__[^{;]*?(kv_\w+_kernel|rope_kernel)\(", text):
            body = text[text.index("{", found.end()) + 1:]
            depth, flat = 1, ""                                         # inner blocks as empty statements
            for c in body:
                depth += (c == "{") - (c == "}")
                if depth == 0:
                    break
                flat += ";" if c == "}" else c if depth == 1 else ""
            seen.append(found[1])
            assert "grid_dep_wait();" in flat, (path, found[1])
            before = flat[:flat.index("grid_dep_wait();")]
            for memory in (r"c\.(start|length|table|pages)\[", r"\bstats\[", r"kv_sequence_of", r"unit_of", r"\.data\)"):
                assert not re.search(memory, before), (path, found[1], memory)
            assert not re.search(r"\b(if|else|for|while)\b[^;]*$", before.rstrip()), (path, found[1])
    assert len(seen) == 13 and "kv_weigh_rows_kernel" in seen


def test_slots_without_new_tokens_need_no_operands(mmq_lib):
    """Rows as operands: a tile of 128 of them more for each sequence that has any, not for each slot of the batch."""
    def need(batch, ntok=2048, dtype=0):
        c = cache(kv_heads=32, batch=batch, max_pages=64)
        return (mmq.mmq_kv_attend_weights_workspace_bytes(c, dtype, 32, ntok, 2048, 4096)
                - mmq.mmq_kv_attend_workspace_bytes(c, dtype, 32, ntok, 2048, 4096))
    for dtype, tile in ((0, 2 * 128 * 128 * 2 + 128 * 4), (1, 128 * 128 * 2 + 128 * 4)):
        for ntok in (2048, 200, 300):
            stats = ntok * 32 * 8
            for batch in (1, 16, 1024, 1 << 20):
                assert need(batch, ntok, dtype) <= stats + (ntok // 128 + min(batch, ntok) + 1) * 32 * tile
        assert need(1 << 20, 2048, dtype) == need(2048, 2048, dtype)


def test_numbers_far_below_zero_stay_below(mmq_lib, monkeypatch):
    """Their low 32 bits may be none, but they are not taken for 0: the library is given negative ones, which it
    refuses."""
    import torch

    class OnZero(torch.Tensor):
        def get_device(self):
            return 0

    def at(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnZero)

    calls = {}

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.update({name: a}) or 0

    monkeypatch.setattr(mmq, "_lib", Library())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    q, kv = at(3, 2, 64, dtype=torch.float32), (at(4, 2, 72 * 64, dtype=torch.uint8), at(1, 4), at(2), at(1))
    w, ws = at(4, 2, 64, dtype=torch.float32), at(1 << 16, dtype=torch.uint8)
    place = dict(max_q=5, max_kv=6, window=8, sinks=9)
    for name, i in place.items():
        for more in ({}, {"max_kv": 1 << 40}, {"max_q": 1 << 40}):
            args = {**dict(max_q=3, max_kv=64, window=0, sinks=0), **more, name: -(1 << 40)}
            mmq.kv_attend(q, *kv, out=q, workspace=ws, **args)
            mmq.kv_attend_weights(q, w, *kv, out=q, workspace=ws, **args)
            for call in ("mmq_kv_attend", "mmq_kv_attend_weights"):
                assert -(1 << 31) <= calls[call][i] < 0, (call, args)
                assert all(calls[call][k] < 1 << 31 for k in place.values())
            assert -(1 << 31) <= calls["mmq_kv_attend_weights_workspace_bytes"][{5: 4, 6: 5, 8: 6, 9: 7}[i]] < 0
    mmq.kv_evict(w, *kv, at(1, 1), 8, 1, 2, max_kv=-(1 << 40), new_length=at(1), kept=at(1, 2, 8))
    assert -(1 << 31) <= calls["mmq_kv_evict"][7] < 0


def test_sizes_past_64_bits_are_not_small_ones(mmq_lib):
    """Scores of the largest batch that the checks let through are no room for a few."""
    for heads in (1020, 1021, 1023, 1024):
        for q in (1, 3, 4, 16, 32):
            c = cache(kv_heads=heads, batch=1 << 20, max_pages=1 << 24)
            size = mmq.mmq_kv_attend_weights_workspace_bytes(c, 0, heads, q, q, (1 << 31) - 1)
            few = mmq.mmq_kv_attend_workspace_bytes(c, 0, heads, q, q, (1 << 31) - 1) + q * heads * 8 + 16
            assert size <= few, (heads, q)                              # the keys are read again


def test_operands_take_the_room_of_their_rows(mmq_lib):
    """Rows, up to 7 more for each sequence, and 128: a long prompt in a batch of many slots is not a tile of 128 a slot."""
    for dtype, row in ((0, 2 * 128 * 2 + 4), (1, 128 * 2 + 4)):
        for heads in (8, 32):
            for ntok in (200, 2048, 4000):
                for batch in (1, 16, 1024, 1 << 20):
                    c = cache(kv_heads=8, batch=batch, max_pages=64)
                    size = (mmq.mmq_kv_attend_weights_workspace_bytes(c, dtype, heads, ntok, ntok, 4096)
                            - mmq.mmq_kv_attend_workspace_bytes(c, dtype, heads, ntok, ntok, 4096))
                    rows = ntok * heads // 8
                    assert 8 * rows * row <= size <= ntok * heads * 8 + 8 * row * (rows + 8 * min(batch, ntok) + 128)


def test_rows_of_sequences_do_not_meet():
    """first_row of kv_weigh.cu: from the first row of a sequence on there is room for all of its rows before the next
    one's, and for 128 past the last, whatever sequences without rows lie between."""
    import random
    rng = random.Random(1)
    for _ in range(2000):
        group, batch = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 129]), rng.randint(1, 40)
        new = [rng.choice([0, 0, 1, 1, 2, 7, 8, 9, 127, 128, 300]) for _ in range(batch)]
        ntok = sum(new) + rng.choice([0, 0, 5])
        start, end = rng.choice([0, ntok - sum(new)]), 0
        for b, n in enumerate(new):
            if n:
                at = (start * group // 8 + min(b, start)) * 8
                assert at >= end
                end = at + n * group
            start += n
        assert end + 127 <= (ntok * group // 8 + min(batch, ntok)) * 8 + 128
