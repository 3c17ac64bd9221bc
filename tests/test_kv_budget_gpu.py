"""Rotary positions, attention with the weight each key receives, and eviction, on the GPU, against the
definitions of tests/budget_reference.py in 64 bits.

A turned value is off by its cosine's and sine's rounding, its products' and its sum's (each 2^-24
relative, and 2^-24 twice more where a magnitude other than 1 is rounded and multiplied), 2^-33 of the
values for the angle, and the rounding to the rows' type.  A weight: a score's error is at most 2^-20 (S + 1)
as in the attention's tests, it moves a row's softmax by at most twice that, and a sum of n terms adds
n 2^-24 of itself.  What is moved is exact.
"""
import math

import numpy as np
import pytest
import torch

import quant_int8_mmq_gb300 as mmq
from tests import budget_reference as ref
from tests.test_kv_gpu import BF16, DEV, F16, F32, HALF_ULP, Batch, hard_rows, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(mmq_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.synchronize()
    mmq.mmq_get_device_error()
    yield


def rand(*shape, dtype=F32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def turns_of(plan):
    return [int(t) % (1 << 64) for t in plan.held.cpu().tolist()]


def check_turned(x, out, pos, plan):
    rot, m = plan.rot_dim, plan.magnitude
    want, size = ref.turn(x.double(), ref.angles(turns_of(plan), pos.tolist()), rot, bool(plan.interleaved), m)
    far = x.double().abs().amax(-1, keepdim=True) * 2.0 ** -32 * max(abs(m), 1)
    tiny = 2.0 ** -25 if x.dtype == F16 else 2.0 ** -130
    tol = (2 if m == 1 else 4) * 2.0 ** -24 * 1.01 * size + (2.0 ** -24 + HALF_ULP[x.dtype] * (x.dtype != F32)) * want.abs() \
        + far + tiny
    err = (out.double() - want).abs()
    assert out.dtype == x.dtype and out.shape == x.shape
    assert (err <= tol).all(), (err / tol).max().item()
    assert torch.equal(out[..., rot:], x[..., rot:])


# ------------------------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot,heads", [(128, 128, 5), (64, 64, 1), (80, 32, 3), (128, 34, 2), (96, 96, 7), (130, 66, 1),
                                           (6, 2, 4), (256, 250, 1), (1024, 1024, 2), (66, 64, 33), (7, 4, 3)])
def test_rows_turn(dtype, interleaved, dim, rot, heads):
    plan = mmq.rope_plan(rot, interleaved=interleaved)
    for n in (1, 37):
        x = rand(n, heads, dim, dtype=dtype, seed=n)
        pos = torch.randint(0, 200000, (n,), dtype=torch.int32, generator=torch.Generator().manual_seed(3)).to(DEV)
        pos[0] = 0
        check_turned(x, mmq.rope(x, pos, plan), pos, plan)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn", "bands"])
def test_scalings_turn_by_their_frequencies(scaling):
    plan = mmq.rope_plan(64, 5e5, scaling=scaling, factor=8.0, original=2048)
    freq, m = mmq.mmq_rope_frequencies(scaling, 64, 5e5, 8.0, 2048)
    assert abs(plan.magnitude - m) == 0
    pos = torch.tensor([1, 77, 5000, 16383], dtype=torch.int32, device=DEV)
    x = rand(4, 2, 64)
    out = mmq.rope(x, pos, plan)
    check_turned(x, out, pos, plan)
    angle = np.outer(pos.cpu().numpy().astype(np.float64), freq)
    want, _ = ref.turn(x.double(), angle, 64, False, m)
    assert (out.double() - want).abs().max() < 4e-6


def test_positions_of_any_size_and_sign():
    for interleaved in (False, True):
        plan = mmq.rope_plan(128, interleaved=interleaved, freq=[2.0 * 0.87 ** i for i in range(64)], magnitude=0.7)
        pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 1 << 20, -65537], dtype=torch.int32, device=DEV)
        x = rand(8, 3, 128)
        check_turned(x, mmq.rope(x, pos, plan), pos, plan)


def test_cosine_and_sine_are_the_nearest_but_for_few():
    """x = (1, 0) gives them.  Off by 2^-33 before the rounding, so another f32 number comes out where the true
    one is within that of the middle of two: 2^-8 of numbers in [1/2, 1), 2^-7 in [1/4, 1/2) and so on; the
    numbers of uniform angles lie there with 2/3, 1/6, 1/12, ..., which makes 2/3 2^-8 + 1/6 2^-7 + ... with k
    terms of about 2^-8 / 3 each; counted to 2^-12, under 2^-8 (2/3 + 12/3) = 1.9 %."""
    n = 1 << 15
    plan = mmq.rope_plan(128)
    x = torch.zeros(n, 1, 128, device=DEV)
    x[..., :64] = 1.0
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (n,), dtype=torch.int32, device=DEV)
    out = mmq.rope(x, pos, plan)
    phase = pos.long()[:, None] * plan.held[None]                      # wraps as the definition does
    angle = phase.double() * (2 * math.pi / 2.0 ** 64)
    for got, want in ((out[:, 0, :64], angle.cos()), (out[:, 0, 64:], angle.sin())):
        assert ((got.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -33).all()
        assert (got != want.float()).float().mean() < 0.019


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("shift", [0, 1, 4, 8])
def test_rows_of_any_stride_and_in_place(dtype, shift):
    for interleaved in (False, True):
        plan = mmq.rope_plan(48, interleaved=interleaved)
        wide = rand(19, 500 + shift, dtype=dtype)
        x = wide[:, shift:shift + 192].view(19, 3, 64)
        pos = torch.arange(19, dtype=torch.int32, device=DEV) * 1000
        want = mmq.rope(x.contiguous(), pos, plan)
        check_turned(x, want, pos, plan)
        outer = torch.full((3, 19, 64 + shift), 9.0, device=DEV, dtype=dtype)
        out = outer[..., :64].transpose(0, 1)
        assert mmq.rope(x, pos, plan, out=out) is out
        assert torch.equal(out, want) and (outer[..., 64:] == 9.0).all()
        before = wide.clone()
        mmq.rope(x, pos, plan, out=x)
        assert torch.equal(x, want)
        wide[:, shift:shift + 192] = before[:, shift:shift + 192]
        assert torch.equal(wide, before)
        one = rand(1, 1, 64, dtype=dtype).expand(19, 3, 64)            # the same row everywhere
        check_turned(one, mmq.rope(one, pos, plan), pos, plan)


def test_no_number_touches_its_pair_alone():
    for interleaved in (False, True):
        plan = mmq.rope_plan(32, interleaved=interleaved)
        x, pos = rand(5, 2, 64), torch.arange(5, dtype=torch.int32, device=DEV)
        want = mmq.rope(x, pos, plan)
        x[3, 1, 4], x[4, 0, 60] = float("nan"), float("inf")
        got = mmq.rope(x, pos, plan)
        bad = torch.zeros_like(x, dtype=torch.bool)
        bad[3, 1, [4, 5] if interleaved else [4, 20]] = True
        assert got[bad].isnan().all() and got[4, 0, 60] == float("inf")
        bad[4, 0, 60] = True
        assert torch.equal(got[~bad], want[~bad])


def test_rope_on_a_stream_in_a_graph_and_empty():
    plan = mmq.rope_plan(64)
    x, pos = rand(6, 4, 64), torch.arange(6, dtype=torch.int32, device=DEV)
    want = mmq.rope(x, pos, plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mmq.rope(x, pos, plan, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mmq.rope(x, pos, plan, out=out)
        mmq.rope(out, pos, plan, out=out)
    for _ in range(2):
        x.copy_(rand(6, 4, 64, seed=5))
        graph.replay()
    assert torch.equal(out, mmq.rope(mmq.rope(x, pos, plan), pos, plan))
    assert mmq.rope(x[:0], pos[:0], plan).shape == (0, 4, 64)


# ------------------------------------------------------------------------------------ into the cache
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (128, 64, False), (128, 34, False), (128, 128, True),
                                                 (64, 64, False), (64, 64, True), (64, 16, False), (64, 6, True),
                                                 (64, 50, False)])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (5, 5), (3, 1)])
def test_writing_turned_rows_is_turning_and_writing(dtype, dim, rot, interleaved, heads, kv_heads):
    """Byte for byte: a turned key is quantised as it is in f32."""
    plan = mmq.rope_plan(rot, interleaved=interleaved, scaling="yarn", factor=4.0, original=1000)
    b = Batch([1, 7, 0, 70], [1, 70, 5, 131], kv_heads, dim, dtype, fill=False)
    other = b.pages.clone()
    q, k, v = (rand(b.rows, h, dim, dtype=dtype, seed=s) for s, h in ((1, heads), (2, kv_heads), (3, kv_heads)))
    pos = torch.randint(0, 100000, (b.rows,), dtype=torch.int32, device=DEV)
    out = mmq.kv_write_rope(q, k, v, pos, plan, *b.cache)
    mmq.kv_write(mmq.rope(k.float(), pos, plan), v.float(), other, *b.cache[1:])
    assert status() == 0
    assert torch.equal(b.pages, other)
    assert torch.equal(out, mmq.rope(q, pos, plan))
    b.pages.fill_(0xFF)
    mmq.kv_write_rope(q, k, v, pos, plan, *b.cache, out=q)
    assert torch.equal(b.pages, other) and torch.equal(q, out)


@pytest.mark.parametrize("rows", [1, 2431, 4863, 9731])
@pytest.mark.parametrize("interleaved,rot", [(False, 64), (True, 64), (False, 20)])
def test_many_tokens_enter(rows, interleaved, rot):
    """Every number of tokens a CTA takes, the last CTA not full."""
    plan = mmq.rope_plan(rot, interleaved=interleaved)
    b = Batch([rows // 3, rows - rows // 3], [rows // 3 + 10, rows], 1, 64, fill=False)
    other = b.pages.clone()
    q, k, v = (rand(rows, h, 64, seed=s) for s, h in ((1, 3), (2, 1), (3, 1)))
    pos = torch.arange(rows, dtype=torch.int32, device=DEV)
    out = mmq.kv_write_rope(q, k, v, pos, plan, *b.cache)
    mmq.kv_write(mmq.rope(k, pos, plan), v, other, *b.cache[1:])
    assert status() == 0 and torch.equal(b.pages, other) and torch.equal(out, mmq.rope(q, pos, plan))


@pytest.mark.parametrize("rows", [205, 403, 811])
@pytest.mark.parametrize("kv_heads,dim", [(1, 64), (3, 128)])
def test_some_tokens_enter(rows, kv_heads, dim):
    """Two, four and eight tokens a CTA, the last one not full, queries of other CTAs."""
    plan = mmq.rope_plan(dim)
    b = Batch([rows // 3, rows - rows // 3], [rows // 3 + 10, rows], kv_heads, dim, F16, fill=False)
    other = b.pages.clone()
    q, k, v = (rand(rows, h, dim, dtype=F16, seed=s) for s, h in ((1, 3), (2, kv_heads), (3, kv_heads)))
    pos = torch.arange(rows, dtype=torch.int32, device=DEV)
    out = mmq.kv_write_rope(q, k, v, pos, plan, *b.cache)
    mmq.kv_write(mmq.rope(k.float(), pos, plan), v.float(), other, *b.cache[1:])
    assert status() == 0 and torch.equal(b.pages, other) and torch.equal(out, mmq.rope(q, pos, plan))


def test_rows_of_any_stride_enter_and_those_without_a_place_turn():
    plan = mmq.rope_plan(128)
    b = Batch([3, 70], [2, 70], 2, 128, max_pages=2, fill=False)         # the first row is before its sequence
    wide = rand(73, 1001)
    q, k, v = (wide[:, 1 + 128 * i:1 + 128 * (i + h)].view(73, h, 128) for i, h in ((0, 3), (3, 2), (5, 2)))
    pos = torch.arange(73, dtype=torch.int32, device=DEV)
    other = b.pages.clone()
    out = mmq.kv_write_rope(q, k, v, pos, plan, *b.cache)
    assert status() == 1 and status() == 0
    mmq.kv_write(mmq.rope(k, pos, plan), v, other, *b.cache[1:])
    assert status() == 1
    assert torch.equal(b.pages, other) and torch.equal(out, mmq.rope(q, pos, plan))
    table = b.table.clone()
    table[1, 1] = b.pages.shape[0]
    mmq.kv_write_rope(q, k, v, pos, plan, b.pages, table, b.start, b.length)
    assert status() == 1 and torch.equal(b.pages, other)


# ------------------------------------------------------------------------------------ weights
def weights_for(b, seed=7):
    return torch.rand(b.pages.shape[0], b.hk, 64, generator=torch.Generator().manual_seed(seed)).to(DEV)


def check_weights(b, q, before, after, scale=None, window=0, sinks=0, decay=1.0, max_q=None):
    scale = b.dim ** -0.5 if scale is None else scale
    want, tol = before.double(), torch.zeros_like(before, dtype=torch.float64)
    lo = 0
    for s, (n, m) in enumerate(zip(b.new, b.len)):
        if n and m > 0:
            k, _ = held_of(b, s)
            got, bound = torch.zeros(b.hk, m, device=DEV, dtype=torch.float64), torch.zeros(b.hk, m, device=DEV, dtype=torch.float64)
            counted = min(n, max_q or n)
            for i in range(0, counted, 256):
                c = min(256, counted - i)
                pos = torch.arange(m - n + i, m - n + i + c, device=DEV)
                g, e = ref.received(q[lo + i:lo + i + c].double(), k, pos, scale, window, sinks)
                got += g
                bound += e
            j = torch.arange(m, device=DEV)
            page = b.table[s, j // 64].long()
            old = torch.where(j < m - n, before[page, :, j % 64].double().T * decay, 0.0)
            terms = n * q.shape[1] // b.hk + 2
            want[page, :, j % 64] = (old + got).T
            tol[page, :, j % 64] = (2.0 ** -19 * bound + terms * 2.0 ** -24 * (got + old) + 2.0 ** -126).T
        lo += n
    err = (after.double() - want).abs()
    assert (err <= tol).all(), ((err / tol.clamp(min=1e-300)).max().item(), err.max().item())


def held_of(b, s):
    from tests import kv_reference
    return tuple(torch.from_numpy(kv_reference.values(x[s].double().cpu().numpy())).to(DEV) for x in (b.k, b.v))


def weigh_and_check(b, heads, seed=1, factor=1.5, **kw):
    q = b.q(heads, seed, factor)
    before = weights_for(b)
    mine = before.clone()
    out, into = mmq.kv_attend_weights(q, mine, *b.cache, max_q=max(b.new), **kw)
    assert into is mine and status() == 0
    decay = kw.pop("decay", 1.0)
    assert torch.equal(out, mmq.kv_attend(q, *b.cache, max_q=max(b.new), **kw))
    kw.pop("max_kv", None)
    check_weights(b, q, before, mine, decay=decay, **kw)
    return q, before, mine


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 8, 2), (64, 4, 4), (128, 5, 1), (64, 48, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (100, 3), (64, 65)])
def test_keys_receive_their_weight(dtype, dim, heads, kv_heads, window, sinks):
    b = Batch([1, 3, 0, 70, 5], [1, 200, 64, 70, 777], kv_heads, dim, dtype)
    weigh_and_check(b, heads, window=window, sinks=sinks, decay=0.75)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("new,length", [(1, 64), (1, 65), (1, 63), (2, 2), (64, 64), (65, 65), (33, 97), (300, 300), (129, 1000)])
def test_sequences_of_every_length(dtype, new, length):
    weigh_and_check(Batch([new], [length], 2, 128, dtype), 6)


def test_a_whole_prompt_and_a_long_cache():
    weigh_and_check(Batch([1500], [1500], 2, 64, F16), 4)
    weigh_and_check(Batch([1, 1], [30001, 7], 2, 128, F32), 8, decay=0.5)
    weigh_and_check(Batch([700, 1], [2000, 900], 1, 128, BF16), 3, window=300, sinks=5)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim,window,sinks", [(64, 0, 0), (128, 0, 0), (64, 200, 3), (128, 130, 70)])
def test_more_scores_than_are_kept(dtype, dim, window, sinks):
    """A table so wide that scores for all of it would be over a gigabyte: the keys are read again."""
    lens = [1, 64, 129, 300, 5, 1000, 128, 2500]
    b = Batch([1, 2, 1, 2, 1, 1, 1, 2], lens, 2, dim, dtype, max_pages=(1 << 30) // (256 * 8 * 2 * 8) + 1)
    weigh_and_check(b, 8, window=window, sinks=sinks, decay=0.5)
    q = b.q(8)
    w = [weights_for(b) for _ in range(2)]
    for x, most in zip(w, (2500, None)):                                # kept, and not
        mmq.kv_attend_weights(q, x, *b.cache, 2, most, window=window, sinks=sinks)
    assert not torch.equal(*w) and (w[0] - w[1]).abs().max() < 1e-4


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hint", [1, 100, 130])
def test_a_length_hint_that_is_too_low(dtype, dim, hint):
    b = Batch([1, 2, 3], [200, 700, 90], 2, dim, dtype)
    weigh_and_check(b, 6, max_kv=hint, decay=0.5)
    weigh_and_check(b, 6, max_kv=hint, window=100, sinks=2)
    weigh_and_check(Batch([40, 90], [300, 700], 2, dim, dtype), 4, max_kv=hint)
    weigh_and_check(Batch([400], [900], 1, dim, dtype), 4, max_kv=hint)


def test_every_row_gives_one_and_heads_add_up():
    b = Batch([9], [500], 2, 64)
    w = weights_for(b).zero_()
    mmq.kv_attend_weights(b.q(6), w, *b.cache, 9)
    # 9 rows of 3 heads a kv head; a sum of 500 numbers that are each within 2^-18 of theirs
    assert (w.sum((0, 2)) - 27).abs().max() < 27 * 2.0 ** -17


@pytest.mark.parametrize("dtype", [F32, F16])
def test_steps_add_up_and_may_be_taken_back(dtype):
    b = Batch([2], [150], 1, 64, dtype)
    q, before = b.q(4), weights_for(b)
    into = torch.full_like(before, 5.0)
    out, got = mmq.kv_attend_weights(q, before, *b.cache, 2, decay=0.5, into=into)
    assert got is into
    check = before.clone()
    mmq.kv_attend_weights(q, check, *b.cache, 2, decay=0.5)
    j = torch.arange(150, device=DEV)
    page = b.table[0, j // 64].long()
    assert torch.equal(into[page, :, j % 64], check[page, :, j % 64])
    untouched = torch.ones_like(into, dtype=torch.bool)
    untouched[page, :, j % 64] = False
    assert (into[untouched] == 5.0).all() and torch.equal(check[untouched], before[untouched])
    # nothing of the old weights matters to tokens that are new, not even what is no number
    before[b.table[0, 2].long(), :, 148 % 64:150 % 64] = float("nan")
    mmq.kv_attend_weights(q, before, *b.cache, 2, decay=0.5)
    assert torch.equal(before[page, :, j % 64], check[page, :, j % 64])
    assert status() == 0


def test_rows_that_see_nothing_and_rows_without_a_number():
    b = Batch([5, 2], [3, 70], 1, 64)                                   # two rows before the sequence's first token
    w = weights_for(b)
    before = w.clone()
    q = b.q(2)
    mmq.kv_attend_weights(q, w, *b.cache, 5)
    j = torch.arange(3, device=DEV)
    page = b.table[0, 0].long()
    assert abs(w[page, 0, :3].sum().item() - 3 * 2) < 1e-4              # three rows of two heads, all keys new
    # a row that is no number: the others' weights as if it were not there
    for dtype in (F32, F16, BF16):
        for n in (3, 200):
            b = Batch([n], [300], 1, 128, dtype)
            q = b.q(2)
            w0 = weights_for(b)
            want = w0.clone()
            alone = q.clone()
            alone[1, 1] = 0.0
            mmq.kv_attend_weights(alone, want, *b.cache, n)
            zero = w0.clone()
            seen = 300 - n + 2                                          # the zero row gives 1 / seen to each
            q[1, 1, 3] = float("nan")
            mmq.kv_attend_weights(q, zero, *b.cache, n)
            j = torch.arange(300, device=DEV)
            page = b.table[0, j // 64].long()
            diff = want[page, 0, j % 64] - zero[page, 0, j % 64]
            expect = torch.where(j < seen, 1.0 / seen, 0.0)
            assert zero[page, 0, j % 64].isfinite().all() and (diff - expect).abs().max() < 1e-4
    assert status() == 0


def test_rows_past_max_q_and_of_no_sequence_add_nothing():
    b = Batch([40], [400], 2, 128)
    q, before = b.q(2), weights_for(b)
    w = before.clone()
    mmq.kv_attend_weights(q, w, *b.cache, 8)                            # 8 rows a tile: the rest are left out
    assert status() == 1
    check_weights(b, q, before, w, max_q=8)
    b = Batch([3, 4], [100, 200], 2, 64)
    q, before = b.q(4), weights_for(b)
    w = before.clone()
    start = torch.tensor([0, 3, 9], dtype=torch.int32, device=DEV)      # past the rows
    mmq.kv_attend_weights(q, w, b.pages, b.table, start, b.length, 6)
    assert status() == 1
    two = b.table[1, :4].long()
    assert torch.equal(w[two], before[two]) and not torch.equal(w, before)


def test_pages_that_are_not_there_are_left_out():
    b = Batch([2], [300], 1, 128)
    bad = b.table.clone()
    bad[0, 1] = b.pages.shape[0] + 5
    w = weights_for(b)
    before = w.clone()
    mmq.kv_attend_weights(b.q(2), w, b.pages, bad, b.start, b.length, 2)
    assert status() == 1
    gone = b.table[0, 1].long()
    assert torch.equal(w[gone], before[gone])
    rest = b.table[0, [0, 2, 3, 4]].long()
    assert abs((w[rest] - before[rest])[:, 0, :].double().sum().item()) < 1e3 and w[rest].isfinite().all()
    assert not torch.equal(w[rest], before[rest])


def test_weights_do_not_vary_and_replay():
    b = Batch([1, 90, 2], [2000, 90, 700], 2, 128)
    q, before = b.q(8), weights_for(b)
    a, c = before.clone(), before.clone()
    mmq.kv_attend_weights(q, a, *b.cache, 90)
    mmq.kv_attend_weights(q, c, *b.cache, 90)
    assert torch.equal(a, c)
    static = before.clone()
    out = torch.empty_like(q)
    need = mmq.mmq_kv_attend_weights_workspace_bytes(mmq._kv_cache(*b.cache)[0], 0, 8, b.rows, 90, b.max_pages * 64)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]                 # two graphs that share a workspace
    for graph in graphs:
        with torch.cuda.graph(graph):
            mmq.kv_attend_weights(q, static, *b.cache, 90, decay=0.5, out=out, workspace=ws)
    static.copy_(before)
    for graph in graphs:
        graph.replay()
    want = before.clone()
    for _ in range(2):
        mmq.kv_attend_weights(q, want, *b.cache, 90, decay=0.5)
    assert torch.equal(static, want) and status() == 0


# ------------------------------------------------------------------------------------ eviction
def evict_and_check(b, w, keep, first, last, bytes_too=True, **kw):
    """Pages for the new tables come from a pool that is grown for them."""
    n = -(-keep // 64)
    num = b.pages.shape[0]
    pages = torch.cat([b.pages, torch.full((n * len(b.len) + 1, b.hk, 72 * b.dim), 0xAB, dtype=torch.uint8, device=DEV)])
    weights = torch.cat([w, torch.full((n * len(b.len) + 1, b.hk, 64), -5.0, device=DEV)])
    perm = torch.randperm(n * len(b.len), generator=torch.Generator().manual_seed(3)).to(torch.int32) + num
    table = perm.view(len(b.len), n).to(DEV)
    p0, w0 = pages.cpu().numpy().copy(), weights.cpu().numpy().copy()
    length, kept = mmq.kv_evict(weights, pages, b.table, b.start, b.length, table, keep, first, last, **kw)
    assert status() == 0
    got_p, got_w, got_l, got_k = (x.cpu().numpy() for x in (pages, weights, length, kept))
    old_t, new_t = b.table.cpu().numpy(), table.cpu().numpy()
    want_p, want_w = p0.copy(), w0.copy()
    for s, m in enumerate(b.len):
        assert got_l[s] == min(m, keep)
        for h in range(b.hk):
            j = np.arange(m)
            stays = ref.stays(w0[old_t[s, j // 64], h, j % 64], keep, first, last)
            assert got_k[s, h, :len(stays)].tolist() == stays and (got_k[s, h, len(stays):] == -1).all()
            for i, o in enumerate(stays):
                want_w[new_t[s, i // 64], h, i % 64] = w0[old_t[s, o // 64], h, o % 64]
                if bytes_too:
                    ref.move(p0[old_t[s, o // 64], h], want_p[new_t[s, i // 64], h], i % 64, o % 64, b.dim)
    assert np.array_equal(got_w, want_w, equal_nan=True)
    if bytes_too:
        assert np.array_equal(got_p, want_p)
    return pages, weights, table, length, kept


@pytest.mark.parametrize("dim,kv_heads", [(64, 1), (128, 2), (64, 3)])
@pytest.mark.parametrize("keep,first,last", [(64, 4, 16), (65, 0, 0), (1, 0, 0), (1, 1, 0), (100, 0, 100), (100, 60, 40),
                                             (130, 1, 65), (63, 63, 0), (200, 4, 64)])
def test_what_stays_moves(dim, kv_heads, keep, first, last):
    b = Batch([1, 1, 0, 1], [199, 64, 0, 131], kv_heads, dim)
    evict_and_check(b, weights_for(b), keep, first, last)


@pytest.mark.parametrize("kind", ["equal", "zero", "signed", "odd", "two", "bits"])
@pytest.mark.parametrize("keep,first,last", [(100, 4, 16), (333, 0, 1), (64, 0, 0)])
def test_ties_and_weights_of_any_kind(kind, keep, first, last):
    b = Batch([1, 1], [1000, 401], 2, 64, fill=False)
    w = weights_for(b)
    g = torch.Generator().manual_seed(9)
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "zero":
        w.copy_(torch.where(torch.rand(w.shape, generator=g) < 0.5, 0.0, -0.0))
    elif kind == "signed":
        w.copy_(torch.randn(w.shape, generator=g) * 10.0 ** torch.randint(-44, 38, w.shape, generator=g))
    elif kind == "odd":
        odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, 3e38, -1.0])
        w.copy_(odd[torch.randint(0, 8, w.shape, generator=g)])
    elif kind == "two":
        w.copy_((torch.rand(w.shape, generator=g) < 0.2).float())
    else:           # neighbours that differ in the last bits
        w.copy_((torch.randint(0, 50, w.shape, generator=g) + (1 << 29)).to(torch.int32).view(torch.float32))
    evict_and_check(b, w, keep, first, last, bytes_too=False)


@pytest.mark.parametrize("length,kv_heads,keep", [(20001, 1, 5000), (70000, 2, 333), (300001, 1, 200000), (5000, 40, 1)])
@pytest.mark.parametrize("hint", [None, 1])
def test_long_sequences_and_any_hint(length, kv_heads, keep, hint):
    """Clusters of every size; with a hint far too low, weights are read again from memory."""
    b = Batch([1], [length], kv_heads, 64, fill=False)
    w = weights_for(b)
    w[::3] = w[::3].round()                                              # many equal ones
    evict_and_check(b, w, keep, 65, min(100, keep - 65) if keep > 65 else 0, bytes_too=False, max_kv=hint) if keep > 65 else \
        evict_and_check(b, w, keep, 0, 0, bytes_too=False, max_kv=hint)


def test_a_batch_of_many_sequences():
    lens = [(i * 37) % 300 for i in range(200)]
    b = Batch([1] * 200, lens, 2, 64, fill=False)
    evict_and_check(b, weights_for(b), 77, 3, 20, bytes_too=False)


def test_the_new_length_may_be_the_old_one_and_pages_may_be_shared():
    b = Batch([1, 1], [300, 200], 1, 64)
    b.table[1, :3] = b.table[0, :3]                                      # a shared prefix
    w = weights_for(b)
    pages = torch.cat([b.pages, torch.zeros(4, 1, 72 * 64, dtype=torch.uint8, device=DEV)])
    weights = torch.cat([w, torch.zeros(4, 1, 64, device=DEV)])
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2) + b.pages.shape[0]
    first = mmq.kv_evict(weights.clone(), pages.clone(), b.table, b.start, b.length, table, 120, 4, 30)
    length = b.length.clone()
    got, kept = mmq.kv_evict(weights, pages, b.table, b.start, length, table, 120, 4, 30, new_length=length)
    assert got is length and length.tolist() == [120, 120] and torch.equal(kept, first[1])
    assert torch.equal(pages[:-4], b.pages) and torch.equal(weights[:-4], w) and status() == 0


def test_pages_that_are_not_there_when_tokens_move():
    b = Batch([1], [200], 1, 64)
    w = weights_for(b)
    pages = torch.cat([b.pages, torch.full((2, 1, 72 * 64), 0xCD, dtype=torch.uint8, device=DEV)])
    weights = torch.cat([w, torch.full((2, 1, 64), 9.0, device=DEV)])
    num = b.pages.shape[0]
    bad = b.table.clone()
    bad[0, 1] = -3
    table = torch.tensor([[num, num + 1]], dtype=torch.int32, device=DEV)
    _, kept = mmq.kv_evict(weights, pages, bad, b.start, b.length, table, 128, 70, 0)
    assert status() == 1 and status() == 0
    assert kept[0, 0, :70].tolist() == list(range(70))                   # the first ones stay, whatever they are
    assert (kept[0, 0, 70:] >= 128).all()
    assert (weights[num + 1, 0, :6] == 0).all() and (weights[num, 0] == w[b.table[0, 0].long(), 0]).all()
    k, v = mmq.kv_read(pages, table, torch.tensor([0, 128], dtype=torch.int32, device=DEV),
                       torch.tensor([128], dtype=torch.int32, device=DEV), 128, dtype=F32)
    assert (k[64:70] == 0).all() and (v[64:70] == 0).all()
    before = pages.clone(), weights.clone()
    table = torch.tensor([[num + 2, -1]], dtype=torch.int32, device=DEV)  # new pages that are none
    mmq.kv_evict(weights, pages, b.table, b.start, b.length, table, 128, 4, 0)
    assert status() == 1 and torch.equal(pages, before[0]) and torch.equal(weights, before[1])
    # lengths that the table has no pages for, or below zero
    for m, n in ((100000, 128), (-5, 0)):
        length = torch.tensor([m], dtype=torch.int32, device=DEV)
        got, _ = mmq.kv_evict(weights, pages, b.table, b.start, length, torch.tensor([[num, num + 1]], dtype=torch.int32,
                                                                                      device=DEV), 128, 4, 0)
        assert got.item() == n and status() == 1


def test_eviction_replays_in_a_graph():
    b = Batch([1], [500], 2, 64, fill=False)
    w = weights_for(b)
    pages = torch.cat([b.pages, torch.zeros(2, 2, 72 * 64, dtype=torch.uint8, device=DEV)])
    weights = torch.cat([w, torch.zeros(2, 2, 64, device=DEV)])
    table = torch.arange(2, dtype=torch.int32, device=DEV)[None] + b.pages.shape[0]
    length, kept = mmq.kv_evict(weights, pages, b.table, b.start, b.length, table, 128)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mmq.kv_evict(weights, pages, b.table, b.start, b.length, table, 128, new_length=length, kept=kept)
    weights[:-2] = torch.rand(w.shape, device=DEV)
    graph.replay()
    again = mmq.kv_evict(weights, pages, b.table, b.start, b.length, table, 128)
    assert torch.equal(kept, again[1]) and torch.equal(length, again[0]) and status() == 0


# ------------------------------------------------------------------------------------ all together
def test_a_conversation_within_a_budget():
    """A prompt and single tokens through rotation, cache, weighed attention and eviction, against 64 bits that
    keep their own list of (position, key, value, weight) per head."""
    heads, hk, dim, keep, first, last = 4, 2, 64, 100, 4, 20
    plan = mmq.rope_plan(32, scaling="bands", factor=4.0, original=64)
    pages, weights = mmq.kv_pages(12, hk, dim), mmq.kv_weights(12, hk)
    pages.fill_(0xFF)
    free = list(range(12))
    from tests import kv_reference
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)     # noqa: E731
    mine, length, far = [], 0, 0                                        # pages, slots in use, positions so far
    keys = [torch.zeros(0, dim, dtype=torch.float64, device=DEV) for _ in range(hk)]
    values, sums = [x.clone() for x in keys], [torch.zeros(0, dtype=torch.float64, device=DEV) for _ in range(hk)]
    for step, new in enumerate([130, 1, 1, 3, 1, 70, 1, 1]):
        if length > keep:
            table = ints([mine + [-1] * (8 - len(mine))])
            to = [free.pop() for _ in range(2)]
            got, kept = mmq.kv_evict(weights, pages, table, ints([0, 0]), ints([length]), ints([to]), keep, first, last)
            for h in range(hk):
                j = kept[0, h].long()
                # of weights nearer to each other than their errors either may stay: all that left are below
                # the least that stayed, to within them
                gone = torch.ones(length, dtype=torch.bool, device=DEV)
                gone[j] = False
                middle = sums[h][j][first:keep - last]
                assert j[:first].tolist() == list(range(first)) and j[-last:].tolist() == list(range(length - last, length))
                assert sums[h][gone].max() <= middle.min() * (1 + 1e-4)
                keys[h], values[h], sums[h] = keys[h][j], values[h][j], sums[h][j]
            free += mine
            mine, length = to, int(got)
        while len(mine) * 64 < length + new:
            mine.append(free.pop())
        length += new
        q, k, v = (rand(new, n, dim, seed=10 * step + i) for i, n in enumerate((heads, hk, hk)))
        pos = torch.arange(far, far + new, dtype=torch.int32, device=DEV)
        far += new
        cache = pages, ints([mine + [-1] * (8 - len(mine))]), ints([0, new]), ints([length])
        turned = mmq.kv_write_rope(q, k, v, pos, plan, *cache)
        out, _ = mmq.kv_attend_weights(turned, weights, *cache, max_q=new, decay=0.9)
        check_turned(q, turned, pos, plan)
        kt = mmq.rope(k, pos, plan)                                     # codes depend on its last bits
        for h in range(hk):
            keys[h] = torch.cat([keys[h], torch.from_numpy(kv_reference.values(kt[:, h].double().cpu().numpy())).to(DEV)])
            values[h] = torch.cat([values[h], torch.from_numpy(kv_reference.values(v[:, h].double().cpu().numpy())).to(DEV)])
            p = torch.arange(length - new, length, device=DEV)
            mineq = turned[:, 2 * h:2 * h + 2].double()
            want, S = kv_reference.attend(mineq, keys[h][:, None], values[h][:, None], p, dim ** -0.5)
            assert (out[:, 2 * h:2 * h + 2].double() - want).abs().max() < 2 ** -19 * (S.max() + 1) * values[h].abs().max() + 1e-6
            got, _ = ref.received(mineq, keys[h][:, None], p, dim ** -0.5)
            sums[h] = torch.cat([0.9 * sums[h], torch.zeros(new, dtype=torch.float64, device=DEV)]) + got[0]
            j = torch.arange(length, device=DEV)
            held = weights[cache[1][0, j // 64].long(), h, j % 64]
            assert (held.double() - sums[h]).abs().max() < 1e-4 * sums[h].max()
    assert status() == 0


# ------------------------------------------------------------------------------------ as programs use them
@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("new,lens,window,sinks,wide", [
    ([1, 2, 1], [5000, 90, 700], 0, 0, 0), ([1, 2, 1], [5000, 90, 700], 130, 70, 0), ([2, 1], [9000, 20000], 0, 0, 0),
    ([1, 2, 1, 1, 1, 1, 2, 1], [500, 90, 700, 1, 64, 65, 128, 40], 100, 0, 1), ([9, 20], [300, 1000], 200, 1, 0),
    ([150, 1, 70], [1000, 30, 70], 0, 0, 0), ([300, 40], [2000, 555], 333, 7, 0)])
def test_a_workspace_may_hold_anything(dtype, new, lens, window, sinks, wide):
    """Scores, statistics and operands of other calls, or no numbers, change nothing."""
    b = Batch(new, lens, 2, 128, dtype, max_pages=(1 << 30) // (256 * 8 * 2 * 8) + 1 if wide else None)
    q, most = b.q(8), b.max_pages * 64
    need = mmq.mmq_kv_attend_weights_workspace_bytes(mmq._kv_cache(*b.cache)[0], mmq.DTYPES[str(dtype)[6:]], 8, b.rows,
                                                     max(new), most, window, sinks)
    got = []
    for byte in (0, 0xFF, 0x43):                                        # 0x43434343 is 195.26
        w = weights_for(b)
        out, _ = mmq.kv_attend_weights(q, w, *b.cache, max(new), window=window, sinks=sinks,
                                       workspace=torch.full((need,), byte, dtype=torch.uint8, device=DEV))
        got.append((out, w))
    assert status() == 0
    for out, w in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(w, got[0][1])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (128, 64, False), (128, 34, False), (128, 128, True),
                                                 (64, 64, False), (64, 20, True)])
def test_keys_of_any_kind_enter_turned(dtype, dim, rot, interleaved):
    """Ties, zeros, huge, tiny and infinite values and no numbers, byte for byte as turning and writing."""
    plan = mmq.rope_plan(rot, interleaved=interleaved)
    b = Batch([120], [150], 2, dim, dtype, fill=False)
    k, v = (hard_rows(120, 2, dim, dtype, s).to(DEV) for s in (5, 6))
    pos = torch.randint(0, 5, (120,), dtype=torch.int32, device=DEV)    # many rows at 0, where ties stay ties
    q, other = rand(120, 3, dim, dtype=dtype), b.pages.clone()
    mmq.kv_write_rope(q, k, v, pos, plan, *b.cache)
    mmq.kv_write(mmq.rope(k.float(), pos, plan), v.float(), other, *b.cache[1:])
    assert status() == 0 and torch.equal(b.pages, other)


def turn_weigh_evict(b, q, k, v, pos, plan, table, w, keep, stream=None):
    turned = mmq.kv_write_rope(q, k, v, pos, plan, *b.cache, stream=stream)
    out, _ = mmq.kv_attend_weights(turned, w, *b.cache, max(b.new), decay=0.5, stream=stream)
    length, kept = mmq.kv_evict(w, b.pages, b.table, b.start, b.length, table, keep, stream=stream)
    return turned, out, length, kept


def budget_case(seed, new, lens, keep, heads, hk, dim, dtype):
    n = -(-keep // 64)
    b = Batch(new, lens, hk, dim, dtype, seed=seed, spare=n * len(lens) + 1)
    used = set(b.table.flatten().tolist())
    free = [i for i in range(b.pages.shape[0]) if i not in used][:n * len(lens)]
    table = torch.tensor(free, dtype=torch.int32, device=DEV).view(len(lens), n)
    q, k, v = (rand(b.rows, h, dim, dtype=dtype, seed=seed + i) for i, h in enumerate((heads, hk, hk)))
    pos = torch.randint(0, 5000, (b.rows,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).to(DEV)
    return b, q, k, v, pos, mmq.rope_plan(dim), table, weights_for(b), keep


def test_calls_on_two_streams_at_once():
    shapes = [(1, [1, 1, 2], [700, 3000, 90], 200, 8, 2, 128, F16), (2, [150, 40], [900, 4000], 300, 4, 2, 64, F32)]
    want = []
    for s in shapes:
        case = budget_case(*s)
        want.append((turn_weigh_evict(*case), case))
    torch.cuda.synchronize()
    cases, streams = [budget_case(*s) for s in shapes], [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    got = [turn_weigh_evict(*c, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    assert status() == 0
    for (w, wc), g, gc in zip(want, got, cases):
        for x, y in zip(w, g):
            assert torch.equal(x, y)
        assert torch.equal(wc[0].pages, gc[0].pages) and torch.equal(wc[7], gc[7])


def test_a_whole_step_replays():
    b, q, k, v, pos, plan, table, w, keep = budget_case(3, [1, 2, 1], [700, 300, 65], 128, 8, 2, 128, BF16)
    pages0, w0 = b.pages.clone(), w.clone()
    want = turn_weigh_evict(b, q, k, v, pos, plan, table, w, keep)
    pages1, w1 = b.pages.clone(), w.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = turn_weigh_evict(b, q, k, v, pos, plan, table, w, keep)
    for _ in range(2):
        b.pages.copy_(pages0)
        w.copy_(w0)
        graph.replay()
        assert torch.equal(b.pages, pages1) and torch.equal(w, w1)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert status() == 0


def test_pools_past_32_bits():
    """Page ids whose bytes are past 2^32, against the same tokens in a small pool."""
    b, q, k, v, pos, plan, table, w, keep = budget_case(4, [1, 20], [300, 200], 128, 16, 8, 64, F16)
    far = 2 ** 32 // (8 * 64 * 72) + 1
    n = b.pages.shape[0]
    big = mmq.kv_pages(far + n, 8, 64)
    wide = mmq.kv_weights(far + n, 8)
    big[far:] = b.pages
    wide[far:] = w
    other = Batch([1, 20], [300, 200], 8, 64, F16, fill=False)
    other.pages, other.table = big, torch.where(b.table >= 0, b.table + far, -1)
    got = turn_weigh_evict(other, q, k, v, pos, plan, table + far, wide, keep)
    want = turn_weigh_evict(b, q, k, v, pos, plan, table, w, keep)
    assert status() == 0 and all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(big[far:], b.pages) and torch.equal(wide[far:], w)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("new", [2, 40, 150])
def test_lengths_that_are_no_lengths(dtype, new):
    """Below zero nobody has a key; past the table its pages are all there are.  The other sequence is as ever."""
    b = Batch([new, new], [200, 200], 1, 128, dtype)
    q, before = b.q(2), weights_for(b)
    alone = before.clone()
    mmq.kv_attend_weights(q, alone, *b.cache, new)
    second, first = b.table[1].long(), b.table[0].long()
    for m in (-7, 0):
        w = before.clone()
        length = torch.tensor([m, 200], dtype=torch.int32, device=DEV)
        out, _ = mmq.kv_attend_weights(q, w, b.pages, b.table, b.start, length, new)
        status()
        assert torch.equal(w[second], alone[second]) and torch.equal(w[first], before[first])
        assert (out[:new] == 0).all()


@pytest.mark.parametrize("length", [8191, 8192, 8193, 16385, 32769])
def test_clusters_begin(length):
    """One CTA and clusters of two, four and eight, whose last has hardly a token."""
    b = Batch([1], [length], 1, 64, fill=False)
    evict_and_check(b, weights_for(b), 4000, 3, 100, bytes_too=False)


@pytest.mark.parametrize("budget", [1, 100, 400])
def test_the_example_keeps_a_budget(budget):
    """It runs; a budget that all of the prompt fits in changes nothing that the cache's own rounding does not."""
    from examples import attention_block
    args = ["--hidden", "512", "--heads", "4", "--kv-heads", "2", "--dim", "128", "--prompt", "300", "--steps", "3",
            "--batch", "2"]
    worst = attention_block.main(args + ["--budget", str(budget)])
    assert math.isfinite(worst)
    if budget == 400:
        assert worst == pytest.approx(attention_block.main(args), abs=1e-5)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("new,length,batch", [(1, 9000, 40), (40, 700, 4), (300, 900, 2)])
def test_a_wait_that_runs_out_ends_every_kernel_of_the_call(dtype, new, length, batch):
    """A fill that the attention's first CTA leaves out: the kernels behind it see the error and end, and the
    next call is right."""
    b = Batch([new] * batch, [length] * batch, 2, 128, dtype)
    q, before = b.q(4), weights_for(b)
    want = before.clone()
    mmq.kv_attend_weights(q, want, *b.cache, new, length, decay=0.5)
    torch.cuda.synchronize()
    assert status() == 0
    try:
        mmq.mmq_debug_inject_wait_timeout(0, 1_000_000)
        mmq.kv_attend_weights(q, before.clone(), *b.cache, new, length, decay=0.5)
        assert status() == 5
        assert status() == 0
        got = before.clone()
        mmq.kv_attend_weights(q, got, *b.cache, new, length, decay=0.5)
        assert status() == 0
    finally:
        mmq.mmq_debug_inject_wait_timeout(-1)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("factor,scale", [(4e37, 1.2e-38), (1e-38, 2e37), (1e-30, 1.5e29)])
@pytest.mark.parametrize("new,length,hint", [([1, 2], [700, 300], None), ([1, 2], [700, 300], 100), ([40], [700], None),
                                             ([200], [700], None)])
def test_rows_of_any_size_weigh(dtype, factor, scale, new, length, hint):
    """q . k alone passes f32 where its product with the scale is an ordinary number, as does a row's size."""
    b = Batch(new, length, 2, 128, dtype)
    weigh_and_check(b, 6, factor=factor, scale=scale, max_kv=hint, decay=0.5)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("new", [[0] * 90 + [300] + [0] * 200 + [1, 0, 1, 129, 0, 2] + [0] * 40 + [128],
                                 [1] * 140 + [0] * 300 + [200], [1, 200] + [0] * 50 + [1] * 20 + [0, 255, 1]])
def test_many_slots_and_few_with_new_tokens(dtype, new):
    """Operand tiles of sequences lie side by side however many slots without rows are between them."""
    b = Batch(new, [n + (i * 37) % 150 for i, n in enumerate(new)], 2, 64, dtype)
    weigh_and_check(b, 6, decay=0.5)
