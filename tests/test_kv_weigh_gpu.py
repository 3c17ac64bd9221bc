"""The weights of keys where a CTA has many tiles, heads and sequences to walk through, where pages are missing and
where lengths are none, and eviction by clusters of every size: on the GPU, against the definitions of
tests/budget_reference.py in 64 bits, with the tolerances of tests/test_kv_budget_gpu.py.
"""
from types import SimpleNamespace

import pytest
import torch

import quant_int8_mmq_gb300 as mmq
from tests.test_kv_budget_gpu import check_weights, evict_and_check, held_of, weigh_and_check, weights_for
from tests.test_kv_gpu import BF16, DEV, F16, F32, Batch, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(mmq_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.synchronize()
    mmq.mmq_get_device_error()
    yield


# ------------------------------------------------------------------------------------ few rows, many tiles
# 128 keys a tile, 152 CTAs: more than 16 tiles a CTA go round its ring of codes, whichever size that has, and every
# one of its warpgroups has several; shares end inside heads and sequences.
LONG, RAGGED = [30000, 9000, 17000], [3000, 30000, 700, 12345, 129]


@pytest.mark.parametrize("dtype,dim,heads,new,lens", [
    (F16, 128, 32, [32, 17, 25], LONG),            # 128 columns
    (BF16, 128, 32, [20, 32, 1, 9, 31], RAGGED),
    (F16, 128, 8, [20, 32, 1, 9, 31], RAGGED),     # 32
    (F16, 64, 32, [32, 17, 25], LONG),
    (F32, 128, 32, [32, 17, 25], LONG),            # 128 and their low parts, by two products: two buffers of K
    (F32, 128, 16, [30, 17, 25], LONG),            # 64 and theirs side by side: two buffers of K
    (F32, 128, 8, [40, 17, 33], LONG),             # 48 and theirs
    (F32, 64, 8, [40, 17, 33], LONG),
    (F32, 64, 32, [20, 32, 1, 9, 31], RAGGED)])
def test_a_cta_has_many_tiles(dtype, dim, heads, new, lens):
    weigh_and_check(Batch(new, lens, 8, dim, dtype), heads, decay=0.5)


@pytest.mark.parametrize("dtype,dim", [(F16, 128), (F32, 128), (F32, 64), (BF16, 64)])
@pytest.mark.parametrize("window,sinks,decay", [(3000, 0, 0.75), (700, 200, 1.0), (129, 1000, 0.5), (20000, 3, 1.0)])
def test_many_tiles_of_which_some_are_not_seen(dtype, dim, window, sinks, decay):
    """In place, and into another buffer, where what is not seen has to be written too."""
    new, lens = [28, 17, 1, 31], [30000, 9000, 300, 20000]
    b = Batch(new, lens, 8, dim, dtype)
    q, before, mine = weigh_and_check(b, 32, window=window, sinks=sinks, decay=decay)
    into = torch.full_like(before, 5.0)
    mmq.kv_attend_weights(q, before, *b.cache, max(new), window=window, sinks=sinks, decay=decay, into=into)
    want = torch.full_like(before, 5.0)
    for s, m in enumerate(lens):
        j = torch.arange(m, device=DEV)
        page = b.table[s, j // 64].long()
        want[page, :, j % 64] = mine[page, :, j % 64]
    assert status() == 0 and torch.equal(into, want)


@pytest.mark.parametrize("dtype,dim", [(F16, 128), (F32, 128), (F32, 64), (BF16, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 70)])
def test_a_cta_has_many_short_sequences(dtype, dim, window, sinks):
    """Runs of one to four tiles, dozens a CTA, of other rows each; sequences without new tokens between them."""
    lens = [1 + (i * 61) % 450 for i in range(400)]
    new = [0 if i % 11 == 5 else min(m, 1 + (i * 7) % 16) for i, m in enumerate(lens)]
    new[3] = min(lens[3], 16)
    weigh_and_check(Batch(new, lens, 8, dim, dtype), 32 if dim == 128 else 56, window=window, sinks=sinks, decay=0.5)


@pytest.mark.parametrize("dtype,dim", [(F16, 128), (F32, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (5000, 130)])
def test_many_tiles_of_single_tokens(dtype, dim, window, sinks):
    """More scores than are kept: the same kernel, 16 columns."""
    b = Batch([2, 1, 2], LONG, 8, dim, dtype, max_pages=(1 << 30) // (256 * 8 * 8 * 3) + 1)
    weigh_and_check(b, 32, window=window, sinks=sinks, decay=0.5)


@pytest.mark.parametrize("dtype,dim", [(F16, 128), (F32, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("window,sinks,hint", [(0, 0, None), (0, 0, 1), (0, 0, 600), (400, 300, None), (400, 300, 1)])
def test_many_rows_and_a_buffer_of_their_own(dtype, dim, window, sinks, hint):
    """One group of 256 keys a CTA, or, by a low hint, all of them; tiles that some rows do not see."""
    new, lens = [300, 0, 129, 65], [3000, 90, 129, 1000]
    b = Batch(new, lens, 2, dim, dtype)
    q, before, mine = weigh_and_check(b, 6, window=window, sinks=sinks, decay=0.5, max_kv=hint)
    into = torch.full_like(before, 5.0)
    mmq.kv_attend_weights(q, before, *b.cache, max(new), hint, window=window, sinks=sinks, decay=0.5, into=into)
    want = torch.full_like(before, 5.0)
    for s, m in enumerate(lens):
        if new[s]:
            j = torch.arange(m, device=DEV)
            page = b.table[s, j // 64].long()
            want[page, :, j % 64] = mine[page, :, j % 64]
    assert status() == 0 and torch.equal(into, want)


# ------------------------------------------------------------------------------------ pages and lengths that are none
def received(q, k, pos, scale, there):
    """budget_reference.received without a window, of the keys that are there."""
    n, heads, D = q.shape
    qg = q.reshape(n, k.shape[1], heads // k.shape[1], D)
    ok = ((torch.arange(k.shape[0], device=DEV)[None] <= pos[:, None]) & there[None])[:, None, None, :]
    x = torch.where(ok, torch.einsum("nhgd,jhd->nhgj", qg, k) * scale, float("-inf"))
    w = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e300))
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    S = torch.where(ok, torch.einsum("nhgd,jhd->nhgj", qg.abs(), k.abs()) * scale, 0.0).amax(-1, keepdim=True)
    return w.sum((0, 2)), (w * (1.0 + S)).sum((0, 2))


WIDE = (1 << 30) // (256 * 8 * 2) + 1          # pages of a table whose scores of 8 rows of 2 heads would pass a gigabyte


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,wide", [(2, None), (2, WIDE), (40, None), (150, None)])
@pytest.mark.parametrize("gone", [[1], [0], [4], [0, 1, 2], [2, 3], [0, 1, 2, 3, 4]])
def test_the_keys_that_are_there_share_the_weight(dtype, dim, new, wide, gone):
    """Pages that the pool has not, below zero and above: their keys are left out, and their weights as they were."""
    b = Batch([new], [300], 2, dim, dtype, max_pages=wide)
    table = b.table.clone()
    for i, page in enumerate(gone):
        table[0, page] = (b.pages.shape[0] + 5, -1, -2 ** 31, 2 ** 31 - 1, b.pages.shape[0])[i]
    q, before = b.q(8), weights_for(b)
    w = before.clone()
    out, _ = mmq.kv_attend_weights(q, w, b.pages, table, b.start, b.length, new, decay=0.5)
    assert status() == 1 and status() == 0
    assert torch.equal(out, mmq.kv_attend(q, b.pages, table, b.start, b.length, new)) and status() == 1
    j = torch.arange(300, device=DEV)
    there = torch.tensor([i not in gone for i in range(5)], device=DEV)[j // 64]
    k, _ = held_of(b, 0)
    got, bound = received(q.double(), k, torch.arange(300 - new, 300, device=DEV), dim ** -0.5, there)
    page = b.table[0, j // 64].long()
    old = torch.where(j < 300 - new, 0.5 * before[page, :, j % 64].double().T, 0.0)
    want, tol = before.double(), torch.zeros_like(before, dtype=torch.float64)
    at = page[there], slice(None), j[there] % 64
    want[at] = (old + got).T[there]
    tol[at] = (2.0 ** -19 * bound + (4 * new + 2) * 2.0 ** -24 * (got + old) + 2.0 ** -126).T[there]
    err = (w.double() - want).abs()
    assert (err <= tol).all(), ((err / tol.clamp(min=1e-300)).max().item(), err.max().item())


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("new,wide", [(2, False), (2, True), (40, False), (150, False)])
@pytest.mark.parametrize("length", [257, 258, 300, 2 ** 30, 2 ** 31 - 1])
def test_lengths_past_the_table(dtype, new, wide, length):
    """Rows past what the table has pages for see all of them, and it is reported; the other sequence is as ever."""
    b = Batch([new, new], [256, 200], 2, 64, dtype)
    if wide:        # the same pages, a batch of so many slots without rows that scores would pass a gigabyte
        more = (1 << 30) // (256 * 8 * 2 * 4) - 1
        b.table = torch.cat([b.table, torch.full((more, 4), -1, dtype=torch.int32, device=DEV)])
        b.start = torch.cat([b.start, torch.full((more,), 2 * new, dtype=torch.int32, device=DEV)])
        b.length = torch.cat([b.length, torch.zeros(more, dtype=torch.int32, device=DEV)])
    q, before = b.q(8), weights_for(b)
    alone = before.clone()
    mmq.kv_attend_weights(q, alone, *b.cache, new, decay=0.5)
    assert status() == 0
    b.length[0] = length
    w = before.clone()
    mmq.kv_attend_weights(q, w, *b.cache, new, decay=0.5)
    assert status() == 1 and status() == 0
    second = b.table[1, :4].long()
    assert torch.equal(w[second], alone[second])
    j = torch.arange(256, device=DEV)
    k, _ = held_of(b, 0)
    pos = torch.arange(length - new, length, device=DEV)
    got, bound = received(q[:new].double(), k, pos, 0.125, torch.ones(256, dtype=torch.bool, device=DEV))
    page = b.table[0, j // 64].long()
    old = torch.where(j < length - new, 0.5 * before[page, :, j % 64].double().T, 0.0)
    want = (old + got).T
    tol = (2.0 ** -19 * bound + (4 * new + 2) * 2.0 ** -24 * (got + old) + 2.0 ** -126).T
    err = (w[page, :, j % 64].double() - want).abs()
    assert (err <= tol).all(), ((err / tol).max().item(), err.max().item())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,length", [([3, 2], [2, 70]), ([40, 33], [25, 700]), ([40], [1]), ([300, 1, 200], [100, 9, 650]),
                                        ([200], [3])])
def test_more_new_tokens_than_tokens(dtype, dim, new, length):
    """Rows before a sequence's first token see nothing and give nothing."""
    b = Batch(new, length, 2, dim, dtype)
    q, before = b.q(8), weights_for(b)
    w = before.clone()
    out, _ = mmq.kv_attend_weights(q, w, *b.cache, max(new), decay=0.5)
    assert status() == 0 and (out[:new[0] - length[0]] == 0).all()
    check_weights(b, q, before, w, decay=0.5)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[2, 1], [40, 9], [200, 3]])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_rows_of_any_stride_weigh(dtype, dim, new, shift):
    """Rows of a wider buffer, at any alignment, the result by heads: the same bits as of rows that lie together."""
    b = Batch(new, [300, 90], 2, dim, dtype)
    q, before = b.q(6), weights_for(b)
    wide = torch.full((b.rows, 8 * dim + 7), 3.0, device=DEV, dtype=dtype)
    x = wide[:, shift:shift + 6 * dim].view(b.rows, 6, dim)
    x.copy_(q)
    outer = torch.full((6, b.rows, dim + shift), 9.0, device=DEV, dtype=dtype)
    out = outer[..., :dim].transpose(0, 1)
    want, w = before.clone(), before.clone()
    there, _ = mmq.kv_attend_weights(q, want, *b.cache, max(new))
    mmq.kv_attend_weights(x, w, *b.cache, max(new), out=out)
    assert status() == 0 and torch.equal(w, want) and torch.equal(out, there) and (outer[..., dim:] == 9.0).all()
    check_weights(b, q, before, w)
    one = q[:1, :1].expand(b.rows, 6, dim)                              # the same row everywhere
    w = before.clone()
    mmq.kv_attend_weights(one, w, *b.cache, max(new))
    check_weights(b, one, before, w)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("heads,kv_heads,new,lens", [(300, 1, [1, 2], [900, 77]), (1024, 4, [1], [500]), (129, 1, [1, 1, 1], [70, 900, 1]),
                                                     (70, 2, [3, 1], [600, 64]), (14, 2, [37, 5], [800, 129])])
def test_many_heads_on_one(dtype, heads, kv_heads, new, lens):
    weigh_and_check(Batch(new, lens, kv_heads, 64, dtype), heads, decay=0.5)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("new,max_q", [([40, 7], 20), ([300, 129, 2], 150), ([300, 129, 2], 1000000)])
def test_rows_past_max_q_of_many(dtype, new, max_q):
    """They add nothing, and it is reported; a number past the rows is none too many."""
    b = Batch(new, [700, 200, 90][:len(new)], 2, 128, dtype)
    q, before = b.q(4), weights_for(b)
    w = before.clone()
    mmq.kv_attend_weights(q, w, *b.cache, max_q, decay=0.5)
    assert status() == (1 if max_q < max(new) else 0)
    check_weights(b, q, before, w, decay=0.5, max_q=max_q)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("new", [2, 40, 150])
def test_sequences_that_share_pages_weigh_one_by_one(dtype, new):
    """Not in one call; in a call each, both add to what the pages of the prefix hold."""
    b = Batch([new, new], [400, 360], 2, 64, dtype)
    b.table[1, :3] = b.table[0, :3]
    b.k[1][:192], b.v[1][:192] = b.k[0][:192], b.v[0][:192]
    q, w = b.q(8), weights_for(b)
    start = torch.tensor([0, new], dtype=torch.int32, device=DEV)
    for s in range(2):
        one, rows, before = slice(s, s + 1), slice(s * new, (s + 1) * new), w.clone()
        mmq.kv_attend_weights(q[rows], w, b.pages, b.table[one], start, b.length[one], new, decay=0.5)
        assert status() == 0
        alone = SimpleNamespace(new=[new], len=b.len[one], hk=b.hk, dim=b.dim, table=b.table[one], k=b.k[one], v=b.v[one])
        check_weights(alone, q[rows], before, w, decay=0.5)


# ------------------------------------------------------------------------------------ eviction
@pytest.mark.parametrize("batch,heads,length,keep", [(50, 2, 12001, 3000), (77, 1, 8300, 8000), (152, 1, 9001, 65),
                                                     (38, 2, 9000, 4500), (25, 2, 17000, 5000)])
@pytest.mark.parametrize("kind", ["equal", "some", "random"])
def test_clusters_of_two_and_four(batch, heads, length, keep, kind):
    """77 to 152 sequences' heads: two CTAs each; 39 to 76: four.  Equal weights on both sides of a CTA's border."""
    lens = [length - (i * 613) % 3000 for i in range(batch)]
    lens[1] = keep
    b = Batch([1] * batch, lens, heads, 64, fill=False)
    w = weights_for(b)
    if kind == "equal":
        w.fill_(1.0)
    elif kind == "some":
        w.mul_(4).round_()
    evict_and_check(b, w, keep, 3, 60, bytes_too=False)
