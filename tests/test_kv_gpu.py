"""The 4-bit key/value cache and the attention over it, on the GPU, against the definitions of
tests/kv_reference.py in 64 bits.

Written bytes and values read back are exact.  Attention: a score's error is at most
2^-20 (S + 1) with S = scale * sum |q| |k| (operands of 22 bits, f32 sums of up to 2 * 128 terms, the
exponential's 2^-22), and moves the result by at most twice that times the largest |v|; weights
that enter the products in 16 bits (16-bit rows only) add 2^-11 of it, and the result's own
rounding half a unit of its last place.
"""
import numpy as np
import pytest
import torch

import quant_int8_mmq_gb300 as mmq
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF_ULP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib(mmq_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.synchronize()
    mmq.mmq_get_device_error()
    yield


def status():
    return mmq.mmq_get_device_error()


class Batch:
    """Sequences of the given lengths whose last new[b] tokens are the packed rows, in pages in no
    order; unwritten slots hold 0xFF (their scales are no numbers)."""

    def __init__(self, new, length, kv_heads, dim, dtype=F32, seed=0, max_pages=None, spare=2, fill=True):
        g = torch.Generator().manual_seed(seed)
        self.new, self.len, self.hk, self.dim, self.dtype = new, length, kv_heads, dim, dtype
        need = [-(-max(m, 0) // 64) for m in length]
        self.max_pages = max_pages or max(max(need), 1)
        num = sum(need) + spare
        perm = torch.randperm(num, generator=g).to(torch.int32)
        table = torch.full((len(new), self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table = table.to(DEV)
        self.start = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
        self.length = torch.tensor(length, dtype=torch.int32, device=DEV)
        self.rows = sum(new)
        self.pages = torch.full((num, kv_heads, 72 * dim), 0xFF, dtype=torch.uint8, device=DEV)
        self.k, self.v = [], []
        if fill:   # every token of every sequence, written by the package (checked bit for bit elsewhere)
            self.k = [torch.randn(max(m, 0), kv_heads, dim, generator=g).to(dtype).to(DEV) for m in length]
            self.v = [torch.randn(max(m, 0), kv_heads, dim, generator=g).to(dtype).to(DEV) for m in length]
            whole = torch.tensor([0] + list(np.cumsum([max(m, 0) for m in length])), dtype=torch.int32, device=DEV)
            if sum(max(m, 0) for m in length):
                mmq.kv_write(torch.cat(self.k), torch.cat(self.v), self.pages, self.table, whole,
                             self.length.clamp(min=0))

    @property
    def cache(self):
        return self.pages, self.table, self.start, self.length

    def q(self, heads, seed=1, factor=1.5):
        g = torch.Generator().manual_seed(seed)
        return (factor * torch.randn(self.rows, heads, self.dim, generator=g)).to(self.dtype).to(DEV)

    def held(self, b):
        """What the cache holds of sequence b, f64."""
        return tuple(torch.from_numpy(ref.values(x[b].double().cpu().numpy())).to(DEV) for x in (self.k, self.v))

    def check(self, q, out, scale=None, window=0, sinks=0):
        scale = self.dim ** -0.5 if scale is None else scale
        assert out.dtype == self.dtype
        lo = 0
        for b, (n, m) in enumerate(zip(self.new, self.len)):
            k, v = self.held(b)
            for i in range(0, n, 512):
                c = min(512, n - i)
                rows = slice(lo + i, lo + i + c)
                pos = torch.arange(m - n + i, m - n + i + c, device=DEV)
                want, S = ref.attend(q[rows].double(), k, v, pos, scale, window, sinks)
                big = v.abs().max() if v.numel() else 0.0
                # f32 rounding of the scale itself moves every score by a factor within 2^-23
                tol = (2 ** -19 * (S + 1) + (2 ** -11 if self.dtype != F32 else 0))[..., None] * big \
                    + HALF_ULP[self.dtype] * want.abs() + 2.0 ** -25
                err = (out[rows].double() - want).abs()
                assert torch.isfinite(out[rows]).all()
                assert (err <= tol).all(), (b, i, err.max().item(), (err / tol).max().item())
            lo += n
        assert status() == 0


# ------------------------------------------------------------------------------------ write, read
def hard_rows(n, heads, dim, dtype, seed):
    """Rows with what quantising can get wrong: ties, zeros, huge, tiny, no numbers."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, dim, generator=g)
    x[0::5] *= 10.0 ** torch.randint(-9, 6, (len(x[0::5]), heads, 1), generator=g)
    x[1::5] = torch.randint(-15, 16, (len(x[1::5]), heads, dim), generator=g).float() / 2     # exact ties
    x[2, :, :32] = 0.0
    x[2, :, 32:64] = -0.0
    x[3, :, 5] = float("nan")
    x[3, :, 40] = float("inf")
    x[4, :, 7] = float("-inf")
    x[4, :, 33:] = 7000.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim,heads", [(64, 3), (128, 2), (128, 1)])
def test_written_bytes_are_the_definition(dtype, dim, heads):
    new, length = [1, 7, 0, 70], [1, 70, 5, 131]
    b = Batch(new, length, heads, dim, dtype, fill=False)
    k, v = (hard_rows(b.rows, heads, dim, dtype, s) for s in (1, 2))
    want = b.pages.cpu().numpy()
    r = 0
    for s, (n, m) in enumerate(zip(new, length)):
        for p in range(m - n, m):
            ref.put(want, int(b.table[s, p // 64]), p % 64, k[r].double().numpy(), v[r].double().numpy())
            r += 1
    mmq.kv_write(k.to(DEV), v.to(DEV), *b.cache)
    assert status() == 0
    got = b.pages.cpu().numpy()
    assert np.array_equal(got, want)          # slots of no new token are untouched too
    for out, x in zip(mmq.kv_read(*b.cache, b.rows, dtype=F32), (k, v)):
        assert np.array_equal(out.double().cpu().numpy(), ref.values(x.double().numpy()))
    for t in (F16, BF16):
        for out, x in zip(mmq.kv_read(*b.cache, b.rows, dtype=t), (k, v)):
            assert torch.equal(out.cpu(), torch.from_numpy(ref.values(x.double().numpy())).to(t))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_rows_of_any_stride_and_alignment(dtype, shift):
    """k and v as parts of one wide row, shifted by single elements; heads outside tokens; broadcasts."""
    heads, dim, n = 2, 128, 67
    b = Batch([n], [n], heads, dim, dtype, fill=False)
    wide = torch.randn(n, 1000 + shift, device=DEV).to(dtype)
    k = wide[:, shift:shift + 256].view(n, heads, dim)
    v = wide[:, shift + 300:shift + 300 + 256].view(n, heads, dim)
    mmq.kv_write(k, v, *b.cache)
    out = [x.double().cpu().numpy() for x in mmq.kv_read(*b.cache, n, dtype=F32)]
    for o, x in zip(out, (k, v)):
        assert np.array_equal(o, ref.values(x.double().cpu().numpy()))
    outer = torch.full((heads, n, dim + shift), 9.0, device=DEV, dtype=dtype)
    both = [x[..., :dim].transpose(0, 1) for x in (outer.clone(), outer.clone())]
    mmq.kv_read(*b.cache, n, k=both[0], v=both[1])
    for o, x in zip(both, out):
        assert torch.equal(o.cpu(), torch.from_numpy(x).to(dtype))
    assert all((o.transpose(0, 1)._base[..., dim:] == 9.0).all() for o in both)
    one = torch.randn(1, 1, dim, device=DEV).to(dtype).expand(n, heads, dim)
    mmq.kv_write(one, one, *b.cache)
    got = mmq.kv_read(*b.cache, n, dtype=F32)
    want = torch.from_numpy(ref.values(one[:1, :1].double().cpu().numpy())).float().to(DEV)
    assert all(torch.equal(g, want.expand(n, heads, dim)) for g in got)
    assert status() == 0


def test_tokens_without_a_place_are_reported_and_read_as_zero():
    b = Batch([3, 70], [2, 70], 2, 64, max_pages=2)         # the first row of sequence 0 is before it
    before = b.pages.clone()
    bad = b.table.clone()
    bad[1, 1] = b.pages.shape[0]                            # a page past the pool
    x = torch.randn(73, 2, 64, device=DEV)
    mmq.kv_write(x, x, b.pages, bad, b.start, b.length)
    assert status() == 1 and status() == 0
    touched = (b.pages != before).flatten(1).any(1)
    assert touched.sum() == 2
    k, v = mmq.kv_read(b.pages, bad, b.start, b.length, 73, dtype=F32)
    assert status() == 1
    want = torch.from_numpy(ref.values(x.double().cpu().numpy())).float().to(DEV)
    want[0] = 0
    want[3 + 64:] = 0
    assert torch.equal(k, want) and torch.equal(v, want)
    bad[1, 1] = -7
    mmq.kv_read(b.pages, bad, b.start, torch.tensor([3, 200], dtype=torch.int32, device=DEV), 73)
    assert status() == 1


def test_many_sequences_find_their_rows():
    """Row to sequence over more sequences than a warp probes at once, some without rows."""
    new = [(i * 7) % 4 for i in range(1500)]
    length = [n + (i * 13) % 50 for i, n in enumerate(new)]
    b = Batch(new, length, 1, 64, fill=False)
    x = torch.randn(b.rows, 1, 64, device=DEV)
    mmq.kv_write(x, 2 * x, *b.cache)
    k, v = mmq.kv_read(*b.cache, b.rows, dtype=F32)
    want = torch.from_numpy(ref.values(x.double().cpu().numpy())).float().to(DEV)
    assert torch.equal(k, want) and torch.equal(v, 2 * want) and status() == 0


def test_pool_past_32_bits():
    heads, dim, num = 8, 128, 60000                          # 4.4 GB of pages
    pages = mmq.kv_pages(num, heads, dim)
    assert pages.numel() > 1 << 32
    table = torch.tensor([[num - 1, 3, num - 2]], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 150], dtype=torch.int32, device=DEV)
    length = torch.tensor([150], dtype=torch.int32, device=DEV)
    x = torch.randn(150, heads, dim, device=DEV)
    mmq.kv_write(x, -x, pages, table, start, length)
    k, v = mmq.kv_read(pages, table, start, length, 150, dtype=F32)
    want = torch.from_numpy(ref.values(x.double().cpu().numpy())).to(DEV)
    assert torch.equal(k.double(), want)
    assert torch.equal(v.double(), torch.from_numpy(ref.values(-x.double().cpu().numpy())).to(DEV))
    q = torch.randn(150, heads, dim, device=DEV)
    out = mmq.kv_attend(q, pages, table, start, length, 150)
    want, S = ref.attend(q.double(), want, v.double(), torch.arange(150, device=DEV), dim ** -0.5)
    assert ((out.double() - want).abs() <= 2 ** -19 * (S + 1)[..., None] * v.abs().max() + 2.0 ** -25).all()
    assert status() == 0


# ----------------------------------------------------------------------------------------- attention
STEP = [  # new, length, heads, kv heads, dim
    ([1], [1], 1, 1, 128),
    ([1], [64], 4, 4, 64),
    ([1], [65], 8, 1, 128),
    ([1, 1, 1], [63, 200, 1], 6, 2, 128),
    ([1], [5000], 32, 8, 128),
    ([3, 0, 5, 1], [3, 7, 700, 130], 10, 2, 64),
    ([2], [4097], 48, 3, 128),
    ([1] * 40, [1 + 97 * i for i in range(40)], 8, 8, 64),
]
PROMPT = [
    ([65], [65], 2, 2, 128),
    ([129, 1, 0, 300], [129, 64, 9, 1000], 6, 2, 128),
    ([500], [511], 5, 1, 64),
    ([1000], [1300], 4, 2, 128),
    ([33, 257], [2000, 257], 16, 2, 64),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("new,length,heads,kv_heads,dim", STEP + PROMPT)
def test_attention(new, length, heads, kv_heads, dim, dtype):
    b = Batch(new, length, kv_heads, dim, dtype, seed=len(new) + heads)
    q = b.q(heads)
    b.check(q, mmq.kv_attend(q, *b.cache, max_q=max(new)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length", [63, 64, 65, 127, 128, 129, 193, 256, 257, 385, 700])
def test_every_number_of_pages(length, dim, dtype):
    """Rows of one tile (both tiles take every other step), of two, and of two and a rest, with
    odd and even numbers of pages and steps."""
    for rows in (min(length, 40), min(length, 100), min(length, 190)):
        b = Batch([rows], [length], 1, dim, dtype, seed=length)
        q = b.q(2)
        b.check(q, mmq.kv_attend(q, *b.cache, max_q=rows))


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("new,heads,kv_heads", [(1, 4, 1), (2, 12, 1), (1, 32, 4), (40, 2, 1), (300, 1, 1)])
@pytest.mark.parametrize("length", [257, 700, 1500, 3000, 6000, 20000])
def test_parts_of_any_number(length, new, heads, kv_heads, dtype):
    """Few rows on caches that are cut into one part, one cluster, or many parts and a join."""
    new = min(new, length)
    b = Batch([new], [length], kv_heads, 128, dtype, seed=length)
    q = b.q(heads)
    b.check(q, mmq.kv_attend(q, *b.cache, max_q=new, max_kv=length))


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (65, 0), (100, 64), (100, 65), (700, 4),
                                          (333, 200), (1 << 30, 3), (50, 1 << 30)])
@pytest.mark.parametrize("new,length,heads,kv_heads,dim", [([1, 2], [1000, 64], 4, 1, 128), ([1], [3001], 4, 4, 64),
                                                           ([400, 3], [900, 400], 4, 2, 128),
                                                           ([300], [300], 8, 1, 64)])
def test_window_and_first_tokens(new, length, heads, kv_heads, dim, window, sinks, dtype):
    b = Batch(new, length, kv_heads, dim, dtype, seed=window % 97)
    q = b.q(heads)
    out = mmq.kv_attend(q, *b.cache, max_q=max(new), window=window, sinks=sinks)
    b.check(q, out, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new,length", [([5, 2], [3, 0]), ([200, 1], [100, 0]), ([1], [0])])
def test_rows_that_see_no_key_are_zero(new, length, dtype):
    b = Batch(new, length, 2, 64, dtype)
    q = b.q(4)
    out = mmq.kv_attend(q, *b.cache, max_q=max(new))
    b.check(q, out)
    assert (out[:new[0] - length[0]] == 0).all()


@pytest.mark.parametrize("hint", [0, 1, 64, 5000, 1 << 30])
def test_any_length_hint_is_right(hint):
    b = Batch([1, 2], [5000, 100], 2, 128)
    q = b.q(4)
    b.check(q, mmq.kv_attend(q, *b.cache, max_q=2, max_kv=hint))


@pytest.mark.parametrize("factor,scale", [(1e-30, 1e28), (1e25, 3e-26), (40.0, None), (0.0, None), (1.0, 1e-20)])
@pytest.mark.parametrize("new,length", [([2], [300]), ([150], [300])])
def test_queries_and_scales_of_any_size(new, length, factor, scale):
    """Large logits (one key takes all the weight), zero queries, magnitudes far from 1."""
    b = Batch(new, length, 1, 128)
    q = b.q(4, factor=factor)
    b.check(q, mmq.kv_attend(q, *b.cache, max_q=max(new), scale=scale), scale=scale)


@pytest.mark.parametrize("new,length", [([2, 3], [300, 90]), ([150, 140], [300, 140])])
def test_a_row_that_is_no_number_stays_alone(new, length):
    b = Batch(new, length, 1, 64)
    q = b.q(2)
    clean = mmq.kv_attend(q, *b.cache, max_q=max(new))
    q[1, 1, 7] = float("nan")
    out = mmq.kv_attend(q, *b.cache, max_q=max(new))
    assert torch.isnan(out[1, 1]).all()
    out[1, 1] = clean[1, 1]
    assert torch.equal(out, clean) and status() == 0


@pytest.mark.parametrize("new,length", [([1], [700]), ([200], [700])])
def test_keys_of_a_page_outside_the_pool_are_not_there(new, length):
    b = Batch(new, length, 2, 128)
    q = b.q(2)
    table = b.table.clone()
    table[0, 3] = 1 << 20
    out = mmq.kv_attend(q, b.pages, table, b.start, b.length, max_q=max(new))
    assert status() == 1 and status() == 0
    k, v = b.held(0)
    keep = torch.cat([torch.arange(0, 192), torch.arange(256, length[0])]).to(DEV)
    # without page 3 later keys move up by 64, so do the positions that look at them
    pos = torch.arange(length[0] - new[0], length[0], device=DEV) - 64
    want, S = ref.attend(q.double(), k[keep], v[keep], pos, 128 ** -0.5)
    assert ((out.double() - want).abs() <= 2 ** -19 * (S + 1)[..., None] * v.abs().max() + 2.0 ** -25).all()


def test_length_past_the_table_is_reported():
    b = Batch([1], [128], 1, 64)
    q = b.q(1)
    mmq.kv_attend(q, b.pages, b.table, b.start, b.length + 64, max_q=1)
    assert status() == 1
    b2 = Batch([40], [128], 1, 64)
    mmq.kv_attend(b2.q(1), *b2.cache, max_q=1)               # more rows than the caller said
    assert status() == 1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new,length", [([1, 1], [900, 65]), ([200, 30], [300, 64])])
def test_strided_queries_and_results(new, length, dtype):
    heads, dim = 6, 128
    b = Batch(new, length, 2, dim, dtype)
    q = b.q(heads)
    plain = mmq.kv_attend(q, *b.cache, max_q=max(new))
    for shift in (0, 1):
        wide = torch.zeros(b.rows, 1200 + shift, device=DEV, dtype=dtype)
        part = wide[:, 7 * 4 + shift:7 * 4 + shift + heads * dim].view(b.rows, heads, dim)
        part.copy_(q)
        out = torch.full((heads, b.rows, dim + shift), 5.0, device=DEV, dtype=dtype)
        mmq.kv_attend(part, *b.cache, max_q=max(new), out=out[..., :dim].transpose(0, 1))
        assert torch.equal(out[..., :dim].transpose(0, 1), plain)
        assert (out[..., dim:] == 5.0).all()


@pytest.mark.parametrize("new,length,heads", [([1], [20000], 8), ([1] * 9, [777] * 9, 4), ([300], [1500], 4)])
def test_results_do_not_vary(new, length, heads):
    b = Batch(new, length, 2, 128)
    q = b.q(heads)
    first = mmq.kv_attend(q, *b.cache, max_q=max(new))
    for _ in range(5):
        assert torch.equal(mmq.kv_attend(q, *b.cache, max_q=max(new)), first)
    b.check(q, first)


def test_other_streams_and_graphs():
    """Work on a stream that is not the current one; a captured step replayed over new tokens."""
    b = Batch([1, 1], [600, 90], 2, 128, spare=4)
    q = b.q(4)
    want = mmq.kv_attend(q, *b.cache, max_q=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = mmq.kv_attend(q, *b.cache, max_q=1, stream=side)
    side.synchronize()
    assert torch.equal(out, want)

    k, v = (torch.randn(2, 2, 128, device=DEV) for _ in range(2))
    warm = mmq.kv_attend(q, *b.cache, max_q=1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mmq.kv_write(k, v, *b.cache)
        got = mmq.kv_attend(q, *b.cache, max_q=1)
    del warm
    for step in range(3):
        b.length += 1
        b.len = [m + 1 for m in b.len]
        k.normal_()
        v.normal_()
        q.normal_()
        for s in range(2):
            b.k[s] = torch.cat([b.k[s], k[s:s + 1]])
            b.v[s] = torch.cat([b.v[s], v[s:s + 1]])
        graph.replay()
        b.check(q, got)


def test_a_prompt_and_its_tokens_one_by_one_agree():
    """The same rows as one prompt, as chunks and as single tokens."""
    n, heads = 260, 4
    b = Batch([n], [n], 2, 64)
    q = b.q(heads)
    whole = mmq.kv_attend(q, *b.cache, max_q=n)
    b.check(q, whole)
    parts = []
    for lo, hi in ((0, 1), (1, 2), (2, 9), (9, 140), (140, 259), (259, 260)):
        start = torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV)
        length = torch.tensor([hi], dtype=torch.int32, device=DEV)
        parts.append(mmq.kv_attend(q[lo:hi], b.pages, b.table, start, length, max_q=hi - lo))
    b.check(q, torch.cat(parts))


@pytest.mark.parametrize("kv_heads,dim,hidden", [(2, 128, 512), (1, 64, 256)])
def test_example_block(kv_heads, dim, hidden):
    """The example's prompt and steps agree up to what the products before the attention differ by
    (their kernels for few and many tokens, 1e-5 of a row, which may move a 4-bit code)."""
    from examples import attention_block
    worst = attention_block.main(["--hidden", str(hidden), "--heads", str(hidden // dim), "--kv-heads", str(kv_heads),
                                  "--dim", str(dim), "--prompt", "150", "--steps", "3"])
    assert worst < 1e-3


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,heads,kv_heads", [(300, 2, 1), (100, 1, 1), (70, 6, 2)])
@pytest.mark.parametrize("length,hint", [(20000, 64), (20000, 20000), (4300, 64), (2050, 64)])
@pytest.mark.parametrize("shift", [0, 1])
def test_sums_over_long_caches_keep_32_bits(length, hint, new, heads, kv_heads, dim, shift):
    """Values of one sign, whose sums lose the most to a sum that is cut toward zero: 1e-5 of every
    element, which a single such sum over 20000 keys exceeds (2500 products, each cutting half of
    2^-23 of what is there, half of the whole on average: 4e-5 and more).  Scores of small
    queries add at most 2^-19 * 1.7.  A low hint leaves the keys in one part.  Results in place
    of rows of another stride and alignment too."""
    b = Batch([new], [length], kv_heads, dim, F32, seed=length)
    g = torch.Generator().manual_seed(3)
    b.v = [(1.0 + 0.25 * torch.randn(length, kv_heads, dim, generator=g)).to(DEV)]
    whole = torch.tensor([0, length], dtype=torch.int32, device=DEV)
    mmq.kv_write(b.k[0], b.v[0], b.pages, b.table, whole, b.length)
    q = b.q(heads, factor=0.1)
    room = torch.full((new, heads, dim + 4 * shift + shift), 7.0, device=DEV)
    out = room[..., shift:shift + dim]
    mmq.kv_attend(q, *b.cache, max_q=new, max_kv=hint, out=out)
    k, v = b.held(0)
    want, _ = ref.attend(q.double(), k, v, torch.arange(length - new, length, device=DEV), dim ** -0.5)
    err = ((out.double() - want).abs() / want.abs()).max().item()
    assert err <= 1e-5, err
    assert (room[..., :shift] == 7).all() and (room[..., shift + dim:] == 7).all()
    assert status() == 0


def test_long_sums_of_f16_rows_lose_less_than_their_rounding():
    """160 sequences on the same 65536 tokens, values of one sign: enough tiles to fill the chip, so
    that nothing but the sums' length cuts them.  Rounding the results averages out over the
    elements, sums cut toward zero do not: less than half a unit of f16's last place, 2^-12."""
    batch, new, length, dim = 160, 200, 65536, 64   # more than 128 rows: each tile sums up all keys
    b = Batch([new], [length], 1, dim, F16, seed=1)
    g = torch.Generator().manual_seed(3)
    b.v = [(1.0 + 0.25 * torch.randn(length, 1, dim, generator=g)).to(F16).to(DEV)]
    mmq.kv_write(b.k[0], b.v[0], b.pages, b.table, torch.tensor([0, length], dtype=torch.int32, device=DEV), b.length)
    q = b.q(1, factor=0.1)
    out = mmq.kv_attend(q.repeat(batch, 1, 1), b.pages, b.table.repeat(batch, 1),
                        torch.arange(batch + 1, dtype=torch.int32, device=DEV) * new, b.length.repeat(batch),
                        max_q=new, max_kv=length)
    k, v = b.held(0)
    want, _ = ref.attend(q.double(), k, v, torch.arange(length - new, length, device=DEV), dim ** -0.5)
    off = ((out.double().view(batch, new, 1, dim) - want) / want).mean().item()
    assert abs(off) < 2.0 ** -12, off
    assert status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new,length,heads", [([1, 2], [200, 90], 4), ([1, 1], [3000, 90], 4),      # a CTA, a cluster a part,
                                              ([1, 1], [20000, 90], 4), ([1] * 70, [90] * 70, 2),   # many parts;
                                              ([150, 3], [300, 90], 2), ([60, 3], [20000, 90], 2)])  # prompts
def test_rows_of_no_sequence_are_zero_and_reported(new, length, heads, dtype):
    """Packed rows before the first sequence's and past the last's, as a padded batch has them."""
    b = Batch(new, length, 2, 64, dtype)
    front, back = 3, 5
    q = b.q(heads)
    wide = torch.cat([torch.ones(front, heads, 64, device=DEV).to(dtype), q, torch.ones(back, heads, 64, device=DEV).to(dtype)])
    for lo, hi in ((front, back), (0, back), (front, 0)):
        part = wide[front - lo:wide.shape[0] - back + hi]
        out = torch.full_like(part, 7.0)
        mmq.kv_attend(part, b.pages, b.table, b.start + lo, b.length, max_q=max(new), max_kv=max(length), out=out)
        assert status() == 1 and status() == 0
        assert (out[:lo] == 0).all() and (out[lo + b.rows:] == 0).all()
        b.check(q, out[lo:lo + b.rows])


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("new,length", [([2, 3], [200, 90]), ([1, 2], [20000, 90]), ([300, 40], [300, 90])])
def test_sequences_that_lead_outside_the_rows_are_zero_and_reported(new, length, dtype):
    b = Batch(new, length, 2, 64, dtype)
    q = b.q(4)
    right = mmq.kv_attend(q, *b.cache, max_q=max(new), max_kv=max(length))
    b.check(q, right)
    n = new[0]
    for start, lo, hi in (([-1, n, b.rows], 0, n), ([0, n, b.rows + 2], n, b.rows), ([-5, -5, -5], 0, b.rows)):
        out = torch.full_like(q, 7.0)
        mmq.kv_attend(q, b.pages, b.table, torch.tensor(start, dtype=torch.int32, device=DEV), b.length, max_q=max(new),
                      max_kv=max(length), out=out)
        assert status() == 1 and status() == 0
        assert (out[lo:hi] == 0).all()
        assert torch.equal(out[:lo], right[:lo]) and torch.equal(out[hi:], right[hi:])
    out = mmq.kv_attend(q, b.pages, b.table, torch.tensor([0, n, n - 1], dtype=torch.int32, device=DEV), b.length,
                        max_q=max(new), max_kv=max(length), out=torch.full_like(q, 7.0))
    assert status() == 1
    assert torch.equal(out[:n - 1], right[:n - 1]) and (out[n:] == 0).all()


@pytest.mark.parametrize("length", [128, 20000])
def test_rows_past_max_q_are_zero_and_reported(length):
    b = Batch([40, 2], [length, 70], 1, 64)
    q = b.q(1)
    out = torch.full_like(q, 7.0)
    mmq.kv_attend(q, *b.cache, max_q=2, max_kv=length, out=out)
    assert status() == 1 and status() == 0
    left = (out[:40] == 0).flatten(1).all(1)
    assert left.any() and not left[0]
    want = mmq.kv_attend(q, *b.cache, max_q=40, max_kv=length)
    out[:40][left] = want[:40][left]
    b.check(q, out)


@pytest.mark.parametrize("batch,new,length,heads,kv_heads,dim,hint", [
    (9, 1, 65536, 4, 4, 128, 65536), (7, 1, 65536, 8, 8, 64, 65536),             # clusters of twice the pages
    (1, 1, 20000, 1, 1, 128, 64), (1, 3, 70000, 8, 2, 64, 64), (1, 1, 131072, 4, 1, 128, 64)])   # all keys in one CTA
def test_sums_of_few_rows_over_long_caches_keep_32_bits(batch, new, length, heads, kv_heads, dim, hint):
    """Values of one sign under few rows, as above for many: 1e-5 of every element.  Where a CTA has
    128 pages a warp sums up 256 products, each cutting up to 2^-23 of what is there, half of it
    on average; sequences share their pages, so that a batch costs one sequence's memory."""
    b = Batch([new], [length], kv_heads, dim, F32, seed=length)
    g = torch.Generator().manual_seed(3)
    b.v = [(1.0 + 0.25 * torch.randn(length, kv_heads, dim, generator=g)).to(DEV)]
    whole = torch.tensor([0, length], dtype=torch.int32, device=DEV)
    mmq.kv_write(b.k[0], b.v[0], b.pages, b.table, whole, b.length)
    q = b.q(heads, factor=0.1)
    out = mmq.kv_attend(q.repeat(batch, 1, 1), b.pages, b.table.repeat(batch, 1),
                        torch.arange(batch + 1, dtype=torch.int32, device=DEV) * new, b.length.repeat(batch),
                        max_q=new, max_kv=hint)
    k, v = b.held(0)
    want, _ = ref.attend(q.double(), k, v, torch.arange(length - new, length, device=DEV), dim ** -0.5)
    err = ((out.double().view(batch, new, heads, dim) - want).abs() / want.abs()).max().item()
    assert err <= 1e-5, err
    assert status() == 0


@pytest.mark.parametrize("new,heads,length,dim,products,run", [(1, 4, 400000, 64, 128, 4 * 1024),
                                                               (70, 1, 131072, 64, 160, 1280),
                                                               (300, 1, 131072, 128, 160, 1280)])
def test_one_loud_key_before_a_long_tail(new, heads, length, dim, products, run):
    """f32 rows whose first key outweighs each of the others by 2^28 .. 2^40, all keys in one part.
    The tail must not be lost key by key: each may be off by 2^-38 of the largest weight, and its
    value is up to 8 times that of the first; the products that meet in one tensor-core sum cut 2^-23 of
    it each; products and weights so far are added up in f32 once a run of keys (of four warps under
    few rows), the weights of a run in up to 16 steps."""
    b = Batch([new], [length], 1, dim, F32, seed=length, fill=False)
    g = torch.Generator().manual_seed(3)
    b.k = [torch.zeros(length, 1, dim, device=DEV)]
    b.k[0][0] = 1.0
    b.v = [(1.0 + 0.25 * torch.randn(length, 1, dim, generator=g)).clamp(min=0.5).to(DEV)]
    b.v[0][0] = 0.25
    whole = torch.tensor([0, length], dtype=torch.int32, device=DEV)
    mmq.kv_write(b.k[0], b.v[0], b.pages, b.table, whole, b.length)
    k, v = b.held(0)
    below = torch.linspace(28, 40, new * heads, device=DEV).view(new, heads, 1)
    below[-1, -1] = 32.05
    q = (below / k[0].sum()).float().expand(new, heads, dim).contiguous()
    scale = float(np.float32(np.log(2.0)))
    out = mmq.kv_attend(q, *b.cache, max_q=new, max_kv=64, scale=scale)
    want, _ = ref.attend(q.double(), k, v, torch.arange(length - new, length, device=DEV), scale)
    err = ((out.double() - want).abs() / want.abs()).max().item()
    # the scores' own errors change what the tail adds, which is little
    assert err <= products * 2.0 ** -23 + 8 * length * 2.0 ** -38 + 2 * (length / run + 16) * 2.0 ** -24 + 2.0 ** -19, err
    assert status() == 0


def test_calls_on_empty_tensors_do_nothing():
    b = Batch([0, 0], [70, 5], 2, 64)
    before = b.pages.clone()
    x, q = torch.empty(0, 2, 64, device=DEV), torch.empty(0, 4, 64, device=DEV)
    mmq.kv_write(x, x, *b.cache)
    k, v = mmq.kv_read(*b.cache, 0)
    out = mmq.kv_attend(q, *b.cache, max_q=0)
    assert k.shape == v.shape == (0, 2, 64) and out.shape == q.shape
    assert torch.equal(b.pages, before) and status() == 0


@pytest.mark.parametrize("dtype,new,length,heads,kv_heads,dim,batch,fill", [
    (F32, 1, 200, 4, 4, 128, 1, 0), (F16, 4, 250, 16, 4, 128, 1, 0), (BF16, 1, 9000, 16, 8, 64, 40, 0),   # few rows
    (F32, 1, 9000, 8, 8, 128, 40, 3),
    (F32, 100, 900, 2, 1, 128, 1, 0), (F32, 400, 2000, 1, 1, 64, 1, 3), (BF16, 100, 900, 2, 1, 128, 1, 1),
    (F16, 400, 2000, 1, 1, 64, 1, 5), (F16, 400, 500, 2, 2, 128, 30, 2)])
def test_expired_wait_is_reported_then_cleared(dtype, new, length, heads, kv_heads, dim, batch, fill):
    """One copy of the first CTA is left out and every wait of the launch gives up after 1 ms (launches
    without clusters of CTAs): the launch ends, the report says why and clears, the next is right."""
    b = Batch([new], [length], kv_heads, dim, dtype)
    q = b.q(heads)
    call = dict(max_q=new, max_kv=length)
    many = (b.pages, b.table.repeat(batch, 1), torch.arange(batch + 1, dtype=torch.int32, device=DEV) * new,
            b.length.repeat(batch))
    torch.cuda.synchronize()
    assert status() == 0
    try:
        mmq.mmq_debug_inject_wait_timeout(fill, 1_000_000)
        mmq.kv_attend(q.repeat(batch, 1, 1), *many, **call)
        assert status() == 5
        assert status() == 0
        out = mmq.kv_attend(q.repeat(batch, 1, 1), *many, **call)
        assert status() == 0
    finally:
        mmq.mmq_debug_inject_wait_timeout(-1)
    b.check(q, out[:new])
    b.check(q, out[-new:])


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,window,sinks", [(1, 0, 0), (1, 19000, 70), (3, 0, 0), (3, 12000, 4)])
def test_many_pages_of_one_warp(new, window, sinks, dim, dtype):
    """A hint far too low leaves 20000 keys, 79 pages a warp, in one CTA of the step kernel, which
    fetches page ids 32 at a time."""
    b = Batch([new], [20000], 2, dim, dtype, seed=dim)
    q = b.q(6)
    out = mmq.kv_attend(q, *b.cache, max_q=new, max_kv=64, window=window, sinks=sinks)
    b.check(q, out, window=window, sinks=sinks)
