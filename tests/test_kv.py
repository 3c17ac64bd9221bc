"""Refusals and size queries of the 4-bit key/value cache and its attention (no GPU needed)."""
import ctypes

import pytest

import quant_int8_mmq_gb300 as mmq

P16 = 0x10000          # an aligned address that the error paths never follow
OK, ARG, SHAPE, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 6


def cache(**kw):
    f = dict(pages=P16, table=P16, start=P16, length=P16, num_pages=8, kv_heads=2, head_dim=128, batch=1, max_pages=8)
    f.update(kw)
    return mmq.KVCache(*(f[n] for n, _ in mmq.KVCache._fields_))


def rows(heads=2, dim=128, dtype=0, **kw):
    f = dict(data=P16, dtype=dtype, token_stride=heads * dim, head_stride=dim)
    f.update(kw)
    return mmq.Rows(*(f[n] for n, _ in mmq.Rows._fields_))


def write(c=None, k=None, v=None, n=4):
    return mmq.load().mmq_kv_write(c or cache(), k or rows(), v or rows(), n, None)


def read(c=None, k=None, v=None, n=4):
    return mmq.load().mmq_kv_read(c or cache(), k or rows(), v or rows(), n, None)


def attend(c=None, q=None, out=None, heads=2, n=4, max_q=4, max_kv=256, scale=0.1, window=0, sinks=0, ws=P16,
           size=1 << 40):
    return mmq.load().mmq_kv_attend(c or cache(), q or rows(), out or rows(), heads, n, max_q, max_kv, scale, window,
                                    sinks, ws, size, None)


def test_page_bytes(mmq_lib):
    assert mmq.mmq_kv_page_bytes(1, 64) == 4608
    assert mmq.mmq_kv_page_bytes(8, 128) == 8 * 9216
    for heads, dim in ((0, 128), (1025, 128), (1, 96), (1, 256), (1, 0)):
        with pytest.raises(mmq.MMQError) as e:
            mmq.mmq_kv_page_bytes(heads, dim)
        assert e.value.status == SHAPE
    assert mmq.load().mmq_kv_page_bytes(1, 64, None) == ARG


@pytest.mark.parametrize("call", [write, read, attend])
def test_cache_is_checked_by_every_call(mmq_lib, call):
    for kw, st in ((dict(head_dim=80), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=1025), SHAPE),
                   (dict(num_pages=0), SHAPE), (dict(batch=0), SHAPE), (dict(batch=(1 << 20) + 1), SHAPE),
                   (dict(max_pages=0), SHAPE), (dict(max_pages=(1 << 24) + 1), SHAPE),
                   (dict(pages=None), ARG), (dict(table=None), ARG), (dict(start=None), ARG), (dict(length=None), ARG),
                   (dict(pages=P16 + 8), ALIGN), (dict(table=P16 + 2), ALIGN), (dict(start=P16 + 1), ALIGN),
                   (dict(length=P16 + 2), ALIGN)):
        assert call(c=cache(**kw)) == st, kw
    lib = mmq.load()
    assert lib.mmq_kv_write(None, rows(), rows(), 4, None) == ARG
    assert lib.mmq_kv_read(None, rows(), rows(), 4, None) == ARG
    assert lib.mmq_kv_attend(None, rows(), rows(), 2, 4, 4, 256, 0.1, 0, 0, P16, 0, None) == ARG


@pytest.mark.parametrize("call,names", [(write, ("k", "v")), (read, ("k", "v")), (attend, ("q", "out"))])
def test_rows_are_checked_by_every_call(mmq_lib, call, names):
    for name in names:
        for kw, st in ((dict(data=None), ARG), (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(token_stride=-256), ARG),
                       (dict(head_stride=-128), ARG), (dict(token_stride=1 << 41), SHAPE), (dict(data=P16 + 2), ALIGN)):
            assert call(**{name: rows(**kw)}) == st, (name, kw)
        assert call(**{name: rows(dtype=1)}) == ARG          # one type for both
    both = {name: rows(dtype=2, data=P16 + 1) for name in names}
    assert call(**both) == ALIGN


def test_written_rows_may_not_overlap(mmq_lib):
    unsupported_or_launched = (OK, UNSUPPORTED)
    for kw in (dict(token_stride=0), dict(head_stride=0), dict(token_stride=200), dict(token_stride=64, head_stride=64)):
        assert read(v=rows(**kw)) == ARG, kw
        assert attend(out=rows(**kw)) == ARG, kw
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses below are no memory")
    # heads outside tokens, gaps, and (for rows that are only read) broadcasts
    for kw in (dict(token_stride=128, head_stride=512), dict(token_stride=300, head_stride=130)):
        assert read(v=rows(**kw)) in unsupported_or_launched, kw
        assert attend(out=rows(**kw)) in unsupported_or_launched, kw
    assert write(k=rows(token_stride=0), v=rows(head_stride=0)) in unsupported_or_launched


def test_counts_scale_window_and_workspace(mmq_lib):
    assert write(n=-1) == SHAPE and read(n=(1 << 22) + 1) == SHAPE and attend(n=-1) == SHAPE
    for kw, st in ((dict(heads=3), SHAPE), (dict(heads=0), SHAPE), (dict(heads=2048), SHAPE), (dict(scale=0.0), ARG),
                   (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
                   (dict(window=-1), ARG), (dict(sinks=-1), ARG), (dict(max_q=-1), ARG), (dict(max_kv=-1), ARG)):
        assert attend(**kw) == st, kw
    # a call that is cut into parts needs its workspace
    many = dict(c=cache(max_pages=4096), n=1, max_q=1, max_kv=4096 * 64)
    need = mmq.mmq_kv_attend_workspace_bytes(many["c"], 0, 2, 1, 1, 4096 * 64)
    assert need > 0 and need % 16 == 0
    assert attend(**many, ws=None) == ARG
    assert attend(**many, size=need - 1) == ARG
    assert attend(**many, ws=P16 + 8) == ALIGN
    assert mmq.load().mmq_kv_attend_workspace_bytes(many["c"], 0, 2, 1, 1, 64, 0, 0, None) == ARG
    assert mmq.load().mmq_kv_attend_workspace_bytes(None, 0, 2, 1, 1, 64, 0, 0,
                                                    ctypes.byref(ctypes.c_size_t())) == ARG


def test_no_rows_is_no_work(mmq_lib):
    before = mmq.mmq_launch_count()
    assert write(n=0) == OK and read(n=0) == OK and attend(n=0, ws=None, size=0) == OK
    assert mmq.mmq_kv_attend_workspace_bytes(cache(), 0, 2, 0, 1, 64) == 0
    assert mmq.mmq_launch_count() == before


def test_without_a_gpu_calls_are_unsupported(mmq_lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert write() == UNSUPPORTED and read() == UNSUPPORTED and attend() == UNSUPPORTED


def test_tensor_helpers_refuse(mmq_lib):
    import torch
    pages = mmq.kv_pages(4, 2, 64, device="cpu")
    assert pages.shape == (4, 2, 4608) and pages.dtype == torch.uint8
    table, start, length = (torch.zeros(s, dtype=torch.int32) for s in ((1, 4), (2,), (1,)))
    x = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        mmq.kv_write(x, x, pages, table, start, length)
    for bad, what in (((pages.float(), table, start, length), "pages"), ((pages[..., :-1], table, start, length), "pages"),
                      ((pages, table.long(), start, length), "table"), ((pages, table[0], start, length), "table"),
                      ((pages, table, start[:1], length), "start"), ((pages, table, start, length.long()), "length"),
                      ((pages, table, start, start), "length")):
        for call in (lambda c: mmq.kv_write(x, x, *c), lambda c: mmq.kv_read(*c, 3), lambda c: mmq.kv_attend(x, *c, 3)):
            with pytest.raises(ValueError, match=what):
                call(bad)


@pytest.mark.parametrize("heads,kv_heads,dim,batch,new,dtype", [(32, 8, 128, 64, 1, 2), (4, 2, 128, 2, 2, 0),
                                                                (32, 8, 128, 1, 16384, 1), (1, 1, 64, 1, 1, 0)])
@pytest.mark.parametrize("max_pages", [1, 79, 2048])
def test_a_length_hint_past_the_table_counts_as_the_table(mmq_lib, heads, kv_heads, dim, batch, new, dtype, max_pages):
    """No sequence has more keys than its row of the table has pages for, so a larger max_kv cuts
    the work no finer and asks for no more workspace."""
    c = cache(kv_heads=kv_heads, head_dim=dim, batch=batch, max_pages=max_pages)

    def need(max_kv):
        return mmq.mmq_kv_attend_workspace_bytes(c, dtype, heads, batch * new, new, max_kv)

    assert need(1 << 30) == need((1 << 31) - 1) == need(64 * max_pages)
    # a part holds 4 pages or more: sums, reference and weight of each row for so many parts at most
    assert need(1 << 30) <= (max_pages // 4 + 1) * batch * new * heads * (4 * dim + 8) + 16


def test_the_size_query_checks_the_tables_width(mmq_lib):
    for max_pages in (0, -1, (1 << 24) + 1):
        with pytest.raises(mmq.MMQError) as e:
            mmq.mmq_kv_attend_workspace_bytes(cache(max_pages=max_pages), 0, 2, 4, 4, 256)
        assert e.value.status == SHAPE


def test_tensors_of_another_device_than_the_current_are_refused(mmq_lib, monkeypatch):
    """The library launches on the current device.  The tensors here are host memory that claims to
    be on cuda:1; the library is replaced too, so that nothing can reach a GPU."""
    import torch

    class OnOne(torch.Tensor):
        def get_device(self):
            return 1

    def at(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnOne)

    class Stream:
        def __init__(self, device):
            self.device_index, self.cuda_stream = device, 0

    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(mmq, "_lib", Library())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    x = at(3, 2, 64, dtype=torch.float32)
    cache = at(4, 2, 72 * 64, dtype=torch.uint8), at(1, 4), at(2), at(1)

    def everything(stream):
        yield lambda: mmq.kv_write(x, x, *cache, stream=stream)
        yield lambda: mmq.kv_read(*cache, 3, k=x, v=x, stream=stream)
        yield lambda: mmq.kv_attend(x, *cache, 3, out=x, stream=stream)

    for current, stream, what in ((0, None, "current device"), (0, Stream(0), "current device"),
                                  (0, Stream(1), "current device"), (1, Stream(0), "stream")):
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
        for call in everything(stream):
            with pytest.raises(ValueError, match=what):
                call()
    assert calls == []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    for stream in (None, Stream(1)):
        for call in everything(stream):
            call()
    assert calls == ["mmq_kv_write", "mmq_kv_read", "mmq_kv_attend"] * 2


def test_rows_without_an_address_are_no_rows(mmq_lib):
    """An empty tensor's data pointer is null; a call on it is as little work as on any other."""
    before = mmq.mmq_launch_count()
    none = rows(data=None)
    assert write(k=none, v=none, n=0) == OK and read(k=none, v=none, n=0) == OK
    assert attend(q=none, out=none, n=0, ws=None, size=0) == OK
    assert mmq.mmq_launch_count() == before
    assert write(k=none, n=1) == ARG and read(v=none, n=1) == ARG and attend(out=none, n=1) == ARG


def test_numbers_past_32_bits_are_not_cut_off(mmq_lib, monkeypatch):
    """A window of 2^32 is a wide one, not none.  Host memory that claims to be on a device, and no
    library behind it."""
    import torch

    class OnZero(torch.Tensor):
        def get_device(self):
            return 0

    def at(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnZero)

    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: seen.append(a) or 0

    monkeypatch.setattr(mmq, "_lib", Library())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    x = at(3, 2, 64, dtype=torch.float32)
    cache = at(4, 2, 72 * 64, dtype=torch.uint8), at(1, 4), at(2), at(1)
    big = (1 << 31) - 1
    for given, taken in (((3, 70, 5, 1), (3, 70, 5, 1)), ((1 << 32, 70, 0, 1 << 33), (big, 70, 0, big)),
                         ((3, (1 << 40) + 1, (1 << 32) + 7, 1 << 31), (3, big, big, big)), ((3, 70, -1, 0), (3, 70, -1, 0))):
        max_q, max_kv, window, sinks = given
        mmq.kv_attend(x, *cache, max_q, max_kv, window=window, sinks=sinks, out=x)
        a = seen.pop()
        assert (a[5], a[6], a[8], a[9]) == taken
    many = x[:1].expand((1 << 32) + 1, 2, 64).as_subclass(OnZero)
    with pytest.raises(ValueError, match="rows"):
        mmq.kv_write(many, many, *cache)
    assert seen == []
