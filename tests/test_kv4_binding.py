"""The Python side of the 4-bit cache without a GPU: stand-ins for device tensors, a library that records its calls."""
import contextlib
import math
import types

import pytest
import torch

import entropy_coding_02_amd as kvc

STREAMS = []  # what torch.cuda.stream has entered, innermost last


class Fake:
    """What the binding asks of a device tensor.  `home`: the stream that was current when it was made."""
    made = 0

    def __init__(self, shape, dtype, device=0, strides=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", device)
        if strides is None:
            strides = [math.prod(shape[i + 1:]) for i in range(len(shape))]
        self.strides, self.is_cuda = tuple(strides), True
        Fake.made += 1
        self.address = Fake.made << 32
        self.home = STREAMS[-1] if STREAMS else None

    def dim(self): return len(self.shape)
    def numel(self): return self.shape.numel()
    def element_size(self): return torch.empty(0, dtype=self.dtype).element_size()
    def stride(self, i=None): return self.strides if i is None else self.strides[i]
    def data_ptr(self): return self.address
    def get_device(self): return self.device.index

    def is_contiguous(self):
        return self.strides == Fake(self.shape, self.dtype).strides

    def new_empty(self, shape, dtype=None):
        t = Fake(shape if isinstance(shape, (tuple, torch.Size)) else (shape,), dtype or self.dtype, self.device.index)
        ALLOCATED.append(t)
        return t


ALLOCATED = []


@pytest.fixture
def calls(monkeypatch):
    """The launches of the library, as (name, arguments); sizes come from the library itself."""
    real, made = kvc._load(), []

    def record(name):
        return lambda *a: made.append((name, a)) or kvc.KVC_OK

    lib = types.SimpleNamespace(**{n: getattr(real, n) for n in kvc.EXPORTED})
    for n in ("kvc_kv4_append", "kvc_kv4_read", "kvc_kv4_attention"):
        setattr(lib, n, record(n))

    @contextlib.contextmanager
    def stream(s):
        STREAMS.append(s)
        yield
        STREAMS.pop()

    monkeypatch.setattr(kvc, "_load", lambda: lib)
    monkeypatch.setattr(kvc, "_RAW_STREAM", lambda i: 77 + i)
    monkeypatch.setattr(kvc, "_CURRENT_DEVICE", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: types.SimpleNamespace(cuda_stream=h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0))
    ALLOCATED.clear()
    return made


def pool(H=2, D=64, P=64, n=200, G=64, device=0):
    return kvc.Kv4Cache(H, D, n, page_tokens=P, group=G,
                        codes=Fake((n, 2, H, P * D // 2), torch.uint8, device),
                        params=Fake((n, 2, H, D // G, P, 2), torch.float16, device),
                        dev_status=Fake((1,), torch.int32, device))


def attention(cache, **kw):
    """One query over a table of 200 pages: split, so that a workspace is wanted."""
    a = dict(q=Fake((1, 4, cache.head_dim), torch.float16), page_table=Fake((1, 200), torch.int32),
             kv_len=Fake((1,), torch.int32))
    a.update(kw)
    return kvc.kv4_attention(cache, a.pop("q"), a.pop("page_table"), a.pop("kv_len"), **a)


@pytest.mark.parametrize("handle", [False, True])
def test_what_a_call_allocates_belongs_to_its_stream(calls, handle):
    s = types.SimpleNamespace(cuda_stream=1234)
    attention(pool(), return_lse=True, stream=1234 if handle else s)
    kvc.kv4_read(pool(), Fake((5,), torch.int64), stream=1234 if handle else s)
    assert len(ALLOCATED) == 5  # out, lse, workspace; k, v
    assert all(t.home is not None and t.home.cuda_stream == 1234 for t in ALLOCATED)
    assert all(a[-1] == 1234 for _, a in calls)


def test_without_a_stream_the_current_one_is_used(calls):
    attention(pool(), return_lse=True)
    kvc.kv4_read(pool(), Fake((5,), torch.int64))
    assert len(ALLOCATED) == 5 and all(t.home is None for t in ALLOCATED)
    assert all(a[-1] == 77 for _, a in calls)
    attention(pool(), stream=0)  # the default stream's handle
    assert calls[-1][1][-1] == 0 and ALLOCATED[-1].home.cuda_stream == 0


def launched(calls, n=1):
    return [a for _, a in calls[-n:]]


def test_an_assigned_buffer_is_the_one_used(calls):
    cache = pool()
    new = Fake(cache.codes.shape, torch.uint8), Fake(cache.params.shape, torch.float16), Fake((1,), torch.int32)
    cache.codes, cache.params, cache.dev_status = new
    assert (cache.codes, cache.params, cache.dev_status) == new
    slots, rows = Fake((5,), torch.int64), (Fake((5, 2, 64), torch.float16), Fake((5, 2, 64), torch.float16))
    kvc.kv4_append(cache, *rows, slots)
    kvc.kv4_read(cache, slots)
    attention(cache)
    for args in launched(calls, 3):
        for t in new:
            assert t.data_ptr() in args


@pytest.mark.parametrize("name,bad", [
    ("codes", lambda c: Fake((1,), torch.uint8)), ("codes", lambda c: Fake(c.codes.shape, torch.int8)),
    ("codes", lambda c: Fake(c.codes.shape, torch.uint8, strides=(1, 1, 1, 1))),
    ("params", lambda c: Fake((1,), torch.float16)), ("params", lambda c: Fake(c.params.shape, torch.bfloat16)),
    ("codes", lambda c: torch.empty(c.codes.shape, dtype=torch.uint8)),
    ("dev_status", lambda c: Fake((1,), torch.int64)), ("dev_status", lambda c: Fake((0,), torch.int32)),
    ("dev_status", lambda c: torch.zeros(1, dtype=torch.int32))])
def test_an_assigned_buffer_is_checked(calls, name, bad):
    cache = pool()
    kept = getattr(cache, name)
    with pytest.raises(ValueError):
        setattr(cache, name, bad(cache))
    assert getattr(cache, name) is kept and kept.data_ptr() in (cache.codes_ptr, cache.params_ptr, cache.status_ptr)


@pytest.mark.parametrize("strides", [(0, 64, 1), (128, 0, 1), (128, 63, 1), (-63, 640, 1), (0, 0, 1)])
def test_written_rows_may_not_overlap(calls, strides):
    cache = pool()
    ok = Fake((2, 2, 64), torch.float16)
    bad = Fake((2, 2, 64), torch.float16, strides=strides)
    for kw in (dict(k=bad, v=ok), dict(k=ok, v=bad)):
        with pytest.raises(ValueError):
            kvc.kv4_read(cache, Fake((2,), torch.int64), **kw)
    with pytest.raises(ValueError):
        attention(cache, q=ok, page_table=Fake((2, 9), torch.int32), kv_len=Fake((2,), torch.int32), out=bad)
    assert not calls
    kvc.kv4_append(cache, bad, bad, Fake((2,), torch.int64))  # what is only read may be broadcast
    attention(cache, q=bad, page_table=Fake((2, 9), torch.int32), kv_len=Fake((2,), torch.int32), out=ok)
    assert len(calls) == 2


def test_strides_that_no_row_uses_and_negative_ones(calls):
    cache = pool(H=1)
    kvc.kv4_read(cache, Fake((3,), torch.int64), k=Fake((3, 1, 64), torch.float16, strides=(-64, 0, 1)),
                 v=Fake((3, 1, 64), torch.float16, strides=(64, 1, 1)))
    kvc.kv4_read(cache, Fake((1,), torch.int64), k=Fake((1, 1, 64), torch.float16, strides=(0, 0, 1)),
                 v=Fake((1, 1, 64), torch.float16, strides=(1, 64, 1)))
    assert len(calls) == 2


def test_tensors_of_another_device_are_refused(calls):
    cache, f16, i32, i64 = pool(), torch.float16, torch.int32, torch.int64
    here, there = Fake((2, 2, 64), f16), Fake((2, 2, 64), f16, device=1)
    for call in (lambda: kvc.kv4_append(cache, there, here, Fake((2,), i64)),
                 lambda: kvc.kv4_append(cache, here, there, Fake((2,), i64)),
                 lambda: kvc.kv4_append(cache, here, here, Fake((2,), i64, device=1)),
                 lambda: kvc.kv4_read(cache, Fake((2,), i64, device=1)),
                 lambda: kvc.kv4_read(cache, Fake((2,), i64), k=there, v=here),
                 lambda: attention(cache, q=Fake((1, 4, 64), f16, device=1)),
                 lambda: attention(cache, out=Fake((1, 4, 64), f16, device=1)),
                 lambda: attention(cache, lse=Fake((1, 4), torch.float32, device=1)),
                 lambda: attention(cache, page_table=Fake((1, 200), i32, device=1)),
                 lambda: attention(cache, kv_len=Fake((1,), i32, device=1)),
                 lambda: attention(cache, cu_q=Fake((2,), i32, device=1), max_q=1),
                 lambda: attention(cache, work=Fake((1 << 20,), torch.uint8, device=1)),
                 lambda: setattr(cache, "codes", Fake(cache.codes.shape, torch.uint8, device=1)),
                 lambda: setattr(cache, "params", Fake(cache.params.shape, f16, device=1)),
                 lambda: setattr(cache, "dev_status", Fake((1,), i32, device=1))):
        with pytest.raises(ValueError):
            call()
    assert not calls


def test_the_cache_s_device_is_current_at_the_launch(calls, monkeypatch):
    entered = []

    @contextlib.contextmanager
    def device(i):
        entered.append(i)
        n = len(calls)
        yield
        assert len(calls) == n + 1

    monkeypatch.setattr(torch.cuda, "device", device)
    cache = pool(device=1)
    rows = Fake((2, 2, 64), torch.float16, device=1)
    kvc.kv4_append(cache, rows, rows, Fake((2,), torch.int64, device=1))
    assert entered == [1] and calls[-1][1][-1] == 78  # the current stream of that device
    kvc.kv4_append(pool(), Fake((2, 2, 64), torch.float16), Fake((2, 2, 64), torch.float16), Fake((2,), torch.int64))
    assert entered == [1] and calls[-1][1][-1] == 77
