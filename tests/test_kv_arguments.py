"""What the Python layer of the cache refuses and how it passes tensors on
(no GPU: stand-ins that have a tensor's shape, strides, type and place)."""
import math

import pytest
import torch

import draft_token_verification_sv_gb300 as sv
from draft_token_verification_sv_gb300 import build as _build


@pytest.fixture(scope="module", autouse=True)
def _library():
    _build.build()


class Stand:
    """A CUDA tensor as the argument checks see it."""

    def __init__(self, shape, dtype=torch.float32, strides=None, device="cuda:0", address=1 << 20):
        self.shape, self.dtype, self._address = torch.Size(shape), dtype, address
        self._strides = strides or tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))
        self.device = torch.device(device)
        self.is_cuda = self.device.type == "cuda"

    def stride(self):
        return self._strides

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def is_contiguous(self):
        return self._strides == tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def data_ptr(self):
        return self._address

    def numel(self):
        return self.shape.numel()


def _ints(*shape, **kw):
    return Stand(shape, torch.int32, **kw)


def _cache(**kw):
    codes = lambda: Stand((9, 2, 16, 64), torch.uint8, **kw)
    scales = lambda: Stand((9, 2), **kw)
    return dict(k=codes(), v=codes(), k_scale=scales(), v_scale=scales())


def _calls(table, cache=None, **kw):
    """The four entry points on 4 sequences of 3 new tokens, as functions."""
    cache = cache or _cache()
    rows = lambda heads: Stand((4, 3, heads, 64))
    return {
        "append": lambda: sv.kv_append(cache, rows(2), rows(2), table, _ints(4), **kw),
        "read": lambda: sv.kv_read(cache, table, _ints(4), 3, out=(rows(2), rows(2)), **kw),
        "commit": lambda: sv.kv_commit(cache, table, _ints(4), _ints(4, 5), _ints(4), 8, new_lens=_ints(4), **kw),
        "attention": lambda: sv.kv_attention(rows(8), cache, table, _ints(4), out=rows(8),
                                             ws=Stand((1 << 30,), torch.uint8), **kw),
    }


CALLS = ("append", "read", "commit", "attention")


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("strides", [(0, 1), (4, 1), (1, 1)])
def test_rows_of_a_page_table_that_overlap_are_refused(call, strides):
    """An expanded row of page ids is not five rows of memory."""
    with pytest.raises(ValueError, match="page_table"):
        _calls(_ints(4, 5, strides=strides))[call]()


@pytest.fixture
def fake_streams(monkeypatch):
    """torch's streams and allocations replaced by stand-ins: yields the list
    of (stream that memory was allocated on, streams recorded on it)."""
    import contextlib

    from draft_token_verification_sv_gb300 import _native as N
    current, made = ["main"], []

    class Fake:
        def __init__(self, name):
            self.name, self.cuda_stream, self.device_index = name, hash(name) & 0xffff, 0

    class Made(Stand):
        def record_stream(self, stream):
            made[self.at][1].append(stream.name)

    @contextlib.contextmanager
    def on(stream):
        current.append(stream.name)
        yield
        current.pop()

    def allocate(shape, dtype=torch.float32, device="cuda:0"):
        t = Made((shape,) if isinstance(shape, int) else shape, dtype)
        t.at = len(made)
        made.append((current[-1], []))
        return t
    class Lib:
        def __getattr__(self, name):
            return lambda *args: 1000 if name.endswith("size") else N.SV_OK
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Fake("main"))
    monkeypatch.setattr(sv.kvcache, "_current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(torch, "zeros", allocate)
    monkeypatch.setattr(sv.kvcache, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(N, "lib", Lib)
    monkeypatch.setattr(sv.verify, "_WORKSPACES", {})
    monkeypatch.setattr(sv.kvcache, "_WORKSPACES", sv.verify._WORKSPACES)
    for plan in (sv.kvcache._append_plan, sv.kvcache._read_plan, sv.kvcache._commit_plan, sv.kvcache._attention_plan):
        plan.cache_clear()
    yield Fake, made
    sv.kvcache._attention_plan.cache_clear()


def test_results_and_workspaces_belong_to_the_calls_stream(fake_streams):
    """With stream=, memory is allocated there (a fill of the workspace and
    earlier users of the memory are then ordered with the call), and results
    are kept until the current stream is done with them."""
    Fake, made = fake_streams
    side, cache, q = Fake("side"), _cache(), Stand((4, 3, 8, 64))
    sv.kv_attention(q, cache, _ints(4, 5), _ints(4), lse=True, stream=side)
    assert sorted(made) == [("side", []), ("side", ["main"]), ("side", ["main"])]  # workspace, out, lse
    made.clear()
    sv.kv_attention(q, cache, _ints(4, 5), _ints(4), lse=True, stream=side)
    assert made == [("side", ["main"])] * 2
    made.clear()
    sv.kv_read(cache, _ints(4, 5), _ints(4), 3, stream=side)
    sv.kv_commit(cache, _ints(4, 5), _ints(4), _ints(4, 5), _ints(4), 8, stream=side)
    assert made == [("side", ["main"])] * 3


@pytest.mark.parametrize("what,call", [
    ("window", lambda c, q, x: sv.kv_attention(q, c, _ints(4, 5), _ints(4), window=2 ** 32 + 1)),
    ("sinks", lambda c, q, x: sv.kv_attention(q, c, _ints(4, 5), _ints(4), window=8, sinks=2 ** 32)),
    ("max_new", lambda c, q, x: sv.kv_append(c, x, x, _ints(4, 5), _ints(4), new_start=_ints(5), max_new=2 ** 32 + 3)),
    ("tokens", lambda c, q, x: sv.kv_read(c, _ints(4, 5), _ints(4), 2 ** 32 + 3, new_start=_ints(5), out=(x, x))),
    ("nodes", lambda c, q, x: sv.kv_commit(c, _ints(4, 5), _ints(4), _ints(4, 5), _ints(4), 2 ** 32 + 8, new_lens=_ints(4))),
    ("rows", lambda c, q, x: sv.kv_append(c, Stand((2 ** 32 + 1, 2, 64)), Stand((2 ** 32 + 1, 2, 64)), _ints(4, 5), _ints(4),
                                          new_start=_ints(5), max_new=1))])
def test_numbers_beyond_32_bits_are_refused(fake_streams, what, call):
    """They lost their upper bits on the way into the descriptors (a window of 2^32 + 1 became one of 1)."""
    with pytest.raises(ValueError, match="32 bits"):
        call(_cache(), Stand((4, 3, 8, 64)), Stand((12, 2, 64)))


OTHER = dict(device="cuda:1")


@pytest.mark.parametrize("what", ["table", "lens", "cache", "q", "parents", "status", "out"])
def test_tensors_of_two_gpus_are_refused(what):
    place = lambda name: OTHER if name == what else {}
    with pytest.raises(ValueError, match="one GPU"):
        sv.kv_attention(Stand((4, 3, 8, 64), **place("q")), _cache(**place("cache")), _ints(4, 5, **place("table")),
                        _ints(4, **place("lens")), parents=_ints(4, 3, **place("parents")), out=Stand((4, 3, 8, 64), **place("out")),
                        row_status=_ints(4, **place("status")), ws=Stand((1 << 30,), torch.uint8))


@pytest.mark.parametrize("ws", [Stand((1 << 30,), torch.uint8, device="cpu"), Stand((1 << 30,), torch.uint8, **OTHER),
                                Stand((1 << 30,), torch.uint8, strides=(0,))],
                         ids=["host", "other GPU", "expanded"])
def test_workspaces_the_call_cannot_write_are_refused(monkeypatch, ws):
    monkeypatch.setattr(sv.kvcache, "_raw_stream", lambda index: 0)
    with pytest.raises(ValueError, match="ws"):
        sv.kv_attention(Stand((4, 3, 8, 64)), _cache(), _ints(4, 5), _ints(4), out=Stand((4, 3, 8, 64)), ws=ws)


def test_the_tensors_gpu_is_made_current(fake_streams, monkeypatch):
    import contextlib
    entered = []

    @contextlib.contextmanager
    def device(index):
        entered.append(index)
        yield
    monkeypatch.setattr(torch.cuda, "device", device)
    x, one = Stand((4, 3, 2, 64), **OTHER), lambda *shape: _ints(*shape, **OTHER)
    sv.kv_append(_cache(**OTHER), x, x, one(4, 5), one(4))
    assert entered == [1]
    sv.kv_append(_cache(), Stand((4, 3, 2, 64)), Stand((4, 3, 2, 64)), _ints(4, 5), _ints(4))
    assert entered == [1]
    with pytest.raises(ValueError, match="stream"):
        sv.kv_append(_cache(**OTHER), x, x, one(4, 5), one(4), stream=fake_streams[0]("side"))
