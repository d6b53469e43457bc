"""What the Python layer of the cache refuses and how it passes tensors on
(no GPU: stand-ins that have a tensor's shape, strides, type and place)."""
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
        t = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype, self._strides, self._address = t.shape, dtype, strides or t.stride(), address
        self.device = torch.device(device)
        self.is_cuda = self.device.type == "cuda"

    def stride(self):
        return self._strides

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
