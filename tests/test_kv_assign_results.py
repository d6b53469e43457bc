"""Results that a caller of kv_assign brings: both or none, each of the type
and size that the kernels write (no GPU: nothing may get as far as a launch)."""
import pytest
import torch

import draft_token_verification_sv_gb300 as sv

from test_kv_arguments import Stand, _ints, _library  # noqa: F401
from test_prompt_refusals import _assign_py


@pytest.fixture(autouse=True)
def called(monkeypatch):
    """What reaches the library."""
    made = []
    monkeypatch.setattr(sv.kvcache, "_call", lambda device, entry, *args: made.append(entry))
    monkeypatch.setattr(sv.kvcache, "_raw_stream", lambda index: 0)
    return made


SLOTS, POSITIONS = Stand((4, 3), torch.int64), _ints(4, 3)
ONE = [(None, POSITIONS), (None, _ints(1)), (None, Stand((12,), torch.int16)), (None, Stand((12,), torch.int64)),
       (None, _ints(4, 3, strides=(6, 2))), (None, _ints(4, 3, device="cpu")), (SLOTS, None), (Stand((1,), torch.int64), None), (None, None)]


@pytest.mark.parametrize("out", ONE, ids=range(len(ONE)))
@pytest.mark.parametrize("kw", [{}, dict(max_new=0), dict(new_start=_ints(5), total=12), dict(new_start=_ints(5), total=0, max_new=0)], ids=range(4))
def test_one_result_alone_is_refused(called, out, kw):
    with pytest.raises(ValueError):
        _assign_py(out=out, **kw)()
    assert not called


@pytest.mark.parametrize("kw", [{}, dict(new_start=_ints(5)), dict(new_start=_ints(5), total=12)], ids=range(3))
def test_both_are_taken(called, kw):
    got = _assign_py(out=(SLOTS, POSITIONS), **kw)()
    assert called == ["sv_kv_assign"] and got == dict(slots=SLOTS, positions=POSITIONS)


@pytest.mark.parametrize("out", [(Stand((4, 2), torch.int64), _ints(4, 2)), (Stand((12,), torch.int64), _ints(4, 3)), (SLOTS, Stand((4, 3), torch.int16)),
                                 (Stand((4, 3), torch.int32), POSITIONS), (SLOTS, _ints(4, 3, strides=(6, 2))), (SLOTS, _ints(4, 3, device="cpu"))],
                         ids=range(6))
def test_of_both_each_is_checked(called, out):
    with pytest.raises(ValueError):
        _assign_py(out=out)()
    assert not called
