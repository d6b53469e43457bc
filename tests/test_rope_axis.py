"""Which position turns which pair, where the axes are interleaved over the
pairs (no GPU: what the descriptor holds)."""
import pytest

import draft_token_verification_sv_gb300 as sv

from test_kv_arguments import Stand, _ints, _library  # noqa: F401


@pytest.fixture
def axes_of(monkeypatch):
    made = []
    monkeypatch.setattr(sv.prompt, "_call", lambda device, entry, desc, *args: made.append((desc._obj.axes, list(desc._obj.axis[:32]))))
    monkeypatch.setattr(sv.kvcache, "_raw_stream", lambda index: 0)

    def call(axes, **kw):
        rows = Stand((7, 4, 64))
        sv.rope(rows, None, _ints(7) if axes == 1 else _ints(axes, 7), Stand((32,)), out=(rows, None), **kw)
        return made[-1]
    return call


@pytest.mark.parametrize("axis", [[i % 3 for i in range(32)], [2] * 32, [0] * 20 + [1, 2] * 6])
def test_an_axis_for_each_pair(axes_of, axis):
    assert axes_of(3, axis=axis) == (3, axis) and axes_of(3, axis=tuple(axis)) == (3, axis)


def test_sections_are_the_same_in_order(axes_of):
    assert axes_of(3, sections=(8, 12, 12)) == axes_of(3, axis=[0] * 8 + [1] * 12 + [2] * 12)
    assert axes_of(1) == axes_of(1, axis=[0] * 32) == (1, [0] * 32)


@pytest.mark.parametrize("axes,kw", [(3, dict(axis=[0] * 31)), (3, dict(axis=[0] * 33)), (3, dict(axis=[0] * 31 + [3])), (3, dict(axis=[-1] + [0] * 31)),
                                     (1, dict(axis=[1] * 32)), (3, dict(axis=[])), (3, dict(axis=[0] * 32, sections=(32, 0, 0))), (3, {})],
                         ids=range(8))
def test_refused(axes_of, axes, kw):
    with pytest.raises(ValueError):
        axes_of(axes, **kw)
