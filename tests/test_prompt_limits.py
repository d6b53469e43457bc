"""max_new of packed prompts is a bound that may be any (no GPU: what the
descriptor holds)."""
import pytest

import draft_token_verification_sv_gb300 as sv

from test_kv_arguments import Stand, _ints, _library  # noqa: F401


def _max_new(monkeypatch, **kw):
    made = []
    monkeypatch.setattr(sv.prompt, "_call", lambda device, entry, desc, *args: made.append(desc._obj.max_new))
    monkeypatch.setattr(sv.kvcache, "_raw_stream", lambda index: 0)
    args = dict(q=Stand((12, 8, 64)), k=Stand((12, 2, 64)), v=Stand((12, 2, 64)), out=Stand((12, 8, 64)), new_start=_ints(5))
    args.update(kw)
    sv.prompt_attention(**args)
    return made[0]


@pytest.mark.parametrize("max_new,want", [(2 ** 31 - 1, 12), (1 << 30, 12), (13, 12), (12, 12), (11, 11), (0, 0), (-1, -1)])
def test_a_packed_call_s_bound_is_its_rows_at_most(monkeypatch, max_new, want):
    """(A sequence of more tokens than there are rows is left out either way; a negative bound is the library's to refuse.)"""
    assert _max_new(monkeypatch, max_new=max_new) == want


@pytest.mark.parametrize("heads", [8, 128])
def test_no_bound_is_no_refusal(monkeypatch, heads):
    assert _max_new(monkeypatch, max_new=2 ** 31 - 1, q=Stand((12, heads, 64)), out=Stand((12, heads, 64)), k=Stand((12, 1, 64)), v=Stand((12, 1, 64))) * heads < 2 ** 31 - 256


def test_more_than_32_bits_are_refused(monkeypatch):
    with pytest.raises(ValueError):
        _max_new(monkeypatch, max_new=2 ** 31)


def test_a_padded_call_has_its_own(monkeypatch):
    rows = {n: Stand((4, 3, h, 64)) for n, h in (("q", 8), ("k", 2), ("v", 2), ("out", 8))}
    assert _max_new(monkeypatch, new_start=None, **rows) == 3
