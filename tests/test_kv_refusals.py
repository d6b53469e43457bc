"""Refusals of the cache's C entry points beyond those of single arguments (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def N():
    from draft_token_verification_sv_gb300 import build as b
    b.build()
    from draft_token_verification_sv_gb300 import _native
    _native.lib()
    return _native


def _kv(N):
    return N.KvDesc(4, 2, 64, 16, 100, 8, 2 * 16 * 64, 16 * 64, 64, 10)


@pytest.mark.parametrize("place", [dict(ctx=0), dict(ctx=12), dict(ctx=-12), dict(accept=0), dict(accept=4), dict(path=0),
                                   dict(path=-60), dict(path=12), dict(table=0), dict(table=-148), dict(table=12)],
                         ids=lambda p: "".join(f"{k}{v}" for k, v in p.items()))
def test_commit_refuses_new_lengths_over_its_inputs(N, place):
    """4 sequences, paths of 4 nodes, page table rows of 8 entries 10 apart: `place` is how many bytes an input begins behind new_lens."""
    new = 0x200000
    at = {n: ctypes.c_void_p(new + place[n] if n in place else 0x100000) for n in ("table", "ctx", "path", "accept")}
    A = ctypes.c_void_p(0x100000)
    assert N.lib().sv_kv_commit(ctypes.byref(_kv(N)), 8, 4, at["table"], at["ctx"], at["path"], at["accept"], A, A, A, A,
                                ctypes.c_void_p(new), None, None) == N.SV_ERR_INVALID_ARGUMENT


A, MIS = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100002)


@pytest.mark.parametrize("i", range(3))
def test_append_and_read_refuse_words_off_their_boundary(N, i):
    """ctx_lens (first), new_start, row_status."""
    rows = N.KvRowsDesc(3, 12, N.SV_BF16, 0, 128, 64, 128, 64)
    w = [MIS if j == i else (A if j == 0 else None) for j in range(3)]
    assert N.lib().sv_kv_append(ctypes.byref(_kv(N)), ctypes.byref(rows), A, A, A, w[0], w[1], A, A, A, A, w[2], None) == N.SV_ERR_INVALID_ARGUMENT
    assert N.lib().sv_kv_read(ctypes.byref(_kv(N)), ctypes.byref(rows), A, A, A, A, A, w[0], w[1], A, A, w[2], None) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("i", range(5))
def test_commit_refuses_words_off_their_boundary(N, i):
    """ctx_lens, path, accept_len, new_lens, row_status."""
    w = [A, A, A, ctypes.c_void_p(0x200000), None]
    w[i] = ctypes.c_void_p(0x300002)
    assert N.lib().sv_kv_commit(ctypes.byref(_kv(N)), 8, 4, A, w[0], w[1], w[2], A, A, A, A, w[3], w[4], None) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("i", range(5))
def test_attention_refuses_words_off_their_boundary(N, i):
    """ctx_lens, new_start, parents, lse, row_status."""
    a = N.KvAttentionDesc(_kv(N), 8, 3, 12, N.SV_BF16, 0.125, 0, 0, 0, 512, 64, 512, 64)
    w = [MIS if j == i else (A if j == 0 else None) for j in range(5)]
    assert N.lib().sv_kv_attention(ctypes.byref(a), A, A, A, A, A, A, w[0], w[1], w[2], A, w[3], w[4], A, ctypes.c_size_t(1 << 40),
                                   None) == N.SV_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("max_new,group", [(2 ** 31 - 1, 1), (2 ** 31 - 128, 1), (2 ** 29, 4), (2 ** 24, 128)])
def test_more_rows_than_32_bits_count_are_refused(N, max_new, group):
    """Rounded up to whole tiles of up to 128 rows; one row less is taken."""
    a = N.KvAttentionDesc(_kv(N), 2 * group, max_new, 12, N.SV_BF16, 0.125, 0, 0, 0, 512, 64, 512, 64)
    assert N.lib().sv_kv_attention_workspace_size(ctypes.byref(a)) == 0
    a.max_new = (2 ** 31 - 129) // group
    assert N.lib().sv_kv_attention_workspace_size(ctypes.byref(a)) > 0
