"""The cache's entry points at the ends of what they take."""
import numpy as np
import pytest

from oracle import kv_oracle as KO

from _kv import cache_gpu, copy, make_cache, make_table, same_cache, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


def test_commit_of_zeros_out_of_a_page_of_huge_values(sv):
    """Zeros on a page whose scale is 2^40 become a page of their own, whose
    scale is 2^-100: the quotient of the two is beyond float32."""
    g = np.random.default_rng(0)
    page, dim, heads, ctx, nodes = 16, 32, 2, 32, 20
    table, pages = make_table(g, [ctx + nodes], page)
    cache = make_cache(g, pages, heads, page, dim)
    cache["k_scale"][table[0, 2]] = 2.0 ** 40
    cache["v_scale"][table[0, 2]] = 2.0 ** 90
    for name in ("k", "v"):
        cache[name][table[0, 2], :, :6] = 0
        cache[name][table[0, 2], :, 1, ::2] = 0x80  # -0
    path = np.array([[0, 1, 3, 5]], np.int32)
    want, dev = copy(cache), cache_gpu(cache)
    KO.commit(want, table[0], page, ctx, path[0])
    new = sv.kv_commit(dev, to_gpu(table), to_gpu(np.array([ctx], np.int32)), to_gpu(path), to_gpu(np.array([3], np.int32)), nodes)
    assert new.tolist() == [ctx + 4]
    same_cache(dev, want)


@pytest.mark.parametrize("call", ["append", "read", "attention"])
@pytest.mark.parametrize("ragged", [False, True])
def test_lengths_are_flagged_without_new_tokens_too(sv, call, ragged):
    import torch
    g = np.random.default_rng(0)
    table, pages = make_table(g, [32] * 5, 16)
    dev = cache_gpu(make_cache(g, pages, 2, 16, 64))
    lens = to_gpu(np.array([0, -1, 32, 33, 5], np.int32))
    st = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    rows = lambda heads: torch.empty((0, heads, 64) if ragged else (5, 0, heads, 64), device="cuda")
    kw, want = dict(row_status=st), [0, 128, 0, 128, 0]
    if ragged:
        kw.update(new_start=to_gpu(np.array([0, 0, 0, 0, 0, 2], np.int32)))  # two rows that are not there
        want[4] = 128
        kw.update({} if call == "read" else dict(max_new=3))
    if call == "append":
        sv.kv_append(dev, rows(2), rows(2), to_gpu(table), lens, **kw)
    elif call == "read":
        sv.kv_read(dev, to_gpu(table), lens, 3 if ragged else 0, out=(rows(2), rows(2)), **kw)
    else:
        sv.kv_attention(rows(4), dev, to_gpu(table), lens, **kw)
    assert st.tolist() == want
