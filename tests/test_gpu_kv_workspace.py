"""Workspaces and streams of the attention over the 8-bit cache."""
import ctypes

import numpy as np
import pytest

from _kv import cache_gpu, make_cache, make_table, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


@pytest.mark.parametrize("dtype,heads", [("bf16", 2), ("f32", 6), ("bf16", 12)])
@pytest.mark.parametrize("shift", [0, 16, 32, 48])
def test_any_workspace_on_a_16_byte_boundary(sv, dtype, heads, shift):
    """Of exactly the size that is asked for, with nothing written behind it."""
    import torch
    from draft_token_verification_sv_gb300 import _native as N
    g = np.random.default_rng(heads)
    page, dim, ctx, n = 64, 128, 5003, 5
    table, pages = make_table(g, [ctx + n], page)
    dev = cache_gpu(make_cache(g, pages, 1, page, dim))
    q = to_gpu(g.normal(0, 1, (1, n, heads, dim)).astype(np.float32), dtype)
    lens = to_gpu(np.array([ctx], np.int32))
    want = sv.kv_attention(q, dev, to_gpu(table), lens)
    kv = N.KvDesc(1, 1, dim, page, pages, table.shape[1], page * dim, page * dim, dim, table.shape[1])
    a = N.KvAttentionDesc(kv, heads, n, n, N.SV_BF16 if dtype == "bf16" else N.SV_F32, dim ** -0.5, 0, 0, 0, heads * dim, dim, heads * dim, dim)
    need = N.lib().sv_kv_attention_workspace_size(ctypes.byref(a))
    whole = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    assert whole.data_ptr() % 256 == 0
    got = sv.kv_attention(q, dev, to_gpu(table), lens, ws=whole[1024 + shift:1024 + shift + need])
    assert torch.equal(got, want)
    assert (whole[:1024 + shift] == 0xa5).all() and (whole[1024 + shift + need:] == 0xa5).all()


@pytest.mark.parametrize("dtype,heads", [("bf16", 2), ("f32", 6), ("bf16", 12)])
def test_stream_argument_beside_a_busy_current_stream(sv, dtype, heads):
    """A first call on a stream, then one that needs a larger workspace, both
    while the current stream is held up."""
    import torch
    g = np.random.default_rng(heads)
    page, dim, n = 64, 128, 5
    table, pages = make_table(g, [5003 + n], page)
    dev = cache_gpu(make_cache(g, pages, 1, page, dim))
    t, lens, zero, side = to_gpu(table), to_gpu(np.array([5003], np.int32)), to_gpu(np.zeros(1, np.int32)), torch.cuda.Stream()
    for rows in (1, heads):
        q = to_gpu(g.normal(0, 1, (1, n, rows, dim)).astype(np.float32), dtype)
        want, sums = sv.kv_attention(q, dev, t, lens, lse=True)
        back = sv.kv_read(dev, t, zero, 700)
        spoilt = torch.empty(1 << 24, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        spoilt.fill_(float("nan"))
        del spoilt  # its memory is free for what the current stream allocates, and still to be written by it
        got, lse = sv.kv_attention(q, dev, t, lens, lse=True, stream=side)
        k, v = sv.kv_read(dev, t, zero, 700, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(lse, sums)
        assert torch.equal(k, back[0]) and torch.equal(v, back[1])
