"""The attention over the 8-bit cache with queries and results of any layout,
and with more sequences than a block has threads, against the fp64 oracle."""
import numpy as np
import pytest

from oracle import kv_oracle as KO

from _kv import attention_tolerance, cache_gpu, make_cache, make_table, round_to, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


def _within(out, lse, q, cache, table, page, ctx, new, dtype):
    dim, at = q.shape[-1], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        want, wlse, absolute, largest = KO.attention(q[at:at + n].astype(np.float64), cache, table[b], page, c, None, dim ** -0.5, 0, 0)
        tol, ltol = attention_tolerance(want, absolute, largest, c + n, dim, dtype)
        assert (np.abs(out[at:at + n] - want) <= tol).all(), b
        assert (np.abs(lse[at:at + n] - wlse) <= ltol).all(), b
        at += n


def _wide(rows, heads, dim, shift, dtype, fill):
    """[rows, heads, dim] inside a larger array: rows and heads further apart, `shift` values off the array's start."""
    import torch
    whole = torch.full((rows, heads + 1, dim + 16 + shift), fill, dtype=dtype, device="cuda")
    return whole, whole[:, 1:, shift:shift + dim]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("new", [1, 5, 21])
@pytest.mark.parametrize("shift", [1, 8, 16])
def test_strided_queries_and_results(sv, dtype, dim, new, shift):
    """Off 16-byte boundaries, on 16- and on 32-byte ones; whole items and items
    in parts; nothing else of the results' array is written."""
    import torch
    g = np.random.default_rng(dim + new + shift)
    page, heads, kv_heads = 32, 6, 2
    ctx, counts = [20, 2477, 300], [new, max(1, new - 2), new]
    table, pages = make_table(g, [c + n for c, n in zip(ctx, counts)], page)
    cache = make_cache(g, pages, kv_heads, page, dim)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q = round_to(g.normal(0, 1.5, (start[-1], heads, dim)), dtype)
    qd = to_gpu(q, dtype)
    _, queries = _wide(start[-1], heads, dim, shift, qd.dtype, float("nan"))
    queries.copy_(qd)
    for place in (shift, 0):  # 0: aligned results of unaligned queries
        whole, out = _wide(start[-1], heads, dim, place, qd.dtype, 7.0)
        got, lse = sv.kv_attention(queries, cache_gpu(cache), to_gpu(table), to_gpu(np.array(ctx, np.int32)), new_start=to_gpu(start),
                                   max_new=new, out=out, lse=True)
        assert got.data_ptr() == out.data_ptr()
        _within(out.double().cpu().numpy(), lse.double().cpu().numpy(), q, cache, table, page, ctx, counts, dtype)
        out.fill_(7.0)
        assert (whole == 7.0).all()


@pytest.mark.parametrize("dtype,heads", [("bf16", 2), ("f32", 6), ("bf16", 12)])
def test_more_sequences_than_threads_against_the_oracle(sv, dtype, heads):
    """Empty sequences among them, lengths from nothing on, and a long one that is in parts."""
    g = np.random.default_rng(heads)
    ctx, new = g.integers(0, 40, 700), g.integers(0, 4, 700)
    new[:3] = new[300:420] = 0
    ctx[650], new[650] = 2000, 3
    table, pages = make_table(g, [int(n) for n in ctx + new], 16)
    cache = make_cache(g, pages, 1, 16, 64)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = round_to(g.normal(0, 0.7, (int(start[-1]), heads, 64)), dtype)
    out, lse = sv.kv_attention(to_gpu(q, dtype), cache_gpu(cache), to_gpu(table), to_gpu(ctx.astype(np.int32)),
                               new_start=to_gpu(start), max_new=3, lse=True)
    _within(out.double().cpu().numpy(), lse.double().cpu().numpy(), q, cache, table, 16, [int(c) for c in ctx], [int(n) for n in new], dtype)
