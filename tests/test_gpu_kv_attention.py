"""Attention over the 8-bit cache on the GPU against the fp64 oracle, within
bounds derived from the operations (tests/_kv.py)."""
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


def _tree(g, n):
    return [-1][:n] + [int(g.integers(max(0, i - 6), i)) for i in range(1, n)]


def _check(sv, g, dtype, dim, page, heads, kv_heads, ctx, new, tree=False, window=0, sinks=0, scale=None, layout="hnd",
           ragged=True, peak=1.5, shift=0, spread=2, harm=None, garbage=False):
    """One call against the oracle; returns what the GPU gave."""
    import torch
    table, pages = make_table(g, [c + n for c, n in zip(ctx, new)], page)
    cache = make_cache(g, pages, kv_heads, page, dim, spread)
    total = sum(new)
    q = round_to(g.normal(0, peak, (total, heads, dim)), dtype)
    parents = [_tree(g, n) for n in new] if tree else [None] * len(ctx)
    if harm:
        harm(table, cache)
    dev = dict(cache)
    if garbage:  # what lies behind the last token may be anything
        dev = {n: a.copy() for n, a in cache.items()}
        for b, (c, n) in enumerate(zip(ctx, new)):
            if (c + n) % page:
                for name in ("k", "v"):
                    dev[name][table[b, (c + n) // page], :, (c + n) % page:] = 0x7f
        for name in ("k", "v"):
            unused = np.setdiff1d(np.arange(pages), np.concatenate([table[b, :-(-(c + n) // page)] for b, (c, n) in enumerate(zip(ctx, new))]))
            dev[name][unused] = 0x7f
            dev[name + "_scale"][unused] = np.nan
    dev = cache_gpu(dev, layout)
    qd = to_gpu(q, dtype)
    if shift:
        wide = torch.zeros((total, heads + 1, dim + shift), dtype=qd.dtype, device="cuda")
        wide[:, 1:, shift:] = qd
        qd = wide[:, 1:, shift:]
    st = torch.full((len(ctx),), -7, dtype=torch.int32, device="cuda")
    pd = to_gpu(np.array([p for row in parents for p in row], np.int32)) if tree else None
    kw = dict(parents=pd, window=window, sinks=sinks, scale=scale, lse=True, row_status=st)
    if ragged:
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        out, lse = sv.kv_attention(qd, dev, to_gpu(table), to_gpu(np.array(ctx, np.int32)), new_start=to_gpu(start), max_new=max(new), **kw)
    else:
        out, lse = sv.kv_attention(qd.reshape(len(ctx), new[0], heads, dim), dev, to_gpu(table), to_gpu(np.array(ctx, np.int32)), **kw)
        out, lse = out.reshape(total, heads, dim), lse.reshape(total, heads)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        want, wlse, absolute, largest = KO.attention(q[at:at + n].astype(np.float64), cache, table[b], page, c, parents[b],
                                                     dim ** -0.5 if scale is None else scale, window, sinks)
        tol, ltol = attention_tolerance(want, absolute, largest, c + n, dim, dtype)
        off = np.abs(out[at:at + n] - want)
        assert np.isfinite(out[at:at + n]).all(), (b, "not finite")
        assert (off <= tol).all(), (b, float((off / tol).max()))
        none = np.isneginf(wlse)
        assert (np.isneginf(lse[at:at + n]) == none).all()
        assert (np.abs(lse[at:at + n] - wlse)[~none] <= ltol[~none]).all(), (b, float((np.abs(lse[at:at + n] - wlse) / ltol)[~none].max()))
        at += n
    return out, lse, st.cpu().tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page,heads,kv_heads", [(16, 16, 1, 1), (48, 32, 6, 2), (64, 16, 8, 1), (80, 64, 3, 3),
                                                     (128, 128, 8, 2), (128, 64, 16, 1), (192, 16, 4, 2), (256, 128, 5, 1)])
def test_one_token(sv, dtype, dim, page, heads, kv_heads):
    """Decoding: contexts of nothing, one token, and odd lengths about the page's."""
    g = np.random.default_rng(dim + heads)
    ctx = [0, 1, page - 1, page, page + 1, 15, 16, 17, 333]
    st = _check(sv, g, dtype, dim, page, heads, kv_heads, ctx, [1] * len(ctx), ragged=False)[2]
    assert st == [0] * len(ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dim,page,heads,kv_heads,new", [(64, 16, 8, 2, 6), (128, 64, 8, 2, 8), (128, 32, 4, 4, 33), (80, 64, 10, 2, 20),
                                                         (128, 128, 8, 1, 16), (256, 64, 4, 1, 9), (32, 16, 16, 1, 65), (128, 64, 12, 4, 2)])
def test_chains_and_trees(sv, dtype, tree, dim, page, heads, kv_heads, new):
    g = np.random.default_rng(dim + heads + new)
    ctx = [0, 1, 63, 64, 200, 37]
    counts = [new, 1, max(1, new - 1), new, (new + 1) // 2, 0]
    _check(sv, g, dtype, dim, page, heads, kv_heads, ctx, counts, tree=tree)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (16, 4), (100, 17), (7, 1000), (1000, 4)])
def test_window_and_sinks(sv, dtype, tree, window, sinks):
    g = np.random.default_rng(window + sinks)
    _check(sv, g, dtype, 64, 16, 4, 2, [0, 3, 50, 129, 260], [9, 12, 7, 12, 12], tree=tree, window=window, sinks=sinks, layout="nhd")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [100, 257])
def test_stretches_of_a_prompt(sv, dtype, new):
    g = np.random.default_rng(new)
    _check(sv, g, dtype, 64, 32, 4, 2, [0, 45], [new, new - 31])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_contexts(sv, dtype):
    """Split over many blocks: one long context beside short ones."""
    g = np.random.default_rng(12)
    _check(sv, g, dtype, 64, 16, 2, 1, [5003, 17, 0, 1203], [4, 4, 4, 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,dim", [(2, 64), (6, 128), (16, 64), (12, 128)])
def test_long_contexts_of_more_rows(sv, dtype, heads, dim):
    """Items of up to 16, 32, 128 and more rows in parts of several blocks."""
    g = np.random.default_rng(heads + dim)
    _check(sv, g, dtype, dim, 64, heads, 1, [5003, 17, 0, 1203, 2600], [5, 4, 2, 5, 1] if heads < 8 else [11, 2, 4, 5, 3])


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (100, 17), (7, 1000), (700, 4)])
def test_window_and_sinks_of_many_rows(sv, tree, dim, window, sinks):
    g = np.random.default_rng(window + sinks + dim)
    _check(sv, g, "bf16", dim, 16, 8, 1, [0, 3, 50, 129, 1260], [9, 40, 7, 0, 12], tree=tree, window=window, sinks=sinks, layout="nhd")


@pytest.mark.parametrize("dtype,heads", [("bf16", 2), ("f32", 6), ("bf16", 12)])
def test_more_sequences_than_threads(sv, dtype, heads):
    """Empty sequences among them, and lengths from nothing on: the results of
    calls of 50 sequences each, bit for bit (no sequence is in parts here)."""
    import torch
    g = np.random.default_rng(heads)
    ctx, new = g.integers(0, 40, 700).astype(np.int32), g.integers(0, 4, 700).astype(np.int32)
    new[:3] = new[300:420] = 0
    table, pages = make_table(g, [int(n) for n in ctx + new], 16)
    cache = cache_gpu(make_cache(g, pages, 1, 16, 64))
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = to_gpu(g.normal(0, 1.5, (int(start[-1]), heads, 64)).astype(np.float32), dtype)
    out, lse = sv.kv_attention(q, cache, to_gpu(table), to_gpu(ctx), new_start=to_gpu(start), max_new=3, lse=True)
    for b in range(0, 700, 50):
        lo, hi = int(start[b]), int(start[b + 50])
        some, sums = sv.kv_attention(q[lo:hi], cache, to_gpu(table[b:b + 50]), to_gpu(ctx[b:b + 50]),
                                     new_start=to_gpu(start[b:b + 51] - lo), max_new=3, lse=True)
        assert torch.equal(out[lo:hi], some) and torch.equal(lse[lo:hi], sums), b


@pytest.mark.parametrize("dtype,heads", [("bf16", 2), ("f32", 2), ("bf16", 6), ("f32", 6), ("bf16", 12)])
@pytest.mark.parametrize("dim", [64, 128])
def test_small_weights(sv, dtype, heads, dim):
    """Scores that differ by more than fp16 weights can hold.  Weights are
    multiplied by 2^6 at least against a row's largest and their steps end at
    2^-24, so each is off by at most 2^-25 2^-6 of the largest, with the value's
    code and the largest scale of V behind it.  (The weight of a token whose
    rivals all hold exactly 0 in a dim is all that is left there.)"""
    g = np.random.default_rng(heads + dim)
    ctx, n, page = [1, 28, 300], 3, 16
    table, pages = make_table(g, [c + n for c in ctx], page)
    cache = make_cache(g, pages, 1, page, dim)
    cache["v"][g.random(cache["v"].shape) < 0.3] = 0
    q = round_to(g.normal(0, 4, (len(ctx), n, heads, dim)), dtype)
    out = sv.kv_attention(to_gpu(q, dtype), cache_gpu(cache), to_gpu(table), to_gpu(np.array(ctx, np.int32))).double().cpu().numpy()
    for b, c in enumerate(ctx):
        want, _, absolute, largest = KO.attention(q[b].astype(np.float64), cache, table[b], page, c, None, dim ** -0.5, 0, 0)
        tol, _ = attention_tolerance(want, absolute, largest, c + n, dim, dtype)
        used = table[b, :-(-(c + n) // page)]
        codes = np.abs(KO.read(dict(cache, v_scale=np.ones_like(cache["v_scale"])), "v", table[b], page, 0, c + n)).sum(0)[0]
        tol += 2.0 ** -31 * cache["v_scale"][used].max() * codes
        off = np.abs(out[b] - want)
        assert (off <= tol).all(), (b, float((off / tol).max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("peak,spread,scale", [(0.0, 2, None), (40.0, 2, None), (1.5, 12, None), (1.5, 2, -0.3), (1.5, 2, 0.0), (1e-20, 2, 1e18), (3e4, 2, 1e-6)])
def test_scores_and_scales(sv, dtype, peak, spread, scale):
    """Equal scores, scores that leave one token, page scales that differ by
    powers of two up to 2^24, negative and zero factors, queries far from 1."""
    g = np.random.default_rng(13)
    _check(sv, g, dtype, 64, 16, 4, 2, [130, 400], [5, 1], peak=peak, spread=spread, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 8, 40])
def test_bytes_behind_the_last_token(sv, dtype, new):
    g = np.random.default_rng(14)
    _check(sv, g, dtype, 128, 64, 8, 2, [0, 10, 70, 125], [new] * 4, garbage=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 8])
def test_strided_queries(sv, dtype, shift):
    g = np.random.default_rng(15)
    _check(sv, g, dtype, 80, 16, 6, 3, [20, 77], [7, 3], shift=shift)


@pytest.mark.parametrize("new", [1, 12, 40])
def test_bad_pages_are_not_seen(sv, new):
    """Tokens on pages outside the pool are left out, which leaves some rows empty."""
    g = np.random.default_rng(16)

    def harm(table, cache):
        table[0, 1] = cache["k"].shape[0]
        table[1, :] = -1
        table[2, 0] = -5
    st = _check(sv, g, "bf16", 64, 16, 4, 2, [40, 40, 3, 20], [new] * 4, harm=harm)[2]
    assert st == [64, 64, 64, 0]


def test_bad_lengths(sv):
    """Flagged sequences' rows are cleared where they are known."""
    import torch
    g = np.random.default_rng(17)
    page, dim, heads = 16, 64, 4
    table, pages = make_table(g, [32] * 4, page)
    dev = cache_gpu(make_cache(g, pages, 2, page, dim))
    q = to_gpu(g.normal(0, 1, (4, 3, heads, dim)).astype(np.float32), "bf16")
    out = torch.full_like(q, 2.0 ** 100)
    st = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    _, lse = sv.kv_attention(q, dev, to_gpu(table), to_gpu(np.array([5, -1, 30, 29], np.int32)), out=out, lse=True, row_status=st)
    assert st.cpu().tolist() == [0, 128, 128, 0]
    assert (out[1:3] == 0).all() and torch.isneginf(lse[1:3]).all()
    assert torch.isfinite(lse[[0, 3]]).all()
    start = to_gpu(np.array([0, 3, 2, 9, 12], np.int32))
    out = torch.full_like(q.reshape(12, heads, dim), 2.0 ** 100)
    sv.kv_attention(q.reshape(12, heads, dim), dev, to_gpu(table), to_gpu(np.array([5, 5, 5, 5], np.int32)), new_start=start, max_new=4, out=out, row_status=st)
    assert st.cpu().tolist() == [0, 128, 128, 0]
    untouched = (out == 2.0 ** 100).flatten(1)
    assert untouched[3:9].all().item() and not untouched[:3].any().item() and not untouched[9:].any().item()


def test_bad_parents(sv):
    """A parent outside [0, i) counts as none, and is flagged."""
    import torch
    g = np.random.default_rng(18)
    page, dim = 16, 64
    table, pages = make_table(g, [16] * 2, page)
    cache = make_cache(g, pages, 1, page, dim)
    q = round_to(g.normal(0, 1, (2, 4, 2, dim)), "bf16")
    parents = np.array([[-1, 0, 1, 1], [0, 1, 5, -1]], np.int32)
    st = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    out = sv.kv_attention(to_gpu(q, "bf16"), cache_gpu(cache), to_gpu(table), to_gpu(np.array([3, 3], np.int32)), parents=to_gpu(parents), row_status=st)
    assert st.cpu().tolist() == [0, 2]
    for b in range(2):
        want, _, absolute, largest = KO.attention(q[b].astype(np.float64), cache, table[b], page, 3, parents[b], dim ** -0.5, 0, 0)
        tol, _ = attention_tolerance(want, absolute, largest, 7, dim, "bf16")
        assert (np.abs(out[b].double().cpu().numpy() - want) <= tol).all()


def test_queries_that_are_not_finite_stay_in_their_rows(sv):
    import torch
    g = np.random.default_rng(19)
    page, dim = 16, 64
    for n in (1, 6, 40):
        table, pages = make_table(g, [50 + n], page)
        dev = cache_gpu(make_cache(g, pages, 2, page, dim))
        q = to_gpu(g.normal(0, 1, (1, n, 4, dim)).astype(np.float32), "bf16")
        bad = q.clone()
        bad[0, 0, 1, 3] = float("nan")
        args = (dev, to_gpu(table), to_gpu(np.array([50], np.int32)))
        a, b = sv.kv_attention(q, *args), sv.kv_attention(bad, *args)
        assert torch.isnan(b[0, 0, 1]).all()
        keep = torch.ones((n, 4), dtype=torch.bool, device="cuda")
        keep[0, 1] = False
        assert torch.equal(a[0][keep], b[0][keep])


def test_repeatable_on_other_streams_and_in_graphs(sv):
    """The same bits from run to run, on a stream of its own with a workspace
    of its own, and replayed from a graph after the lengths changed."""
    import torch
    g = np.random.default_rng(20)
    page, dim, heads, kv = 32, 128, 8, 2
    table, pages = make_table(g, [900, 900, 900], page)
    dev = cache_gpu(make_cache(g, pages, kv, page, dim))
    t = to_gpu(table)
    for n in (1, 8, 40):
        q = to_gpu(g.normal(0, 1, (3, n, heads, dim)).astype(np.float32), "bf16")
        ctx = to_gpu(np.array([700, 3, 333], np.int32))
        first = sv.kv_attention(q, dev, t, ctx)
        assert torch.equal(first, sv.kv_attention(q, dev, t, ctx))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = sv.kv_attention(q, dev, t, ctx)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(first, other)
        out = torch.empty_like(q)
        ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sv.kv_attention(q, dev, t, ctx, out=out, ws=ws)
        ws.fill_(255)
        ctx.copy_(to_gpu(np.array([5, 850, 64], np.int32)))
        graph.replay()
        assert torch.equal(out, sv.kv_attention(q, dev, t, ctx))


def test_chain_as_a_tree(sv):
    """Parents i - 1 give what no parents give."""
    import torch
    g = np.random.default_rng(21)
    page, dim = 16, 64
    for n in (2, 20, 65):
        table, pages = make_table(g, [100 + n] * 2, page)
        dev = cache_gpu(make_cache(g, pages, 2, page, dim))
        q = to_gpu(g.normal(0, 1, (2, n, 6, dim)).astype(np.float32), "bf16")
        ctx = to_gpu(np.array([100, 31], np.int32))
        parents = to_gpu(np.tile(np.arange(-1, n - 1, dtype=np.int32), (2, 1)))
        for window, sinks in ((0, 0), (20, 3)):
            a = sv.kv_attention(q, dev, to_gpu(table), ctx, window=window, sinks=sinks)
            b = sv.kv_attention(q, dev, to_gpu(table), ctx, parents=parents, window=window, sinks=sinks)
            assert torch.equal(a, b)


def test_nothing_to_do(sv):
    import torch
    g = np.random.default_rng(22)
    table, pages = make_table(g, [10], 16)
    dev = cache_gpu(make_cache(g, pages, 2, 16, 64))
    zero = to_gpu(np.zeros(1, np.int32))
    q = torch.empty((1, 0, 4, 64), device="cuda")
    assert sv.kv_attention(q, dev, to_gpu(table), zero).shape == q.shape
    empty = to_gpu(np.zeros((0, 1), np.int32))
    q = torch.empty((0, 3, 4, 64), device="cuda")
    assert sv.kv_attention(q, dev, empty, zero[:0]).shape == q.shape
