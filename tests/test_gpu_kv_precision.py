"""What the attention over the 8-bit cache keeps of weights and queries whose
sizes differ widely, against the fp64 oracle within bounds derived from the
operations (tests/_kv.py)."""
import numpy as np
import pytest

from oracle import kv_oracle as KO

from _kv import attention_tolerance, cache_gpu, make_cache, make_table, round_to, to_gpu

pytestmark = pytest.mark.gpu

# (type, heads of one kv head): up to 16 rows, up to 32, and more
ROWS = [("bf16", 2), ("f32", 2), ("bf16", 24), ("f32", 24), ("bf16", 48)]


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


def _compare(sv, cache, table, page, ctx, q, dtype, scale, copies=1):
    """One sequence, one new token, one kv head (or so many sequences on the
    same pages, each then the work of a block or two)."""
    heads, dim = q.shape[1:]
    lens = to_gpu(np.full(copies, ctx, np.int32))
    outs, sums = sv.kv_attention(to_gpu(np.stack([q] * copies), dtype), cache_gpu(cache), to_gpu(np.repeat(table, copies, 0)), lens,
                                 scale=scale, lse=True)
    want, wlse, absolute, largest = KO.attention(q.astype(np.float64), cache, table[0], page, ctx, None, scale, 0, 0)
    tol, ltol = attention_tolerance(want, absolute, largest, ctx + 1, dim, dtype)
    # weights end at 2^-31 of the row's largest, counted with the scales of V
    k = KO.read(cache, "k", table[0], page, 0, ctx + 1)[:, 0]
    codes = np.abs(KO.read(dict(cache, v_scale=np.ones_like(cache["v_scale"])), "v", table[0], page, 0, ctx + 1))[:, 0]
    unit = cache["v_scale"][table[0][np.arange(ctx + 1) // page], 0]
    p = np.exp(q[0].astype(np.float64) @ k.T * scale - wlse[0][:, None])
    tol[0] += 2.0 ** -31 * (p * unit).max(1)[:, None] * codes.sum(0)
    off = np.abs(outs.double().cpu().numpy() - want)
    assert (off <= tol).all(), float((off / tol).max())
    loff = np.abs(sums.double().cpu().numpy() - wlse)
    assert (loff <= ltol).all(), float((loff / ltol).max())


@pytest.mark.parametrize("dtype,heads", ROWS)
@pytest.mark.parametrize("dim", [64, 128])
def test_weights_and_values_that_rise_together(sv, dtype, heads, dim):
    """Every page has larger values and larger weights than the one before, so
    that both units change within a tile, again and again."""
    g = np.random.default_rng(dim + heads)
    page, ctx = 16, 700
    table, pages = make_table(g, [ctx + 1], page)
    cache = make_cache(g, pages, 1, page, dim)
    cache["k"][:] = 0
    cache["k_scale"][:] = 1.0
    for i, p in enumerate(table[0]):
        cache["v_scale"][p] = 2.0 ** (i - 20)
        cache["k"][p, 0, :, 0] = KO.encode(np.full(page, 10.0 * (i - 20)))
    q = np.zeros((1, heads, dim), np.float32)
    q[0, :, 0] = np.linspace(0.05, 0.7, heads)
    _compare(sv, cache, table, page, ctx, round_to(q, dtype), dtype, 1.0)


@pytest.mark.parametrize("dtype,heads", ROWS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("r", [0, 10, 16, 24, 60])
def test_pages_of_large_values_without_weight(sv, dtype, heads, dim, where, r):
    """One token of much weight and a long even tail 2^-12 below it, on pages
    whose scale of V lies 2^-r below that of pages that weigh 2^-40 and less."""
    g = np.random.default_rng(r + dim)
    page, ctx = 16, 2999
    table, pages = make_table(g, [ctx + 1], page)
    cache = make_cache(g, pages, 1, page, dim)
    cache["k"][:] = 0
    cache["k_scale"][:] = 1.0
    cache["k"][..., 0] = KO.encode(-12.0)
    cache["v"] = np.maximum(cache["v"] & 0x7f, 0x20).astype(np.uint8) | (cache["v"] & 0x80)
    cache["v_scale"][:] = 2.0 ** -6
    at = {"first": 0, "middle": 101, "last": (ctx + 1) // page - 8}[where]
    heavy = table[0, at:at + 8]  # enough for every warp to meet one
    cache["v_scale"][heavy] *= 2.0 ** r
    cache["k"][heavy, 0, :, 0] = KO.encode(-(40.0 + min(r, 40)))
    peak = 1234
    cache["k"][table[0, peak // page], 0, peak % page, 0] = 0
    q = np.zeros((1, heads, dim), np.float32)
    q[0, :, 0] = np.log(2.0) * (1 + np.arange(heads) / 200)
    _compare(sv, cache, table, page, ctx, round_to(q, dtype), dtype, 1.0, copies=600)


@pytest.mark.parametrize("dtype,heads", ROWS)
@pytest.mark.parametrize("dim", [64, 128])
def test_pages_of_zeros_among_large_values(sv, dtype, heads, dim):
    """Appended zeros have the smallest scale, 2^-100; their weights count all the same."""
    g = np.random.default_rng(dim + heads)
    page, ctx = 16, 400
    table, pages = make_table(g, [ctx + 1], page)
    cache = make_cache(g, pages, 1, page, dim)
    zeros = table[0, ::3]
    cache["v"][zeros] = 0
    cache["v_scale"][zeros] = 2.0 ** -100
    cache["v_scale"][table[0, 1::3]] = 2.0 ** 20
    _compare(sv, cache, table, page, ctx, round_to(g.normal(0, 1.5, (1, heads, dim)), dtype), dtype, dim ** -0.5)


@pytest.mark.parametrize("dtype,heads", ROWS)
@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("key", [0.0, 1.0])
@pytest.mark.parametrize("factor", [100.0, 300.0, 3000.0, 3e6])
def test_one_dim_of_the_queries_is_far_larger(sv, dtype, heads, dim, key, factor):
    """The rest keeps its bits, whether the keys have anything in that dim or not."""
    g = np.random.default_rng(dim + heads)
    page, ctx, at = 32, 500, 17
    table, pages = make_table(g, [ctx + 1], page)
    cache = make_cache(g, pages, 1, page, dim)
    cache["k"][..., at] = KO.encode(KO.VALUE[cache["k"][..., at]] * key)
    q = g.normal(0, 1, (1, heads, dim))
    q[..., at] = factor * np.sign(q[..., at])
    _compare(sv, cache, table, page, ctx, round_to(q, dtype), dtype, dim ** -0.5)
