"""The 8-bit cache on the GPU against the fp64 oracle: codes and scales must
be equal (power-of-two scales leave one rounding, which is exact to decide),
values read back too."""
import numpy as np
import pytest

from oracle import kv_oracle as KO

from _kv import cache_gpu, copy, make_cache, make_table, round_to, same_cache, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


def _status(b):
    import torch
    return torch.full((b,), -7, dtype=torch.int32, device="cuda")


def _append_case(sv, g, dtype, dim, page, heads, ctx, new, layout="hnd", ragged=True, spread=1.0, shift=0, poke=None):
    """Appends to random caches and compares everything, the untouched pages too."""
    table, pages = make_table(g, [c + n for c, n in zip(ctx, new)], page)
    cache = make_cache(g, pages, heads, page, dim)
    total = sum(new)
    x = [round_to(g.normal(0, 1, (total, heads, dim)) * np.exp(g.normal(0, spread, (total, heads, 1))), dtype)
         for _ in range(2)]
    if poke:
        poke(x)
    want = copy(cache)
    at = 0
    odd = []
    for b, (c, n) in enumerate(zip(ctx, new)):
        with np.errstate(invalid="ignore"):
            odd.append(KO.append(want, x[0][at:at + n], x[1][at:at + n], table[b], page, c))
        at += n
    dev = cache_gpu(cache, layout)
    if shift:  # rows of a wider array that start off a 16-byte boundary
        import torch
        kv = []
        for a in x:
            wide = torch.zeros((total, heads + 1, dim + shift), dtype=to_gpu(a, dtype).dtype, device="cuda")
            wide[:, 1:, shift:] = to_gpu(a, dtype)
            kv.append(wide[:, 1:, shift:])
    else:
        kv = [to_gpu(a, dtype) for a in x]
    st = _status(len(ctx))
    if ragged:
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        sv.kv_append(dev, *kv, to_gpu(table), to_gpu(np.array(ctx, np.int32)), new_start=to_gpu(start), max_new=max(new), row_status=st)
    else:
        kv = [a.reshape(len(ctx), new[0], heads, dim) for a in kv]
        sv.kv_append(dev, *kv, to_gpu(table), to_gpu(np.array(ctx, np.int32)), row_status=st)
    same_cache(dev, want)
    assert st.cpu().tolist() == [256 if o else 0 for o in odd]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page,heads", [(16, 16, 1), (64, 32, 3), (80, 16, 2), (128, 64, 2), (128, 128, 1), (256, 128, 1), (208, 64, 1)])
def test_append_ragged(sv, dtype, dim, page, heads):
    g = np.random.default_rng(dim + page)
    ctx = [0, 1, page - 1, page, 2 * page + 3, 5, 7]
    new = [1, 2 * page + 5, 1, page, page - 3, 0, 3]
    _append_case(sv, g, dtype, dim, page, heads, ctx, new)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 8, 65])
def test_append_uniform_other_layout(sv, dtype, n):
    g = np.random.default_rng(n)
    _append_case(sv, g, dtype, 128, 64, 3, [0, 63, 64, 100, 191], [n] * 5, layout="nhd", ragged=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 3, 8])
def test_append_rows_of_a_wider_array(sv, dtype, shift):
    g = np.random.default_rng(shift)
    _append_case(sv, g, dtype, 96, 32, 2, [3, 40], [37, 5], shift=shift)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_magnitudes(sv, dtype):
    """Pages of zeros, of tiny and of huge values, and growth over many powers of two."""
    g = np.random.default_rng(4)

    def poke(x):
        x[0][0:16] = 0
        x[1][0:16] = round_to(x[1][0:16] * 1e-32, dtype)
        x[0][16:20] = round_to(x[0][16:20] * 1e30, dtype)
        x[1][16:40] = round_to(np.where(g.random(x[1][16:40].shape) < 0.1, 448.0, x[1][16:40] * 1e-3), dtype)
        x[0][40] = 3.3e38 if dtype == "f32" else round_to(np.float32(3.3e38), dtype)
    _append_case(sv, g, dtype, 64, 16, 2, [0, 5, 30], [20, 20, 9], spread=4.0, poke=poke)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_nan_and_infinity(sv, dtype):
    g = np.random.default_rng(5)

    def poke(x):
        x[0][3, 0, 5] = np.nan
        x[1][30, 1, 7] = np.inf
        x[1][31] = -np.inf
        x[0][32] = np.nan
    _append_case(sv, g, dtype, 64, 32, 2, [0, 10, 0], [25, 20, 6], poke=poke)


def test_append_one_token_at_a_time(sv):
    """A sequence grown token by token ends as the oracle's does, and differs
    from one call for all tokens by no more than half of the smallest code."""
    import torch
    g = np.random.default_rng(6)
    page, heads, dim, n = 16, 2, 64, 40
    table, pages = make_table(g, [n], page)
    cache = make_cache(g, pages, heads, page, dim)
    x = round_to(g.normal(0, 1, (n, heads, dim)) * np.exp(np.linspace(-3, 3, n))[:, None, None], "bf16")
    want, dev = copy(cache), cache_gpu(cache)
    t, k = to_gpu(table), to_gpu(x, "bf16")
    for i in range(n):
        KO.append(want, x[i:i + 1], -x[i:i + 1], table[0], page, i)
        sv.kv_append(dev, k[None, i:i + 1], -k[None, i:i + 1], t, torch.tensor([i], dtype=torch.int32, device="cuda"))
    same_cache(dev, want)


def test_append_flags_bad_lengths_and_pages(sv):
    """A flagged sequence leaves its cache alone (bad page: that page's tokens
    are left out); the others are served."""
    g = np.random.default_rng(7)
    page, heads, dim = 16, 2, 32
    ctx, new = np.array([4, -1, 30, 44, 20], np.int32), 6  # 44 + 6 > 48
    table, pages = make_table(g, [48] * 5, page)
    table[4, 1] = pages  # outside the pool
    cache = make_cache(g, pages, heads, page, dim)
    x = round_to(g.normal(0, 1, (5, new, heads, dim)), "bf16")
    want, dev = copy(cache), cache_gpu(cache)
    st = _status(5)
    for b in (0, 2, 4):
        KO.append(want, x[b], x[b], table[b], page, int(ctx[b]))
    sv.kv_append(dev, to_gpu(x, "bf16"), to_gpu(x, "bf16"), to_gpu(table), to_gpu(ctx), row_status=st)
    same_cache(dev, want)
    assert st.cpu().tolist() == [0, 128, 0, 128, 64]


def test_append_flags_bad_rows(sv):
    """Ragged rows that run backwards, beyond max_new or beyond the rows given."""
    g = np.random.default_rng(8)
    page, heads, dim = 16, 1, 32
    table, pages = make_table(g, [48] * 5, page)
    cache = make_cache(g, pages, heads, page, dim)
    x = round_to(g.normal(0, 1, (12, heads, dim)), "f32")
    start, ctx = np.array([0, 3, 2, 9, 11, 14], np.int32), np.zeros(5, np.int32)
    want, dev = copy(cache), cache_gpu(cache)
    KO.append(want, x[0:3], x[0:3], table[0], page, 0)
    KO.append(want, x[9:11], x[9:11], table[3], page, 0)
    st = _status(5)
    sv.kv_append(dev, to_gpu(x), to_gpu(x), to_gpu(table), to_gpu(ctx), new_start=to_gpu(start), max_new=4, row_status=st)
    same_cache(dev, want)
    assert st.cpu().tolist() == [0, 128, 128, 0, 128]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page,heads,layout", [(16, 16, 1, "hnd"), (80, 32, 3, "nhd"), (128, 64, 2, "hnd"), (256, 128, 2, "nhd")])
def test_read(sv, dtype, dim, page, heads, layout):
    import torch
    g = np.random.default_rng(dim)
    first, n = [0, 3, page, 2 * page - 1, 9], [1, 2 * page + 5, page, 300, 0]
    table, pages = make_table(g, [c + m for c, m in zip(first, n)], page)
    cache = make_cache(g, pages, heads, page, dim)
    dev = cache_gpu(cache, layout)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    st = _status(5)
    k, v = sv.kv_read(dev, to_gpu(table), to_gpu(np.array(first, np.int32)), max(n), new_start=to_gpu(start), total=sum(n),
                      dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, row_status=st)
    for name, got in (("k", k), ("v", v)):
        want = np.concatenate([KO.read(cache, name, table[b], page, c, m) for b, (c, m) in enumerate(zip(first, n))])
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)  # 4 significant bits: exact in both types
    assert st.cpu().tolist() == [0] * 5


def test_read_into_a_wider_array_and_bad_pages(sv):
    import torch
    g = np.random.default_rng(9)
    page, heads, dim = 16, 2, 48
    table, pages = make_table(g, [40, 40, 40], page)
    table[1, 1] = -3
    cache = make_cache(g, pages, heads, page, dim)
    first = np.array([2, 2, 20], np.int32)
    wide = [torch.full((3, 30, heads, dim + 3), 9.0, device="cuda") for _ in range(2)]
    st = _status(3)
    sv.kv_read(cache_gpu(cache), to_gpu(table), to_gpu(first), 30, out=tuple(w[..., 3:] for w in wide), dtype=torch.float32, row_status=st)
    for name, w in zip(("k", "v"), wide):
        got = w.double().cpu().numpy()
        assert (got[..., :3] == 9).all()
        for b in range(2):
            np.testing.assert_array_equal(got[b, ..., 3:], KO.read(cache, name, table[b], page, 2, 30))
        assert (got[2, ..., 3:] == 0).all()  # 20 + 30 > 48: left out, rows cleared
    assert st.cpu().tolist() == [0, 64, 128]


@pytest.mark.parametrize("dim,page,heads,layout", [(16, 16, 1, "hnd"), (64, 16, 3, "nhd"), (128, 64, 2, "hnd"), (256, 32, 1, "hnd")])
def test_commit(sv, dim, page, heads, layout):
    g = np.random.default_rng(page + dim)
    nodes, deep = 64, 17
    ctx = np.array([0, 1, page - 1, page, 3 * page + 5, 2, 77, 8], np.int32)
    accept = np.array([0, 16, 5, 9, 16, 3, 0, 12], np.int32)
    paths = np.full((8, deep), -1, np.int32)
    for b, a in enumerate(accept):
        paths[b, :a + 1] = [0] + sorted(g.choice(np.arange(1, nodes), a, replace=False))
    paths[5, :4] = [0, 1, 2, 3]  # nothing moves
    table, pages = make_table(g, [int(c) + nodes for c in ctx], page)
    cache = make_cache(g, pages, heads, page, dim, spread=4)
    want, dev = copy(cache), cache_gpu(cache, layout)
    lens = [KO.commit(want, table[b], page, int(ctx[b]), paths[b, :accept[b] + 1].tolist()) for b in range(8)]
    st = _status(8)
    got = sv.kv_commit(dev, to_gpu(table), to_gpu(ctx), to_gpu(paths), to_gpu(accept), nodes, row_status=st)
    assert got.cpu().tolist() == lens
    assert st.cpu().tolist() == [0] * 8
    same_cache(dev, want)


def test_commit_flags_and_keeps_nothing(sv):
    g = np.random.default_rng(10)
    page, heads, dim, nodes = 16, 2, 32, 8
    paths = np.array([[0, 2, 5], [-1, -1, -1], [0, 5, 2], [1, 2, 3], [0, 2, 8], [0, 2, 5], [0, 2, 5], [0, 2, 5], [0, 0, 1]], np.int32)
    accept = np.array([2, 0, 2, 1, 2, 3, -1, 2, 2], np.int32)
    ctx = np.array([3, 3, 3, 3, 3, 3, 3, 41, 3], np.int32)
    table, pages = make_table(g, [48] * 9, page)
    cache = make_cache(g, pages, heads, page, dim)
    want, dev = copy(cache), cache_gpu(cache)
    KO.commit(want, table[0], page, 3, [0, 2, 5])
    st = _status(9)
    got = sv.kv_commit(dev, to_gpu(table), to_gpu(ctx), to_gpu(paths), to_gpu(accept), nodes, row_status=st)
    assert got.cpu().tolist() == [6, 3, 3, 3, 3, 3, 3, 41, 3]
    assert st.cpu().tolist() == [0, 0, 512, 512, 512, 512, 512, 128, 512]
    same_cache(dev, want)


def test_far_pages(sv):
    """Codes beyond 2^32 bytes into the pool."""
    import torch
    g = np.random.default_rng(11)
    page, heads, dim, far = 16, 2, 64, 70000
    stride = 1 << 16  # bytes between pages: page 70000 lies 4.6e9 bytes in
    pool = [torch.zeros(stride * far + heads * page * dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    view = [p.as_strided((far + 1, heads, page, dim), (stride, page * dim, dim, 1)) for p in pool]
    dev = dict(k=view[0], v=view[1], k_scale=torch.ones((far + 1, heads), device="cuda"), v_scale=torch.ones((far + 1, heads), device="cuda"))
    table = np.array([[far, far - 1]], np.int32)
    small = make_cache(g, 2, heads, page, dim)
    x = round_to(g.normal(0, 1, (1, 20, heads, dim)), "bf16")
    KO.append(small, x[0], -x[0], [0, 1], page, 0)
    k = to_gpu(x, "bf16")
    zero = to_gpu(np.zeros(1, np.int32))
    sv.kv_append(dev, k, -k, to_gpu(table), zero)
    rk, rv = sv.kv_read(dev, to_gpu(table), zero, 20, dtype=torch.float32)
    np.testing.assert_array_equal(rk[0].double().cpu().numpy(), KO.read(small, "k", [0, 1], page, 0, 20))
    np.testing.assert_array_equal(rv[0].double().cpu().numpy(), KO.read(small, "v", [0, 1], page, 0, 20))
    q = to_gpu(round_to(g.normal(0, 1, (1, 3, 4, dim)), "bf16"), "bf16")
    near = cache_gpu(small)
    ctx = to_gpu(np.array([17], np.int32))
    a = sv.kv_attention(q, dev, to_gpu(table), ctx)
    b = sv.kv_attention(q, near, to_gpu(np.array([[0, 1]], np.int32)), ctx)
    assert torch.equal(a, b)
