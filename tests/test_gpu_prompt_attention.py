"""Attention of prompts on the GPU against the fp64 oracle, within bounds
derived from the operations (tests/_prompt.py)."""
import numpy as np
import pytest

from _kv import round_to, to_gpu
from _prompt import near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


def _inputs(g, dtype, total, heads, kv_heads, dim, peak=1.5):
    return [round_to(g.normal(0, s, (total, h, dim)), dtype) for h, s in ((heads, peak), (kv_heads, 1), (kv_heads, 1))]


def _check(sv, dtype, lengths, heads=4, kv_heads=2, dim=64, window=0, sinks=0, scale=None, peak=1.5, seed=0, behind=0, ahead=0, place=None,
           ragged=True, harm=None):
    """One call against the oracle; `ahead` and `behind`: rows that belong to no sequence."""
    import torch
    g = np.random.default_rng(seed)
    starts = (ahead + np.concatenate([[0], np.cumsum(lengths)])).astype(np.int32)
    total = int(starts[-1]) + behind
    q, k, v = _inputs(g, dtype, total, heads, kv_heads, dim, peak)
    dev = [to_gpu(x, dtype) for x in (q, k, v)]
    if harm:
        harm(*dev, starts)
    if place:
        dev = place(*dev)
    st = torch.full((len(lengths),), -7, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks, scale=scale, lse=True, row_status=st)
    if ragged:
        out = torch.full((total, heads, dim), 9.0, dtype=dev[0].dtype, device="cuda")
        out, lse = sv.prompt_attention(*dev, new_start=to_gpu(starts), max_new=max(lengths), out=out, **kw)
        assert (out[:ahead] == 9).all() and (out[total - behind:] == 9).all()
    else:
        out, lse = sv.prompt_attention(*(x.reshape(len(lengths), lengths[0], *x.shape[1:]) for x in dev), **kw)
        out, lse = out.reshape(total, heads, dim), lse.reshape(total, heads)
    assert st.tolist() == [0] * len(lengths)
    near(out.double().cpu().numpy(), lse.double().cpu().numpy(), q, k, v, starts, dim ** -0.5 if scale is None else scale, window, sinks, dtype)
    return out, lse


DIMS = [16, 32, 48, 64, 80, 96, 112, 128, 144, 160, 192, 208, 256]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", DIMS)
def test_head_dims(sv, dtype, dim):
    _check(sv, dtype, [150, 1, 37], dim=dim)


@pytest.mark.parametrize("dim", [16, 64, 128, 144, 192, 208, 256])
def test_what_float32_scores_lose(sv, dim):
    """Alone in its sequence a token's lse is its score.  Of positive terms the
    sum grows evenly, so that what is cut off with each 16 of them (less than
    the last place, 2^-23 of the sum so far; half of that in the mean) comes to
    (dim / 16 + 1) / 4 of 2^-23 of the score; scaling, to base 2 and back, and
    the products that are left out take less than 2 of 2^-23."""
    g = np.random.default_rng(dim)
    q, k, v = (round_to(g.uniform(0.5, 2, (300, 2, dim)), "f32") for _ in range(3))
    starts = np.arange(301, dtype=np.int32)
    _, lse = sv.prompt_attention(*(to_gpu(x, "f32") for x in (q, k, v)), new_start=to_gpu(starts), max_new=1, lse=True)
    want = (q.astype(np.float64) * k).sum(-1) * float(np.float32(dim ** -0.5))
    assert abs((lse.double().cpu().numpy() / want - 1).mean()) <= ((dim / 16 + 1) / 4 + 2) * 2.0 ** -23


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (8, 2), (6, 2), (5, 1), (7, 1), (14, 2), (16, 1), (40, 1), (100, 1), (128, 1)])
def test_shared_heads(sv, dtype, heads, kv_heads):
    _check(sv, dtype, [1, 130, 0, 16], heads=heads, kv_heads=kv_heads, dim=32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 257, 300, 384, 511, 513])
def test_lengths(sv, dtype, length):
    _check(sv, dtype, [length], heads=2, kv_heads=1, dim=64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[0], [0, 0, 5, 0], [3, 200, 0, 64, 65, 1], [1] * 70, [257, 3, 128, 128]])
def test_packed_lengths(sv, dtype, lengths):
    _check(sv, dtype, lengths, heads=4, kv_heads=1, dim=128, ahead=3, behind=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded_batch(sv, dtype):
    _check(sv, dtype, [77] * 3, dim=80, ragged=False)
    _check(sv, dtype, [1] * 5, dim=128, heads=8, ragged=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (64, 0), (63, 4), (65, 130), (100, 1), (128, 128), (200, 300), (1000, 5),
                                          (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (7, 2 ** 31 - 1)])
def test_windows_and_sinks(sv, dtype, window, sinks):
    _check(sv, dtype, [520, 129, 7], heads=2, kv_heads=1, dim=64, window=window, sinks=sinks)


@pytest.mark.parametrize("heads", [5, 16])
@pytest.mark.parametrize("window,sinks", [(30, 0), (300, 70)])
def test_windows_with_many_heads_to_a_kv_head(sv, heads, window, sinks):
    _check(sv, "bf16", [530, 64], heads=heads, kv_heads=1, dim=48, window=window, sinks=sinks)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_long_prompt(sv, dim):
    _check(sv, "bf16", [1411, 40], heads=3, kv_heads=1, dim=dim)
    _check(sv, "f32", [1100, 40], heads=2, kv_heads=1, dim=dim)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 1e-30])
def test_scales(sv, dtype, scale):
    _check(sv, dtype, [140], scale=scale, peak=0.7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("peak", [1e-20, 20.0, 3000.0])
def test_flat_and_sharp_softmax(sv, dtype, peak):
    _check(sv, dtype, [300], peak=peak, heads=2, kv_heads=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_rise_all_the_way(sv, dtype):
    """Every tile's largest score is far above the one before, and far below in the other sequence."""
    import torch
    g = np.random.default_rng(0)
    n, dim = 600, 64
    q = np.ones((2 * n, 1, dim), np.float32)
    along = np.concatenate([np.arange(n), -np.arange(n)]) * 0.5
    k = round_to(np.ones((2 * n, 1, dim)) * along[:, None, None], dtype)
    v = round_to(g.normal(size=(2 * n, 1, dim)), dtype)
    starts = np.array([0, n, 2 * n], np.int32)
    out, lse = sv.prompt_attention(*(to_gpu(x, dtype) for x in (q, k, v)), new_start=to_gpu(starts), max_new=n, lse=True)
    near(out.double().cpu().numpy(), lse.double().cpu().numpy(), q, k, v, starts, dim ** -0.5, 0, 0, dtype)


def _strided(*dev):
    """Slices of one projection's output."""
    import torch
    every = torch.cat(dev, 1).contiguous()
    h, hk = dev[0].shape[1], dev[1].shape[1]
    return every[:, :h], every[:, h:h + hk], every[:, h + hk:]


def _shifted(by):
    def place(*dev):
        import torch
        made = []
        for x in dev:
            wide = torch.zeros((x.shape[0], x.shape[1] + 1, x.shape[2] + by), dtype=x.dtype, device="cuda")
            wide[:, 1:, by:] = x
            made.append(wide[:, 1:, by:])
        return made
    return place


def _heads_first(*dev):
    return [x.transpose(0, 1).contiguous().transpose(0, 1) for x in dev]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("place", [_strided, _shifted(1), _shifted(2), _shifted(4), _shifted(8), _heads_first],
                         ids=["fused", "by1", "by2", "by4", "by8", "heads_first"])
@pytest.mark.parametrize("dim", [64, 80, 256])
def test_strides_and_alignments(sv, dtype, place, dim):
    _check(sv, dtype, [150, 33], dim=dim, heads=6, kv_heads=2, place=place)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("stride", [2 ** 38, 2 ** 39, 2 ** 40 - 8])
def test_strides_beyond_those_of_a_tensor_map(sv, dtype, which, stride):
    """(Of a single row, which are never stepped over.)"""
    import torch
    g = np.random.default_rng(0)
    x = [to_gpu(x, dtype) for x in _inputs(g, dtype, 1, 4, 2, 64)]
    kw = dict(new_start=to_gpu(np.array([0, 1], np.int32)), max_new=1)
    want = sv.prompt_attention(*x, **kw)
    x[which] = x[which].as_strided(x[which].shape, (stride, 64, 1))
    assert torch.equal(sv.prompt_attention(*x, **kw), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 2, 4, 8, 16])
def test_results_with_strides_of_their_own(sv, dtype, shift):
    import torch
    g = np.random.default_rng(0)
    q, k, v = (to_gpu(x, dtype) for x in _inputs(g, dtype, 140, 4, 2, 64))
    kw = dict(new_start=to_gpu(np.array([0, 140], np.int32)), max_new=140)
    want = sv.prompt_attention(q, k, v, **kw)
    wide = torch.full((140, 5, 64 + shift), 9.0, dtype=q.dtype, device="cuda")
    out = sv.prompt_attention(q, k, v, out=wide[:, 1:, shift:], **kw)
    assert torch.equal(out, want)
    wide[:, 1:, shift:] = 9
    assert (wide == 9).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf"), "lowest"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_what_is_not_seen_has_no_influence(sv, dtype, dim, what, window, sinks):
    """Rows between and behind the sequences, and the next sequence, may hold anything."""
    import torch
    worst = torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min if what == "lowest" else what
    g = np.random.default_rng(1)
    heads, kv_heads = 4, 2
    lengths = [150, 97, 130]  # the second one is spoilt
    q, k, v = _inputs(g, dtype, sum(lengths) + 9, heads, kv_heads, dim)
    starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    dev = [to_gpu(x, dtype) for x in (q, k, v)]
    for x in dev:
        x[150:247] = worst
        x[377:] = worst
    out, lse = sv.prompt_attention(*dev, new_start=to_gpu(starts), max_new=150, window=window, sinks=sinks, lse=True)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for first, last in ((0, 150), (247, 377)):
        at = slice(first, last)
        near(out[at], lse[at], q[at], k[at], v[at], [0, last - first], dim ** -0.5, window, sinks, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads", [2, 6, 48])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (64, 3)])
def test_a_token_that_is_not_finite_spoils_those_that_see_it_alone(sv, dtype, dim, what, heads, window, sinks):
    import torch
    g = np.random.default_rng(2)
    n, kv_heads = 300, 2
    q, k, v = _inputs(g, dtype, n, heads, kv_heads, dim)
    i = np.arange(n)
    for bad in (0, 140, 257, 299):
        dev = [to_gpu(x, dtype) for x in (q, k, v)]
        dev[2][bad, 1, 5] = what
        sees = (i >= bad) & ((window == 0) | (i - bad < window) | (bad < sinks))
        out = sv.prompt_attention(*(x[None] for x in dev), window=window, sinks=sinks)[0].double().cpu().numpy()
        hit = np.zeros(out.shape, bool)
        hit[sees, heads // 2:, 5] = True
        assert (np.isfinite(out) == ~hit).all(), (bad, np.argwhere(np.isfinite(out) == hit)[:5].tolist())
        clean = sv.prompt_attention(*(to_gpu(x, dtype)[None] for x in (q, k, v)), window=window, sinks=sinks)[0].double().cpu().numpy()
        assert (np.where(hit, 0, out) == np.where(hit, 0, clean)).all()
        dev = [to_gpu(x, dtype) for x in (q, k, v)]
        dev[1][bad, 1, 5] = what
        out = sv.prompt_attention(*(x[None] for x in dev), window=window, sinks=sinks)[0].double().cpu().numpy()
        free = np.ones((n, heads), bool)
        free[sees, heads // 2:] = False
        assert (np.where(free[..., None], out, 0) == np.where(free[..., None], clean, 0)).all()
        if what != what:
            assert np.isnan(out[~free]).all()


def test_a_query_that_is_not_finite_spoils_its_row_alone(sv):
    g = np.random.default_rng(2)
    q, k, v = (to_gpu(x, "bf16")[None] for x in _inputs(g, "bf16", 200, 4, 2, 128))
    clean = sv.prompt_attention(q, k, v)
    q[0, 57, 2, 9] = float("nan")
    out = sv.prompt_attention(q, k, v)
    assert out[0, 57, 2].isnan().all()
    out[0, 57, 2] = clean[0, 57, 2]
    assert (out == clean).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_sequences_are_left_out(sv, dtype):
    import torch
    g = np.random.default_rng(0)
    q, k, v = _inputs(g, dtype, 60, 2, 1, 64)
    dev = [to_gpu(x, dtype) for x in (q, k, v)]
    for starts, max_new, flags in (([0, 20, 10, 30, 60], 30, [0, 128, 0, 0]), ([-1, 5, 30, 61, 60], 30, [128, 0, 128, 128]),
                                   ([0, 31, 32, 2 ** 31 - 1, -2 ** 31], 30, [128, 0, 128, 128])):
        st = torch.full((4,), -7, dtype=torch.int32, device="cuda")
        out = torch.full((60, 2, 64), 9.0, dtype=dev[0].dtype, device="cuda")
        sv.prompt_attention(*dev, new_start=to_gpu(np.array(starts, np.int32)), max_new=max_new, out=out, row_status=st)
        assert st.tolist() == flags
        out = out.double().cpu().numpy()
        untouched = np.ones(60, bool)
        for (a, b), bad in zip(zip(starts, starts[1:]), flags):
            if not bad:
                untouched[a:b] = False
                if starts[1] != 20 or a == 30:  # (rows of two sequences are one's or the other's)
                    near(out[a:b], None, q[a:b], k[a:b], v[a:b], [0, b - a], 64 ** -0.5, 0, 0, dtype)
        assert (out[untouched] == 9).all()


def test_bad_lengths_are_flagged_without_a_token_too(sv):
    import torch
    st = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    x = torch.zeros(0, 2, 64, device="cuda")
    sv.prompt_attention(x, x, x, new_start=to_gpu(np.array([0, 0, 1, 0], np.int32)), max_new=5, row_status=st)
    assert st.tolist() == [0, 128, 128]
    sv.prompt_attention(x, x, x, new_start=to_gpu(np.array([0, 0, 1, 0], np.int32)), max_new=0, row_status=st)
    assert st.tolist() == [0, 128, 128]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(sv, dtype):
    g = np.random.default_rng(8)
    _check(sv, dtype, [int(n) for n in g.integers(0, 9, 1500)], heads=2, kv_heads=1, dim=16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_call_gives_the_same_bits(sv, dtype):
    import torch
    g = np.random.default_rng(0)
    lengths = [int(n) for n in g.integers(1, 700, 20)]
    starts = to_gpu(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32))
    q, k, v = (to_gpu(x, dtype) for x in _inputs(g, dtype, sum(lengths), 8, 2, 128))
    first = sv.prompt_attention(q, k, v, new_start=starts, max_new=700, lse=True)
    for _ in range(10):
        again = sv.prompt_attention(q, k, v, new_start=starts, max_new=700, lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed_beside_another_stream(sv, dtype):
    import torch
    g = np.random.default_rng(0)
    q, k, v = (to_gpu(x, dtype) for x in _inputs(g, dtype, 500, 8, 2, 64))
    start = to_gpu(np.array([0, 200, 500], np.int32))
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        sv.prompt_attention(q, k, v, new_start=start, max_new=500, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            sv.prompt_attention(q, k, v, new_start=start, max_new=500, out=out)
    for at in (1, 250, 499):
        start[1] = at
        q.mul_(-1.25)
        want = sv.prompt_attention(q, k, v, new_start=start, max_new=500)
        torch.cuda.synchronize()
        graph.replay()
        beside = sv.prompt_attention(q, k, v, new_start=start, max_new=500)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(beside, want)
    with torch.cuda.stream(torch.cuda.default_stream()):
        other = sv.prompt_attention(q, k, v, new_start=start, max_new=500, stream=side)
    side.synchronize()
    assert torch.equal(other, want)


@pytest.mark.parametrize("dtype,shift", [("bf16", 0), ("bf16", 1), ("f32", 0)])
def test_offsets_beyond_32_bits(sv, dtype, shift):
    import torch
    g = np.random.default_rng(5)
    n, step = 40, 1 << 26
    dev = [to_gpu(x, dtype) for x in _inputs(g, dtype, n, 4, 2, 64)]
    memory = torch.empty(n * step, dtype=dev[0].dtype, device="cuda")
    far = [memory.as_strided((n, h, 64), (step, 64, 1), 1024 * i + shift) for i, h in enumerate((4, 2, 2, 4))]
    for x, y in zip(far, dev):
        x.copy_(y)
    out = sv.prompt_attention(*far[:3], out=far[3], new_start=to_gpu(np.array([0, n], np.int32)), max_new=n)
    near(out.double().cpu().numpy(), None, *(x.double().cpu().numpy() for x in dev), [0, n], 64 ** -0.5, 0, 0, dtype)
