"""Prompt attention of more sequences than a block sorts: each item is found,
and what finding costs grows with the number of sequences, not with its square."""
import numpy as np
import pytest

from _kv import to_gpu
from _prompt import near
from test_gpu_prompt_attention import _check, _inputs, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch", [96, 97, 129, 192, 193, 1000])
@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (48, 48), (60, 1)])
def test_packed(sv, dtype, batch, heads, kv_heads):  # noqa: F811
    """Lengths that differ much, none at all among them; with 48 kv heads more items than blocks."""
    g = np.random.default_rng(batch)
    lengths = [int(n) for n in g.integers(0, 5, batch)]
    for at, n in zip(g.permutation(batch)[:5], (0, 300, 129, 64, 513)):
        lengths[at] = n
    _check(sv, dtype, lengths, heads=heads, kv_heads=kv_heads, dim=32, ahead=1, behind=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,n,heads,kv_heads", [(97, 1, 2, 1), (97, 130, 4, 2), (200, 9, 48, 48), (1000, 3, 6, 2), (300, 2, 64, 1)])
def test_padded(sv, dtype, batch, n, heads, kv_heads):  # noqa: F811
    _check(sv, dtype, [n] * batch, heads=heads, kv_heads=kv_heads, dim=32, ragged=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch", [5000, 65_535])
@pytest.mark.parametrize("ragged", [False, True])
def test_single_tokens_get_their_values(sv, dtype, batch, ragged):  # noqa: F811
    """(Weights of 1: results are the values themselves; float32 ones to 2^-21, of parts of 8 bits.)"""
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    make = lambda h: torch.randn(batch, h, 16, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)  # noqa: E731
    q, k, v = make(6), make(3), make(3)
    if ragged:
        gone = torch.arange(batch, device="cuda") % 7 == 3  # these have none, the one before them has two
        lengths = torch.where(gone, 0, torch.where(gone.roll(-1), 2, 1))
        start = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)]).int()
        total = int(start[-1])
        out = sv.prompt_attention(q[:total], k[:total], v[:total], new_start=start, max_new=5)
        first = start[:-1][lengths > 0].long()
        out, v = out[first], v[first]
    else:
        out = sv.prompt_attention(*(x[:, None] for x in (q, k, v)))[:, 0]
    want = v.repeat_interleave(2, 1)
    assert torch.equal(out, want) if dtype == "bf16" else ((out - want).abs() <= 2.0 ** -21 * want.abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_that_are_left_out_among_many(sv, dtype):  # noqa: F811
    import torch
    g = np.random.default_rng(1)
    lengths = g.integers(0, 9, 700)
    starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    total = int(starts[-1])
    given = starts.copy()
    given[[50, 333, 334, 600]] = [total + 5, -3, 2 ** 31 - 1, -2 ** 31]
    n = np.diff(given.astype(np.int64))
    good = (n >= 0) & (n <= 12) & (given[:-1] >= 0) & (given[:-1] + n <= total)
    q, k, v = _inputs(g, dtype, total, 4, 2, 32)
    st = torch.full((700,), -7, dtype=torch.int32, device="cuda")
    out = torch.full((total, 4, 32), 9.0, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    sv.prompt_attention(*(to_gpu(x, dtype) for x in (q, k, v)), new_start=to_gpu(given), max_new=12, out=out, row_status=st)
    assert (st.cpu().numpy() == np.where(good, 0, 128)).all() and (~good).sum() >= 6
    out = out.double().cpu().numpy()
    untouched = np.ones(total, bool)
    for b in np.flatnonzero(good):
        rows = slice(given[b], given[b + 1])
        untouched[rows] = False
        near(out[rows], None, q[rows], k[rows], v[rows], [0, int(n[b])], 32 ** -0.5, 0, 0, dtype)
    assert untouched.any() and (out[untouched] == 9).all()


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_four_times_the_sequences_take_about_four_times_as_long(sv, dtype, ragged):  # noqa: F811
    """(Fifteen times when each search went through all sequences.)"""
    import torch

    def best(batch):
        x = torch.randn(batch, 8, 24, 16, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        kw = {}
        if ragged:
            x = x.flatten(0, 1)
            kw = dict(new_start=torch.arange(batch + 1, dtype=torch.int32, device="cuda") * 8, max_new=8)
        q, k, v = x[..., :8, :], x[..., 8:16, :], x[..., 16:, :]
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            sv.prompt_attention(q, k, v, **kw)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    assert best(16_000) <= 8 * best(4000)
