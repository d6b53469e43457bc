"""Rotary positions on the GPU against the oracle.

The angle's sine and cosine are off by 2^-23 at most, so a result before its
last rounding is off by at most (2 * 2^-23 + 2 * 2^-24) of |a| + |b|, which is
within sqrt(2) of the pair's length; the last rounding is 2^-24 of the value
(float32, with 2^-149 below the smallest normal value) or 2^-8 (bfloat16)."""
import numpy as np
import pytest

from oracle import prompt_oracle as PO

from _kv import round_to, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


def _freq(half, base=10000.0):
    return (base ** (-np.arange(half) / half)).astype(np.float32)


def _near(got, x, positions, freq, axis, adjacent, dtype):
    want, size = PO.rope(x, positions, freq, axis, adjacent)
    last = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = last * np.abs(want) + 1.4143 * 3 * 2.0 ** -23 * size * (1 + last) + 2.0 ** -133
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= np.where(size > 0, tol, 0)).all(), float((off / tol).max())


def _check(sv, dtype="bf16", rows=7, heads=5, kv_heads=2, dim=64, half=None, adjacent=False, sections=None, positions=None, base=10000.0,
           pad=0, shift=0, inplace=False, seed=0, freq=None):
    import torch
    g = np.random.default_rng(seed)
    half = dim // 2 if half is None else half
    axes = 1 if sections is None else len(sections)
    axis = [0] * half if sections is None else [a for a, n in enumerate(sections) for _ in range(n)]
    positions = g.integers(0, 5000, (axes, rows)) if positions is None else np.broadcast_to(positions, (axes, rows))
    freq = _freq(half, base) if freq is None else freq
    x = [round_to(g.normal(size=(rows, h, dim)), dtype) for h in (heads, kv_heads)]
    dev = []
    for y in x:
        t = to_gpu(y, dtype)
        wide = torch.full((rows, y.shape[1] + 1, dim + pad), 3.0, dtype=t.dtype, device="cuda")
        flat = torch.full((wide.numel() + shift,), 3.0, dtype=t.dtype, device="cuda")
        view = flat[shift:].view(wide.shape)[:, 1:, :dim]
        view.copy_(t)
        dev.append((flat, view))
    p = to_gpu(positions.astype(np.int32))
    p = p[0].contiguous() if axes == 1 else p
    kw = dict(sections=sections, adjacent=adjacent)
    if inplace:
        kw["out"] = (dev[0][1], dev[1][1])
    q, k = sv.rope(dev[0][1], dev[1][1], p, to_gpu(freq), **kw)
    for got, y, (flat, view) in zip((q, k), x, dev):
        _near(got, y, positions, freq, axis, adjacent, dtype)
        rest = flat.clone()
        rest[shift:].view(rows, y.shape[1] + 1, dim + pad)[:, 1:, :dim] = 3.0
        assert (rest == 3.0).all()
        if not inplace:
            assert torch.equal(view, to_gpu(y, dtype))
    return q, k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 160, 192, 256])
def test_head_dims(sv, dtype, adjacent, dim):
    _check(sv, dtype, dim=dim, adjacent=adjacent, heads=dim // 16 + 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dim,half", [(16, 1), (16, 7), (64, 8), (80, 24), (128, 33), (128, 32), (128, 16), (256, 96), (256, 5)])
def test_part_of_the_dims(sv, dtype, adjacent, dim, half):
    _check(sv, dtype, dim=dim, half=half, adjacent=adjacent)


@pytest.mark.parametrize("sections", [(16, 24, 24), (64, 0), (1, 2, 3, 58), (0, 0, 64), (64,)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_axes(sv, sections, adjacent, dtype):
    _check(sv, dtype, dim=128, sections=sections, adjacent=adjacent, rows=11)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (8, 0), (16, 0), (3, 0), (2, 2), (0, 8), (0, 4)])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("half", [32, 16])
def test_strides_and_alignments(sv, dtype, pad, shift, inplace, half):
    _check(sv, dtype, pad=pad, shift=shift, inplace=inplace, half=half)
    _check(sv, dtype, pad=pad, shift=shift, inplace=inplace, half=half, adjacent=True)


@pytest.mark.parametrize("position", [0, 1, -1, 131_071, 16_777_217, 2 ** 31 - 1, -2 ** 31, -987_654_321])
def test_far_positions(sv, position):
    _check(sv, "f32", dim=128, positions=position, base=500000.0)
    _check(sv, "f32", dim=128, positions=position, freq=np.linspace(-7, 7, 64).astype(np.float32))


@pytest.mark.parametrize("rows,heads,kv_heads", [(1, 1, 1), (1, 64, 8), (3, 200, 1), (1000, 3, 3), (5001, 28, 4), (65_537, 1, 1)])
def test_numbers_of_rows_and_heads(sv, rows, heads, kv_heads):
    _check(sv, "bf16", rows=rows, heads=heads, kv_heads=kv_heads, dim=64)


def test_queries_alone_batches_and_none(sv):
    import torch
    g = np.random.default_rng(0)
    x = to_gpu(g.normal(size=(3, 5, 4, 64)).astype(np.float32))
    positions = to_gpu(g.integers(0, 99, (3, 5)).astype(np.int32))
    freq = to_gpu(_freq(32))
    q, k = sv.rope(x, None, positions, freq)
    assert k is None and q.shape == x.shape
    _near(q.reshape(15, 4, 64), x.reshape(15, 4, 64).cpu().numpy(), positions.reshape(1, 15).cpu().numpy(), _freq(32), [0] * 32, False, "f32")
    both = sv.rope(x, x[:, :, :2], positions, freq)
    assert torch.equal(both[0], q) and torch.equal(both[1], q[:, :, :2])
    three = sv.rope(x, None, positions.expand(3, 3, 5).contiguous(), freq, sections=(4, 8, 20))
    assert torch.equal(three[0], q)
    empty = sv.rope(x[:0], x[:0], positions[:0], freq)
    assert empty[0].shape == (0, 5, 4, 64)


def test_values_that_are_not_finite_stay_in_their_pair(sv):
    import torch
    x = torch.ones(1, 2, 64, device="cuda")
    x[0, 0, 3] = float("inf")
    x[0, 1, 40] = float("nan")
    q, _ = sv.rope(x, None, to_gpu(np.array([5], np.int32)), to_gpu(_freq(32)))
    assert sorted(torch.nonzero(~q[0, 0].isfinite()).flatten().tolist()) == [3, 35]
    assert sorted(torch.nonzero(~q[0, 1].isfinite()).flatten().tolist()) == [8, 40]


def test_captured_and_replayed(sv):
    import torch
    g = np.random.default_rng(0)
    x = to_gpu(g.normal(size=(9, 4, 64)).astype(np.float32), "bf16")
    positions, freq = to_gpu(np.arange(9, dtype=np.int32)), to_gpu(_freq(32))
    out = (torch.empty_like(x), None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.rope(x, None, positions, freq, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            sv.rope(x, None, positions, freq, out=out)
    positions.add_(1000)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], sv.rope(x, None, positions, freq)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_offsets_beyond_32_bits(sv, dtype, shift):
    import torch
    g = np.random.default_rng(5)
    n, step = 40, 1 << 26
    rows, positions, freq = [round_to(g.normal(0, 1, (n, h, 64)), dtype) for h in (4, 2)], np.arange(n, dtype=np.int32), _freq(32)
    memory = torch.empty(n * step, dtype=to_gpu(rows[0], dtype).dtype, device="cuda")
    far = [memory.as_strided((n, h, 64), (step, 64, 1), 1024 * i + shift) for i, h in enumerate((4, 2))]
    for x, y in zip(far, rows):
        x.copy_(to_gpu(y, dtype))
    for x, y in zip(sv.rope(*far, to_gpu(positions), to_gpu(freq), out=tuple(far)), rows):
        _near(x, y, positions[None], freq, np.zeros(32, int), False, dtype)
