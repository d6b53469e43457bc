"""Rotary positions at angles next to a multiple of a quarter turn, and at
frequencies that are none.

An angle is a number of 2^-64 turns, at most one of them too small for each
position; the rest behind the nearest quarter turn becomes a float by two
conversions and two products (4 roundings of 2^-24 with the constant's), the
sine takes two more and leaves out a term below 2^-29: 2^-21 of the value, and
2 pi 2^-64 for each position.  A result of one pair value alone is that times
the value, rounded once."""
import numpy as np
import pytest

from _kv import to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


PI = "3.14159265358979323846264338327950288419716939937510582097494459230781640628620899"


def _cos_sin(position, freq):
    """Of position * freq (a float32), by series in 60 digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi = Decimal(PI)
    t = Decimal(int(position)) * Decimal(float(freq))
    quarters = (t / (pi / 2)).to_integral_value()
    t -= quarters * (pi / 2)

    def series(x, n):
        total, n0 = Decimal(0), n
        while abs(x) > Decimal(10) ** -45 or n == n0:
            total += x
            x = -x * t * t / ((n + 1) * (n + 2))
            n += 2
            if x == 0:
                break
        return total
    c, s = series(Decimal(1), 0), series(t, 1) if t else Decimal(0)
    for _ in range(int(quarters) % 4):
        c, s = -s, c
    return float(c), float(s)


HALF = float(np.float32(np.pi / 2))
FREQS = [2.4e-6, 1e-7, 3.3e-8, 7.1e-5, 1e-3, HALF, -HALF, -2.4e-6, 2 * HALF, 3 * HALF, 0.37, 1.0]


@pytest.mark.parametrize("half", [16, 12])  # whole vectors; pairs one by one
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("position", [0, 1, -1, 2, 3, 37, -1000, 65_537])
def test_small_angles_keep_their_bits(sv, half, adjacent, position):
    import torch
    freq = np.array((FREQS + [5e-9, 1.0, 1e-6, 0.25])[:half], np.float32)
    x = torch.zeros(1, 2, 64, device="cuda")
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if adjacent else (slice(0, half), slice(half, 2 * half))
    x[0, 0, first] = 1  # (cos, sin)
    x[0, 1, second] = 1  # (-sin, cos)
    q, _ = sv.rope(x, None, to_gpu(np.array([position], np.int32)), to_gpu(freq), adjacent=adjacent)
    got = q[0].double().cpu().numpy()
    c, s = np.array([_cos_sin(position, f) for f in freq]).T
    lost = abs(position) * 2 * np.pi * 2.0 ** -64
    for have, want in ((got[0, first], c), (got[0, second], s), (got[1, first], -s), (got[1, second], c)):
        off, tol = np.abs(have - want), (2.0 ** -21 + 2.0 ** -24) * np.abs(want) + lost
        assert (off <= tol).all(), (freq[off > tol].tolist(), (off / np.maximum(np.abs(want), 1e-300))[off > tol].tolist())


NONE = [np.nan, np.inf, -np.inf, 2.0 ** 60, -2.0 ** 60, 2.0 ** 63, 2.0 ** 64, 1e30, float(np.finfo(np.float32).max)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,half", [(64, 32), (64, 31), (128, 16)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
def test_pairs_of_a_frequency_that_is_none_are_nan(sv, dtype, dim, half, adjacent, axes):
    import torch
    g = np.random.default_rng(0)
    freq = (10000.0 ** (-np.arange(half) / half)).astype(np.float32)
    bad = g.permutation(half)[:len(NONE)]
    freq[np.setdiff1d(np.arange(half), bad)[0]] = np.nextafter(np.float32(2.0 ** 60), np.float32(0))
    x = to_gpu(g.normal(size=(5, 6, dim)).astype(np.float32), dtype)
    positions = to_gpu(g.integers(0, 1000, (axes, 5)).astype(np.int32))
    kw = dict(adjacent=adjacent, sections=None if axes == 1 else (half - 2, 1, 1))
    positions = positions[0].contiguous() if axes == 1 else positions
    clean = sv.rope(x[:, :4], x[:, 4:], positions, to_gpu(freq), **kw)
    assert all(y.isfinite().all() for y in clean)
    freq[bad] = NONE
    for y, want in zip(sv.rope(x[:, :4], x[:, 4:], positions, to_gpu(freq), **kw), clean):
        hit = torch.zeros(dim, dtype=torch.bool, device="cuda")
        for i in bad.tolist():
            hit[[2 * i, 2 * i + 1] if adjacent else [i, i + half]] = True
        assert y[..., hit].isnan().all()
        assert torch.equal(y[..., ~hit], want[..., ~hit])
