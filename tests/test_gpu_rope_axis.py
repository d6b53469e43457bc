"""Rotary positions with axes that are interleaved over the pairs, against the oracle."""
import numpy as np
import pytest

from _kv import round_to, to_gpu
from test_gpu_rope import _freq, _near, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dim,half", [(128, 64), (64, 24), (48, 21), (256, 128)])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_interleaved(sv, dtype, adjacent, dim, half, axes):  # noqa: F811
    g = np.random.default_rng(dim)
    x, positions = round_to(g.normal(size=(11, 6, dim)), dtype), g.integers(0, 5000, (axes, 11))
    for axis in ([i % axes for i in range(half)], g.integers(0, axes, half).tolist()):
        dev = to_gpu(x, dtype)
        for y, at in zip(sv.rope(dev[:, :4], dev[:, 4:], to_gpu(positions.astype(np.int32)), to_gpu(_freq(half)), axis=axis, adjacent=adjacent),
                         (slice(0, 4), slice(4, 6))):
            _near(y, x[:, at], positions, _freq(half), axis, adjacent, dtype)
