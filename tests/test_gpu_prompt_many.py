"""Prompt attention of many packed sequences and of long ones."""
import numpy as np
import pytest

from _kv import round_to, to_gpu
from _prompt import tolerance
from test_gpu_prompt_attention import _check, _inputs, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch", [90, 200, 700])
@pytest.mark.parametrize("dim", [16, 256])
def test_more_items_than_blocks(sv, dtype, batch, dim):  # noqa: F811
    """A launch has blocks for 4096 / kv_heads + 1 sequences more than their tokens fill; blocks take what is beyond."""
    g = np.random.default_rng(batch)
    _check(sv, dtype, [int(n) for n in g.integers(0, 4, batch - 1)] + [150], heads=32, kv_heads=32, dim=dim, ahead=2, behind=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_of_many_heads(sv, dtype):  # noqa: F811
    _check(sv, dtype, [1] * 300, heads=512, kv_heads=512, dim=16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bound_far_above_what_comes(sv, dtype):  # noqa: F811
    import torch
    g = np.random.default_rng(0)
    x = [to_gpu(x, dtype) for x in _inputs(g, dtype, 200, 4, 2, 64)]
    start = to_gpu(np.array([0, 70, 70, 200], np.int32))
    want = sv.prompt_attention(*x, new_start=start, max_new=130)
    assert torch.equal(sv.prompt_attention(*x, new_start=start, max_new=2 ** 31 - 1), want)


@pytest.mark.parametrize("dtype,dim,n", [("bf16", 64, 50_001), ("bf16", 128, 20_001), ("bf16", 256, 9_001), ("f32", 64, 9_001)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (5000, 7)])
def test_rows_of_a_long_prompt(sv, dtype, dim, n, window, sinks):  # noqa: F811
    """Some rows of it, the last ones among them, against float64."""
    g = np.random.default_rng(dim)
    q, k, v = _inputs(g, dtype, n, 2, 1, dim)
    out, lse = sv.prompt_attention(*(to_gpu(x, dtype)[None] for x in (q, k, v)), window=window, sinks=sinks, lse=True)
    out, lse = out[0].double().cpu().numpy(), lse[0].double().cpu().numpy()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    kk, vv = k[:, 0].astype(np.float64), v[:, 0].astype(np.float64)
    for i in sorted({0, 1, 4999, 5000, n - 1, n - 2, *g.integers(0, n, 20).tolist()}):
        j = np.arange(i + 1)
        seen = j if not window else j[(i - j < window) | (j < sinks)]
        for h in range(2):
            s = kk[seen] @ q[i, h].astype(np.float64) * dim ** -0.5
            w = np.exp(s - s.max())
            wlse, w = s.max() + np.log(w.sum()), w / w.sum()
            want, absolute = w @ vv[seen], w @ np.abs(vv[seen])
            largest = (np.abs(kk[seen]) @ np.abs(q[i, h].astype(np.float64))).max() * dim ** -0.5
            tol, ltol = tolerance(want[None], absolute[None], np.array([largest]), len(seen), dim, dtype)
            assert (np.abs(out[i, h] - want) <= tol[0]).all() and abs(lse[i, h] - wlse) <= ltol[0], (i, h)


@pytest.mark.parametrize("dim", [64, 256])
def test_what_sums_of_a_long_bf16_prompt_lose(sv, dim):  # noqa: F811
    """Values of 1 have sums of 1: what a row's result is less, beyond its rounding, is lost in the sums over values, at most 2^-23
    with each 16 tokens, of weights that are bf16's to 2^-8 each, evenly to both sides.  Beside 1 bf16 has steps of 2^-8 below and
    2^-7 above: a result may be half a step and that off."""
    import torch
    n = 200_000 if dim == 64 else 60_000
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k = (torch.randn(1, n, 1, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    out = sv.prompt_attention(q, k, torch.ones_like(k))[0].double()
    i = torch.arange(n, device="cuda", dtype=torch.float64)
    # (a row's weights are rounded with errors that are evenly spread: their sum's is well within 2^-8 / 8 from 1000 tokens on)
    tol = 2.0 ** -8 + (i / 16 + 1) * 2.0 ** -23 + torch.where(i < 1000, 2.0 ** -8, 2.0 ** -11)
    off = (out - 1).abs().amax((1, 2))
    assert (off <= tol).all(), (off - tol).max().item()
