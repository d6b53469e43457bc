"""Infinities and NaN in the queries and keys of prompt attention.

bf16 calls take the formula as it stands: a score of -inf has weight 0, a row
that sees no other is NaN with a log-sum-exp of -inf, and a score that is NaN or
inf makes NaN of both.  float32 calls, which multiply parts of the values, make
NaN of all that such a query or key enters."""
import numpy as np
import pytest

from _kv import round_to, to_gpu
from _prompt import near, tolerance
from oracle import prompt_oracle as PO

pytestmark = pytest.mark.gpu

N, HEADS, KV_HEADS = 300, 4, 2


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


def _call(sv, rows, dtype, shift, window, sinks):
    """shift: elements that rows lie off their boundary, which takes the other kernel of bf16 rows."""
    import torch
    dev = []
    for x in rows:
        wide = torch.zeros(N, x.shape[1], x.shape[2] + 8, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
        wide[..., shift:shift + x.shape[2]] = to_gpu(x, dtype)
        dev.append(wide[None, ..., shift:shift + x.shape[2]])
    out, lse = sv.prompt_attention(*dev, window=window, sinks=sinks, lse=True)
    return out[0].double().cpu().numpy(), lse[0].double().cpu().numpy()


def _formula(q, k, v, scale, window, sinks):
    """out, lse in float64; of rows that are NaN both are, of rows that see scores of -inf alone the lse is -inf."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    sees = PO.sees(N, window, sinks)
    outs, sums = [], []
    with np.errstate(all="ignore"):
        for h in range(HEADS):
            g = h // (HEADS // KV_HEADS)
            s = np.where(sees, (q[:, None, h] * k[None, :, g]).sum(-1) * scale, -np.inf)
            top = s.max(-1, keepdims=True)
            w = np.where(sees, np.exp(s - top), 0)
            total = w.sum(-1, keepdims=True)
            bad = np.isnan(total) | (top == np.inf)
            none = (top == -np.inf) & ~np.isnan(s).any(-1, keepdims=True)
            outs.append(np.where(bad | none, np.nan, w @ v[:, g] / total))
            sums.append(np.where(none, -np.inf, np.where(bad, np.nan, top + np.log(total)))[:, 0])
    return np.stack(outs, 1), np.stack(sums, 1)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_bf16_follows_the_formula(sv, dim, shift, what, window, sinks):
    g = np.random.default_rng(dim)
    rows = [round_to(g.normal(0, s, (N, h, dim)), "bf16") for h, s in ((HEADS, 1.5), (KV_HEADS, 1), (KV_HEADS, 1))]
    for tokens in ((0,), (0, 1, 2), (140,), (3, 257, 299)):
        q, k, v = (x.copy() for x in rows)
        k[list(tokens), 1, 5] = what
        q[:, :, 5] = np.where(np.arange(N)[:, None] % 3 == 0, -1, 1) * np.abs(q[:, :, 5])
        q[::7, 2, 5] = 0
        want, wlse = _formula(q, k, v, dim ** -0.5, window, sinks)
        assert np.isfinite(want[:, :2]).all() and np.isnan(want[:, 2:]).any()
        out, lse = _call(sv, (q, k, v), "bf16", shift, window, sinks)
        assert (np.isnan(out) == np.isnan(want)).all(), (tokens, np.argwhere(np.isnan(out) != np.isnan(want))[:4].tolist())
        assert (np.isnan(lse) == np.isnan(wlse)).all() and ((lse == -np.inf) == (wlse == -np.inf)).all()
        # (a key of weight 0 leaves the others their error bounds: those of the same call without infinities)
        _, _, absolute, largest = PO.attention(q, rows[1], v, dim ** -0.5, window, sinks)
        known = np.isfinite(want).all(-1)
        spread = np.abs(v).max()
        tol, ltol = tolerance(want, np.minimum(absolute + spread, 2 * spread), largest, N, dim, "bf16")
        assert (np.abs(out[known] - want[known]) <= tol[known]).all() and (np.abs(lse[known] - wlse[known]) <= ltol[known]).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_float32_results_that_a_key_enters_are_nan(sv, dim, what, window, sinks):
    g = np.random.default_rng(dim)
    q, k, v = (round_to(g.normal(0, s, (N, h, dim)), "f32") for h, s in ((HEADS, 1.5), (KV_HEADS, 1), (KV_HEADS, 1)))
    # values whose second and third parts have their sign, or are 0: such infinities gave scores of their own
    q[::2, :, 5] = np.float32(1 + 2 ** -10 + 2 ** -18)
    q[1::4, :, 5] = 2
    i = np.arange(N)
    for bad in (0, 140, 257, 299):
        spoilt = k.copy()
        spoilt[bad, 1, 5] = what
        sees = (i >= bad) & ((window == 0) | (i - bad < window) | (bad < sinks))
        out, lse = _call(sv, (q, spoilt, v), "f32", 0, window, sinks)
        hit = np.zeros((N, HEADS), bool)
        hit[sees, HEADS // 2:] = True
        assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all(), (bad, np.argwhere(hit & ~np.isnan(lse))[:4].tolist())
        out[hit], lse[hit] = 0, 0
        clean = _call(sv, (q, k, v), "f32", 0, window, sinks)
        assert (out[~hit] == clean[0][~hit]).all() and (lse[~hit] == clean[1][~hit]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
def test_a_query_s_row_is_nan(sv, dtype, dim, what):
    """(Its scores are inf for some keys, or -inf for all that it sees.)"""
    g = np.random.default_rng(dim)
    q, k, v = (round_to(g.normal(0, s, (N, h, dim)), dtype) for h, s in ((HEADS, 1.5), (KV_HEADS, 1), (KV_HEADS, 1)))
    rows = [0, 1, 57, 130, 299]
    spoilt = q.copy()
    spoilt[rows, 2, 9] = what
    out, lse = _call(sv, (spoilt, k, v), dtype, 0, 0, 0)
    assert np.isnan(out[rows, 2]).all()
    if dtype == "f32":
        assert np.isnan(lse[rows, 2]).all()
    hit = np.zeros((N, HEADS), bool)
    hit[rows, 2] = True
    clean = _call(sv, (q, k, v), dtype, 0, 0, 0)
    assert (out[~hit] == clean[0][~hit]).all() and (lse[~hit] == clean[1][~hit]).all()
    near(*(np.where(hit[..., None] if x.ndim == 3 else hit, y, x) for x, y in zip((out, lse), clean)), q, k, v, [0, N], dim ** -0.5, 0, 0, dtype)
