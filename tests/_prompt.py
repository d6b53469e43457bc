"""Checks shared by the tests of prompt attention."""
import numpy as np

from oracle import prompt_oracle as PO


def tolerance(want, absolute, largest, length, dim, dtype):
    """Bounds of |out - want| and |lse - want_lse|, from the operations:
    scores are fp32 sums of dim exact products (float32 inputs: of products of
    three parts each, of which those below 2^-24 are left out), added 16 at a
    time with at most 2^-22 of the running sum of magnitudes lost each time,
    and are scaled and shifted in base 2 (a few roundings of 2^-24 of their
    size); exp2 is off by 2^-22; bf16 calls' weights are rounded to bf16
    (2^-8), fp32 ones' to 2^-22 at least; the value sums lose 2^-22 for each 16
    tokens; the result is rounded once more."""
    score = (dim / 16 + 10) * 2.0 ** -22 * largest + 2.0 ** -21
    weight = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22
    last = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    out = last * np.abs(want) + (1 + last) * (weight + 2 * score[..., None] + (length / 16 + 64) * 2.0 ** -22) * absolute + 1e-30
    lse = score + (length / 16 + 64) * 2.0 ** -22 + 2.0 ** -22 * (largest + 16)
    return out, lse


def near(out, lse, q, k, v, starts, scale, window, sinks, dtype):
    """out and lse (numpy) of packed sequences against the oracle."""
    dim = q.shape[-1]
    for b, (first, last) in enumerate(zip(starts, starts[1:])):
        rows = slice(first, last)
        want, wlse, absolute, largest = PO.attention(q[rows], k[rows], v[rows], scale, window, sinks)
        tol, ltol = tolerance(want, absolute, largest, last - first, dim, dtype)
        off = np.abs(out[rows] - want)
        assert np.isfinite(out[rows]).all(), (b, "not finite", np.argwhere(~np.isfinite(out[rows]))[:4].tolist())
        assert (off <= tol).all(), (b, float((off / tol).max()), np.argwhere(off > tol)[:4].tolist())
        if lse is not None:
            loff = np.abs(lse[rows] - wlse)
            assert (loff <= ltol).all(), (b, float((loff / ltol).max()))
