"""Inputs and checks shared by the cache and attention tests."""
import numpy as np

from oracle import kv_oracle as KO

TYPES = ("bf16", "f32")


def round_to(x, dtype):
    """x as the type holds it (float32 array)."""
    x = np.asarray(x, np.float32)
    if dtype == "f32":
        return x
    import torch
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy()


def to_gpu(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def lay(codes, layout):
    """A [pages, heads, page, dim] uint8 array on the GPU with the memory order ``layout``."""
    t = to_gpu(codes)
    return t.transpose(1, 2).contiguous().transpose(1, 2) if layout == "nhd" else t


def make_cache(g, pages, heads, page, dim, spread=2):
    """A host cache with codes of every kind but NaN and scales about 2^-6."""
    def codes():
        c = KO.encode(np.clip(g.normal(0, 75, (pages, heads, page, dim)), -448, 448))
        return np.where(g.random(c.shape) < 0.02, g.integers(0, 0x7f, c.shape).astype(np.uint8), c)

    def scales():
        return 2.0 ** g.integers(-6 - spread, -6 + spread + 1, (pages, heads)).astype(np.float64)
    return dict(k=codes(), v=codes(), k_scale=scales(), v_scale=scales())


def copy(cache):
    return {n: a.copy() for n, a in cache.items()}


def cache_gpu(cache, layout="hnd"):
    return dict(k=lay(cache["k"], layout), v=lay(cache["v"], layout),
                k_scale=to_gpu(cache["k_scale"].astype(np.float32)), v_scale=to_gpu(cache["v_scale"].astype(np.float32)))


def same_cache(got, want):
    for n in ("k", "v"):
        np.testing.assert_array_equal(got[n].cpu().numpy(), want[n])
        np.testing.assert_array_equal(got[n + "_scale"].cpu().numpy().astype(np.float64), want[n + "_scale"])


def make_table(g, lengths, page, free=2):
    """Page table of sequences that own disjoint, shuffled pages, and the pool's size."""
    used = [-(-n // page) for n in lengths]
    pool = g.permutation(sum(used) + free)
    table = np.zeros((len(lengths), max(1, max(used))), np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = pool[at:at + n]
        at += n
    return table, len(pool)


def attention_tolerance(want, absolute, largest, length, dim, dtype):
    """Bounds of |out - want| and |lse - want_lse|, from the operations:
    scores are fp32 sums of dim exact products, added 16 at a time with at most
    2^-22 of the running sum of magnitudes lost each time, and are scaled and
    shifted in base 2 (a few roundings of 2^-24 of their size); exp2 is off by
    2^-22; bf16 queries' weights are rounded to half the step of fp16 (2^-11),
    fp32 ones' to 2^-21; the value sums lose 2^-22 for each 16 tokens; the
    result is rounded once more."""
    score = (dim / 16 + 8) * 2.0 ** -22 * largest + 2.0 ** -21
    weight = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    last = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    out = last * np.abs(want) + (weight + 2 * score[..., None] + (length / 16 + 64) * 2.0 ** -22) * absolute + 1e-30
    lse = score + (length / 16 + 64) * 2.0 ** -22 + 2.0 ** -22 * (largest + 16)
    return out, lse
