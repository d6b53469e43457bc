"""The cache oracle against statements of its own parts (no GPU)."""
import numpy as np
import pytest

from oracle import kv_oracle as KO


def test_code_values_match_the_framework_type():
    import torch
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(codes, KO.VALUE)


def test_encode_matches_the_type_conversion():
    import torch
    g = np.random.default_rng(0)
    x = np.concatenate([g.normal(0, s, 20000) for s in (1e-3, 0.02, 1, 100)] + [KO._POSITIVE, (KO._POSITIVE[1:] + KO._POSITIVE[:-1]) / 2])
    x = np.clip(np.concatenate([x, -x]), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(KO.encode(x), want)
    assert KO.encode(np.nan) == 0 and KO.encode(np.inf) == 0x7e and KO.encode(-np.inf) == 0xfe


@pytest.mark.parametrize("a,s", [(0.0, 2.0 ** -100), (448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8),
                                 (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (3e38, 2.0 ** 120)])
def test_need(a, s):
    assert KO.need(a) == s


def test_append_keeps_the_page_invariants():
    """Tokens one at a time: every stored value is within half a step (2^-4
    relative) of its input, or 2^-10 of the page's scale."""
    g = np.random.default_rng(1)
    page, table = 16, np.array([2, 0])
    cache = dict(k=np.full((3, 2, page, 16), 0x55, np.uint8), v=np.full((3, 2, page, 16), 0x55, np.uint8),
                 k_scale=np.full((3, 2), 8.0), v_scale=np.full((3, 2), 8.0))
    x = g.normal(0, 1, (20, 2, 16)) * np.exp(g.normal(0, 1.5, (20, 1, 1)))
    for t in range(20):
        assert not KO.append(cache, x[t:t + 1], -x[t:t + 1], table, page, t)
    back = KO.read(cache, "k", table, page, 0, 20)
    scale = cache["k_scale"][table[np.arange(20) // page]][:, :, None]
    # each growth may round once more, but only what is subnormal under the new scale
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -9 * scale)).all()
    np.testing.assert_array_equal(KO.read(cache, "v", table, page, 0, 20), -back)
    assert (cache["k"][1] == 0x55).all()  # no page of the sequence


def test_visible_by_hand():
    #      0
    #     / \
    #    1   2
    #    |
    #    3
    parents = [-1, 0, 0, 1]
    v = KO.visible(2, 4, parents, 0, 0).astype(int).tolist()
    assert v == [[1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 0], [1, 1, 1, 0, 1, 0], [1, 1, 1, 1, 0, 1]]
    v = KO.visible(2, 4, parents, 2, 1).astype(int).tolist()  # the last two positions, and token 0
    assert v == [[1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 1, 0, 1, 0], [1, 0, 0, 1, 0, 1]]
    assert KO.visible(0, 1, None, 1, 0).tolist() == [[True]]


def test_attention_of_equal_scores_is_the_mean():
    g = np.random.default_rng(2)
    page, table = 16, np.array([1, 0, 2])
    cache = dict(k=np.zeros((3, 1, page, 16), np.uint8), v=KO.encode(g.normal(0, 50, (3, 1, page, 16))),
                 k_scale=np.ones((3, 1)), v_scale=np.ones((3, 1)))
    q = g.normal(0, 1, (2, 2, 16))
    out, lse, _, _ = KO.attention(q, cache, table, page, 38, None, 0.25, 0, 0)
    v = KO.read(cache, "v", table, page, 0, 40)[:, 0]
    for i in range(2):
        np.testing.assert_allclose(out[i], np.stack([v[:39 + i].mean(0)] * 2), rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(lse[i], np.log(39 + i), rtol=1e-12)


def test_commit_is_read_then_append():
    g = np.random.default_rng(3)
    page, table = 16, np.array([3, 1, 0])
    cache = dict(k=KO.encode(g.normal(0, 60, (4, 2, page, 16))), v=KO.encode(g.normal(0, 60, (4, 2, page, 16))),
                 k_scale=2.0 ** g.integers(-3, 3, (4, 2)).astype(float), v_scale=2.0 ** g.integers(-3, 3, (4, 2)).astype(float))
    before = {n: KO.read(cache, n, table, page, 0, 40) for n in ("k", "v")}
    assert KO.commit(cache, table, page, 13, [0, 2, 3, 11]) == 17
    for n in ("k", "v"):
        after = KO.read(cache, n, table, page, 0, 17)
        scale = cache[n + "_scale"][table[np.arange(17) // page]][:, :, None]
        want = np.concatenate([before[n][:13], before[n][[13, 15, 16, 24]]])
        assert (np.abs(after - want) <= 2.0 ** -10 * scale).all()
