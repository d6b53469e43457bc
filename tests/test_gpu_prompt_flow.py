"""A request's way, as a serving loop takes it: pages, rotary positions, the
prompt's attention, the cache; then draft trees with their positions, the
commit, and pages that go back.  Against the oracles, one operator after the
other on what the one before it gave."""
import numpy as np
import pytest

from oracle import kv_oracle as KO
from oracle import prompt_oracle as PO

from _kv import round_to, to_gpu
from _prompt import near

pytestmark = pytest.mark.gpu

HEADS, KV_HEADS, DIM, PAGE = 8, 2, 64, 16


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


def _ints(x):
    return to_gpu(np.array(x, np.int32))


def _turned(x, positions, freq):
    want, size = PO.rope(x, [positions], freq, [0] * len(freq), False)
    return want, 2.0 ** -8 * np.abs(want) + 1.5 * 3 * 2.0 ** -23 * size * 1.01 + 1e-30


@pytest.mark.parametrize("seed", [0, 1])
def test_prompts_then_trees(sv, seed):
    import torch
    g = np.random.default_rng(seed)
    lengths = [150, 1, 77, 33]
    B, nodes = len(lengths), 12
    freq = (10000.0 ** (-np.arange(DIM // 2) / (DIM // 2))).astype(np.float32)
    pool, table, held = sv.kv_pool(64, "cuda"), torch.full((B, 14), -1, dtype=torch.int32, device="cuda"), _ints([0] * B)
    cache = sv.kv_cache(64, KV_HEADS, DIM, PAGE, "cuda")
    host = dict(k=np.zeros((64, KV_HEADS, PAGE, DIM), np.uint8), k_scale=np.ones((64, KV_HEADS)),
                v=np.zeros((64, KV_HEADS, PAGE, DIM), np.uint8), v_scale=np.ones((64, KV_HEADS)))
    free, count, otable, oheld = list(range(63, -1, -1)), 64, [[-1] * 14 for _ in range(B)], [0] * B

    def same_places(got, want_slots, want_positions):
        assert table.tolist() == otable and held.tolist() == oheld and pool["count"].tolist() == [count]
        assert got["slots"].flatten().tolist() == [want_slots[r] for r in range(len(want_slots))]
        assert got["positions"].flatten().tolist() == [want_positions[r] for r in range(len(want_positions))]

    # the prompts: packed rows of one projection's output
    starts = np.concatenate([[0], np.cumsum(lengths)])
    n = int(starts[-1])
    x = round_to(g.normal(size=(n, HEADS + 2 * KV_HEADS, DIM)), "bf16")
    dev = to_gpu(x, "bf16")
    q, k, v = dev[:, :HEADS], dev[:, HEADS:HEADS + KV_HEADS], dev[:, HEADS + KV_HEADS:]
    lens, start = _ints([0] * B), _ints(starts)
    got = sv.kv_assign(pool, table, held, lens, PAGE, new_start=start, max_new=max(lengths), total=n)
    count, slots, positions, flags = PO.assign(free, count, otable, oheld, [0] * B, PAGE, lengths, starts[:-1].tolist(), n, max(lengths))
    assert flags == [0] * B
    same_places(got, slots, positions)
    sv.rope(q, k, got["positions"], to_gpu(freq), out=(q, k))  # in place, in the projection
    for part, at in ((q, slice(0, HEADS)), (k, slice(HEADS, HEADS + KV_HEADS))):
        want, tol = _turned(x[:, at], got["positions"].cpu().numpy(), freq)
        assert (np.abs(part.double().cpu().numpy() - want) <= tol).all()
    assert torch.equal(v, to_gpu(x, "bf16")[:, HEADS + KV_HEADS:])
    qh, kh, vh = (t.float().cpu().numpy() for t in (q, k, v))
    out, lse = sv.prompt_attention(q, k, v, new_start=start, max_new=max(lengths), lse=True)
    near(out.double().cpu().numpy(), lse.double().cpu().numpy(), qh, kh, vh, starts, DIM ** -0.5, 0, 0, "bf16")
    sv.kv_append(cache, k, v, table, lens, new_start=start, max_new=max(lengths))
    for b in range(B):
        at = slice(starts[b], starts[b + 1])
        KO.append(host, kh[at], vh[at], np.array(otable[b]), PAGE, 0)
    # each slot holds its token: the cache is where the slots say
    flat = cache["k"].transpose(1, 2).reshape(64 * PAGE, KV_HEADS, DIM)
    read, _ = sv.kv_read(cache, table, lens, max(lengths), new_start=start, total=n)
    scale = cache["k_scale"].repeat_interleave(PAGE, 0)
    assert torch.equal((flat.float() * scale[..., None])[got["slots"]].bfloat16(), read)

    # trees behind them, twice; the last sequence leaves in between
    lens = _ints(lengths)
    ctx = list(lengths)
    for step in range(2):
        parents = [[-1] + [int(g.integers(max(0, i - 4), i)) for i in range(1, nodes)] for _ in range(B)]
        flat_parents = [p for row in parents for p in row]
        got = sv.kv_assign(pool, table, held, lens, PAGE, max_new=nodes, parents=_ints(parents))
        count, slots, positions, flags = PO.assign(free, count, otable, oheld, ctx, PAGE, [nodes] * B, [b * nodes for b in range(B)], B * nodes,
                                                   nodes, flat_parents)
        assert flags == [0] * B
        same_places(got, slots, positions)
        x = round_to(g.normal(size=(B, nodes, HEADS + 2 * KV_HEADS, DIM)), "bf16")
        dev = to_gpu(x, "bf16")
        q, k = sv.rope(dev[:, :, :HEADS], dev[:, :, HEADS:HEADS + KV_HEADS], got["positions"], to_gpu(freq))
        v = dev[:, :, HEADS + KV_HEADS:]
        sv.kv_append(cache, k, v, table, lens)
        seen, slse = sv.kv_attention(q, cache, table, lens, parents=_ints(parents), lse=True)
        for b in range(B):
            KO.append(host, k[b].float().cpu().numpy(), v[b].float().cpu().numpy(), np.array(otable[b]), PAGE, ctx[b])
            want, wlse, absolute, _ = KO.attention(q[b].double().cpu().numpy(), host, np.array(otable[b]), PAGE, ctx[b], parents[b], DIM ** -0.5, 0, 0)
            assert (np.abs(seen[b].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * absolute).all()
        paths = []
        for b in range(B):
            path, node = [0], 0
            for i in range(1, nodes):
                if parents[b][i] == node and len(path) < 5:
                    path.append(i)
                    node = i
            paths.append(path)
        deep = max(map(len, paths))
        lens = sv.kv_commit(cache, table, lens, _ints([p + [-1] * (deep - len(p)) for p in paths]), _ints([len(p) - 1 for p in paths]), nodes)
        ctx = [KO.commit(host, np.array(otable[b]), PAGE, ctx[b], paths[b]) for b in range(B)]
        assert lens.tolist() == ctx
        if step == 0:
            ctx[-1] = 0  # it leaves: all of its pages go back
            lens[-1] = 0
        sv.kv_assign(pool, table, held, lens, PAGE)
        count, _, _, _ = PO.assign(free, count, otable, oheld, ctx, PAGE, [0] * B, [0] * B, 0, 0)
        assert held.tolist() == oheld == [-(-c // PAGE) for c in ctx] and pool["count"].tolist() == [count]
        assert pool["free"].tolist() == free
