"""Pages for lengths, slots and positions on the GPU against the oracle: all of it whole numbers."""
import numpy as np
import pytest

from oracle import prompt_oracle as PO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import draft_token_verification_sv_gb300 as sv
    return sv


def _gpu(x, dtype=np.int32):
    import torch
    return torch.from_numpy(np.array(x, dtype)).cuda()


class Both:
    """A pool and page table on the GPU and the oracle's beside it."""

    def __init__(self, sv, size, batch, columns, page, g, pad=0):
        import torch
        self.sv, self.page, self.size, self.columns, self.batch = sv, page, size, columns, batch
        self.free = g.permutation(size).tolist()
        self.count, self.held = size, [0] * batch
        self.table = [[-5 - c for c in range(columns)] for _ in range(batch)]
        self.pool = dict(free=_gpu(self.free), count=_gpu([size]))
        whole = torch.full((batch, columns + pad), -9, dtype=torch.int32, device="cuda")
        whole[:, :columns] = _gpu(self.table)
        self.whole, self.dev_table, self.dev_held = whole, whole[:, :columns], _gpu(self.held)

    def call(self, ctx, new, parents=None, ragged=True, starts=None, total=None, max_new=None, rows_behind=0):
        import torch
        given = starts
        starts = np.concatenate([[0], np.cumsum(new)]).tolist() if starts is None else starts
        total = starts[-1] + rows_behind if total is None else total
        max_new = max(new, default=0) if max_new is None else max_new
        counts = [b - a for a, b in zip(starts, starts[1:])]
        self.count, slots, positions, flags = PO.assign(self.free, self.count, self.table, self.held, list(ctx), self.page, counts, starts,
                                                        total, max_new, None if parents is None else parents)
        st = torch.full((self.batch,), -7, dtype=torch.int32, device="cuda")
        kw = dict(row_status=st, parents=None if parents is None else _gpu(parents), max_new=max_new)
        out = (torch.full((total,), -77, dtype=torch.int64, device="cuda"), torch.full((total,), -77, dtype=torch.int32, device="cuda"))
        if ragged:
            kw.update(new_start=_gpu(starts), total=total, out=out)
        got = self.sv.kv_assign(self.pool, self.dev_table, self.dev_held, _gpu(ctx), self.page, **kw)
        self.same()
        assert st.tolist() == flags
        if max_new == 0 and not ragged:
            assert got == dict(slots=None, positions=None)
            return flags
        want = [np.array([d.get(r, -77) for r in range(total)]) for d in (slots, positions)]
        assert got["slots"].dtype == torch.int64 and got["positions"].dtype == torch.int32
        claims = np.zeros(total, int)  # (a row that two sequences claim is one's or the other's)
        for first, n in zip(starts, counts):
            claims[max(first, 0):max(first + n, 0)] += 0 <= n <= max_new and 0 <= first <= total - n
        for have, expect in zip((got["slots"], got["positions"]), want):
            np.testing.assert_array_equal(have.flatten().cpu().numpy()[claims < 2], expect[claims < 2])
        assert given is not None or ragged or tuple(got["slots"].shape) == (self.batch, max_new)
        return flags

    def same(self):
        assert self.pool["count"].tolist() == [self.count]
        assert self.pool["free"].tolist() == list(self.free)
        assert self.dev_held.tolist() == self.held
        assert self.dev_table.tolist() == self.table
        assert (self.whole[:, self.columns:] == -9).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("batch,most", [(1, 1), (3, 40), (33, 300), (70, 5)])
def test_calls_in_a_row(sv, page, batch, most):
    g = np.random.default_rng(batch)
    columns = 700 // page + 2
    b = Both(sv, batch * (350 // page + 1) + 1, batch, columns, page, g, pad=3)
    for step in range(8):
        ctx = [int(x) for x in g.integers(0, 700 - most, batch)]
        if step % 2:
            new = [int(x) for x in g.integers(0, most + 1, batch)]
            b.call(ctx, new, rows_behind=step)
        else:
            b.call(ctx, [most] * batch, ragged=False)
    b.call([0] * batch, [0] * batch, ragged=False)  # all leave
    assert b.count == b.size


@pytest.mark.parametrize("n", [1, 2, 33, 500])
def test_trees(sv, n):
    g = np.random.default_rng(n)
    b = Both(sv, 400, 4, 70, 16, g)
    new = [n, max(1, n // 2), n, 0]
    parents = [p for m in new for p in [-1][:m] + [int(g.integers(max(0, i - 9), i)) for i in range(1, m)]]
    assert b.call([5, 0, 31, 99], new, parents) == [0] * 4
    bad = list(parents)
    bad[0] = 0
    bad[-1] = n if n > 2 else -3
    flags = b.call([5, 0, 31, 99], new, bad)
    assert flags[0] & PO.BAD_PARENT and flags[2] & PO.BAD_PARENT and not flags[1]


def test_a_chain_as_a_tree(sv):
    g = np.random.default_rng(5)
    b = Both(sv, 200, 1, 150, 16, g)
    b.call([3], [2000], list(range(-1, 1999)))


def test_more_sequences_than_a_block_scans_at_once(sv):
    """Shortage in the middle, gives and takes on both sides of 1024 sequences."""
    g = np.random.default_rng(3)
    batch = 2500
    b = Both(sv, 4000, batch, 8, 16, g)
    for step in range(4):
        ctx = [int(x) for x in g.integers(0, 100, batch)]
        flags = b.call(ctx, [int(x) for x in g.integers(0, 29, batch)])
        if step == 1:
            assert PO.NO_PAGE in flags
    assert b.call([0] * batch, [0] * batch, ragged=False) == [0] * batch
    assert b.count == 4000


def test_a_largest_number_of_tokens_far_above_what_comes(sv):
    g = np.random.default_rng(3)
    batch = 1100
    both = Both(sv, 9000, batch, 700, 16, g)
    new = g.integers(0, 30, batch)
    new[[5, 900]] = 11_000, 5_003
    both.call(np.zeros(batch, int), new, max_new=2 ** 31 - 1)


@pytest.mark.parametrize("short", [0, 1, 7])
def test_what_a_call_gives_back_a_later_sequence_takes(sv, short):
    g = np.random.default_rng(1)
    b = Both(sv, 20, 3, 20, 16, g)
    b.call([16 * 9, 16 * 8, 0], [0] * 3, ragged=False)
    flags = b.call([16, 16 * 5, 16 * (14 + short)], [0] * 3, ragged=False)
    # (21 pages are more than a row of the table has room for)
    assert flags == [0, 0, {0: 0, 1: PO.NO_PAGE, 7: PO.BAD_LENGTH}[short]]


def test_bad_lengths_are_left_out(sv):
    g = np.random.default_rng(2)
    b = Both(sv, 64, 6, 8, 16, g)
    b.call([20] * 6, [0] * 6, ragged=False)
    flags = b.call([-1, 8 * 16, 8 * 16 - 2, 2 ** 31 - 1, 20, 20], [3, 1, 2, 1, 0, 4])
    assert flags == [128, 128, 0, 128, 0, 0]
    # starts that go back, beyond the rows, or give more than max_new
    flags = b.call([0] * 6, [], starts=[0, 3, 1, 4, 9, 9, 40], total=30, max_new=4)
    assert flags == [0, 128, 0, 128, 0, 128]
    flags = b.call([0] * 6, [], starts=[-2, 3, 3, 4, 4, 4, 4], total=30, max_new=8)
    assert flags == [128, 0, 0, 0, 0, 0]
    b.held[2] = 9
    b.dev_held[2] = 9
    b.held[3] = -1
    b.dev_held[3] = -1
    assert b.call([0, 1, 2, 3, 4, 5], [2] * 6) == [0, 0, 128, 128, 0, 0]


@pytest.mark.parametrize("count", [-3, 30])
def test_a_count_outside_the_stack(sv, count):
    g = np.random.default_rng(2)
    b = Both(sv, 20, 2, 8, 16, g)
    b.count = count
    b.pool["count"].fill_(count)
    b.call([30, 40], [3, 0])


def test_more_pages_than_the_stack_has_room_for_are_lost(sv):
    g = np.random.default_rng(2)
    b = Both(sv, 10, 2, 8, 16, g)
    b.call([64, 64], [0, 0], ragged=False)
    b.count = 7  # as if some had been put back by hand
    b.pool["count"].fill_(7)
    b.call([0, 0], [0, 0], ragged=False)
    assert b.count == 10


def test_pages_outside_the_pool_have_no_slots(sv):
    g = np.random.default_rng(2)
    b = Both(sv, 10, 2, 8, 16, g)
    b.call([40, 40], [0, 0], ragged=False)
    for page, col in ((99, 2), (-1, 1)):
        b.table[1][col] = page
        b.dev_table[1, col] = page
    assert b.call([20, 20], [20, 20]) == [0, PO.BAD_PAGE]


def test_slots_beyond_32_bits(sv):
    """Page ids of a pool whose slots pass 2^31."""
    import torch
    page, size = 128, (1 << 25) + 5
    pool = dict(free=torch.arange(size, dtype=torch.int32, device="cuda"), count=_gpu([size]))
    table, held = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), _gpu([0])
    got = sv.kv_assign(pool, table, held, _gpu([0]), page, max_new=300)
    want = (size - 1 - np.arange(300) // page) * np.int64(page) + np.arange(300) % page
    np.testing.assert_array_equal(got["slots"].cpu().numpy()[0], want)
    assert want.max() > 2 ** 31


@pytest.mark.parametrize("batch,columns", [(2, 20), (40, 500), (1100, 20)])
def test_captured_on_another_stream_and_replayed(sv, batch, columns):
    """One launch of a block, of many, and of more sequences than that takes."""
    import torch
    g = np.random.default_rng(4)
    b = Both(sv, 20 * batch, batch, columns, 16, g)
    new = [int(x) for x in g.integers(0, 6, batch)]
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    total = starts[-1]
    ctx, start = _gpu([0] * batch), _gpu(starts)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kw = dict(new_start=start, max_new=5, total=total)
        got = sv.kv_assign(b.pool, b.dev_table, b.dev_held, ctx, 16, **kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            sv.kv_assign(b.pool, b.dev_table, b.dev_held, ctx, 16, out=(got["slots"], got["positions"]), **kw)
    b.count, slots, positions, _ = PO.assign(b.free, b.count, b.table, b.held, [0] * batch, 16, new, starts[:-1], total, 5)
    for step in range(3):
        lens = [int(x) for x in g.integers(0, 16 * 20 - 5, batch)]
        ctx.copy_(_gpu(lens))
        graph.replay()
        torch.cuda.synchronize()
        b.count, slots, positions, _ = PO.assign(b.free, b.count, b.table, b.held, lens, 16, new, starts[:-1], total, 5)
        b.same()
        assert got["slots"].tolist() == [slots[r] for r in range(total)] and got["positions"].tolist() == [positions[r] for r in range(total)]


@pytest.mark.parametrize("batch,columns,most", [(3, 6000, 90_000), (1000, 17, 200), (1024, 40, 33)])
def test_calls_that_several_blocks_share(sv, batch, columns, most):
    """Many pages or tokens: gives, takes and places of more than one block."""
    g = np.random.default_rng(batch)
    b = Both(sv, int(0.8 * batch * columns), batch, columns, 16, g)
    for step in range(4):
        ctx = [int(x) for x in g.integers(0, 16 * columns - most, batch)]
        new = [int(x) for x in g.integers(0, most + 1, batch)]
        parents = [p for m in new for p in [-1][:m] + [int(x) for x in (g.integers(0, 9, max(0, m - 1)) % np.arange(1, max(1, m)))]] + 3 * [-1] if step == 2 else None
        b.call(ctx, new, parents, rows_behind=3)
    b.call([0] * batch, [0] * batch, ragged=False)
    assert b.count == b.size
