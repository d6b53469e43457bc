"""Which form pages and places take: by what a call brings, not by the room of
its table, and each form gives what the oracle does."""
import numpy as np
import pytest

from oracle import prompt_oracle as PO
from test_gpu_kv_assign import Both, _gpu, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def _launches(sv, call):  # noqa: F811
    before = sv.lib().sv_launch_count()
    call()
    return sv.lib().sv_launch_count() - before


@pytest.mark.parametrize("columns", [10, 2048, 100_000])
@pytest.mark.parametrize("batch", [1, 64, 1024])
def test_a_step_of_few_tokens_is_one_launch_whatever_the_table_s_room(sv, batch, columns):  # noqa: F811
    import torch
    g = np.random.default_rng(batch)
    size = 9 * batch
    b = Both(sv, size, batch, 10, 16, g)
    room = torch.full((batch, columns), -3, dtype=torch.int32, device="cuda")
    room[:, :10] = b.dev_table
    b.table = [row + [-3] * (columns - 10) for row in b.table] if columns <= 2048 else b.table
    b.whole, b.dev_table, b.columns = room, room[:, :columns], columns
    if columns > 2048:  # the oracle sees the columns that it can reach
        b.same = lambda: None
    new = [int(x) for x in g.integers(0, 3, batch)]
    parents = [p for m in new for p in [-1, 0][:m]]
    assert _launches(sv, lambda: b.call([60] * batch, new)) == 1
    assert _launches(sv, lambda: b.call([62] * batch, new, parents)) == 1
    assert _launches(sv, lambda: b.call([63] * batch, [1] * batch, ragged=False)) == 1
    assert _launches(sv, lambda: b.call([16] * batch, [0] * batch, ragged=False)) == 1
    assert b.dev_held.tolist() == b.held == [1] * batch
    assert room[:, :10].tolist() == [row[:10] for row in b.table] and (room[:, 10:] == -3).all()


@pytest.mark.parametrize("new", [4000, 4001, 9000])
def test_captured_with_many_tokens(sv, new):  # noqa: F811
    import torch
    g = np.random.default_rng(new)
    b = Both(sv, 900, 3, 700, 16, g)
    lengths = [new - 17, 0, 17]
    starts = [0, new - 17, new - 17, new]
    ctx, start = _gpu([0] * 3), _gpu(starts)
    st = _gpu([-7] * 3)
    out = (torch.full((new,), -77, dtype=torch.int64, device="cuda"), torch.full((new,), -77, dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call = lambda: sv.kv_assign(b.pool, b.dev_table, b.dev_held, ctx, 16, new_start=start, max_new=new, total=new, out=out, row_status=st)  # noqa: E731
        assert _launches(sv, call) == (1 if new <= 4000 else 2)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    b.count, _, _, _ = PO.assign(b.free, b.count, b.table, b.held, [0] * 3, 16, lengths, starts[:-1], new, new)
    b.same()
    for lens in ([5, 40, 900], [900, 0, 0], [1300, 33, 16], [12_000, 0, 0]):
        ctx.copy_(_gpu(lens))
        graph.replay()
        torch.cuda.synchronize()
        b.count, slots, positions, flags = PO.assign(b.free, b.count, b.table, b.held, lens, 16, lengths, starts[:-1], new, new)
        b.same()
        assert st.tolist() == flags
        assert out[0].tolist() == [slots[r] for r in range(new)] and out[1].tolist() == [positions[r] for r in range(new)]
