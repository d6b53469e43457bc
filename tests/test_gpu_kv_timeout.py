"""What a call reports when a wait inside the many-row attention kernel runs out.

The library is built once more with waits of about 2 ms and with one tile of
every block that is never planned: the roles that need it wait in vain, give
up, and the call ends.  Every wait has that limit, so the GPU stays usable,
which the same child process checks."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import numpy as np
import torch
sys.path[:0] = [{root!r}, {tests!r}]
import draft_token_verification_sv_gb300 as sv
from _kv import cache_gpu, make_cache, make_table, to_gpu

def call(ctx, n, heads, seed=0, status=True):
    g = np.random.default_rng(seed)
    table, pages = make_table(g, [c + n for c in ctx], 64)
    dev = cache_gpu(make_cache(g, pages, 2, 64, 128))
    q = to_gpu(g.normal(0, 1, (len(ctx), n, heads, 128)).astype(np.float32), "bf16")
    st = torch.full((len(ctx),), -7, dtype=torch.int32, device="cuda")
    out, lse = sv.kv_attention(q, dev, to_gpu(table), to_gpu(np.array(ctx, np.int32)), lse=True, row_status=st if status else None)
    torch.cuda.synchronize()
    return out, lse, st

# every block has more tiles than the lost one's number
ctx = np.random.default_rng(1).integers(3000, 9000, 40).tolist()
out, lse, st = call(ctx, 10, 8)
assert st.tolist() == [1024] * 40, st
assert torch.isnan(out).all() and torch.isnan(lse).all()
# without a status the results say so themselves
out, lse, _ = call(ctx, 10, 8, status=False)
assert torch.isnan(out).all() and torch.isnan(lse).all()
# one long sequence over all blocks: all of it in parts
out, lse, st = call([60000], 10, 8)
assert st.tolist() == [1024] and torch.isnan(out).all() and torch.isnan(lse).all()
# few tiles a block: nothing is lost, on the same context
out, lse, st = call([100, 70, 5], 10, 8)
assert st.tolist() == [0] * 3 and torch.isfinite(out).all() and torch.isfinite(lse).all()
# and the other kernel
out, lse, st = call(ctx, 1, 8)
assert st.tolist() == [0] * 40 and torch.isfinite(out).all()
print("child ok")
"""


def test_waits_that_run_out_are_reported_for_every_sequence():
    from draft_token_verification_sv_gb300 import build as b
    library = b.build(variant="lost_tile", defines=("SV_LOST_TILE=3", "SV_WAIT_CYCLES=(1ll<<22)"))
    child = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", child], cwd=ROOT, env=dict(os.environ, SPEC_VERIFY_LIBRARY=library),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
