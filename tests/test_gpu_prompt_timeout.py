"""What a call reports when a wait inside the kernels of prompt attention runs
out.

The library is built once more with waits of about 2 ms and with one tile of
keys or values of every block that is never loaded: the roles that need it wait
in vain, give up, and the call ends.  Every wait has that limit, so the GPU stays
usable, which the same child process checks."""
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
from _kv import round_to, to_gpu
from _prompt import near

def call(lengths, heads, kv_heads, dim, dtype, status=True):
    g = np.random.default_rng(0)
    n = sum(lengths)
    q, k, v = (round_to(g.normal(0, 1, (n, h, dim)), dtype) for h in (heads, kv_heads, kv_heads))
    starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    st = torch.full((len(lengths),), -7, dtype=torch.int32, device="cuda")
    out, lse = sv.prompt_attention(*(to_gpu(x, dtype) for x in (q, k, v)), new_start=to_gpu(starts), max_new=max(lengths), lse=True,
                                   row_status=st if status else None)
    torch.cuda.synchronize()
    return out, lse, st, (q, k, v, starts)

for dtype in ("bf16", "f32"):
    for dim in (64, 128, 256):
        # every item behind the first tokens has more tiles than the lost one's number
        lengths = [700, 300, 128, 0]
        for status in (True, False):
            out, lse, st, (q, k, v, starts) = call(lengths, 4, 2, dim, dtype, status)
            assert not status or st.tolist()[:2] == [1024, 1024] and st.tolist()[3] == 0, st
            for a, b in ((0, 700), (700, 1000)):
                assert torch.isnan(out[a + 128:b]).all() and torch.isnan(lse[a + 128:b]).all(), (dtype, dim)
            # what is not marked is right
            bad = torch.isnan(out).cpu().numpy()
            clean = np.where(bad, 0, out.double().cpu().numpy())
            from oracle import prompt_oracle as PO
            for a, b in zip(starts, starts[1:]):
                if b > a:
                    want = PO.attention(q[a:b][:128], k[a:b][:128], v[a:b][:128], dim ** -0.5, 0, 0)[0]
                    rows = slice(a, a + len(want))
                    assert (np.abs(clean[rows] - np.where(bad[rows], 0, want)) < 0.1).all()
        # one item of one tile: nothing is lost, on the same context
        out, lse, st, (q, k, v, starts) = call([31], 2, 1, dim, dtype)
        assert st.tolist() == [0]
        near(out.double().cpu().numpy(), lse.double().cpu().numpy(), q, k, v, starts, dim ** -0.5, 0, 0, dtype)
print("child ok")
"""


def test_waits_that_run_out_are_reported():
    from draft_token_verification_sv_gb300 import build as b
    library = b.build(variant="lost_prompt_tile", defines=("SV_PROMPT_LOST_TILE=3", "SV_WAIT_CYCLES=(1ll<<22)"))
    child = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", child], cwd=ROOT, env=dict(os.environ, SPEC_VERIFY_LIBRARY=library),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


LONG_CHILD = r"""
import sys
import torch
sys.path[:0] = [{root!r}]
import draft_token_verification_sv_gb300 as sv

n, heads, dim = 20000, 4, 64
for dtype, shift in ((torch.float32, 0), (torch.bfloat16, 0), (torch.bfloat16, 1)):
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(1, n, heads, dim + 8, generator=g, device="cuda").to(dtype)[..., shift:dim + shift] for _ in range(3))
    st = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    clean = sv.prompt_attention(q, k, v)
    assert torch.isfinite(clean).all()
    v[0, 0, :, 5] = float("inf")
    v[0, 3, 1, 7] = float("nan")
    v[0, 9999, 2, 9] = float("-inf")
    out = sv.prompt_attention(q, k, v, row_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0], (dtype, shift, st)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, :, :, 5] = True
    hit[0, 3:, 1, 7] = True
    hit[0, 9999:, 2, 9] = True
    assert torch.equal(torch.isfinite(out), ~hit), (dtype, shift)
    assert torch.equal(out.masked_fill(hit, 0), clean.masked_fill(hit, 0)), (dtype, shift)
print("child ok")
"""


def test_a_value_that_is_not_finite_does_not_hold_a_long_prompt_up():
    """Waits of 17 ms are far more than any role takes for its share, with such values or without."""
    from draft_token_verification_sv_gb300 import build as b
    library = b.build(variant="short_prompt_waits", defines=("SV_WAIT_CYCLES=(1ll<<25)",))
    r = subprocess.run([sys.executable, "-c", LONG_CHILD.format(root=ROOT)], cwd=ROOT, env=dict(os.environ, SPEC_VERIFY_LIBRARY=library),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
