"""The cache's tests of layouts and ends on the bounds-checked debug build
(-DSV_DEBUG): a check that fails there raises a flag, which the child's
fixture asserts is clear."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_debug_build_runs_the_layout_tests():
    from draft_token_verification_sv_gb300 import build as b
    env = dict(os.environ, SPEC_VERIFY_LIBRARY=b.build(debug=True))
    files = [os.path.join(ROOT, "tests", f) for f in ("test_gpu_kv_layouts.py", "test_gpu_kv_edges.py", "test_gpu_kv_workspace.py")]
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *files]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:] + r.stderr[-2000:]
