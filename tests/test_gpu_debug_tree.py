"""The kernels on drafted token trees in the debug build, which checks every global store's index: their
tests in a child process, with results and statuses as in the normal build."""
import os
import subprocess
import sys

import pytest

from test_gpu_debug_build import CHILD, ROOT

pytestmark = pytest.mark.gpu

CASES = ["tests/test_gpu_tree_attention.py", "tests/test_gpu_tree_cache.py", "tests/test_gpu_tree_e4m3.py"]


def test_debug_build_passes_the_tree_cases():
    from tiled_online_softmax_sm_gb300 import build
    lib = build.build(debug=True)
    r = subprocess.run([sys.executable, "-c", CHILD, lib] + CASES, cwd=ROOT,
                       env=dict(os.environ, FA_LIBRARY=lib), capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout
