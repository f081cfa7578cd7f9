"""The C entry points through the binding, in a process that has no torch."""
import os
import subprocess
import sys

from tiled_online_softmax_sm_gb300 import build as fbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import importlib.abc, sys

class NoTorch(importlib.abc.MetaPathFinder):
    def find_spec(self, name, path, target=None):
        if name.split(".")[0] == "torch":
            raise ImportError("no torch here")

sys.meta_path.insert(0, NoTorch())
from tiled_online_softmax_sm_gb300 import binding as fb
assert fb.fa_paged_e4m3_workspace_size(1, 1, 32, 8, 128) > 0
assert fb.fa_paged_decode_workspace_size(1, 32, 128, 4) > 0
for call in (lambda: fb.fa_forward_window(16, 16, 16, 16, None, 1, 0, 1, 8, 8, 128, 128, 0.1, 4, 0, stream=7),
             lambda: fb.fa_paged_decode_e4m3(16, 16, 16, 16, 16, 16, 16, 16, None, 1, 0, 1, 128, 16, 4, 4,
                                             0.1, stream=7),
             lambda: fb.fa_forward(16, 16, 16, 16, None, 1, 0, 1, 8, 8, 128, 128, 0.1, 0, stream=7)):
    try:
        call()
    except fb.FaError as e:
        assert e.status == fb.FA_ERR_INVALID_ARG, e
    else:
        raise AssertionError("not refused")
assert fb.fa_forward(None, None, None, None, None, 0, 4, 2, 0, 0, 128, 128, 0.1, 0, stream=7) is None
assert "torch" not in sys.modules
print("ok")
"""


def test_entry_points_need_no_torch():
    fbuild.build()
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
