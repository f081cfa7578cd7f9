"""The e4m3 cache's and the windowed forward's kernels in the debug build, which checks every global
store's index: a cross-section of their tests, in a child process, with results and statuses as in
the normal build (so every check stays silent, or the status would be FA_ERR_DEBUG_CHECK)."""
import os
import subprocess
import sys

import pytest

from test_gpu_debug_build import CHILD, ROOT

pytestmark = pytest.mark.gpu

CACHE = "tests/test_gpu_e4m3_cache.py::"
CASES = [
    CACHE + "test_write_gives_the_defined_codes_and_leaves_other_slots",
    CACHE + "test_write_skips_what_it_cannot_place",
    CACHE + "test_read_back_is_exact",
    CACHE + "test_decode_groups_and_lengths",                    # clusters
    CACHE + "test_decode_shares_of_a_few_long_sequences",        # shares and their merge
    CACHE + "test_one_long_sequence_is_shared_by_every_warp",
    CACHE + "test_shares_of_short_chunks_skip_bad_sequences",
    CACHE + "test_short_chunks",
    CACHE + "test_chunks",
    CACHE + "test_chunks_window",
    CACHE + "test_chunks_split_over_long_contexts",              # parts and their merge
    CACHE + "test_chunk_status",
    "tests/test_gpu_window.py::test_windows",
    "tests/test_gpu_window.py::test_lengths",
    "tests/test_gpu_window.py::test_varlen",
    "tests/test_gpu_window.py::test_bad_offsets_set_the_status",
]


def test_debug_build_passes_the_cache_and_window_cases():
    from tiled_online_softmax_sm_gb300 import build
    lib = build.build(debug=True)
    r = subprocess.run([sys.executable, "-c", CHILD, lib] + CASES, cwd=ROOT,
                       env=dict(os.environ, FA_LIBRARY=lib), capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout
