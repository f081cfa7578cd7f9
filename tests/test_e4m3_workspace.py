"""Which calls over the e4m3 cache use a workspace, on the CPU: nothing is launched."""
import pytest

from tiled_online_softmax_sm_gb300 import binding as fb
from tiled_online_softmax_sm_gb300 import build as fbuild


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fb.load()


def _decode(lib, S, H, Hkv, d, blocks, ws, bytes_):
    return lib.fa_paged_decode_e4m3(16, 16, 16, 16, 16, 16, 16, 16, 16, S, H, Hkv, d, 16, 100, blocks,
                                    0.1, 0, 0, ws, bytes_, None)


def test_used_is_the_size_or_nothing(lib):
    size, used = fb.fa_paged_e4m3_workspace_size, fb.fa_paged_e4m3_workspace_used
    need = size(1, 1, 32, 8, 128)
    assert used(1, 1, 32, 8, 128, 128) == need > 0
    assert used(1, 1, 32, 8, 128, 127) == 0              # 2032 keys: a cluster has them at once
    assert used(1, 1, 32, 8, 128, 4096, True, 1000) == 0 # nor under a short window,
    assert used(1, 1, 32, 8, 128, 4096, True, 1000, 1100) == need    # unless there are sinks
    assert used(1, 1, 32, 8, 128, 4096, True, 4096 * 16) == need     # a window that hides nothing
    # units (sequences x kv heads) of 8, 16 and 32 rows that clusters of 8 CTAs leave idle SMs for
    for rows, most in ((8, 38), (16, 28), (32, 19)):
        for d in (64, 128):
            assert used(most, 1, rows, 1, d, 4096) == size(most, 1, rows, 1, d) > 0
            assert used(most + 1, 1, rows, 1, d, 4096) == 0
    assert used(64, 1, 32, 8, 128, 512) == 0
    assert used(2, 1, 512, 8, 128, 4096) == 0
    # chunks: cut into parts of at least two tiles of 128 keys
    assert used(1, 64, 32, 8, 128, 512, False) == size(1, 64, 32, 8, 128) > 0
    assert used(1, 64, 32, 8, 128, 31) == 0
    assert used(1, 64, 32, 8, 128, 32) > 0
    assert used(16, 512, 32, 8, 128, 512) == 0
    for bad in ((0, 1, 32, 8, 128, 512), (1, 0, 32, 8, 128, 512), (1, 1, 30, 8, 128, 512),
                (1, 1, 32, 8, 96, 512), (1, 1, 32, 8, 128, 0), (1, 1, 32, 8, 128, 512, True, -1),
                (1, 1, 32, 8, 128, 512, True, 0, -1)):
        assert used(*bad) == 0


def test_a_small_workspace_is_refused_only_where_one_is_used(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    for S, blocks in ((64, 4096), (1000, 8), (5, 1 << 20)):
        assert fb.fa_paged_e4m3_workspace_used(S, 1, 32, 8, 128, blocks) == 0
        assert _decode(lib, S, 32, 8, 128, blocks, 256, 64) == fb.FA_ERR_CUDA      # past the checks
        assert _decode(lib, S, 32, 8, 128, blocks, 257, 64) == fb.FA_ERR_WORKSPACE  # misaligned
    need = fb.fa_paged_e4m3_workspace_size(4, 1, 32, 8, 128)
    assert _decode(lib, 4, 32, 8, 128, 4096, 256, need - 1) == fb.FA_ERR_WORKSPACE
    assert _decode(lib, 4, 32, 8, 128, 4096, 256, need) == fb.FA_ERR_CUDA
