"""Limits of the windowed forward's work units, on the CPU: refused before anything is launched."""
import pytest

from tiled_online_softmax_sm_gb300 import binding as fb
from tiled_online_softmax_sm_gb300 import build as fbuild


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fb.load()


def _packed(lib, S, max_q, H, Hkv, total=64):
    return lib.fa_forward_varlen_window(16, 16, 16, 16, 16, 16, 16, S, total, total, max_q, max_q, H,
                                        Hkv, 64, 64, 0.1, 4, 1, None)


@pytest.mark.parametrize("S,max_q,H,Hkv", [(1 << 25, 1, 128, 128), (1 << 24, 64, 64, 64),
                                           (1 << 30, 1, 1, 1), (1 << 28, 1, 12, 4),
                                           (1 << 29, 64, 4, 2), (2 ** 31 - 1, 64, 128, 1)])
def test_packed_units_stay_in_32_bits(lib, S, max_q, H, Hkv):
    """Mostly empty sequences: their (sequence, head group, query pair) units are numbered in 32 bits."""
    a = 1
    while (H // Hkv) % (2 * a) == 0 and a < 128:
        a *= 2
    units = S * (H // a) * -(-max_q // (256 // a))
    assert units >= 1 << 30
    assert _packed(lib, S, max_q, H, Hkv) == fb.FA_ERR_UNSUPPORTED
    assert "units" in fb.fa_last_error()


def test_units_below_the_limit_pass_the_check(lib):
    """Without a GPU the call then fails on the device, with one it would launch: the check alone."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    for S, max_q, H, Hkv in ((1 << 20, 1, 128, 128), ((1 << 30) - 1, 1, 1, 1), ((1 << 30) - 1, 2, 128, 1)):
        assert _packed(lib, S, max_q, H, Hkv) == fb.FA_ERR_CUDA


def test_dense_units_stay_in_32_bits(lib):
    def dense(B, n, H, Hkv):
        return lib.fa_forward_window(16, 16, 16, 16, 16, B, H, Hkv, n, 1, 64, 64, 0.1, 4, 1, None)
    assert dense(1 << 24, 1, 64, 64) == fb.FA_ERR_UNSUPPORTED
    assert dense(1 << 20, 1, 1 << 12, 1 << 12) == fb.FA_ERR_UNSUPPORTED
