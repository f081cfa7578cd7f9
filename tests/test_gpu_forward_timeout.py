"""The forward's bounded waits: a K tile that never arrives ends every role of every instance.

With FA_TEST_FORCE_WAIT_TIMEOUT=1 each copying warp leaves its first K tile out: a flag that nothing
sets.  The waits for it run out after about a second, FA_ERR_TIMEOUT is recorded, all warps leave
their loops together, and the next call, with the hook unset, gives the bits of the one before."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _e4m3 as E

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _bf16(rng, *shape):
    return E.bf16(rng.standard_normal(shape))[0].cuda()


def _dense(rng, fn, B=2, n=700, H=4, Hkv=2, d=128):
    q, k, v = _bf16(rng, B, n, H, d), _bf16(rng, B, n, Hkv, d), _bf16(rng, B, n, Hkv, d)
    return lambda: fn(q, k, v)


def _packed(rng, fn, d=64):
    new = [300, 1, 513, 129]           # ragged: V tiles whose last rows are zeroed before use
    cu = _i32(np.concatenate([[0], np.cumsum(new)]))
    q, k, v = (_bf16(rng, sum(new), h, d) for h in (4, 2, 2))
    return lambda: fn(q, k, v, cu)


def _fp8(rng):
    q, k, v = (_bf16(rng, 1, 700, 2, 128).to(torch.float8_e4m3fn) for _ in range(3))
    return lambda: fb.forward_fp8(q, k, v, 0.1, 1.0, 1.0, 1.0, True)


def _paged(rng):
    lens, new = np.array([700, 333]), [200, 333]
    table = _i32(rng.permutation(2 * 44).reshape(2, 44))
    kc, vc = _bf16(rng, 88, 2, 16, 128), _bf16(rng, 88, 2, 16, 128)
    q, cu = _bf16(rng, 533, 4, 128), _i32([0, 200, 533])
    return lambda: fb.paged_prefill(q, kc, vc, table, _i32(lens), cu, 333, 0.1)


def _cached(rng, d, lens, new, window=0, blocks=None):
    c = E.Cache(rng, *([E.bf16(rng.standard_normal((L, 2, d)))[1] for L in lens] for _ in "kv"),
                max_blocks=blocks)
    t, q = c.gpu(), _bf16(rng, sum(new), 8, d)
    cu = _i32(np.concatenate([[0], np.cumsum(new)]))
    return lambda: fb.paged_prefill_e4m3(q, *t, cu, max(new), 0.1, window=window, sinks=3)


FORMS = {
    "causal": lambda r: _dense(r, lambda q, k, v: fb.forward(q, k, v, 0.1, True)),
    "split units": lambda r: _dense(r, lambda q, k, v: fb.forward(q, k, v, 0.1, False), B=1, n=1000),
    "e4m3 operands": _fp8,
    "packed": lambda r: _packed(r, lambda q, k, v, cu: fb.forward_varlen(q, k, v, cu, cu, 513, 513, 0.1)),
    "paged": _paged,
    "window": lambda r: _dense(r, lambda q, k, v: fb.forward_window(q, k, v, 0.1, 150, 4)),
    "packed window": lambda r: _packed(
        r, lambda q, k, v, cu: fb.forward_varlen_window(q, k, v, cu, cu, 513, 513, 0.1, 100, 4)),
    "e4m3 chunk": lambda r: _cached(r, 128, [900, 400], [300, 400]),
    "e4m3 chunk d64 window": lambda r: _cached(r, 64, [900, 400], [300, 400], window=200),
    "e4m3 chunk in parts": lambda r: _cached(r, 128, [5000], [60], blocks=320),
}


@pytest.mark.parametrize("form", FORMS)
def test_a_tile_that_never_arrives_sets_the_status(form, monkeypatch):
    call = FORMS[form](np.random.default_rng(len(form)))
    want = call()
    assert fb.fa_get_device_status() == 0
    monkeypatch.setenv("FA_TEST_FORCE_WAIT_TIMEOUT", "1")
    call()
    assert fb.fa_get_device_status() == fb.FA_ERR_TIMEOUT
    monkeypatch.delenv("FA_TEST_FORCE_WAIT_TIMEOUT")
    got = call()
    assert fb.fa_get_device_status() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
