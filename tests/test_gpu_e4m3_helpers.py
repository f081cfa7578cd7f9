"""The torch helpers of the e4m3 cache: which workspace, stream and number types they take."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _e4m3 as E

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


class _Spy:
    """The library with its calls recorded."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)

        def call(*a):
            self.calls.append((name, a))
            return f(*a)
        return call

    def workspace_bytes(self, entry):
        return [a[-2] for name, a in self.calls if name == entry]


@pytest.fixture
def spy(monkeypatch):
    s = _Spy(fb.load())
    monkeypatch.setattr(fb, "_lib", s)
    return s


def _long(rng, d=128, L=5000, Hkv=2):
    return E.Cache(rng, *([E.bf16(rng.standard_normal((L, Hkv, d)))[1]] for _ in "kv"), max_blocks=320)


@pytest.mark.parametrize("tokens,bound", [(60, 60), (60, 512), (60, 8192), (60, 2 ** 31 - 1), (3, 4096)])
def test_a_loose_bound_gets_the_workspace_of_the_rows_at_hand(spy, tokens, bound):
    """A captured step's bound: the call is cut into parts as with the exact one."""
    rng = np.random.default_rng(60)
    c = _long(rng)
    q, cu = E.bf16(rng.standard_normal((tokens, 8, 128)))[0], _i32([0, tokens])
    o, lse = fb.paged_prefill_e4m3(q.cuda(), *c.gpu(), cu, bound, 0.1)
    need = fb.fa_paged_e4m3_workspace_used(1, tokens, 8, 2, 128, 320)
    assert need > 0 and spy.workspace_bytes("fa_paged_prefill_e4m3") == [need]
    ref = E.attend(q.double().numpy(), c.rows["k"][0], c.rows["v"][0], 0.1, vexp=c.vexp[0])
    E.check(o.double().cpu().numpy(), lse.double().cpu().numpy().T, ref, 128, 2.0 ** -7 * 1.01)
    assert fb.fa_get_device_status() == 0


def _given(kind):
    """(what the caller passes, the stream to wait for)"""
    side = torch.cuda.Stream()
    if kind == "handle":
        return side.cuda_stream, side
    if kind == "current":
        return torch.cuda.current_stream(), torch.cuda.current_stream()
    return (0, torch.cuda.default_stream()) if kind == "default" else (side, side)


@pytest.mark.parametrize("kind", ["stream", "handle", "default", "current"])
def test_a_given_stream_has_outputs_and_workspace_of_its_own(spy, kind):
    """The keys are split on a given stream too, and what the helper allocates comes from that
    stream's memory, not from a block that work queued on the current one may still read."""
    rng = np.random.default_rng(61)
    c = _long(rng)
    t, cu = c.gpu(), _i32([0, 60])
    q1, q2 = (E.bf16(rng.standard_normal((n, 8, 128)))[0].cuda() for n in (1, 60))
    k = E.bf16(rng.standard_normal((1, 60, 2, 128)))[0].cuda()
    calls = (lambda **s: fb.paged_decode_e4m3(q1, *t, 0.1, **s),
             lambda **s: fb.paged_prefill_e4m3(q2, *t, cu, 60, 0.1, **s),
             lambda **s: fb.paged_kv_read_e4m3(*t, _i32([0, 60]), 60, **s),
             lambda **s: fb.forward_window(q2[None], k, k, 0.1, 20, 2, **s),
             lambda **s: fb.forward_varlen_window(q2, k[0], k[0], cu, cu, 60, 60, 0.1, 20, 2, **s))
    want = [f() for f in calls]
    torch.cuda.synchronize()
    for f, w in zip(calls, want):
        stream, waited = _given(kind)
        before = torch.empty_like(w[0])      # the block that the next allocation of this size gets
        at = before.data_ptr()
        del before
        got = f(stream=stream)
        if kind in ("stream", "handle"):
            assert got[0].data_ptr() != at
        waited.synchronize()
        for a, b in zip(got, w):
            assert torch.equal(a, b)
    for entry in ("fa_paged_decode_e4m3", "fa_paged_prefill_e4m3"):
        with_ws = spy.workspace_bytes(entry)
        assert len(with_ws) == 2 and with_ws[0] == with_ws[1] > 0
    assert fb.fa_get_device_status() == 0


def test_the_workspace_query_is_kept_by_value():
    """Counts that come as tensors are not kept alive, nor told apart by identity."""
    c = _long(np.random.default_rng(63), L=300)
    t, q = c.gpu(), torch.zeros((60, 8, 128), dtype=torch.bfloat16, device="cuda")
    fb._e4m3_workspace_used.cache_clear()
    for _ in range(3):
        fb.paged_prefill_e4m3(q, *t, _i32([0, 60]), torch.tensor(60), 0.1, window=torch.tensor(50))
    assert fb._e4m3_workspace_used.cache_info().currsize == 1


@pytest.mark.parametrize("scale", [np.float32(0.125), np.float64(0.125), torch.tensor(0.125)])
@pytest.mark.parametrize("integer", [np.int32, np.int64, torch.tensor])
def test_numbers_of_other_types(scale, integer):
    """Scales and counts as numpy and torch give them (a scale of float32(1 / sqrt(d)), a maximum of
    a length tensor), as the other helpers take them."""
    rng = np.random.default_rng(62)
    c = _long(rng, L=300)
    t, cu = c.gpu(), _i32([0, 60])
    q1, q2 = (E.bf16(rng.standard_normal((n, 8, 128)))[0].cuda() for n in (1, 60))
    k = E.bf16(rng.standard_normal((60, 2, 128)))[0].cuda()
    i = integer
    for got, want in (
            (fb.paged_decode_e4m3(q1, *t, scale, window=i(50), sinks=i(2)),
             fb.paged_decode_e4m3(q1, *t, 0.125, window=50, sinks=2)),
            (fb.paged_prefill_e4m3(q2, *t, cu, i(60), scale, window=i(50), sinks=i(2)),
             fb.paged_prefill_e4m3(q2, *t, cu, 60, 0.125, window=50, sinks=2)),
            (fb.paged_kv_read_e4m3(*t, cu, i(60)), fb.paged_kv_read_e4m3(*t, cu, 60)),
            (fb.forward_varlen_window(q2, k, k, cu, cu, i(60), i(60), scale, i(20), i(1)),
             fb.forward_varlen_window(q2, k, k, cu, cu, 60, 60, 0.125, 20, 1)),
            (fb.forward_window(q2[None], k[None], k[None], scale, i(20), i(1)),
             fb.forward_window(q2[None], k[None], k[None], 0.125, 20, 1))):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert fb.fa_get_device_status() == 0
