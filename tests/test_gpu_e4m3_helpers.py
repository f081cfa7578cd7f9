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
