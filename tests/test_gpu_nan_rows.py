"""Rows whose visible scores hold a NaN: O and the LSE are NaN in every form of the windowed forward
and of the e4m3 cache's attention, and never the LSE of a row that sees no key; the other rows of
the call are right (V holds no NaN, so nothing else may spread)."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _e4m3 as E

pytestmark = pytest.mark.gpu
P_ROUND = 2.0 ** -7 * 1.01     # P rounded to bf16 in the value product and in O's divisor
NAN_KEY = 150


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _check(q, k, v, o, lse, d, causal, window, sinks, bad_q, bad_k, vexp=None):
    """q [n,H,d], k, v [L,Hkv,d] without the NaNs; rows bad_q (pairs) and all that see key bad_k of
    kv head 0 must be NaN."""
    n, H = q.shape[:2]
    G = H // k.shape[1]
    ref = E.attend(q, k, v, 0.1, causal, window, sinks, vexp)
    nan = np.zeros((n, H), bool)
    if bad_k is not None:
        nan[:, :G] |= E.visible(n, len(k), causal, window, sinks)[:, bad_k][:, None]
    sees = ref["keys"] > 0
    for i, h in bad_q:
        nan[i, h] |= bool(sees[i])
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(lse[nan]).all() and np.isnan(o[nan]).all()
    # the rest against the plain form, the NaN rows put out of the way
    o, lse = np.where(nan[..., None], ref["o"], o), np.where(nan, ref["lse"], lse)
    E.check(o, lse, ref, d, P_ROUND)
    assert nan.any() and (~nan).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["q", "k"])
def test_window(d, which):
    rng = np.random.default_rng(d)
    n, H, Hkv, window, sinks = 400, 4, 2, 90, 3
    q, k, v = (E.bf16(rng.standard_normal((n, h, d))) for h in (H, Hkv, Hkv))
    qt, kt = q[0].clone(), k[0].clone()
    bad_q, bad_k = [], None
    if which == "q":
        bad_q = [(0, 0), (130, 3), (399, 1)]
        for i, h in bad_q:
            qt[i, h, 5] = float("nan")
    else:
        bad_k = NAN_KEY
        kt[bad_k, 0, 7] = float("nan")
    qt, kt, vt = qt.cuda(), kt.cuda(), v[0].cuda()
    o, lse = fb.forward_window(qt[None], kt[None], vt[None], 0.1, window, sinks)
    _check(q[1], k[1], v[1], o[0], lse[0].T, d, True, window, sinks, bad_q, bad_k)
    cu = _i32([0, n])
    o, lse = fb.forward_varlen_window(qt, kt, vt, cu, cu, n, n, 0.1, window, sinks)
    _check(q[1], k[1], v[1], o, lse.T, d, True, window, sinks, bad_q, bad_k)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,window,sinks", [(1, 0, 0), (3, 0, 0), (60, 0, 0), (60, 300, 3), (300, 0, 0)])
@pytest.mark.parametrize("which", ["q", "k"])
def test_cache(d, new, window, sinks, which):
    """Single tokens, short chunks and long ones, each with a workspace (keys cut into parts) and
    without one."""
    rng = np.random.default_rng(d + new)
    L, H, Hkv = 2400, 8, 2
    c = E.Cache(rng, *([E.bf16(rng.standard_normal((L, Hkv, d)))[1]] for _ in "kv"), max_blocks=160)
    q = E.bf16(rng.standard_normal((new, H, d)))
    qt, t = q[0].clone(), c.gpu()
    bad_q, bad_k = [], None
    if which == "q":
        bad_q = [(0, 0), (new - 1, 6)]
        for i, h in bad_q:
            qt[i, h, 5] = float("nan")
    else:
        bad_k = NAN_KEY if not window else L - new - 200
        t[0].view(torch.uint8)[c.table[0, bad_k // 16], 0, bad_k % 16, 9] = 0x7f
    need = fb.fa_paged_e4m3_workspace_size(1, new, H, Hkv, d)
    for ws in (None, torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")):
        o = torch.full((new, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((H, new), 9.0, device="cuda")
        fb.fa_paged_prefill_e4m3(qt.cuda(), *t, _i32([0, new]), o, lse, 1, new, new, H, Hkv, d, 16,
                                 c.num_pages, 160, 0.1, True, window, sinks, ws, need if ws is not None else 0)
        _check(q[1], c.rows["k"][0], c.rows["v"][0], o, lse.T, d, True, window, sinks, bad_q, bad_k,
               c.vexp[0])
    assert fb.fa_get_device_status() == 0
