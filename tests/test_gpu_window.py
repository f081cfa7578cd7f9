"""fa_forward_window and fa_forward_varlen_window against a plain float64 form.

Bounds of _e4m3.bounds with P rounded to bf16 in the value product and in O's
divisor (2^-8 each)."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _e4m3 as E

pytestmark = pytest.mark.gpu
P_ROUND = 2.0 ** -7 * 1.01


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _f64(t):
    return t.double().cpu().numpy()


def _dense_check(rng, B, n, m, H, Hkv, d, window, sinks, hot=1.0):
    q = E.bf16(hot * rng.standard_normal((B, n, H, d)))[0]
    k = E.bf16(hot * rng.standard_normal((B, m, Hkv, d)))[0]
    v = E.bf16(rng.standard_normal((B, m, Hkv, d)))[0]
    scale = E.softmax_scale(d)
    o, lse = fb.forward_window(q.cuda(), k.cuda(), v.cuda(), scale, window, sinks)
    o, lse = _f64(o), _f64(lse)
    for b in range(B):
        ref = E.attend(q[b].double().numpy(), k[b].double().numpy(), v[b].double().numpy(), scale,
                       True, window, sinks)
        E.check(o[b], lse[b].T, ref, d, P_ROUND, f"n={n} m={m} window={window} sinks={sinks} b={b}")
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 0), (1, 1), (2, 0), (63, 4), (127, 0), (128, 0),
                                          (129, 4), (256, 130), (200, 256), (383, 0), (600, 700),
                                          (100000, 3)])
def test_windows(window, sinks, d):
    rng = np.random.default_rng(window + sinks + d)
    _dense_check(rng, 1, 641, 641, 4, 2, d, window, sinks)


@pytest.mark.parametrize("n,m", [(1, 1), (1, 300), (128, 128), (129, 129), (127, 500), (256, 513),
                                 (300, 200), (257, 1), (300, 0)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 3), (128, 128)])
def test_lengths(n, m, window, sinks):
    """One token, tile borders, fewer and more queries than keys, no keys."""
    _dense_check(np.random.default_rng(n + m), 2, n, m, 2, 1, 128, window, sinks)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (6, 2), (8, 1), (12, 4), (128, 1), (160, 1)])
def test_head_groups(H, Hkv):
    """Groups that pack into tiles whole, in part, or not at all."""
    _dense_check(np.random.default_rng(H), 1, 150, 210, H, Hkv, 64, 40, 2)


@pytest.mark.parametrize("d", [64, 128])
def test_hot_scores(d):
    """Scores of several hundred: references are raised across the sinks' tiles and the window's."""
    _dense_check(np.random.default_rng(7), 1, 400, 700, 4, 1, d, 150, 4, hot=8.0)


def test_wide_window_is_the_causal_forward():
    rng = np.random.default_rng(1)
    q, k, v = (E.bf16(rng.standard_normal((2, 500, 2, 128)))[0].cuda() for _ in range(3))
    o1, l1 = fb.forward_window(q, k, v, 0.1, 500, 0)
    o2, l2 = fb.forward(q, k, v, 0.1, True)
    assert torch.equal(o1.view(torch.int16), o2.view(torch.int16))
    assert torch.equal(l1.view(torch.int32), l2.view(torch.int32))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 4), (128, 0), (333, 140)])
@pytest.mark.parametrize("num_seqs", [9, 600])
def test_varlen(d, window, sinks, num_seqs):
    """Ragged batches on the sorted list and beyond it, empty sequences among them; sequences
    with unequal query and key counts."""
    rng = np.random.default_rng(window + d)
    if num_seqs == 9:
        new = np.array([0, 1, 128, 129, 700, 5, 300, 256, 90])
        lens = np.array([5, 1, 128, 400, 700, 0, 301, 100, 90])
    else:
        new = rng.integers(0, 20, num_seqs)
        lens = new + rng.integers(0, 20, num_seqs)
    cu, cu_k = (np.concatenate([[0], np.cumsum(x)]) for x in (new, lens))
    H, Hkv = 4, 2
    q = E.bf16(rng.standard_normal((cu[-1], H, d)))[0]
    k = E.bf16(rng.standard_normal((cu_k[-1], Hkv, d)))[0]
    v = E.bf16(rng.standard_normal((cu_k[-1], Hkv, d)))[0]
    scale = E.softmax_scale(d)
    o, lse = fb.forward_varlen_window(q.cuda(), k.cuda(), v.cuda(), _i32(cu), _i32(cu_k),
                                      int(new.max()), int(lens.max()), scale, window, sinks)
    o, lse = _f64(o), _f64(lse)
    for s in range(num_seqs):
        r, rk = slice(cu[s], cu[s + 1]), slice(cu_k[s], cu_k[s + 1])
        ref = E.attend(q[r].double().numpy(), k[rk].double().numpy(), v[rk].double().numpy(), scale,
                       True, window, sinks)
        E.check(o[r], lse[:, r].T, ref, d, P_ROUND, f"sequence {s}")
    assert fb.fa_get_device_status() == 0


def test_nan_stays_in_its_batch_element_and_sequence():
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((3, 200, 2, 64)) for _ in range(3))
    v[1] = np.nan
    k[1] = np.inf
    q, k, v = (E.bf16(x)[0] for x in (q, k, v))
    scale = E.softmax_scale(64)
    cu = _i32([0, 200, 400, 600])
    outs = [fb.forward_window(q.cuda(), k.cuda(), v.cuda(), scale, 60, 4)]
    o, lse = fb.forward_varlen_window(*(x.reshape(600, 2, 64).cuda() for x in (q, k, v)), cu, cu, 200,
                                      200, scale, 60, 4)
    outs.append((o.reshape(3, 200, 2, 64), lse.reshape(2, 3, 200).permute(1, 0, 2)))
    for o, lse in outs:
        for b in (0, 2):
            ref = E.attend(*(x[b].double().numpy() for x in (q, k, v)), scale, True, 60, 4)
            E.check(_f64(o[b]), _f64(lse[b]).T, ref, 64, P_ROUND)


def test_captured_and_replayed_on_another_stream():
    rng = np.random.default_rng(4)
    q, k, v = (E.bf16(rng.standard_normal((1, 300, 2, 128)))[0].cuda() for _ in range(3))
    want = fb.forward_window(q, k, v, 0.1, 100, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        o, lse = fb.forward_window(q, k, v, 0.1, 100, 4)
    with torch.cuda.stream(side):
        for _ in range(3):
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_widest_windows():
    big = 2 ** 31 - 1
    for n, m in ((200, 300), (300, 200)):
        for w, s in ((big, 0), (big, big), (60, big)):
            _dense_check(np.random.default_rng(n), 1, n, m, 4, 2, 64, w, s)


def test_wild_offsets_are_refused():
    """Offsets whose sums pass 32 bits: the sequence is skipped and nothing is written."""
    big = 2 ** 31 - 1
    q, k, v = (torch.zeros((100, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for cu in ([0, big - 4, big], [big, 5, 10], [-big, big, 60], [big - 3, -big, 60]):
        o = torch.full((100, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        fb.fa_forward_varlen_window(q, k, v, o, None, _i32(cu), _i32([0, 50, 100]), 2, 100, 100, 60, 60,
                                    2, 2, 64, 64, 0.1, 20, 1)
        assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG, cu
        assert (o[60:] == 9.0).all(), cu


def test_bad_offsets_set_the_status():
    rng = np.random.default_rng(5)
    q, k, v = (E.bf16(rng.standard_normal((100, 2, 64)))[0].cuda() for _ in range(3))
    o, lse = fb.forward_varlen_window(q, k, v, _i32([0, 50, 101]), _i32([0, 50, 100]), 60, 60, 0.1,
                                      20, 1)
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    ref = E.attend(*(x[:50].double().cpu().numpy() for x in (q, k, v)), float(np.float32(0.1)), True,
                   20, 1)
    E.check(_f64(o[:50]), _f64(lse[:, :50]).T, ref, 64, P_ROUND)
