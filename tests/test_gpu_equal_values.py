"""Softmax weights sum to one: where every visible V row is the same, O is that row.

The weights are rounded for the value product, and O is divided by the sum of the rounded ones.  With
V rows of 1.875 (a code, and a bf16 just below 2, where half a step is 2^-9 / 0.9375 = 0.0021 of it)
the sums are fp32 sums of at most 2400 terms of one sign, off by less than 2400 * 2^-24 * 2 = 0.0003,
so O rounds to 1.875 exactly.  A divisor taken from the unrounded weights would be off by up to 2^-8
where one weight carries the row, and rounds to a neighbour.  The rows kernels round their weights
to f16 (2^-11 = 0.0005 against the exact sum), which is inside the half step too."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _e4m3 as E

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _peaked(rng, n, H, L, Hkv, d):
    """Rows of q that two of the keys carry: an early one, which sets the reference, and a later one a
    few powers of two above it, whose weight is then no round number."""
    k = rng.standard_normal((L, Hkv, d)) * 0.02
    k[:, :, 0], k[:, :, 1] = -8.0, -8.0
    k[3, :, 0], k[L // 2 + 9, :, 1] = 8.0, 8.0
    q = rng.standard_normal((n, H, d)) * 0.02
    q[:, :, 0] = 30.0
    q[:, :, 1] = 30.0 + 5.0 * rng.random((n, H))
    return E.bf16(q)[0], E.bf16(k)[1]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [2, 8])
@pytest.mark.parametrize("new,window,sinks", [(1, 0, 0), (2, 0, 0), (50, 0, 0), (300, 0, 0), (300, 1300, 4)])
def test_cache(d, H, new, window, sinks):
    rng = np.random.default_rng(new + d + H)
    L, Hkv = 2400, 2
    q, k = _peaked(rng, new, H, L, Hkv, d)
    c = E.Cache(rng, [k], [np.full((L, Hkv, d), 1.875)], max_blocks=160)
    need = fb.fa_paged_e4m3_workspace_size(1, new, H, Hkv, d)
    for ws in (None, torch.empty(need, dtype=torch.uint8, device="cuda")):
        o = torch.full((new, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
        fb.fa_paged_prefill_e4m3(q.cuda(), *c.gpu(), _i32([0, new]), o, None, 1, new, new, H, Hkv, d, 16,
                                 c.num_pages, 160, 0.1, True, window, sinks, ws,
                                 need if ws is not None else 0)
        assert (o == 1.875).all(), f"{(o != 1.875).float().mean().item():.3f} of O off"
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [2, 8])
def test_window(d, H):
    rng = np.random.default_rng(d + H)
    q, k = _peaked(rng, 300, H, 2400, 2, d)
    k = torch.from_numpy(k.astype(np.float32)).bfloat16().cuda()
    v = torch.full_like(k, 1.875)
    o, _ = fb.forward_window(q.cuda()[None], k[None], v[None], 0.1, 1300, 4)
    assert (o == 1.875).all()
    o, _ = fb.forward_varlen_window(q.cuda(), k, v, _i32([0, 300]), _i32([0, 2400]), 300, 2400, 0.1, 1300, 4)
    assert (o == 1.875).all()


def test_chunk_has_the_bits_of_the_bf16_prefill():
    """Widening a tile is exact: with one query head per kv head O's bits are those of
    fa_paged_prefill on the rows read back into a bf16 cache."""
    rng = np.random.default_rng(30)
    lens, new, d = [300, 77, 513, 20], [200, 77, 60, 33], 128
    c = E.Cache(rng, *([E.bf16(rng.standard_normal((L, 4, d)) * np.exp2(x * rng.standard_normal((L, 4, 1))))[1]
                        for L in lens] for x in (0.3, 2.0)))
    q = E.bf16(rng.standard_normal((sum(new), 4, d)))[0].cuda()
    t, cu = c.gpu(), _i32(np.concatenate([[0], np.cumsum(new)]))
    kc, vc = (torch.from_numpy(E.values(c.codes[x], np.where(c.scales[x] == 255, 0, c.scales[x]))
                               .astype(np.float32)).bfloat16().cuda() for x in "kv")
    o1, l1 = torch.empty_like(q), torch.empty((4, sum(new)), device="cuda")
    fb.fa_paged_prefill_e4m3(q, *t, cu, o1, l1, 4, sum(new), max(new), 4, 4, d, 16, c.num_pages,
                             c.table.shape[1], 0.1)
    o2, l2 = fb.paged_prefill(q, kc, vc, t[4], t[5], cu, max(new), 0.1)
    assert torch.equal(l1.view(torch.int32), l2.view(torch.int32))
    assert torch.equal(o1.view(torch.int16), o2.view(torch.int16))
