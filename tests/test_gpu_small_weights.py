"""A long tail of small weights beside one large one, in the kernels that round weights to f16.

One key of weight 1 whose V row is (1, 0, 0, ...), and L - 1 keys of weight 2^-24.8125 with V = 1: O's
dims from the second on are the tail's share, (L - 1) 2^-24.8125 over the sum.  The kernels hold
weights down to 2^-32 of the largest, in steps of at most 2^-31 there, so each is off by half a step,
2^-32, and O by L 2^-32; the fp32 sum of L terms adds L 2^-23 and the rounding to bf16 2^-8, both
relative.  (Each warp has a reference of its own: only keys that share a warp with the large one
lose anything, a quarter of them in the launches of many sequences.)"""
import math

import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

pytestmark = pytest.mark.gpu
L = 131072
W = 2.0 ** -24.8125


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 70000, L - 1])
@pytest.mark.parametrize("S,new,group", [(1, 1, 1), (700, 1, 1), (500, 1, 12), (400, 1, 20), (500, 4, 4)])
def test_tail(d, at, S, new, group):
    k = torch.zeros((L, 1, d), dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    k[:, 0, 0] = -0.8125          # scores in powers of two: q k scale = k ln 2; all values are codes
    k[at, 0, 0], v[at, 0, 1:] = 24.0, 0.0
    blocks = L // 16
    cache = [torch.zeros((blocks, 1, 16, d), dtype=torch.uint8, device="cuda") for _ in "kv"]
    cache += [torch.zeros((blocks, 1, 16), dtype=torch.uint8, device="cuda") for _ in "kv"]
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").view(1, -1)
    fb.paged_kv_write_e4m3(k, v, *cache, table, _i32([L]), _i32([0, L]))
    cache += [table.expand(S, blocks).contiguous(), _i32([L] * S)]     # the sequences share their pages
    q = torch.zeros((S * new, group, d), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    need = fb.fa_paged_e4m3_workspace_size(S, new, group, 1, d)
    want = (L - 1) * W / (1 + (L - 1) * W)
    bound = 1.01 * (L * 2.0 ** -32 + (2.0 ** -8 + L * 2.0 ** -23) * want)
    for ws in (None, torch.empty(need, dtype=torch.uint8, device="cuda")):
        o = torch.full((S * new, group, d), 9.0, dtype=torch.bfloat16, device="cuda")
        fb.fa_paged_prefill_e4m3(q, *cache, _i32(np.arange(S + 1) * new), o, None, S, S * new, new, group,
                                 1, d, 16, blocks, blocks, math.log(2.0), False, 0, 0, ws,
                                 0 if ws is None else need)
        err = (o[:, :, 1:].double() - want).abs().max().item()
        assert err <= bound, f"O {o[0, 0, 1].item()}, wanted {want}, off by up to {err}, bound {bound}"
        assert (o[:, :, 0] == 1.0).all()
    assert fb.fa_get_device_status() == 0
