"""Drafted nodes whose later keys are much hotter than their first ones: how far a score may pass its
row's reference, and the values of V that fit beside it, against a 64-bit form."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _tree as T

pytestmark = pytest.mark.gpu

LENS, HKV = [3000, 2700, 2900, 3100], 8      # 4-6 K/V tiles of 128 keys a CTA, or (d = 64) as many halves


def _caches(rng, d, hotter, size, e4m3):
    """Rows whose keys of every third and fourth tile score `hotter` log2 units more than the others
    (queries have 1 at value 0), with values of V around `size`."""
    c = T.Cache(rng, LENS, HKV, d)
    unit = hotter * np.log(2.0) / float(np.float32(d ** -0.5))
    flat = []
    for s, n in enumerate(LENS):
        k, v = (torch.from_numpy(x).cuda() for x in c.rows[s])
        hot = (torch.arange(n, device="cuda") // 128) % 4 >= 2
        k[..., 0] = torch.where(hot, unit, 0.0)[:, None]
        flat.append([k.bfloat16(), (v * size).bfloat16()])
        pos = torch.arange(n, device="cuda")
        page = torch.from_numpy(c.bt[s]).cuda().long()[pos // T.PAGE]
        for x, y in zip((c.k, c.v), flat[s]):
            x[page, :, pos % T.PAGE] = y
        c.rows[s] = [T.f64(x) for x in flat[s]]
    args = (c.k, c.v)
    if e4m3:
        shape = c.k.shape
        args = tuple(torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in "kv") + \
            tuple(torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in "kv")
        state = (*args, T.i32(c.bt), T.i32(LENS))
        cu = T.i32(T.offsets(LENS))
        fb.paged_kv_write_e4m3(*(torch.cat([x[i] for x in flat]).contiguous() for i in range(2)), *state, cu)
        k, v = (T.f64(x) for x in fb.paged_kv_read_e4m3(*state, cu, sum(LENS)))
        at = T.offsets(LENS)
        c.rows = [[x[at[s]:at[s + 1]] for x in (k, v)] for s in range(len(LENS))]
    return (*args, T.i32(c.bt), T.i32(LENS)), c.rows


# 20 log2 units more: weights against the first tiles' reference would reach 2^20, and with V around
# 2^110 leave fp32's range, although no output does.  7, 14: the reference stays where it is.
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [5, 40])        # one and two query tiles of 4 heads a kv head
@pytest.mark.parametrize("hotter,power", [(20, 110), (7, 100), (14, 100), (30, 110)])
def test_hot_tiles_behind_cold_ones(hotter, power, n, d, e4m3):
    rng = np.random.default_rng(60)
    H, scale = 4 * HKV, float(np.float32(d ** -0.5))
    state, rows = _caches(rng, d, hotter, 2.0 ** power, e4m3)
    S = len(LENS)
    q = torch.randn((S * n, H, d), device="cuda", generator=torch.Generator(device="cuda").manual_seed(61))
    q[..., 0] = 1
    q = q.bfloat16()
    sees = [T.ancestors(T.random_parents(rng, n))[0] for _ in range(S)]
    words = (n + 31) // 32
    call = fb.paged_tree_attention_e4m3 if e4m3 else fb.paged_tree_attention
    o, lse = call(q, *state, T.i32(T.offsets([n] * S)), n, T.i32(np.concatenate([T.pack(x, words) for x in sees])),
                  scale)
    assert fb.fa_get_device_status() == 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    o, lse, q = T.f64(o), T.f64(lse).T, T.f64(q)
    for s, g in ((0, 0), (1, 5), (3, 7)):
        r, h = slice(s * n, s * n + n), slice(4 * g, 4 * g + 4)
        see = np.concatenate([np.ones((n, LENS[s] - n), bool), sees[s]], 1)
        ref = T.attend(q[r, h], rows[s][0][:, g], rows[s][1][:, g], scale, see)
        T.check_attention(o[r, h], lse[r, h], ref, f"sequence {s} kv head {g}")
