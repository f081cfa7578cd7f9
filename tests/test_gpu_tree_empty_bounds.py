"""A bound of 0 nodes, and caches without layers: no helper hands back outputs that nobody wrote."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _tree as T

pytestmark = pytest.mark.gpu


def _state(e4m3, lens):
    rng = np.random.default_rng(80)
    c = T.Cache(rng, lens, 2, 128)
    if not e4m3:
        return c.args(), c.rows
    shape = c.k.shape
    state = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in "kv"] + \
        [torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in "kv"] + [T.i32(c.bt), T.i32(lens)]
    cu = T.i32(T.offsets(lens))
    fb.paged_kv_write_e4m3(*(torch.from_numpy(np.concatenate([r[i] for r in c.rows])).cuda().bfloat16()
                             for i in range(2)), *state, cu)
    k, v = (T.f64(x) for x in fb.paged_kv_read_e4m3(*state, cu, sum(lens)))
    at = T.offsets(lens)
    return state, [[x[at[s]:at[s + 1]] for x in (k, v)] for s in range(len(lens))]


@pytest.mark.parametrize("own_workspace", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_bound_of_zero_nodes(e4m3, own_workspace):
    """A sequence of several nodes is reported, one of one node computed; without nodes it is no error,
    with the workspace that the library asks for then (0 bytes), too."""
    call = fb.paged_tree_attention_e4m3 if e4m3 else fb.paged_tree_attention
    state, rows = _state(e4m3, [70, 40])
    q = torch.randn((6, 4, 128), device="cuda").bfloat16()
    mask, scale = T.i32(np.full((6, 1), 1)), float(np.float32(0.1))
    size = fb.fa_paged_tree_workspace_size(2, 0, 4, 2, 128)
    kw = {"workspace": torch.empty(size, dtype=torch.uint8, device="cuda")} if own_workspace else {}
    assert fb.fa_get_device_status() == 0
    call(q, *state, T.i32([0, 5, 6]), 0, mask, scale, **kw)
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    o, lse = call(q, *state, T.i32([0, 1, 1]), 0, mask, scale, **kw)
    assert fb.fa_get_device_status() == 0
    for g in range(2):
        h = slice(2 * g, 2 * g + 2)
        ref = T.attend(T.f64(q)[:1, h], rows[0][0][:, g], rows[0][1][:, g], scale, np.ones((1, 70), bool))
        T.check_attention(T.f64(o)[:1, h], T.f64(lse).T[:1, h], ref)
    call(q, *state, T.i32([0, 0, 0]), 0, mask, scale, **kw)
    assert fb.fa_get_device_status() == 0
    with pytest.raises(fb.FaError):
        call(q, *state, T.i32([0, 5, 6]), -1, mask, scale, **kw)
    o, lse = call(q[:0], *state, T.i32([0, 0, 0]), 0, mask[:0], scale, **kw)
    assert o.shape == (0, 4, 128) and lse.shape == (4, 0)
