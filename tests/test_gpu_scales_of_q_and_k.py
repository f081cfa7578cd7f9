"""K rows and q scaled by opposite powers of two give the same bits: the products of the scales stay
in range where either factor alone would not."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _e4m3 as E

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,group", [(1, 1), (1, 12), (3, 4), (60, 4)])
@pytest.mark.parametrize("p", [-110, -60, 60, 115])
def test_opposite_powers(d, new, group, p):
    rng = np.random.default_rng(d + new)
    L, Hkv = 2300, 2
    k, v = (E.bf16(rng.standard_normal((L, Hkv, d)))[1] for _ in "kv")
    # |q| in [0.5, 3]: scaling it is exact, down to 2^-116
    q = E.bf16(np.exp2(rng.uniform(-1, 1.5, (new, Hkv * group, d))) * rng.choice([-1, 1], (new, Hkv * group, d)))[1]
    out = []
    for x in (0, p):
        c = E.Cache(np.random.default_rng(1), [k * 2.0 ** x], [v], max_blocks=160)
        t, qt = c.gpu(), E.bf16(q * 2.0 ** -x)[0].cuda()
        for ws in (None, torch.empty(fb.fa_paged_e4m3_workspace_size(1, new, Hkv * group, Hkv, d),
                                     dtype=torch.uint8, device="cuda")):
            o = torch.full((new, Hkv * group, d), 9.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((Hkv * group, new), 9.0, device="cuda")
            fb.fa_paged_prefill_e4m3(qt, *t, _i32([0, new]), o, lse, 1, new, new, Hkv * group, Hkv, d, 16,
                                     c.num_pages, 160, 0.1, True, 0, 0, ws, 0 if ws is None else ws.numel())
            out.append((o, lse))
    assert torch.isfinite(out[0][1]).all()
    for a, b in zip(out[:2], out[2:]):
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16))
        assert torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))
    assert fb.fa_get_device_status() == 0


def test_zero_rows_under_the_largest_scale():
    """Codes of zero have score 0 under any scale byte, also beside a large q."""
    rng = np.random.default_rng(2)
    L, d = 300, 128
    k, v = np.zeros((L, 1, d)), E.bf16(rng.standard_normal((L, 1, d)))[1]
    c = E.Cache(rng, [k], [v])
    pos = np.arange(L)
    c.scales["k"][c.table[0, pos // 16], :, pos % 16] = 254
    q = E.bf16(rng.standard_normal((1, 4, d)) * 2.0 ** 40)[0]
    o, lse = fb.paged_decode_e4m3(q.cuda(), *c.gpu(), 0.1)
    ref = E.attend(q.double().numpy() * 0, k, c.rows["v"][0], 0.1, vexp=c.vexp[0])
    E.check(o.double().cpu().numpy(), lse.double().cpu().numpy(), ref, d, 2.0 ** -11)
