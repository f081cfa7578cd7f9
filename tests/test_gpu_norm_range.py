"""Norms of heads over the whole range of bf16: squares past fp32's largest value, and (with eps = 0)
below its smallest, against the 64-bit form."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _tree as T

pytestmark = pytest.mark.gpu

# sizes of heads: 1e18 and 3e18 on either side of where 128 squares leave fp32, up to bf16's largest
# value (3.39e38), down to its smallest normal and subnormal ones
SIZES = [1.0, 1e18, 1.5e18, 3e18, 1e19, 1e30, 1e38, 1e-10, 1e-17, 1e-19, 1e-24, 1e-30, 1e-38, 2.0 ** -130, 1e3, 1e-3]


def _heads(total, heads, d, seed):
    """Each head of a size of its own, so that the lanes of a warp hold both kinds; a value of 0 in each."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((total, heads, d), device="cuda", generator=g, dtype=torch.float64).clamp(-3.3, 3.3)
    x[..., 5] = 0
    size = torch.tensor(SIZES, device="cuda", dtype=torch.float64)
    order = torch.randint(0, len(SIZES), (total, heads, 1), device="cuda", generator=g)
    order[0, :, 0] = torch.arange(heads, device="cuda") % len(SIZES)
    return (x * size[order]).float().bfloat16()


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-6, 1.0, 1e31])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 64)])
def test_heads_of_every_size(d, rot, interleaved, eps):
    total, H, Hkv = 9, 16, 2
    q, k = _heads(total, H, d, 70), _heads(total, Hkv, d, 71)
    g = torch.Generator(device="cuda").manual_seed(72)
    w = [(1 + 0.3 * torch.randn(d, device="cuda", generator=g)).bfloat16() for _ in "qk"]
    angle = 7 * torch.randn((50, rot // 2), device="cuda", generator=g)
    cs = torch.stack([angle.cos(), angle.sin()], -1).contiguous()
    pos = torch.randint(0, 50, (1, total), device="cuda", generator=g).to(torch.int32)
    rows = T.f64(cs)[pos[0].cpu().numpy()]
    want = [T.rotate(T.f64(x), T.f64(y), rows, rot, interleaved, eps) for x, y in zip((q, k), w)]
    got = fb.qk_norm_rope(q, k, *w, cs, pos, eps, None, interleaved)
    for x, (y, mag), name in zip(got, want, "qk"):
        T.check_rows(T.f64(x), y, mag, name)
    kc, vc = (torch.zeros((2, Hkv, 16, d), device="cuda").bfloat16() for _ in "kv")
    qo = fb.paged_qkv_write(q, k, k, *w, cs, pos, kc, vc, T.i32([[1]]), T.i32([total]), T.i32([0, total]), eps, None,
                            interleaved)
    assert torch.equal(qo, got[0]) and torch.equal(kc[1, :, :total], got[1].transpose(0, 1))
    assert torch.equal(vc[1, :, :total], k.transpose(0, 1))
    assert fb.fa_get_device_status() == 0


def test_zeros_infinities_and_nan():
    """x / sqrt(mean x^2 + eps): a head of zeros is 0 (0 / 0 with eps = 0), one with an infinity is NaN
    there and 0 elsewhere, one with a NaN is NaN; the heads beside them are as without them."""
    x = torch.randn((1, 8, 128), device="cuda").bfloat16()
    clean = x.clone()
    x[0, 1] = 0
    x[0, 2, 7] = float("inf")
    x[0, 3, 100] = float("nan")
    x[0, 4] *= 2.0 ** 100
    w = torch.ones(128, device="cuda").bfloat16()
    for eps in (0.0, 1e-6):
        (a, _), (b, _) = (fb.qk_norm_rope(y, y, w, w, None, None, eps) for y in (x, clean))
        assert a[0, 1].isnan().all() if eps == 0 else (a[0, 1] == 0).all()
        assert a[0, 2, 7].isnan() and (a[0, 2, :7] == 0).all() and (a[0, 2, 8:] == 0).all()
        assert a[0, 3].isnan().all()
        # a power of two scales out (but for eps, which moves the norm by less than a step)
        assert (a[0, 4].float() - b[0, 4].float()).abs().max() <= 2 * T.BF16 * b[0, 4].float().abs().max()
        assert torch.equal(a[0, [0, 5, 6, 7]], b[0, [0, 5, 6, 7]])
    assert np.isfinite(T.f64(b)).all()
