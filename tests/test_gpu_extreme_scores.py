"""Scores far from zero, in every form of the e4m3 cache's attention: the references that are taken
off them are differences of equals, so equal scores weigh equally wherever they lie."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _e4m3 as E

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _run(c, q, new, d, scale=1.0):
    """O and LSE in float64, with a workspace and without one."""
    S, H = len(c.lens), q.shape[1]
    for ws in (None, torch.empty(fb.fa_paged_e4m3_workspace_size(S, new, H, c.Hkv, d), dtype=torch.uint8,
                                 device="cuda")):
        o = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((H, S * new), 9.0, device="cuda")
        fb.fa_paged_prefill_e4m3(q.cuda(), *c.gpu(), _i32(np.arange(S + 1) * new), o, lse, S, S * new, new, H,
                                 c.Hkv, d, 16, c.num_pages, c.table.shape[1], scale, False, 0, 0, ws,
                                 0 if ws is None else ws.numel())
        assert fb.fa_get_device_status() == 0
        yield o.double().cpu().numpy(), lse.double().cpu().numpy().T


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,group", [(1, 1), (1, 12), (3, 4), (60, 4)])
@pytest.mark.parametrize("L", [1, 2500])
@pytest.mark.parametrize("score", [-2.0 ** 60, -2.0 ** 25, -2.0 ** 12, 2.0 ** 12, 2.0 ** 25, 2.0 ** 120])
def test_equal_scores(d, new, group, L, score):
    """Every key the same K row: O is the mean of V, the LSE the score and ln L."""
    rng = np.random.default_rng(d + L)
    half = 2.0 ** round(np.log2(abs(score)) / 2)
    k = np.zeros((L, 1, d))
    k[:, :, 3] = half
    v = E.bf16(rng.standard_normal((L, 1, d)) * 2.0 ** -5)[1]
    q = np.zeros((new, group, d))
    q[:, :, 3] = np.sign(score) * abs(score) / half
    q = E.bf16(q)[0]
    c = E.Cache(rng, [k], [v], max_blocks=160)
    x = float(q[0, 0, 3].double()) * half
    mean = c.rows["v"][0][:, 0].mean(0)
    a = np.abs(c.rows["v"][0][:, 0]).mean(0)
    for o, lse in _run(c, q, new, d):
        # the equal weights cancel up to their roundings (2^-8 covers f16 and bf16) and L fp32 sums
        bound = 2.0 ** -8 * np.abs(mean) + (2.0 ** -8 + L * 2.0 ** -23) * a
        assert (np.abs(o - mean) <= bound).all(), f"O off by {np.abs(o - mean).max()}"
        assert (np.abs(lse - (x + np.log(L))) <= 2.0 ** -21 * (abs(x) + 20)).all()


# (Not -1e31 on the tcgen05 forward: it takes the rounded reference off the exact product of score
# and log2(e) scale.  Up to 2^-25 of the product is left, which past 2^31 no exponential can hold; a
# power of two leaves nothing.)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,group,score", [(1, 1, -1e31), (1, 12, -1e31), (3, 4, -1e31), (1, 1, -2.0 ** 120),
                                             (1, 12, -2.0 ** 120), (3, 4, -2.0 ** 120), (60, 4, -2.0 ** 120)])
@pytest.mark.parametrize("L", [1, 2500])
def test_most_negative_scores(d, new, group, L, score):
    """A row all of whose scores lie near the end of fp32's range is not one that sees no key."""
    test_equal_scores(d, new, group, L, score)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,group", [(1, 1), (1, 12), (3, 4), (60, 4)])
def test_scores_from_end_to_end(d, new, group):
    """Scores from -2^120 to 2^120 in one row: the largest takes all."""
    rng = np.random.default_rng(d)
    L = 2500
    k = np.zeros((L, 1, d))
    k[:, 0, 3] = -2.0 ** 60 * rng.choice([0.0, 0.5, 1.0], L)
    best = 1700
    k[best, 0, 3] = 2.0 ** 60
    v = E.bf16(rng.standard_normal((L, 1, d)))[1]
    q = np.zeros((new, group, d))
    q[:, :, 3] = 2.0 ** 60
    c = E.Cache(rng, [k], [v], max_blocks=160)
    for o, lse in _run(c, E.bf16(q)[0], new, d):
        assert (o == c.rows["v"][0][best, 0]).all()     # codes times a power of two are bf16 values
        assert (np.abs(lse / 2.0 ** 120 - 1) <= 2.0 ** -21).all()
