"""Rows of prompts: so many tokens that a warp goes through several groups of heads of one token (q, then
k, then v, the next group on its way), against the 64-bit form; and what each kind of unusable token is
reported as."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _tree as T
from test_gpu_debug_build import CHILD, ROOT

pytestmark = pytest.mark.gpu

# (one wave has room for 3040 warps: from half as many tokens on a token has one warp, from a third on
# two; a group is 8 heads of 128 values or 16 of 64)
CASES = [  # total, H, Hkv, d, rot, interleaved, sections
    (1600, 32, 8, 128, 128, False, [24, 20, 20]),
    (1100, 32, 8, 128, 64, False, [32]),
    (3100, 21, 7, 64, 64, False, [32]),
    (1600, 40, 20, 64, 48, True, [10, 14]),
    (700, 37, 9, 128, 128, True, [64]),
    (1600, 1, 1, 128, 0, False, []),
]


def _inputs(total, H, Hkv, d, rot, axes):
    g = torch.Generator(device="cuda").manual_seed(90)
    x = torch.randn((total, H + 2 * Hkv, d), device="cuda", generator=g)
    x *= torch.exp2(2 * torch.randn((total, H + 2 * Hkv, 1), device="cuda", generator=g))
    # one head in fifty so large that its squares leave fp32
    x *= 1 + 2.0 ** 90 * (torch.rand((total, H + 2 * Hkv, 1), device="cuda", generator=g) < 0.02)
    x = x.bfloat16()
    w = [(1 + 0.3 * torch.randn(d, device="cuda", generator=g)).bfloat16() for _ in "qk"]
    angle = 7 * torch.randn((200, rot // 2), device="cuda", generator=g)
    cs = torch.stack([angle.cos(), angle.sin()], -1).contiguous() if rot else None
    pos = torch.randint(0, 200, (axes, total), device="cuda", generator=g).to(torch.int32) if rot else None
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], w, cs, pos


@pytest.mark.parametrize("total,H,Hkv,d,rot,interleaved,sections", CASES)
def test_prompts(total, H, Hkv, d, rot, interleaved, sections):
    axes, eps = max(1, len(sections)), 1e-6
    q, k, v, w, cs, pos = _inputs(total, H, Hkv, d, rot, axes)
    rows = None
    if rot:
        owner, at = np.repeat(np.arange(axes), sections), pos.cpu().numpy()
        rows = np.stack([T.f64(cs)[at[owner[p]], p] for p in range(rot // 2)], 1)
    want = [T.rotate(T.f64(x), T.f64(y), rows, rot, interleaved, eps) for x, y in zip((q, k), w)]
    got = fb.qk_norm_rope(q, k, *w, cs, pos, eps, sections or None, interleaved)
    for x, (y, mag), name in zip(got, want, "qk"):
        T.check_rows(T.f64(x), y, mag, name)
    rng = np.random.default_rng(91)
    new = [total // 3, 0, 1, total - total // 3 - 1]
    lens = [n + int(x) for n, x in zip(new, (37, 5, 0, 130))]
    pool = sum((n + 15) // 16 for n in lens) + 4
    bt, cu = T.table(rng, lens, pool), T.offsets(new)
    kc, vc = (torch.randn((pool, Hkv, 16, d), device="cuda").bfloat16() for _ in "kv")
    want_k, want_v = kc.clone(), vc.clone()
    for s in range(4):
        at = torch.arange(lens[s] - new[s], lens[s], device="cuda")
        page = torch.from_numpy(bt[s]).cuda().long()[at // 16]
        want_k[page, :, at % 16], want_v[page, :, at % 16] = got[1][cu[s]:cu[s + 1]], v[cu[s]:cu[s + 1]]
    qo = fb.paged_qkv_write(q, k, v, *w, cs, pos, kc, vc, T.i32(bt), T.i32(lens), T.i32(cu), eps, sections or None,
                            interleaved)
    assert torch.equal(qo, got[0]) and torch.equal(kc, want_k) and torch.equal(vc, want_v)
    # in place
    q2, k2 = (x.clone(memory_format=torch.contiguous_format) for x in (q, k))
    fb.fa_qk_norm_rope(q2, k2, *w, cs, pos, q2, k2, total, H, Hkv, d, H * d, Hkv * d, rot, interleaved, axes,
                       sections or None, 200 if rot else 0, eps)
    assert torch.equal(q2, got[0]) and torch.equal(k2, got[1])
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("total", [12, 1612])
@pytest.mark.parametrize("what", ["position below", "position above", "page below", "page above", "rows", "length"])
def test_each_unusable_token_has_its_status(what, total):
    H, Hkv, d = 32, 8, 128
    q, k, v, w, cs, pos = _inputs(total, H, Hkv, d, 128, 2)
    new, lens = [5, 4, total - 10], [20, 30, total + 7]      # the last row is nobody's
    pool = sum((n + 15) // 16 for n in lens)
    bt, cu = T.table(np.random.default_rng(92), lens, pool), T.offsets(new)
    table, L, at = bt.copy(), list(lens), pos.clone()
    status, left = fb.FA_ERR_INVALID_ARG, [7]
    if what.startswith("position"):
        at[1, 7] = 200 if what.endswith("above") else -1
    elif what.startswith("page"):
        table[1, 1] = pool if what.endswith("above") else -1   # tokens 26 .. 29 of sequence 1
        status, left = fb.FA_ERR_BAD_BLOCK_TABLE, [5, 6, 7, 8]
    else:
        L[1] = 3 if what == "rows" else 16 * bt.shape[1] + 1
        left = [5, 6, 7, 8]
    left = left + [total - 1]
    written = [i for i in range(total) if i not in left]
    dense_q, dense_k = fb.qk_norm_rope(q, k, *w, cs, pos, 1e-6, [40, 24])
    assert fb.fa_get_device_status() == 0
    qo = torch.full((total, H, d), 5.0, device="cuda").bfloat16()
    kc, vc = (torch.full((pool, Hkv, 16, d), 3.0, device="cuda").bfloat16() for _ in "kv")
    want_k, want_v = kc.clone(), vc.clone()
    for s in range(3):
        for i in range(cu[s], cu[s + 1]):
            if i not in left:
                p = lens[s] - new[s] + i - cu[s]
                page = int(bt[s, p // 16])
                want_k[page, :, p % 16], want_v[page, :, p % 16] = dense_k[i], v[i]
    st = q.stride(0)
    fb.fa_paged_qkv_write(q, k, v, *w, cs, at, qo, kc, vc, T.i32(table), T.i32(L), T.i32(cu), 3, total, H, Hkv, d, st,
                          st, st, 128, False, 2, [40, 24], 200, 1e-6, 16, pool, bt.shape[1])
    assert fb.fa_get_device_status() == status
    assert (qo[left] == 5).all() and torch.equal(qo[written], dense_q[written])
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_debug_build_passes():
    """Here the normal build's tests; in a child process the debug build's, which checks every store's index."""
    if os.environ.get("FA_LIBRARY"):
        return
    from tiled_online_softmax_sm_gb300 import build
    lib = build.build(debug=True)
    r = subprocess.run([sys.executable, "-c", CHILD, lib, "tests/test_gpu_prompt_rows.py"], cwd=ROOT,
                       env=dict(os.environ, FA_LIBRARY=lib), capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
