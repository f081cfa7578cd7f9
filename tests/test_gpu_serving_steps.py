"""A serving loop over the e4m3 cache, every step held to the bound of the kernels that it takes:
weights rounded to f16 (2^-11) for single tokens and short chunks, to bf16 (2^-7, product and
divisor) for long ones."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _e4m3 as E
from test_gpu_e4m3_cache import _f64, _i32, _rounding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (6, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_steps(window, sinks, H, Hkv, d):
    rng = np.random.default_rng(70)
    S, scale = 3, E.softmax_scale(d)
    steps = [[37, 5, 64], [20, 0, 33], [2, 1, 2], [1, 1, 1], [4, 3, 4], [1, 0, 1], [1, 1, 1]]
    blocks = int((np.array(steps).sum(0).max() + 15) // 16)
    table = rng.permutation(S * blocks).reshape(S, blocks).astype(np.int32)
    cache = [torch.zeros((S * blocks, Hkv, 16, d), device="cuda").to(torch.float8_e4m3fn) for _ in "kv"]
    cache += [torch.zeros((S * blocks, Hkv, 16), dtype=torch.uint8, device="cuda") for _ in "kv"]
    rows = {x: [np.zeros((0, Hkv, d))] * S for x in "kv"}
    vexp, lens = [np.zeros((0, Hkv))] * S, np.zeros(S, np.int32)
    seen = set()
    for new in steps:
        n = sum(new)
        qkv = E.bf16(rng.standard_normal((n, H + 2 * Hkv, d)))[0].cuda()
        q, k, v = qkv[:, :H].contiguous(), qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        lens = lens + np.array(new, np.int32)
        cu = np.concatenate([[0], np.cumsum(new)])
        state = (*cache, _i32(table), _i32(lens))
        fb.paged_kv_write_e4m3(k, v, *state, _i32(cu))
        if new == [1, 1, 1]:
            o, lse = fb.paged_decode_e4m3(q, *state, scale, window=window, sinks=sinks)
        else:
            o, lse = fb.paged_prefill_e4m3(q, *state, _i32(cu), max(new), scale, window=window, sinks=sinks)
            lse = lse.T
        rounding = _rounding(max(new), H // Hkv, d)
        seen.add(rounding)
        o, lse, qd = _f64(o), _f64(lse), _f64(q)
        for s in range(S):
            r = slice(cu[s], cu[s + 1])
            for name, x in (("k", k), ("v", v)):
                code, b = E.quantise(_f64(x[r]))
                rows[name][s] = np.concatenate([rows[name][s], E.values(code, b)])
                if name == "v":
                    vexp[s] = np.concatenate([vexp[s], b.astype(float) - 127])
            ref = E.attend(qd[r], rows["k"][s], rows["v"][s], scale, True, window, sinks, vexp[s])
            E.check(o[r], lse[r], ref, d, rounding, f"step {new} sequence {s}")
    assert len(seen) == 2      # both kinds of kernel
    assert fb.fa_get_device_status() == 0
