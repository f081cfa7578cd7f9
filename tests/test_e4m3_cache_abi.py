"""Refusals of the e4m3 paged cache's and the windowed forward's entries, on the CPU: nothing is
launched."""
import pytest

from tiled_online_softmax_sm_gb300 import binding as fb
from tiled_online_softmax_sm_gb300 import build as fbuild


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fb.load()


CACHE = dict(kc=16, vc=16, ks=16, vs=16, bt=16, sl=16, S=4, Hkv=8, d=128, page=16, P=100, maxb=8)


def _write(lib, **kw):
    a = dict(CACHE, k=16, v=16, cu=16, T=10, kst=1024, vst=1024)
    a.update(kw)
    return lib.fa_paged_kv_write_e4m3(a["k"], a["v"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"],
                                      a["sl"], a["cu"], a["S"], a["T"], a["Hkv"], a["d"], a["kst"],
                                      a["vst"], a["page"], a["P"], a["maxb"], None)


def _read(lib, **kw):
    a = dict(CACHE, k=16, v=16, cu=16, T=10)
    a.update(kw)
    return lib.fa_paged_kv_read_e4m3(a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"], a["cu"],
                                     a["k"], a["v"], a["S"], a["T"], a["Hkv"], a["d"], a["page"],
                                     a["P"], a["maxb"], None)


def _decode(lib, **kw):
    a = dict(CACHE, q=16, o=16, lse=16, H=32, scale=0.1, win=0, sinks=0, ws=None, wsb=0)
    a.update(kw)
    return lib.fa_paged_decode_e4m3(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"],
                                    a["o"], a["lse"], a["S"], a["H"], a["Hkv"], a["d"], a["page"],
                                    a["P"], a["maxb"], a["scale"], a["win"], a["sinks"], a["ws"],
                                    a["wsb"], None)


def _prefill(lib, **kw):
    a = dict(CACHE, q=16, o=16, lse=16, cu=16, T=10, mq=4, H=32, scale=0.1, causal=1, win=0, sinks=0,
             ws=None, wsb=0)
    a.update(kw)
    return lib.fa_paged_prefill_e4m3(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"],
                                     a["cu"], a["o"], a["lse"], a["S"], a["T"], a["mq"], a["H"],
                                     a["Hkv"], a["d"], a["page"], a["P"], a["maxb"], a["scale"],
                                     a["causal"], a["win"], a["sinks"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [_write, _read, _decode, _prefill])
def test_cache_refusals(lib, call):
    for kw in (dict(S=-1), dict(P=-1), dict(maxb=-1), dict(Hkv=0), dict(Hkv=-8), dict(kc=None),
               dict(vc=None), dict(ks=None), dict(vs=None), dict(bt=None), dict(sl=None), dict(P=0),
               dict(maxb=0), dict(kc=24), dict(vc=8), dict(ks=4), dict(vs=17), dict(bt=18),
               dict(sl=17)):
        assert call(lib, **kw) == fb.FA_ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(d=256), dict(page=32), dict(P=1 << 24), dict(maxb=1 << 26)):
        assert call(lib, **kw) == fb.FA_ERR_UNSUPPORTED, kw
    assert call(lib, S=0) == fb.FA_OK


@pytest.mark.parametrize("call", [_write, _read])
def test_row_refusals(lib, call):
    for kw in (dict(k=None), dict(v=None), dict(k=24), dict(v=8), dict(cu=None), dict(cu=18),
               dict(T=-1)):
        assert call(lib, **kw) == fb.FA_ERR_INVALID_ARG, kw
    assert call(lib, T=1 << 28) == fb.FA_ERR_UNSUPPORTED
    assert call(lib, T=0) == fb.FA_OK
    if call is _write:
        for kw in (dict(kst=1016), dict(vst=0), dict(kst=-1024), dict(vst=1028)):
            assert call(lib, **kw) == fb.FA_ERR_INVALID_ARG, kw


@pytest.mark.parametrize("call", [_decode, _prefill])
def test_attention_refusals(lib, call):
    for kw in (dict(q=None), dict(o=None), dict(q=8), dict(o=24), dict(lse=2), dict(H=30),
               dict(H=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(win=-1), dict(sinks=-1)):
        assert call(lib, **kw) == fb.FA_ERR_INVALID_ARG, kw
    assert call(lib, H=8 * 33) == fb.FA_ERR_UNSUPPORTED       # group of 33
    need = fb.fa_paged_e4m3_workspace_size(4, 4 if call is _prefill else 1, 32, 8, 128)
    assert need > 0
    assert call(lib, ws=256, wsb=need - 1) == fb.FA_ERR_WORKSPACE
    assert call(lib, ws=272, wsb=need) == fb.FA_ERR_WORKSPACE   # not 256-byte aligned
    assert call(lib, S=1 << 24, T=1 << 24) == fb.FA_ERR_UNSUPPORTED


def test_prefill_refusals(lib):
    for kw in (dict(cu=None), dict(cu=18), dict(T=-1), dict(mq=-1), dict(causal=2),
               dict(causal=0, win=5)):
        assert _prefill(lib, **kw) == fb.FA_ERR_INVALID_ARG, kw
    assert _prefill(lib, T=0) == fb.FA_OK
    assert _prefill(lib, mq=0) == fb.FA_OK


def _win(lib, **kw):
    a = dict(q=16, k=16, v=16, o=16, lse=16, B=1, H=2, Hkv=1, n=8, m=8, d=128, dv=128, scale=0.1,
             win=4, sinks=1)
    a.update(kw)
    return lib.fa_forward_window(a["q"], a["k"], a["v"], a["o"], a["lse"], a["B"], a["H"], a["Hkv"],
                                 a["n"], a["m"], a["d"], a["dv"], a["scale"], a["win"], a["sinks"], None)


def _varwin(lib, **kw):
    a = dict(q=16, k=16, v=16, o=16, lse=16, cq=16, ck=16, S=2, Tq=20, Tk=20, mq=10, mk=10, H=2,
             Hkv=1, d=128, dv=128, scale=0.1, win=4, sinks=1)
    a.update(kw)
    return lib.fa_forward_varlen_window(a["q"], a["k"], a["v"], a["o"], a["lse"], a["cq"], a["ck"],
                                        a["S"], a["Tq"], a["Tk"], a["mq"], a["mk"], a["H"], a["Hkv"],
                                        a["d"], a["dv"], a["scale"], a["win"], a["sinks"], None)


@pytest.mark.parametrize("call", [_win, _varwin])
def test_window_refusals(lib, call):
    for kw in (dict(win=-1), dict(sinks=-2), dict(H=3, Hkv=2), dict(H=0), dict(q=None), dict(o=None),
               dict(k=None), dict(v=None), dict(q=8), dict(o=24), dict(lse=2), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(lib, **kw) == fb.FA_ERR_INVALID_ARG, kw
    for kw in (dict(d=96, dv=96), dict(dv=64)):
        assert call(lib, **kw) == fb.FA_ERR_UNSUPPORTED, kw


def test_window_sizes(lib):
    assert _win(lib, B=-1) == fb.FA_ERR_INVALID_ARG
    assert _win(lib, n=-1) == fb.FA_ERR_INVALID_ARG
    assert _win(lib, B=0) == fb.FA_OK
    assert _win(lib, n=0) == fb.FA_OK
    assert _win(lib, n=1 << 30) == fb.FA_ERR_UNSUPPORTED
    for kw in (dict(S=-1), dict(Tq=-1), dict(Tk=-1), dict(mq=-1), dict(mk=-1), dict(cq=None),
               dict(ck=None), dict(cq=18), dict(ck=17)):
        assert _varwin(lib, **kw) == fb.FA_ERR_INVALID_ARG, kw
    assert _varwin(lib, S=0) == fb.FA_OK
    assert _varwin(lib, Tq=0) == fb.FA_OK
    assert _varwin(lib, mq=0) == fb.FA_OK
    assert _varwin(lib, Tq=1 << 30, mq=1 << 30) == fb.FA_ERR_UNSUPPORTED


def test_workspace_size(lib):
    size = fb.fa_paged_e4m3_workspace_size
    # (warps of one wave + units) x rows x (d values of O; m, r, l and a gap), and page counts
    assert size(64, 1, 32, 8, 128) == (152 * 3 * 4 + 64 * 8) * 8 * 132 * 4 + 1025 * 4
    assert size(64, 4, 32, 8, 128) == (152 * 3 * 4 + 64 * 8) * 16 * 132 * 4 + 1025 * 4
    assert size(3, 1, 9, 1, 64) == (152 * 3 * 4 + 3) * 16 * 68 * 4 + 1025 * 4
    # chunks on the forward: units of 256 rows, cut into parts that fill 152 SMs once (one
    # sequence) or twice, of 256 rows x (d values of O; m, l, l_p and a gap)
    assert size(1, 64, 32, 8, 128) == 8 * 19 * 256 * 132 * 4
    assert size(4, 512, 32, 8, 64) == 0
    # 32 rows a kv head: the forward at d = 128 for groups of a power of two, else the rows kernels
    assert size(2, 8, 32, 8, 128) == 2 * 8 * 19 * 256 * 132 * 4
    assert size(2, 8, 32, 8, 64) == (152 * 2 * 4 + 2 * 8) * 32 * 68 * 4 + 1025 * 4
    assert size(2, 8, 24, 8, 128) == (152 * 2 * 4 + 2 * 8) * 32 * 132 * 4 + 1025 * 4
    assert size(2, 1, 256, 8, 128) == (152 * 2 * 4 + 2 * 8) * 32 * 132 * 4 + 1025 * 4
    assert size(2, 1, 512, 8, 128) == 0
    assert size(2, 65, 16, 4, 64) == 16 * 19 * 256 * 68 * 4
    for bad in ((0, 1, 32, 8, 128), (4, 0, 32, 8, 128), (4, 1, 30, 8, 128), (4, 1, 32, 8, 96),
                (1025, 1, 32, 8, 128), (-1, 1, 8, 8, 64)):
        assert size(*bad) == 0
