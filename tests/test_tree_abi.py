"""Refusals of the entries on drafted token trees, on the CPU: nothing is launched."""
import ctypes
import inspect

import pytest

from tiled_online_softmax_sm_gb300 import binding as fb
from tiled_online_softmax_sm_gb300 import build as fbuild

INV, UNS, WS, OK = fb.FA_ERR_INVALID_ARG, fb.FA_ERR_UNSUPPORTED, fb.FA_ERR_WORKSPACE, fb.FA_OK
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fb.load()


def _ints(*x):
    return (ctypes.c_int * len(x))(*x)


def _layout(lib, parents=16, sl=16, cu=16, mask=16, pos=16, S=4, T=10, words=2):
    return lib.fa_tree_layout(parents, sl, cu, mask, pos, S, T, words, None)


def _rope(lib, q=16, k=16, qw=16, kw=16, cs=16, pos=16, qo=32, ko=32, T=10, H=8, Hkv=2, d=128, qst=1024, kst=256,
          rot=128, inter=0, axes=1, sec=None, rows=100, eps=1e-6):
    return lib.fa_qk_norm_rope(q, k, qw, kw, cs, pos, qo, ko, T, H, Hkv, d, qst, kst, rot, inter, axes, sec, rows, eps,
                               None)


def _write(lib, q=16, k=16, v=16, qw=16, kw=16, cs=16, pos=16, qo=32, kc=16, vc=16, bt=16, sl=16, cu=16, S=4, T=10, H=8,
           Hkv=2, d=128, qst=1024, kst=256, vst=256, rot=128, inter=0, axes=1, sec=None, rows=100, eps=1e-6, page=16,
           P=100, maxb=8):
    return lib.fa_paged_qkv_write(q, k, v, qw, kw, cs, pos, qo, kc, vc, bt, sl, cu, S, T, H, Hkv, d, qst, kst, vst, rot,
                                  inter, axes, sec, rows, eps, page, P, maxb, None)


def _tree(lib, q=16, kc=16, vc=16, bt=16, sl=16, cu=16, mask=16, o=16, lse=16, S=4, T=10, mq=4, words=1, H=8, Hkv=2,
          d=128, page=16, P=100, maxb=8, scale=0.1, ws=256, wsb=1 << 30):
    return lib.fa_paged_tree_attention(q, kc, vc, bt, sl, cu, mask, o, lse, S, T, mq, words, H, Hkv, d, page, P, maxb,
                                       scale, ws, wsb, None)


def _tree8(lib, q=16, kc=16, vc=16, ks=16, vs=16, bt=16, sl=16, cu=16, mask=16, o=16, lse=16, S=4, T=10, mq=4, words=1,
           H=8, Hkv=2, d=128, page=16, P=100, maxb=8, scale=0.1, ws=256, wsb=1 << 30):
    return lib.fa_paged_tree_attention_e4m3(q, kc, vc, ks, vs, bt, sl, cu, mask, o, lse, S, T, mq, words, H, Hkv, d,
                                            page, P, maxb, scale, ws, wsb, None)


def _accept(lib, kc=16, vc=16, ks=None, vs=None, bt=16, sl=16, cu=16, path=16, pl=16, new=32, S=4, T=10, mp=4, layers=1,
            Hkv=2, d=128, page=16, P=100, maxb=8):
    return lib.fa_paged_kv_accept(kc, vc, ks, vs, bt, sl, cu, path, pl, new, S, T, mp, layers, Hkv, d, page, P, maxb,
                                  None)


def _copy(lib, kc=16, vc=16, ks=None, vs=None, pairs=16, N=4, layers=1, Hkv=2, d=128, page=16, P=100):
    return lib.fa_paged_copy_pages(kc, vc, ks, vs, pairs, N, layers, Hkv, d, page, P, None)


def _takes(call, kw):
    return all(x in inspect.signature(call).parameters for x in kw)


# What each entry that has the argument answers.
REFUSED = [(dict(S=-1), INV), (dict(T=-1), INV), (dict(P=-1), INV), (dict(maxb=-1), INV), (dict(layers=-1), INV),
           (dict(N=-1), INV), (dict(mq=-1), INV), (dict(mp=-1), INV), (dict(Hkv=0), INV), (dict(Hkv=-2), INV),
           (dict(H=0), INV), (dict(d=96), UNS), (dict(d=256), UNS), (dict(page=32), UNS), (dict(P=0), INV),
           (dict(maxb=0), INV), (dict(P=1 << 26), UNS), (dict(maxb=1 << 26), UNS), (dict(words=0), INV),
           (dict(rows=-1), INV), (dict(rot=12), UNS), (dict(rot=-8), INV), (dict(rot=136), INV),
           (dict(inter=2), INV), (dict(axes=0), INV), (dict(axes=5), UNS), (dict(axes=2), INV),
           (dict(axes=2, sec=_ints(30, 30)), INV), (dict(axes=2, sec=_ints(70, -6)), INV),
           (dict(axes=2, sec=_ints(-1, 65)), INV), (dict(axes=2, sec=_ints(2147483647, 2147483647)), INV),
           (dict(sec=_ints(63)), INV), (dict(eps=-1.0), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV),
           (dict(qst=1016), INV), (dict(qst=1028), INV), (dict(kst=248), INV), (dict(kst=260), INV),
           (dict(vst=248), INV), (dict(vst=260), INV), (dict(cs=None), INV), (dict(pos=None, rows=100), INV),
           (dict(rows=0), INV), (dict(T=1 << 28, H=8), UNS), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
           (dict(scale=NAN), INV), (dict(scale=INF), INV), (dict(ws=None), WS), (dict(ws=272), WS),
           (dict(wsb=100), WS), (dict(H=9, scale=0.1), INV), (dict(S=4097, scale=0.1), UNS),
           (dict(ks=16), INV), (dict(vs=16), INV), (dict(mp=1025), UNS), (dict(new=16), INV),
           (dict(layers=65536), UNS), (dict(Hkv=65537, kst=65537 * 128, vst=65537 * 128), UNS),
           (dict(Hkv=65537, layers=1, P=1), UNS), (dict(H=65537, qst=65537 * 128), UNS), (dict(H=258, Hkv=2, scale=0.1), UNS), (dict(N=1 << 26, layers=2), UNS), (dict(words=33, parents=16), UNS),
           (dict(T=1 << 27, words=16, mask=16, H=8), UNS), (dict(qo=16, qst=2048), INV), (dict(ko=16, kst=512), INV)]
REFUSED += [({x: None}, INV) for x in ("parents", "sl", "cu", "mask", "q", "k", "v", "qo", "ko", "kc", "vc", "bt", "o",
                                       "path", "pl", "new", "pairs")]
REFUSED += [({x: 24}, INV) for x in ("q", "k", "v", "qw", "kw", "cs", "qo", "ko", "kc", "vc", "o")]
REFUSED += [({x: 18}, INV) for x in ("parents", "sl", "cu", "mask", "bt", "path", "pl", "new", "pairs", "lse", "pos")]
REFUSED += [(dict(ks=24, vs=16), INV), (dict(ks=16, vs=8), INV)]


@pytest.mark.parametrize("call", [_layout, _rope, _write, _tree, _accept, _copy])
def test_refusals(lib, call):
    tried = 0
    for kw, status in REFUSED:
        if not _takes(call, kw):
            continue
        assert call(lib, **kw) == status, kw
        assert lib.fa_last_error(), kw
        tried += 1
    assert tried >= 5


def test_refusals_e4m3(lib):
    for kw, status in REFUSED:
        if _takes(_tree8, kw) and kw not in (dict(ks=16), dict(vs=16)):
            assert _tree8(lib, **kw) == status, kw
    for kw in (dict(ks=None), dict(vs=None), dict(ks=None, vs=None), dict(ks=24), dict(vs=8)):
        assert _tree8(lib, **kw) == INV, kw
    assert _tree8(lib, S=0, ks=None, vs=None) == OK and _tree8(lib, T=0, ks=None, vs=None, ws=None) == OK


def test_empty_calls(lib):
    assert _layout(lib, S=0, parents=None) == OK and _layout(lib, T=0, mask=None) == OK
    assert _rope(lib, T=0, q=None, k=None, qo=None) == OK
    assert _write(lib, T=0, q=None) == OK and _write(lib, S=0, kc=None) == OK
    assert _tree(lib, S=0, q=None) == OK and _tree(lib, T=0, ws=None) == OK and _tree(lib, mq=0, ws=None) == OK
    assert _accept(lib, S=0, kc=None) == OK and _accept(lib, layers=0, kc=None) == OK
    assert _copy(lib, N=0, pairs=None) == OK and _copy(lib, layers=0) == OK


def test_list_of_tiles_is_bounded(lib):
    """The K/V tiles of all units are numbered in 32 bits."""
    assert _tree(lib, S=4096, T=4096 * 1000, mq=1000, words=32, H=64, Hkv=1, maxb=1 << 20) == UNS
    assert _tree(lib, T=2000000, mq=2000000, H=2000, Hkv=20) == UNS


def test_workspace_size(lib):
    size = lib.fa_paged_tree_workspace_size
    for bad in ((0, 4, 8, 2, 128), (4, 0, 8, 2, 128), (4, 4, 9, 2, 128), (4, 4, 8, 0, 128), (4, 4, 8, 2, 96)):
        assert size(*bad) == 0
    assert 0 < size(1, 1, 8, 2, 64) < size(1, 64, 8, 2, 64) < size(1, 64, 8, 2, 128)
    # no more than two row tiles a partial, however many nodes
    assert size(4, 64, 8, 2, 128) == size(4, 100000, 8, 2, 128) == size(4096, 2147483647, 8, 2, 128)
    need = size(4, 4, 8, 2, 128)
    assert _tree(lib, wsb=need - 1) == WS


def test_new_lengths_are_an_array_of_their_own(lib):
    assert _accept(lib, sl=48, cu=64, path=80, pl=96, new=48) == INV
    for x in ("sl", "cu", "path", "pl"):
        a = dict(sl=48, cu=64, path=80, pl=96)
        assert _accept(lib, new=a[x], **a) == INV, x


def test_helpers_refuse_sections_that_do_not_fit():
    with pytest.raises(fb.FaError):
        fb.fa_qk_norm_rope(16, 16, None, None, 16, 16, 32, 32, 10, 8, 2, 128, 1024, 256, 128, False, 2, [64], 100, 1e-6,
                           stream=7)
