"""Layout of drafted trees, norms with rotation, cache writes, accepted paths and page copies."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _tree as T

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ layout
@pytest.mark.parametrize("words", [1, 2, 9, 32])
def test_layout(words):
    rng = np.random.default_rng(30)
    most = 32 * words
    new = [n for n in (0, 1, 2, 31, 32, 33, 100, 257, 1024, 0, most) if n <= most]
    parents = [T.random_parents(rng, n) for n in new]
    parents[-1] = np.arange(-1, most - 1)          # one chain
    if len(new) > 4:
        parents[4] = np.full(new[4], -1)           # only children of the context
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 9000, len(new)))]
    mask, pos = fb.tree_layout(T.i32(np.concatenate(parents)), T.i32(lens), T.i32(T.offsets(new)), words)
    want = [T.ancestors(p) for p in parents]
    assert np.array_equal(mask.cpu().numpy(), np.concatenate([T.pack(s, words) for s, _ in want]))
    assert np.array_equal(pos.cpu().numpy(), np.concatenate(
        [L - n + depth for (_, depth), L, n in zip(want, lens, new)]))
    assert fb.fa_get_device_status() == 0


def test_layout_refuses_and_leaves_alone():
    new, lens = [3, 40, 5, 4], [10, 50, 4, 9]       # 40 nodes: too many for one word; 5 nodes of 4 tokens
    cu = T.offsets(new)
    total = int(cu[-1]) + 2
    parents = np.zeros(total, np.int32)
    for s in range(4):
        parents[cu[s]:cu[s + 1]] = np.arange(new[s]) - 1
    mask = torch.full((total, 1), 99, dtype=torch.int32, device="cuda")
    pos = torch.full((total,), 99, dtype=torch.int32, device="cuda")
    fb.fa_tree_layout(T.i32(parents), T.i32(lens), T.i32(cu), mask, pos, 4, total, 1)
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    m, p = mask.cpu().numpy()[:, 0], pos.cpu().numpy()
    assert m[:3].tolist() == [1, 3, 7] and p[:3].tolist() == [7, 8, 9]
    assert m[cu[3]:cu[4]].tolist() == [1, 3, 7, 15] and p[cu[3]:cu[4]].tolist() == [5, 6, 7, 8]
    assert (m[3:cu[3]] == 99).all() and (m[cu[4]:] == 99).all() and (p[cu[4]:] == 99).all()
    # links that are no earlier node count as children of the context
    bad = T.i32([-1, 1, 0, 7, -9, 2])
    mask, pos = fb.tree_layout(bad, T.i32([6]), T.i32([0, 6]), 1)
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    assert mask[:, 0].tolist() == [1, 2, 5, 8, 16, 37] and pos.tolist() == [0, 0, 1, 0, 0, 2]
    only = torch.full((6, 1), 0, dtype=torch.int32, device="cuda")
    fb.fa_tree_layout(T.i32([-1, 0, 1, 2, 3, 4]), T.i32([6]), T.i32([0, 6]), only, None, 1, 6, 1)
    assert only[:, 0].tolist() == [1, 3, 7, 15, 31, 63]
    assert fb.fa_get_device_status() == 0


# ------------------------------------------------------------ norms, rotation
def _rope_inputs(seed, total, H, Hkv, d, rot, axes, norm, rows=300):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((total, H + 2 * Hkv, d), device="cuda", generator=g)
    qkv *= torch.exp2(3 * torch.randn((total, H + 2 * Hkv, 1), device="cuda", generator=g))
    qkv = qkv.bfloat16()
    w = [(1 + 0.3 * torch.randn(d, device="cuda", generator=g)).bfloat16() if norm else None for _ in "qk"]
    angle = 7 * torch.randn((rows, rot // 2), device="cuda", generator=g)
    cs = torch.stack([angle.cos(), angle.sin()], -1).contiguous() if rot else None
    pos = torch.randint(0, rows, (axes, total), device="cuda", generator=g).to(torch.int32) if rot else None
    return qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], w, cs, pos


def _angles(cs, pos, sections):
    rows = T.f64(cs)
    half = rows.shape[1]
    owner = np.repeat(np.arange(len(sections)), sections)
    p = pos.cpu().numpy()
    return np.stack([rows[p[owner[x]], x] for x in range(half)], 1)


def _check_rope(got, x, w, cs, pos, sections, rot, interleaved, eps, what):
    rows = _angles(cs, pos, sections) if rot else None
    want, mag = T.rotate(T.f64(x), None if w is None else T.f64(w), rows, rot, interleaved, eps)
    T.check_rows(T.f64(got), want, mag, what)


CASES = [  # total, H, Hkv, d, rot, interleaved, sections, norm
    (1, 1, 1, 128, 128, False, [64], True),
    (7, 32, 8, 128, 128, False, [64], True),
    (33, 6, 2, 64, 64, False, [32], True),
    (5, 5, 1, 128, 64, False, [32], True),
    (9, 8, 2, 64, 64, True, [32], True),
    (9, 3, 3, 128, 40, True, [20], False),
    (12, 8, 4, 128, 128, False, [16, 24, 24], True),
    (12, 7, 1, 64, 48, True, [5, 0, 18, 1], True),
    (4, 40, 2, 128, 0, False, [], True),
    (4, 2, 2, 64, 0, False, [], False),
    (3, 2, 2, 64, 8, False, [3, 1], False),
]


@pytest.mark.parametrize("total,H,Hkv,d,rot,interleaved,sections,norm", CASES)
def test_dense_rows(total, H, Hkv, d, rot, interleaved, sections, norm):
    q, k, _, w, cs, pos = _rope_inputs(31, total, H, Hkv, d, rot, max(1, len(sections)), norm)
    eps = 1e-5
    qo, ko = fb.qk_norm_rope(q, k, *w, cs, pos, eps, sections or None, interleaved)
    _check_rope(qo, q, w[0], cs, pos, sections, rot, interleaved, eps, "q")
    _check_rope(ko, k, w[1], cs, pos, sections, rot, interleaved, eps, "k")
    assert fb.fa_get_device_status() == 0
    # only q normalised; in place
    q2, k2 = (x.clone(memory_format=torch.contiguous_format) for x in (q, k))
    half = [None, None] if rot == 0 else [cs, pos]
    fb.fa_qk_norm_rope(q2, k2, w[0], None, *half, q2, k2, total, H, Hkv, d, H * d, Hkv * d, rot, interleaved,
                       max(1, len(sections)), sections or None, 300, eps)
    assert torch.equal(q2, qo)
    _check_rope(k2, k, None, cs, pos, sections, rot, interleaved, eps, "k without a norm")


@pytest.mark.parametrize("total,H,Hkv,d,rot,interleaved,sections,norm", CASES)
def test_rows_into_the_cache(total, H, Hkv, d, rot, interleaved, sections, norm):
    rng = np.random.default_rng(32)
    q, k, v, w, cs, pos = _rope_inputs(33, total, H, Hkv, d, rot, max(1, len(sections)), norm)
    new = [total // 2, 0, total - total // 2]
    lens = [n + int(x) for n, x in zip(new, (37, 5, 0))]
    cu = T.offsets(new)
    pool = 20
    bt = T.table(rng, lens, pool)
    kc, vc = (torch.randn((pool, Hkv, 16, d), device="cuda").bfloat16() for _ in "kv")
    old = T.f64(kc), T.f64(vc)
    qo = fb.paged_qkv_write(q, k, v, *w, cs, pos, kc, vc, T.i32(bt), T.i32(lens), T.i32(cu), 1e-6,
                            sections or None, interleaved)
    assert fb.fa_get_device_status() == 0
    dense_q, dense_k = fb.qk_norm_rope(q, k, *w, cs, pos, 1e-6, sections or None, interleaved)
    assert torch.equal(qo, dense_q)
    _check_rope(qo, q, w[0], cs, pos, sections, rot, interleaved, 1e-6, "q")
    want = old
    for s in range(3):
        at = np.arange(lens[s] - new[s], lens[s])
        page, place = bt[s, at // 16], at % 16
        want[0][page, :, place] = T.f64(dense_k)[cu[s]:cu[s + 1]]
        want[1][page, :, place] = T.f64(v)[cu[s]:cu[s + 1]]
    assert np.array_equal(T.f64(kc), want[0]) and np.array_equal(T.f64(vc), want[1])


def test_what_is_not_rotated_or_normalised_is_copied():
    """Infinities and NaN of v and of values outside the rotation pass through."""
    x = torch.randn((6, 2, 128), device="cuda").bfloat16()
    x[0, 0, 70] = float("inf")
    x[1, 1, 127] = float("nan")
    x[2, 0, 64] = -float("inf")
    cs = torch.ones((4, 32, 2), device="cuda")
    pos = torch.zeros((1, 6), dtype=torch.int32, device="cuda")
    q, k = fb.qk_norm_rope(x, x, None, None, cs, pos)
    assert torch.equal(q[..., 64:].view(torch.int16), x[..., 64:].view(torch.int16))
    assert torch.isfinite(q[..., :64]).all() and torch.equal(k.view(torch.int16), q.view(torch.int16))


def test_skipped_tokens_are_left_alone():
    rng = np.random.default_rng(34)
    H, Hkv, d, total = 4, 2, 64, 12
    q, k, v, w, cs, pos = _rope_inputs(35, total, H, Hkv, d, 64, 2, True)
    pos[1, 3] = 300
    pos[0, 4] = -1
    new, lens = [5, 4, 2], [20, 3, 40]             # sequence 1: more rows than tokens; row 11: nobody's
    bt = T.table(rng, [20, 16, 40], 9)
    bt[2, 2] = 9                                   # token 39 of sequence 2: no such page
    cu = T.offsets(new)
    kc, vc = (torch.full((9, Hkv, 16, d), 3.0, device="cuda").bfloat16() for _ in "kv")
    qo = torch.full((total, H, d), 5.0, device="cuda").bfloat16()
    args = (w[0], w[1], cs, pos)
    st = q.stride(0)
    fb.fa_paged_qkv_write(q, k, v, *args, qo, kc, vc, T.i32(bt), T.i32(lens), T.i32(cu), 3, total, H, Hkv, d, st,
                          st, st, 64, False, 2, [20, 12], 300, 1e-6, 16, 9, bt.shape[1])
    assert fb.fa_get_device_status() in (fb.FA_ERR_INVALID_ARG, fb.FA_ERR_BAD_BLOCK_TABLE)
    left = [3, 4, 5, 6, 7, 8, 10, 11]
    if lens[2] - 1 < 32:
        left.remove(10)
    written = [i for i in range(total) if i not in left and not (i in (9, 10) and (lens[2] - 2 + i - 9) // 16 == 2)]
    assert (qo[[i for i in range(total) if i not in written]] == 5).all()
    pos_ok = pos.clone()
    pos_ok[1, 3] = pos_ok[0, 4] = 0
    want, wk = fb.qk_norm_rope(q, k, w[0], w[1], cs, pos_ok, 1e-6, [20, 12])
    assert torch.equal(qo[written], want[written])
    for i in (0, 1, 2):
        at = 15 + i
        assert torch.equal(kc[int(bt[0, at // 16]), :, at % 16], wk[i])
        assert torch.equal(vc[int(bt[0, at // 16]), :, at % 16], v[i])
    assert int((kc != 3).any(-1).sum()) == 3 * Hkv and int((vc != 3).any(-1).sum()) == 3 * Hkv
    fb.qk_norm_rope(q, k, w[0], w[1], cs, pos, 1e-6, [20, 12])
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG


# ------------------------------------------------------------- moves, copies
def _caches(seed, layers, pool, Hkv, d, e4m3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, pool, Hkv, 16, d)
    if not e4m3:
        return [torch.randn(shape, device="cuda", generator=g).bfloat16() for _ in "kv"]
    return [torch.randint(0, 256, shape, device="cuda", generator=g).to(torch.uint8).view(F8) for _ in "kv"] + \
        [torch.randint(0, 255, shape[:4], device="cuda", generator=g).to(torch.uint8) for _ in "kv"]


def _bits(t):
    return t.view(torch.int16 if t.dtype is torch.bfloat16 else torch.uint8).cpu().numpy().copy()


@pytest.mark.parametrize("layers,Hkv,d,e4m3", [(1, 8, 128, False), (3, 2, 64, False), (2, 1, 128, True),
                                               (1, 20, 64, True), (2, 12, 128, False)])
def test_accept(layers, Hkv, d, e4m3):
    rng = np.random.default_rng(40)
    new = [1, 1, 40, 17, 0, 64, 300, 33]
    lens = [1, 20, 60, 17, 9, 100, 301, 800]
    paths = [[0], [], [0, 1, 2, 30], [3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 16], [], [63],
             sorted(rng.choice(300, 280, replace=False).tolist()), list(range(33))]
    pool = sum((n + 15) // 16 for n in lens) + 3
    bt = T.table(rng, lens, pool)
    c = _caches(41, layers, pool, Hkv, d, e4m3)
    want = [_bits(x) for x in c]
    deepest = 290
    path = np.full((8, deepest), 12345, np.int32)
    for s, p in enumerate(paths):
        path[s, :len(p)] = p
        src = [(lens[s] - new[s] + t) for t in p]
        for x in want:
            old = [x[:, bt[s, t // 16], :, t % 16].copy() for t in src]
            for a, row in enumerate(old):
                t = lens[s] - new[s] + a
                x[:, bt[s, t // 16], :, t % 16] = row
    k, v, ks, vs = c + [None] * (4 - len(c))
    if layers == 1:
        k, v = k[0], v[0]
        ks, vs = (None, None) if ks is None else (ks[0], vs[0])
    out = fb.paged_kv_accept(k, v, T.i32(bt), T.i32(lens), T.i32(T.offsets(new)), T.i32(path),
                             T.i32([len(p) for p in paths]), ks, vs)
    assert out.tolist() == [L - n + len(p) for L, n, p in zip(lens, new, paths)]
    for x, w in zip(c, want):
        assert np.array_equal(_bits(x), w)
    assert fb.fa_get_device_status() == 0


def test_accept_refuses_paths():
    rng = np.random.default_rng(42)
    bad = [([0, 0], 2), ([2, 1], 2), ([-1], 1), ([5], 1), ([0, 1, 2], 4), ([0, 1, 2], -1), ([1, 5], 2)]
    S = len(bad) + 1
    lens, new = [30] * S, [5] * S
    bt = T.table(rng, lens, 2 * S)
    k, v = _caches(43, 1, 2 * S, 2, 64, False)
    want = _bits(k), _bits(v)
    path = np.zeros((S, 3), np.int32)
    for s, (p, _) in enumerate(bad):
        path[s, :len(p)] = p
    path[-1] = [1, 4, 77]
    counts = [n for _, n in bad] + [2]
    for x in want:
        for a, t in enumerate((1, 4)):
            src, dst = 25 + t, 25 + a
            x[:, bt[-1, dst // 16], :, dst % 16] = x[:, bt[-1, src // 16], :, src % 16]
    out = fb.paged_kv_accept(k, v, T.i32(bt), T.i32(lens), T.i32(T.offsets(new)), T.i32(path), T.i32(counts))
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    assert out.tolist() == [30] * (S - 1) + [27]
    assert np.array_equal(_bits(k), want[0]) and np.array_equal(_bits(v), want[1])
    bt[-1, 1] = 2 * S                              # the sources' and destinations' page
    out = fb.paged_kv_accept(k, v, T.i32(bt[-1:]), T.i32([30]), T.i32([0, 5]), T.i32(path[-1:]), T.i32([2]))
    assert fb.fa_get_device_status() == fb.FA_ERR_BAD_BLOCK_TABLE
    assert out.tolist() == [27] and np.array_equal(_bits(k), want[0]) and np.array_equal(_bits(v), want[1])


@pytest.mark.parametrize("layers,Hkv,d,e4m3", [(1, 8, 128, False), (5, 3, 64, False), (2, 1, 128, True),
                                               (1, 20, 64, True), (3, 17, 128, True)])
def test_copy_pages(layers, Hkv, d, e4m3):
    rng = np.random.default_rng(44)
    c = _caches(45, layers, 90, Hkv, d, e4m3)
    want = [_bits(x) for x in c]
    ids = rng.permutation(90)
    pairs = np.stack([ids[:30], ids[40:70]], 1)
    pairs[5, 0] = pairs[6, 0] = pairs[7, 0]        # one source, several forks
    for x in want:
        x[:, pairs[:, 1]] = x[:, pairs[:, 0]]
    bad = np.concatenate([pairs[:10], [[-1, 0], [0, -1], [90, 1], [1, 1 << 30]], pairs[10:], [[ids[80], ids[80]]]])
    fb.paged_copy_pages(c[0], c[1], T.i32(bad), *c[2:])
    assert fb.fa_get_device_status() == fb.FA_ERR_BAD_BLOCK_TABLE
    for x, w in zip(c, want):
        assert np.array_equal(_bits(x), w)
    fb.paged_copy_pages(c[0], c[1], T.i32(np.zeros((0, 2))), *c[2:])
    assert fb.fa_get_device_status() == 0


# ------------------------------------------------------------ a run of them
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (6, 2, 64)])
def test_drafting_steps(H, Hkv, d):
    """Prompts, then drafted trees, each checked against the 64-bit form; the accepted path's rows then
    are the cache that plain decoding of the same tokens would have left, and a forked sequence goes on
    in pages of its own."""
    rng = np.random.default_rng(50)
    S, scale, eps = 3, float(np.float32(d ** -0.5)), 1e-6
    pool, width = 60, 12
    bt = np.full((S, width), -1, np.int32)
    bt[:] = rng.permutation(pool)[:S * width].reshape(S, width)
    kc, vc = (torch.full((pool, Hkv, 16, d), float("nan"), device="cuda").bfloat16() for _ in "kv")
    angle = np.arange(400)[:, None] * 1000.0 ** (-np.arange(d // 2) / (d // 2))
    cs = torch.from_numpy(np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)).cuda()
    w = [(1 + 0.2 * torch.randn(d, device="cuda")).bfloat16() for _ in "qk"]
    lens = np.zeros(S, np.int64)
    rows = [[np.zeros((0, Hkv, d))] * 2 for _ in range(S)]     # the context's K and V
    for step, new in enumerate(([37, 5, 64], [9, 1, 40], [12, 30, 7], [1, 1, 1])):
        prompt = step == 0
        parents = [np.arange(-1, n - 1) if prompt else T.random_parents(rng, n) for n in new]
        total, words = sum(new), (max(new) + 31) // 32
        cu, L = T.offsets(new), lens + np.array(new)
        mask, pos = fb.tree_layout(T.i32(np.concatenate(parents)), T.i32(L), T.i32(cu), words)
        qkv = torch.randn((total, H + 2 * Hkv, d), device="cuda").bfloat16()
        state = (kc, vc, T.i32(bt), T.i32(L))
        q = fb.paged_qkv_write(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], *w, cs, pos[None].contiguous(),
                               *state, T.i32(cu), eps)
        o, lse = fb.paged_tree_attention(q, *state, T.i32(cu), max(new), mask, scale)
        _, kd = fb.qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hkv], *w, cs, pos[None].contiguous(), eps)
        kd, vd, qd = T.f64(kd), T.f64(qkv[:, H + Hkv:]), T.f64(q)
        paths = []
        for s in range(S):
            r = slice(cu[s], cu[s + 1])
            tree, depth = T.ancestors(parents[s])
            assert pos[r].tolist() == (lens[s] + depth).tolist()
            see = np.concatenate([np.ones((new[s], lens[s]), bool), tree], 1)
            k, v = (np.concatenate([rows[s][x], y[r]]) for x, y in enumerate((kd, vd)))
            for g in range(Hkv):
                h = slice(g * H // Hkv, (g + 1) * H // Hkv)
                ref = T.attend(qd[r, h], k[:, g], v[:, g], scale, see)
                T.check_attention(T.f64(o)[r, h], T.f64(lse).T[r, h], ref, f"step {step} sequence {s}")
            leaf = new[s] - 1 if prompt else int(rng.integers(0, new[s]))
            paths.append(np.nonzero(tree[leaf])[0].tolist())
            rows[s] = [np.concatenate([rows[s][x], y[r][paths[s]]]) for x, y in enumerate((kd, vd))]
        deepest = max(len(p) for p in paths)
        out = fb.paged_kv_accept(*state, T.i32(cu), T.i32([p + [0] * (deepest - len(p)) for p in paths]),
                                 T.i32([len(p) for p in paths]))
        lens = lens + np.array([len(p) for p in paths])
        assert out.tolist() == lens.tolist()
        if step == 1:                              # sequence 2 goes on as a fork of sequence 0
            used = (lens[0] + 15) // 16
            fresh = np.setdiff1d(np.arange(pool), bt)[:used]
            fb.paged_copy_pages(kc, vc, T.i32(np.stack([bt[0, :used], fresh], 1)))
            bt[2, :used] = fresh
            lens[2], rows[2] = lens[0], list(rows[0])
        for s in range(S):
            at = np.arange(lens[s])
            for x, c in enumerate((kc, vc)):
                assert np.array_equal(T.f64(c)[bt[s, at // 16], :, at % 16], rows[s][x]), (step, s)
    if d == 128:    # the cache as the library's decode reads it
        q = torch.randn((S, H, d), device="cuda").bfloat16()
        o, lse = fb.paged_decode(q, kc, vc, T.i32(bt), T.i32(lens), 2, scale)
        for s in range(S):
            for g in range(Hkv):
                h = slice(g * H // Hkv, (g + 1) * H // Hkv)
                ref = T.attend(T.f64(q)[s:s + 1, h], *(x[:, g] for x in rows[s]), scale,
                               np.ones((1, lens[s]), bool))
                T.check_attention(T.f64(o)[s:s + 1, h], T.f64(lse)[s:s + 1, h], ref)
    assert fb.fa_get_device_status() == 0


def test_outputs_where_torch_has_no_short_way(monkeypatch):
    """The helpers' outputs, allocated either way: the same tensors."""
    cu, sl, parents = T.i32([0, 3, 7]), T.i32([20, 30]), T.i32([-1, 0, 0, -1, 0, 1, 1])
    q, k = (torch.randn((7, h, 64), device="cuda").bfloat16() for h in (4, 2))

    def outputs():
        return *fb.tree_layout(parents, sl, cu, 2), *fb.qk_norm_rope(q, k, None, None, None, None)

    got = outputs()
    monkeypatch.setattr(fb, "_new", fb._new_strided)
    for a, b in zip(got, outputs()):
        assert torch.equal(a, b) and a.stride() == b.stride() and a.dtype == b.dtype and a.device == b.device
        assert a.is_contiguous()


def test_caches_past_32_bits():
    """Pages whose elements are numbered past 2^31, in every operator."""
    Hkv, d, pool = 8, 128, 140000                  # 2.3e9 elements a cache
    rng = np.random.default_rng(51)
    kc, vc = (torch.empty((pool, Hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    bt = np.array([[139999, 3, 139000]], np.int32)
    cs = torch.stack([torch.ones((64, 64)), torch.zeros((64, 64))], -1).cuda().contiguous()
    n, L = 40, 40
    qkv = torch.randn((n, 32, d), device="cuda").bfloat16()
    pos = torch.zeros((1, n), dtype=torch.int32, device="cuda")
    state = (kc, vc, T.i32(bt), T.i32([L]))
    q = fb.paged_qkv_write(qkv[:, :16], qkv[:, 16:24], qkv[:, 24:], None, None, cs, pos, *state, T.i32([0, n]))
    assert torch.equal(q, qkv[:, :16])
    see = T.ancestors(T.random_parents(rng, n))[0]
    o, lse = fb.paged_tree_attention(q, *state, T.i32([0, n]), n, T.i32(T.pack(see, 2)), 0.1)
    for g in range(Hkv):
        ref = T.attend(T.f64(q)[:, 2 * g:2 * g + 2], T.f64(qkv[:, 16 + g]), T.f64(qkv[:, 24 + g]),
                       float(np.float32(0.1)), see)
        T.check_attention(T.f64(o)[:, 2 * g:2 * g + 2], T.f64(lse).T[:, 2 * g:2 * g + 2], ref)
    fb.paged_kv_accept(*state, T.i32([0, n]), T.i32([[5, 39]]), T.i32([2]))
    assert torch.equal(kc[139999, :, :2], qkv[[5, 39], 16:24].transpose(0, 1))
    fb.paged_copy_pages(kc, vc, T.i32([[139999, 138000], [139000, 7]]))
    assert torch.equal(vc[138000], vc[139999]) and torch.equal(vc[7, :, :8], vc[139000, :, :8])
    assert fb.fa_get_device_status() == 0
