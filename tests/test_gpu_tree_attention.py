"""Attention of drafted nodes over the bf16 paged cache, against a 64-bit form under derived bounds."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _tree as T

pytestmark = pytest.mark.gpu


def _run(seed, lens, new, H, Hkv, d, sees=None, words=None, scale=None, only=None, bound=None, **kw):
    """One call checked row by row; sees: per sequence [n, n] truth values (default: random trees);
    only: the sequences that are compared (all)."""
    rng = np.random.default_rng(seed)
    scale = scale or float(np.float32(d ** -0.5))
    c = T.Cache(rng, lens, Hkv, d, gen=seed, **kw)
    if sees is None:
        sees = [T.ancestors(T.random_parents(rng, n))[0] for n in new]
    words = words or max((max(new) + 31) // 32, 1)
    cu = T.offsets(new)
    mask = np.concatenate([T.pack(x, words) for x in sees] + [np.zeros((0, words), np.int32)])
    q = torch.randn((int(cu[-1]), H, d), device="cuda",
                    generator=torch.Generator(device="cuda").manual_seed(seed + 1)).bfloat16()
    o, lse = fb.paged_tree_attention(q, *c.args(), T.i32(cu), bound or max(max(new), 1), T.i32(mask), scale)
    assert fb.fa_get_device_status() == 0
    o, lse, qd, G = T.f64(o), T.f64(lse).T, T.f64(q), H // Hkv
    for s in range(len(lens)) if only is None else only:
        L, n = lens[s], new[s]
        r = slice(cu[s], cu[s + 1])
        see = np.concatenate([np.ones((n, L - n), bool), sees[s][:, :n]], 1)
        for g in range(Hkv):
            h = slice(g * G, (g + 1) * G)
            ref = T.attend(qd[r, h], c.rows[s][0][:, g], c.rows[s][1][:, g], scale, see)
            T.check_attention(o[r, h], lse[r, h], ref, f"sequence {s} (L {L}, n {n}) kv head {g}")
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (6, 2), (8, 1)])
def test_ragged_trees(H, Hkv, d):
    _run(3, [1, 16, 17, 127, 128, 129, 300, 1000, 64], [1, 16, 3, 20, 1, 31, 40, 8, 0], H, Hkv, d)


@pytest.mark.parametrize("d", [64, 128])
def test_one_token(d):
    """A tree of one node is a decode step."""
    lens, H, Hkv = [1, 5, 128, 700, 2000], 8, 2
    o, lse = _run(4, lens, [1] * 5, H, Hkv, d)
    if d == 128:
        c = T.Cache(np.random.default_rng(4), lens, Hkv, d, gen=4)
        q = torch.randn((5, H, d), device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()
        od, ld = fb.paged_decode(q, *c.args(), 4, float(np.float32(d ** -0.5)))
        # each within half a bf16 step of weights and of its own rounding of the same row
        assert np.abs(T.f64(od) - o).max() <= 4 * T.BF16 * np.abs(o).max()
        assert np.abs(T.f64(ld) - lse).max() <= 1e-4


@pytest.mark.parametrize("H,Hkv,new", [(3, 1, [130, 7]), (8, 1, [33, 70]), (32, 1, [9, 5]), (2, 1, [300, 1]),
                                       (5, 1, [52, 51]), (1, 1, [129, 128])])
def test_rows_of_several_tiles(H, Hkv, new):
    """More rows a kv head than one tile, than two, and groups that end inside one."""
    _run(5, [500, 420], new, H, Hkv, 128)
    _run(6, [400, 71], new[:1] + [min(71, new[1])], H, Hkv, 64)


@pytest.mark.parametrize("G,new", [(128, [3, 1, 5]), (96, [2, 3, 0]), (65, [1, 4, 2]), (43, [2, 5, 7])])
def test_wide_groups(G, new):
    """Groups of heads that fill a query tile alone, or leave rows of it unused."""
    _run(22, [300, 17, 140], new, G, 1, 128)
    _run(23, [300, 17, 1400], new, 2 * G, 2, 64)


def test_most_sequences():
    """4096 sequences, the most a call takes, of 0 to 3 nodes."""
    rng = np.random.default_rng(24)
    new = rng.integers(0, 4, 4096).tolist()
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 150, 4096))]
    _run(25, lens, new, 2, 1, 64, only=range(5, 4096, 331))


@pytest.mark.parametrize("d", [64, 128])
def test_one_and_two_query_tiles_in_one_batch(d):
    """Units of both kinds over cut keys, weighed against each other."""
    _run(26, [6000, 9000, 4000, 128, 7000, 257], [5, 60, 33, 40, 1, 64], 32, 8, d, only=[1, 2, 3, 4, 5])


def test_loose_bounds():
    """More mask words and a larger bound than any sequence needs."""
    _run(27, [300, 64], [9, 40], 4, 2, 128, words=7, bound=5000)


def test_long_context_is_cut():
    _run(7, [9000, 40], [12, 3], 8, 2, 128)
    _run(8, [9000], [70], 8, 2, 128)      # two query tiles over cut keys
    _run(9, [20000], [2], 4, 1, 64)


def test_more_sequences_than_pieces():
    rng = np.random.default_rng(1)
    new = rng.integers(0, 6, 400).tolist()
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 40, 400))]
    _run(10, lens, new, 2, 1, 64)
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 500, 400))]
    _run(11, lens, new, 4, 2, 128, only=range(0, 400, 37))


def test_bits_beyond_trees():
    """Any bits: rows that see nothing (without a context: O = 0, LSE = -inf), bits above the diagonal,
    bits past the last node, words that nobody needs."""
    rng = np.random.default_rng(2)
    new = [40, 33, 64, 5]
    sees = [rng.random((n, 32 * 4)) < 0.3 for n in new]
    for s in sees:
        s[::3] = False
    _run(12, [40, 33, 300, 130], new, 6, 2, 128, sees=sees, words=4)
    _run(13, [40, 33, 300, 130], new, 6, 2, 64, sees=sees, words=4, bound=100)


@pytest.mark.parametrize("d", [64, 128])
def test_hot_scores(d):
    """Scores of several hundred: the reference is raised often, one key has nearly all the weight."""
    _run(14, [700, 300], [9, 30], 4, 2, d, scale=4.0, spread=1.5)
    _run(28, [1700, 300], [70, 30], 8, 2, d, scale=4.0, spread=1.5)    # two query tiles


@pytest.mark.parametrize("H", [2, 16])
def test_nothing_unseen_is_used(H):
    """NaN in nodes that no node sees (in K and in V), and in a page's rows past the end."""
    rng = np.random.default_rng(15)
    L, n, d = 150, 30, 128
    c = T.Cache(rng, [L], 1, d)
    see = np.tril(np.ones((n, n), bool))
    hidden = [3, 10, 29]
    see[:, hidden] = False
    for t in hidden:
        pos = L - n + t
        for x in (c.k, c.v):
            x[int(c.bt[0, pos // 16]), :, pos % 16] = float("nan")
    q = torch.randn((n, H, d), device="cuda").bfloat16()
    o, lse = fb.paged_tree_attention(q, *c.args(), T.i32([0, n]), n, T.i32(T.pack(see, 1)), 0.1)
    full = np.concatenate([np.ones((n, L - n), bool), see], 1)
    k, v = (np.nan_to_num(x[:, 0]) for x in c.rows[0])
    T.check_attention(T.f64(o), T.f64(lse).T, T.attend(T.f64(q), k, v, 0.1, full))
    assert fb.fa_get_device_status() == 0


def test_nan_and_infinite_scores():
    """A NaN in a key makes the rows that see it NaN, and no row that sees neither it nor its V; an
    infinite score likewise; a key whose score is -inf has weight 0."""
    rng = np.random.default_rng(16)
    L, n, d, H = 400, 20, 64, 2
    for value, bad in ((float("nan"), True), (float("inf"), True), (-float("inf"), False)):
        c = T.Cache(rng, [L], 1, d)
        pos = L - n + 7
        c.k[int(c.bt[0, pos // 16]), 0, pos % 16, 0] = value
        see = np.eye(n, dtype=bool)
        see[9, 7] = True
        q = torch.randn((n, H, d), device="cuda").bfloat16()
        q[..., 0] = q[..., 0].abs() + 0.1       # so that the infinite score has the key's sign
        o, lse = fb.paged_tree_attention(q, *c.args(), T.i32([0, n]), n, T.i32(T.pack(see, 1)), 0.2)
        o, lse = T.f64(o), T.f64(lse).T
        if bad:
            assert np.isnan(o[[7, 9]]).all() and np.isnan(lse[[7, 9]]).all()
        see[[7, 9], 7] = bad
        full = np.concatenate([np.ones((n, L - n), bool), see], 1)
        k, v = (x[:, 0] for x in c.rows[0])
        rest = [i for i in range(n) if not (bad and i in (7, 9))]
        ref = T.attend(T.f64(q)[rest], k, v, float(np.float32(0.2)), full[rest])
        T.check_attention(o[rest], lse[rest], ref)


@pytest.mark.parametrize("H", [2, 16])
@pytest.mark.parametrize("at", [0, 100, 300])
def test_nan_in_the_context(at, H):
    """Every node sees it: all rows are NaN, those of the other kv head and sequence are not."""
    rng = np.random.default_rng(29)
    c = T.Cache(rng, [400, 90], 2, 128)
    c.k[int(c.bt[0, at // 16]), 1, at % 16, 5] = float("nan")
    n = 20
    q = torch.randn((2 * n, 2 * H, 128), device="cuda").bfloat16()
    mask = np.concatenate([T.pack(np.tril(np.ones((n, n), bool)), 1)] * 2)
    o, lse = fb.paged_tree_attention(q, *c.args(), T.i32([0, n, 2 * n]), n, T.i32(mask), 0.1)
    assert o[:n, H:].isnan().all() and lse[H:, :n].isnan().all()
    assert not o[:n, :H].isnan().any() and not lse[:H, :n].isnan().any()
    assert not o[n:].isnan().any() and not lse[:, n:].isnan().any()
    assert fb.fa_get_device_status() == 0


def test_rows_behind_the_last_sequence_and_skipped_ones():
    """Rows that no sequence owns, and rows of sequences whose numbers do not fit, keep their contents;
    the others are computed, and the status word says so."""
    rng = np.random.default_rng(17)
    d, H, Hkv = 128, 4, 2
    lens, new = [50, 30, 200, 90], [4, 40, 6, 5]       # sequence 1 has more nodes than tokens
    c = T.Cache(rng, lens, Hkv, d)
    cu = T.offsets(new)
    total = int(cu[-1]) + 3
    sees = [np.tril(np.ones((n, n), bool)) for n in new]
    mask = np.concatenate([T.pack(x, 2) for x in sees] + [np.zeros((3, 2), np.int32)])
    q = torch.randn((total, H, d), device="cuda").bfloat16()
    o = torch.full((total, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, total), 7.0, device="cuda")

    def call(sl, cu, max_q, words=2):
        o.fill_(7.0)
        lse.fill_(7.0)
        ws = torch.empty(fb.fa_paged_tree_workspace_size(4, max_q, H, Hkv, d), dtype=torch.uint8, device="cuda")
        fb.fa_paged_tree_attention(q, c.k, c.v, T.i32(c.bt), T.i32(sl), T.i32(cu), T.i32(mask[:, :words]), o, lse,
                                   4, total, max_q, words, H, Hkv, d, 16, c.k.shape[0], c.bt.shape[1], 0.1, ws,
                                   ws.numel())
        return T.f64(o), T.f64(lse).T

    def check(got, good):
        for s in range(4):
            r = slice(cu[s], cu[s + 1])
            if s in good:
                see = np.concatenate([np.ones((new[s], lens[s] - new[s]), bool), sees[s]], 1)
                for g in range(Hkv):
                    h = slice(2 * g, 2 * g + 2)
                    ref = T.attend(T.f64(q)[r, h], c.rows[s][0][:, g], c.rows[s][1][:, g],
                                   float(np.float32(0.1)), see)
                    T.check_attention(got[0][r, h], got[1][r, h], ref)
            else:
                assert (got[0][r] == 7).all() and (got[1][r] == 7).all(), s
        assert (got[0][cu[4]:] == 7).all() and (got[1][cu[4]:] == 7).all()

    check(call(lens, cu, 40), (0, 2, 3))
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    check(call([50, 30, 16 * c.bt.shape[1] + 1, 90], cu, 40), (0, 3))    # beyond its table
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    check(call([50, 30, -5, 90], cu, 5), (0, 3))                         # 6 nodes, at most 5 were promised
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    check(call(lens, cu, 40, words=1), (0, 2, 3))
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG


def test_bad_page_is_reported():
    rng = np.random.default_rng(18)
    c = T.Cache(rng, [300, 200], 2, 128)
    for bad in (-1, c.k.shape[0], 1 << 30):
        c.bt[0, 3] = bad
        q = torch.randn((9, 4, 128), device="cuda").bfloat16()
        mask = T.i32(T.pack(np.tril(np.ones((9, 9), bool)), 1))
        o, lse = fb.paged_tree_attention(q, *c.args(), T.i32([0, 4, 9]), 5, mask, 0.1)
        assert fb.fa_get_device_status() == fb.FA_ERR_BAD_BLOCK_TABLE
        see = np.concatenate([np.ones((5, 195), bool), np.tril(np.ones((9, 9), bool))[4:, :5]], 1)
        for g in range(2):   # the other sequence is not touched by it
            ref = T.attend(T.f64(q)[4:, 2 * g:2 * g + 2], c.rows[1][0][:, g], c.rows[1][1][:, g],
                           float(np.float32(0.1)), see)
            T.check_attention(T.f64(o)[4:, 2 * g:2 * g + 2], T.f64(lse).T[4:, 2 * g:2 * g + 2], ref)


def test_same_bits_every_time_and_in_a_graph():
    """No atomics: the same call gives the same bits, alone, replayed from a graph on changed inputs, and
    on another stream with a workspace of its own."""
    rng = np.random.default_rng(19)
    lens, new, H, Hkv, d = [3000, 130, 700], [20, 1, 64], 8, 2, 128
    c = T.Cache(rng, lens, Hkv, d)
    cu, total = T.i32(T.offsets(new)), sum(new)
    mask = T.i32(np.concatenate([T.pack(T.ancestors(T.random_parents(rng, n))[0], 2) for n in new]))
    q = [torch.randn((total, H, d), device="cuda").bfloat16() for _ in range(2)]
    args = c.args()
    want = [fb.paged_tree_attention(x, *args, cu, 64, mask, 0.1) for x in q]
    again = fb.paged_tree_attention(q[0], *args, cu, 64, mask, 0.1)
    assert all(torch.equal(a, b) for a, b in zip(again, want[0]))
    static = q[0].clone()
    ws = torch.empty(fb.fa_paged_tree_workspace_size(3, 64, H, Hkv, d), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fb.paged_tree_attention(static, *args, cu, 64, mask, 0.1, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = fb.paged_tree_attention(static, *args, cu, 64, mask, 0.1, workspace=ws)
    for x, w in zip(q[::-1], want[::-1]):
        static.copy_(x)
        ws.random_(0, 256)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    side.wait_stream(torch.cuda.current_stream())
    two = fb.paged_tree_attention(q[1], *args, cu, 64, mask, 0.1, stream=side)
    one = fb.paged_tree_attention(q[0], *args, cu, 64, mask, 0.1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one + two, want[0] + want[1]))


def test_without_lse_and_empty_batches():
    rng = np.random.default_rng(20)
    c = T.Cache(rng, [100], 1, 128)
    q = torch.randn((5, 2, 128), device="cuda").bfloat16()
    mask = T.i32(np.full((5, 1), 31))
    o, _ = fb.paged_tree_attention(q, *c.args(), T.i32([0, 5]), 5, mask, 0.1)
    o2 = torch.empty_like(o)
    ws = torch.empty(fb.fa_paged_tree_workspace_size(1, 5, 2, 1, 128), dtype=torch.uint8, device="cuda")
    fb.fa_paged_tree_attention(q, *c.args(), T.i32([0, 5]), mask, o2, None, 1, 5, 5, 1, 2, 1, 128, 16,
                               c.k.shape[0], c.bt.shape[1], 0.1, ws, ws.numel())
    assert torch.equal(o, o2)
    none = fb.paged_tree_attention(q[:0], *c.args(), T.i32([0, 0]), 5, mask[:0], 0.1)
    assert none[0].shape == (0, 2, 128) and none[1].shape == (2, 0)
    fb.paged_tree_attention(q, *c.args(), T.i32([0, 0]), 5, mask, 0.1)     # every sequence is empty
    assert fb.fa_get_device_status() == 0


def test_a_wait_that_runs_out_is_reported(monkeypatch):
    """The copies' first tile left out: the bounded waits end, the status word says so, and the next
    call is right again."""
    rng = np.random.default_rng(21)
    c = T.Cache(rng, [300], 1, 128)
    q = torch.randn((5, 2, 128), device="cuda").bfloat16()
    mask = T.i32(T.pack(np.tril(np.ones((5, 5), bool)), 1))
    monkeypatch.setenv("FA_TEST_FORCE_WAIT_TIMEOUT", "1")
    fb.paged_tree_attention(q, *c.args(), T.i32([0, 5]), 5, mask, 0.1)
    assert fb.fa_get_device_status() == fb.FA_ERR_TIMEOUT
    monkeypatch.delenv("FA_TEST_FORCE_WAIT_TIMEOUT")
    o, lse = fb.paged_tree_attention(q, *c.args(), T.i32([0, 5]), 5, mask, 0.1)
    see = np.concatenate([np.ones((5, 295), bool), np.tril(np.ones((5, 5), bool))], 1)
    T.check_attention(T.f64(o), T.f64(lse).T,
                      T.attend(T.f64(q), *(x[:, 0] for x in c.rows[0]), float(np.float32(0.1)), see))
    assert fb.fa_get_device_status() == 0
