"""Attention of drafted nodes over the e4m3 paged cache, against a 64-bit form on the codes' values."""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _tree as T

pytestmark = pytest.mark.gpu


class Cache(T.Cache):
    """The same rows through paged_kv_write_e4m3; other slots hold the code and the byte of NaN."""

    def __init__(self, rng, lens, Hkv, d, gen=1, **kw):
        super().__init__(rng, lens, Hkv, d, gen=gen, **kw)
        shape = self.k.shape
        k, v = (torch.from_numpy(np.concatenate([p[i] for p in self.rows])).cuda().bfloat16() for i in range(2))
        self.k, self.v = (torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.full(shape[:3], 0xff, dtype=torch.uint8, device="cuda") for _ in range(2))
        fb.paged_kv_write_e4m3(k, v, *self.args(), T.i32(T.offsets(lens)))
        self.read()

    def read(self):
        """The codes' values: code * 2^(byte - 127), at most 4 significant bits."""
        self.rows = []
        for s, n in enumerate(self.lens):
            pos = torch.arange(n, device="cuda")
            page = torch.from_numpy(self.bt[s]).cuda().long()[pos // T.PAGE]
            pair = []
            for c, b in ((self.k, self.ks), (self.v, self.vs)):
                x = c[page, :, pos % T.PAGE].view(torch.float8_e4m3fn).double()
                pair.append((x * torch.exp2(b[page, :, pos % T.PAGE].double() - 127)[..., None]).cpu().numpy())
            self.rows.append(pair)

    def args(self):
        return self.k, self.v, self.ks, self.vs, T.i32(self.bt), T.i32(self.lens)


def _run(seed, lens, new, H, Hkv, d, scale=None, sees=None, words=None, **kw):
    rng = np.random.default_rng(seed)
    scale = scale or float(np.float32(d ** -0.5))
    c = Cache(rng, lens, Hkv, d, gen=seed, **kw)
    sees = sees or [T.ancestors(T.random_parents(rng, n))[0] for n in new]
    words = words or max((max(new) + 31) // 32, 1)
    cu = T.offsets(new)
    mask = np.concatenate([T.pack(x, words) for x in sees])
    q = torch.randn((int(cu[-1]), H, d), device="cuda",
                    generator=torch.Generator(device="cuda").manual_seed(seed + 1)).bfloat16()
    o, lse = fb.paged_tree_attention_e4m3(q, *c.args(), T.i32(cu), max(new), T.i32(mask), scale)
    assert fb.fa_get_device_status() == 0
    o, lse, qd, G = T.f64(o), T.f64(lse).T, T.f64(q), H // Hkv
    for s in range(len(lens)):
        L, n = lens[s], new[s]
        r = slice(cu[s], cu[s + 1])
        see = np.concatenate([np.ones((n, L - n), bool), sees[s][:, :n]], 1)
        for g in range(Hkv):
            h = slice(g * G, (g + 1) * G)
            ref = T.attend(qd[r, h], c.rows[s][0][:, g], c.rows[s][1][:, g], scale, see)
            T.check_attention(o[r, h], lse[r, h], ref, f"sequence {s} (L {L}, n {n}) kv head {g}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (6, 2), (8, 1)])
def test_ragged_trees(H, Hkv, d):
    _run(3, [1, 16, 17, 127, 128, 129, 300, 1000, 64], [1, 16, 3, 20, 1, 31, 40, 8, 0], H, Hkv, d)


@pytest.mark.parametrize("d", [64, 128])
def test_one_token(d):
    _run(4, [1, 5, 128, 700, 2000], [1] * 5, 8, 2, d)


@pytest.mark.parametrize("H,Hkv,new", [(3, 1, [130, 7]), (8, 1, [33, 70]), (32, 1, [9, 5]), (2, 1, [300, 1]),
                                       (1, 1, [129, 128]), (96, 1, [2, 3])])
def test_rows_of_several_tiles(H, Hkv, new):
    _run(5, [500, 420], new, H, Hkv, 128)
    _run(6, [400, 171], new, H, Hkv, 64)


@pytest.mark.parametrize("d", [64, 128])
def test_one_and_two_query_tiles_in_one_batch(d):
    _run(7, [3000, 2000, 700, 300, 5000], [3, 40, 64, 1, 20], 16, 4, d)


def test_long_context_is_cut():
    _run(8, [60000], [12], 4, 1, 128)
    _run(9, [50000], [40], 8, 1, 64)


def test_more_sequences_than_pieces():
    rng = np.random.default_rng(10)
    new = rng.integers(0, 9, 400).tolist()
    _run(10, [n + int(x) for n, x in zip(new, rng.integers(0, 400, 400))], new, 4, 2, 128)


@pytest.mark.parametrize("d", [64, 128])
def test_hot_scores(d):
    _run(11, [700, 300], [9, 30], 4, 2, d, scale=4.0, spread=1.5)


def test_scales_of_each_size():
    """Rows of 2^-60 to 2^60, and rows of zeros (byte 0)."""
    rng = np.random.default_rng(12)
    L, n, d = 300, 10, 128
    c = Cache(rng, [L], 1, d)
    pages = torch.from_numpy(c.bt[0]).cuda().long()
    for i, e in enumerate((-60, -30, 0, 30, 60)):
        c.vs[pages[i]] = 127 + e
    c.ks[pages[6]] = 0
    c.vs[pages[7]] = 0
    c.k[pages[6]] = 0
    c.v[pages[7]] = 0
    c.read()
    see = np.tril(np.ones((n, n), bool))
    q = torch.randn((n, 3, d), device="cuda").bfloat16()
    o, lse = fb.paged_tree_attention_e4m3(q, *c.args(), T.i32([0, n]), n, T.i32(T.pack(see, 1)), 0.125)
    full = np.concatenate([np.ones((n, L - n), bool), see], 1)
    T.check_attention(T.f64(o), T.f64(lse).T, T.attend(T.f64(q), *(x[:, 0] for x in c.rows[0]), 0.125, full))
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("byte", [0, 1, 7, 100, 127, 134, 135, 200, 240])
def test_every_code(byte):
    """One key, weight 1: o is V as bf16, of every code that is no NaN and with one that is."""
    d = 128
    c = Cache(np.random.default_rng(13), [1, 1, 1], 1, d)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(2, d)
    for s in range(3):
        page = int(c.bt[s, 0])
        c.v[page, 0, 0] = codes[s % 2] if s < 2 else codes[0].clone().masked_fill(codes[0] == 0x7f, 3)
        c.vs[page, 0, 0] = byte
    q = torch.randn((3, 1, d), device="cuda").bfloat16()
    o, _ = fb.paged_tree_attention_e4m3(q, *c.args(), T.i32([0, 1, 2, 3]), 1, T.i32([[1], [1], [1]]), 0.125)
    for s in range(3):
        x = c.v[int(c.bt[s, 0]), 0, 0].view(torch.float8_e4m3fn).float()
        want = (x.double() * 2.0 ** (byte - 127)).float().bfloat16()      # (exact in fp32)
        # the product with the weight 1 and O's scaling are fp32, whose results below 2^-126 may be 0
        same = (o[s, 0] == want) | (o[s, 0].isnan() & want.isnan()) | \
               ((o[s, 0].float().abs() <= 2.0 ** -126) & (want.float().abs() <= 2.0 ** -126))
        assert same.all(), (byte, s, o[s, 0][~same], want[~same])


@pytest.mark.parametrize("H", [2, 16])
def test_nothing_unseen_is_used(H):
    """Codes and scale bytes of NaN in nodes that no node sees; NaN in one that some see reaches those."""
    rng = np.random.default_rng(15)
    L, n, d = 150, 30, 128
    c = Cache(rng, [L], 1, d)
    see = np.tril(np.ones((n, n), bool))
    hidden = [3, 10, 29]
    see[:, hidden] = False
    for t in hidden:
        pos = L - n + t
        for x, b in ((c.k, c.ks), (c.v, c.vs)):
            x[int(c.bt[0, pos // 16]), :, pos % 16] = 0x7f
            b[int(c.bt[0, pos // 16]), :, pos % 16] = 0xff
    q = torch.randn((n, H, d), device="cuda").bfloat16()
    args = (T.i32([0, n]), n, T.i32(T.pack(see, 1)), 0.125)
    o, lse = fb.paged_tree_attention_e4m3(q, *c.args(), *args)
    full = np.concatenate([np.ones((n, L - n), bool), see], 1)
    T.check_attention(T.f64(o), T.f64(lse).T, T.attend(T.f64(q), *(x[:, 0] for x in c.rows[0]), 0.125, full))
    pos = L - n + 20
    c.k[int(c.bt[0, pos // 16]), 0, pos % 16, 5] = 0x7f
    o2, lse2 = fb.paged_tree_attention_e4m3(q, *c.args(), *args)
    assert o2[20:].isnan().all() and lse2[:, 20:].isnan().all() and not lse2[:, :20].isnan().any()
    assert fb.fa_get_device_status() == 0


def test_same_bits_every_time_and_in_a_graph():
    rng = np.random.default_rng(19)
    lens, new, H, Hkv, d = [3000, 130, 700], [20, 1, 64], 8, 2, 128
    c = Cache(rng, lens, Hkv, d)
    cu, total = T.i32(T.offsets(new)), sum(new)
    mask = T.i32(np.concatenate([T.pack(T.ancestors(T.random_parents(rng, n))[0], 2) for n in new]))
    q = [torch.randn((total, H, d), device="cuda").bfloat16() for _ in range(2)]
    args = c.args()
    want = [fb.paged_tree_attention_e4m3(x, *args, cu, 64, mask, 0.1) for x in q]
    static = q[0].clone()
    ws = torch.empty(fb.fa_paged_tree_workspace_size(3, 64, H, Hkv, d), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fb.paged_tree_attention_e4m3(static, *args, cu, 64, mask, 0.1, workspace=ws)
    for x, w in zip(q[::-1], want[::-1]):
        static.copy_(x)
        ws.random_(0, 256)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two = fb.paged_tree_attention_e4m3(q[1], *args, cu, 64, mask, 0.1, stream=side)
    one = fb.paged_tree_attention_e4m3(q[0], *args, cu, 64, mask, 0.1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one + two, want[0] + want[1]))


def test_bad_page_is_reported():
    rng = np.random.default_rng(18)
    c = Cache(rng, [300, 200], 2, 128)
    q = torch.randn((9, 4, 128), device="cuda").bfloat16()
    see = np.tril(np.ones((9, 9), bool))
    full = np.concatenate([np.ones((5, 195), bool), see[4:, :5]], 1)
    full[:, 195:] = np.tril(np.ones((5, 5), bool))
    mask = T.i32(np.concatenate([T.pack(see[:4], 1), T.pack(np.tril(np.ones((5, 5), bool)), 1)]))
    for bad in (-1, c.k.shape[0], 1 << 30):
        c.bt[0, 3] = bad
        o, lse = fb.paged_tree_attention_e4m3(q, *c.args(), T.i32([0, 4, 9]), 5, mask, 0.125)
        assert fb.fa_get_device_status() == fb.FA_ERR_BAD_BLOCK_TABLE
        for g in range(2):   # the other sequence is not touched by it
            h = slice(2 * g, 2 * g + 2)
            ref = T.attend(T.f64(q)[4:, h], c.rows[1][0][:, g], c.rows[1][1][:, g], 0.125, full)
            T.check_attention(T.f64(o)[4:, h], T.f64(lse).T[4:, h], ref)


def test_a_wait_that_runs_out_is_reported(monkeypatch):
    rng = np.random.default_rng(21)
    c = Cache(rng, [300], 1, 128)
    q = torch.randn((5, 2, 128), device="cuda").bfloat16()
    see = np.tril(np.ones((5, 5), bool))
    args = (T.i32([0, 5]), 5, T.i32(T.pack(see, 1)), 0.125)
    monkeypatch.setenv("FA_TEST_FORCE_WAIT_TIMEOUT", "1")
    fb.paged_tree_attention_e4m3(q, *c.args(), *args)
    assert fb.fa_get_device_status() == fb.FA_ERR_TIMEOUT
    monkeypatch.delenv("FA_TEST_FORCE_WAIT_TIMEOUT")
    o, lse = fb.paged_tree_attention_e4m3(q, *c.args(), *args)
    full = np.concatenate([np.ones((5, 295), bool), see], 1)
    T.check_attention(T.f64(o), T.f64(lse).T, T.attend(T.f64(q), *(x[:, 0] for x in c.rows[0]), 0.125, full))
    assert fb.fa_get_device_status() == 0


def test_pages_past_32_bits():
    """Codes past 2^31 bytes: the same pages at the pool's end and at its beginning give the same bits."""
    pool, Hkv, d, n = 140000, 8, 128, 9            # 2.3e9 bytes a cache
    k, v = (torch.empty((pool, Hkv, 16, d), dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.empty((pool, Hkv, 16), dtype=torch.uint8, device="cuda") for _ in "kv")
    near, far = [5, 1, 7], [139999, 137000, 139001]
    for x in (k, v):
        x[near] = torch.randn((3, Hkv, 16, d), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    for x in (ks, vs):
        x[near] = torch.randint(120, 130, (3, Hkv, 16), dtype=torch.uint8, device="cuda")
    for x in (k, v, ks, vs):
        x[far] = x[near]
    q = torch.randn((n, 16, d), device="cuda").bfloat16()
    mask = T.i32(T.pack(T.ancestors(T.random_parents(np.random.default_rng(2), n))[0], 1))
    out = [fb.paged_tree_attention_e4m3(q, k, v, ks, vs, T.i32([pages]), T.i32([45]), T.i32([0, n]), n, mask, 0.125)
           for pages in (near, far)]
    assert all(torch.equal(a, b) for a, b in zip(*out)) and not out[0][0].isnan().any()
    assert fb.fa_get_device_status() == 0


def test_helper_refuses():
    c = Cache(np.random.default_rng(1), [40], 1, 64)
    q = torch.randn((4, 2, 64), device="cuda").bfloat16()
    mask, cu = T.i32(np.full((4, 1), 15)), T.i32([0, 4])
    k, v, ks, vs, bt, sl = c.args()
    good = dict(q=q, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, block_table=bt, seq_lens=sl, cu_seqlens_q=cu,
                max_seqlen_q=4, mask=mask, scale=0.125)
    fb.paged_tree_attention_e4m3(**good)
    fb.paged_tree_attention_e4m3(**dict(good, k_cache=k.view(torch.float8_e4m3fn)))
    for bad in (dict(q=q.float()), dict(q=q.transpose(0, 1)), dict(k_cache=k.bfloat16()), dict(k_scale=ks[:1]),
                dict(mask=mask.long()), dict(mask=mask[:3]), dict(cu_seqlens_q=cu[:1]), dict(v_scale=vs.cpu()),
                dict(scale=0.0), dict(q=q[..., :32])):
        with pytest.raises(fb.FaError):
            fb.paged_tree_attention_e4m3(**dict(good, **bad))
    with pytest.raises(fb.FaError):
        fb.paged_tree_attention_e4m3(**good, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
