"""The e4m3 paged cache on the GPU: writing, reading back, decode and chunks.

Codes, scale bytes and read-back rows are compared bit for bit with a plain
float64 implementation; attention within the bounds that _e4m3.bounds derives.  Slots no query sees hold NaN codes.
"""
import numpy as np
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _e4m3 as E

pytestmark = pytest.mark.gpu
W_ROUND = 2.0 ** -11           # the rows kernels: weights rounded to f16
P_ROUND = 2.0 ** -7 * 1.01     # the forward: P rounded to bf16 (2^-8) in the value product and in O's divisor


def _rounding(max_q, group, d):
    """The weights' rounding in the kernels that the entry takes for max_q tokens of `group` heads."""
    rows = max_q * group
    if max_q == 1 or rows <= 16 or rows <= 32 and (d == 64 or group & (group - 1)):
        return W_ROUND
    return P_ROUND


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _rows(rng, L, Hkv, d, spread=0.7):
    x = rng.standard_normal((L, Hkv, d)) * np.exp2(spread * rng.standard_normal((L, Hkv, 1)))
    return E.bf16(x)[1]


def _cache(rng, lens, Hkv, d, spread=0.7, **kw):
    return E.Cache(rng, [_rows(rng, L, Hkv, d, 0.3) for L in lens],
                   [_rows(rng, L, Hkv, d, spread) for L in lens], **kw)


def _f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------- writing
def _specials(d):
    """bf16 rows at the edges of the format."""
    x = np.zeros((14, d))
    x[1] = np.ldexp(1.0, -130) * (1 + np.arange(d) % 3)       # subnormal: byte 0
    x[2, 0], x[2, 1] = 448.0, 0.5                             # exactly representable maximum
    x[3, 0], x[3, 1] = 450.0, -3.0                            # one bf16 step above it
    x[4, 0], x[4, 1] = 1.75 * 2.0 ** -20, 2.0 ** -30
    x[5, 0], x[5, 1] = 1.7578125 * 2.0 ** -20, 2.0 ** -30
    x[6] = 3e38                                               # near the largest
    x[7], x[7, 3] = 1.0, np.inf
    x[8], x[8, 5] = -2.5, np.nan
    x[9] = np.inf
    x[10] = np.where(np.arange(d) % 2, 17.0, -0.0)            # a tie, and minus zero
    x[11] = np.linspace(-500, 500, d)
    x[12] = np.ldexp(1.0, np.arange(d) % 40 - 30)             # down into e4m3's subnormals
    x[13] = 1.0625                                            # ties in every element
    return x


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8, 11])
def test_write_gives_the_defined_codes_and_leaves_other_slots(d, Hkv):
    rng = np.random.default_rng(d + Hkv)
    lens, new = [40, 0, 17, 16, 300, 1], [5, 0, 17, 1, 131, 1]
    total = sum(new)
    behind = 3                                  # rows no sequence owns
    x = {n: _rows(rng, total + behind, Hkv, d, 3.0) for n in "kv"}
    sp = _specials(d)
    x["k"][5:5 + len(sp), 0] = sp               # rows of the third sequence
    x["v"][5:5 + len(sp), Hkv - 1] = sp[:, ::-1]
    # K and V as parts of a wider projection output
    wide = torch.zeros((total + behind, 2, Hkv + 1, d), dtype=torch.bfloat16)
    wide[:, 0, :Hkv] = E.bf16(x["k"])[0]
    wide[:, 1, :Hkv] = E.bf16(x["v"])[0]
    k, v = wide.cuda()[:, 0, :Hkv], wide.cuda()[:, 1, :Hkv]
    x = {"k": _f64(k), "v": _f64(v)}
    c = _cache(rng, lens, Hkv, d)
    kc, vc, ks, vs, bt, sl = c.gpu()
    cu = np.concatenate([[0], np.cumsum(new)])
    fb.paged_kv_write_e4m3(k, v, kc, vc, ks, vs, bt, sl, _i32(cu))
    assert fb.fa_get_device_status() == 0
    for name, codes, scale in (("k", kc, ks), ("v", vc, vs)):
        want_c, want_b = c.codes[name].copy(), c.scales[name].copy()
        for s, (L, n) in enumerate(zip(lens, new)):
            pos = np.arange(L - n, L)
            qc, qb = E.quantise(x[name][cu[s]:cu[s + 1]])
            want_c[c.table[s, pos // 16], :, pos % 16] = qc
            want_b[c.table[s, pos // 16], :, pos % 16] = qb
        got_c = codes.view(torch.uint8).cpu().numpy()
        # a NaN code's sign says nothing
        got_c = np.where(got_c & 0x7f == 0x7f, 0x7f, got_c)
        want_c = np.where(want_c & 0x7f == 0x7f, 0x7f, want_c)
        assert np.array_equal(got_c, want_c), (name, np.argwhere(got_c != want_c)[:4])
        assert np.array_equal(scale.cpu().numpy(), want_b), name


def test_write_skips_what_it_cannot_place():
    rng = np.random.default_rng(1)
    lens, new = np.array([20, 33, 5, 64]), [4, 3, 9, 2]     # the third has more rows than tokens
    c = _cache(rng, lens, 2, 64, max_blocks=4)
    kc, vc, ks, vs, bt, sl = c.gpu()
    cu = np.concatenate([[0], np.cumsum(new)])
    x = torch.ones((18, 2, 64), dtype=torch.bfloat16, device="cuda")

    def written():
        return [s for s, L in enumerate(lens)
                if (ks[int(c.table[s, (L - 1) // 16]), :, (L - 1) % 16] == 127 - 8).all()]

    fb.paged_kv_write_e4m3(x, x, kc, vc, ks, vs, bt, sl, _i32(cu))
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    assert written() == [0, 1, 3]
    kc, vc, ks, vs, bt, sl = c.gpu()
    bt[0, 1] = c.num_pages                                   # past the pool
    sl[1] = 65                                               # past its row of the table
    fb.paged_kv_write_e4m3(x[:4], x[:4], kc, vc, ks, vs, bt[:1], sl[:1], _i32([0, 4]))
    assert fb.fa_get_device_status() == fb.FA_ERR_BAD_BLOCK_TABLE
    fb.paged_kv_write_e4m3(x, x, kc, vc, ks, vs, bt, sl, _i32([0, 0, 3, 3, 5]))
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    assert written() == [3]
    fb.paged_kv_write_e4m3(x[:2], x[:2], kc, vc, ks, vs, bt[3:], sl[3:], _i32([-1, 2]))
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    fb.paged_kv_write_e4m3(x[:2], x[:2], kc, vc, ks, vs, bt[3:], sl[3:], _i32([0, 7]))
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("num_seqs", [1, 33, 1100])
def test_write_finds_each_rows_sequence(num_seqs):
    """Every row lands in its own sequence, whatever their number and lengths."""
    rng = np.random.default_rng(num_seqs)
    new = rng.integers(0, 4, num_seqs)
    new[-1] = 2
    lens = new + rng.integers(0, 20, num_seqs)
    need = (lens + 15) // 16
    table = np.full((num_seqs, 2), -1, np.int32)
    at = 0
    for s in range(num_seqs):
        table[s, :need[s]] = np.arange(at, at + need[s])
        at += need[s]
    total = int(new.sum())
    x = torch.zeros((total, 1, 64), dtype=torch.bfloat16)
    x[:, 0, 0] = 448                                          # scale byte 127
    x[:, 0, 1] = torch.arange(total) % 16                     # exact in e4m3
    x[:, 0, 2] = torch.arange(total) // 16 % 16
    x[:, 0, 3] = torch.arange(total) // 256
    kc = torch.zeros((int(at), 1, 16, 64), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((int(at), 1, 16), dtype=torch.uint8, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    cu = np.concatenate([[0], np.cumsum(new)])
    fb.paged_kv_write_e4m3(x.cuda(), x.cuda(), kc, vc, ks, vs, _i32(table), _i32(lens), _i32(cu))
    assert fb.fa_get_device_status() == 0
    got = E.values(kc.cpu().numpy(), ks.cpu().numpy())
    seen = 0
    for s in range(num_seqs):
        pos = np.arange(lens[s] - new[s], lens[s])
        rows = got[table[s, pos // 16], 0, pos % 16]
        want = np.arange(cu[s], cu[s + 1])
        assert np.array_equal(rows[:, 1] + 16 * rows[:, 2] + 256 * rows[:, 3], want)
        seen += len(want)
    assert seen == total and (ks != 0).sum() == total
    assert torch.equal(kc, vc) and torch.equal(ks, vs)


# -------------------------------------------------------------- reading back
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 5, 8, 9])
def test_read_back_is_exact(d, Hkv):
    rng = np.random.default_rng(10 * d + Hkv)
    lens, new = [40, 3, 17, 0, 300], [40, 3, 2, 0, 133]
    c = _cache(rng, lens, Hkv, d, spread=4.0)
    cu = np.concatenate([[0], np.cumsum(new)])
    total = int(cu[-1])
    t = c.gpu()
    k = torch.full((total + 2, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    fb.fa_paged_kv_read_e4m3(*t, _i32(cu), k, v, len(lens), total + 2, Hkv, d, 16, c.num_pages,
                             c.table.shape[1])
    assert fb.fa_get_device_status() == 0
    for name, got in (("k", k), ("v", v)):
        for s, (L, n) in enumerate(zip(lens, new)):
            assert np.array_equal(_f64(got[cu[s]:cu[s + 1]]), c.rows[name][s][L - n:])
        assert (got[total:] == 7.0).all()      # rows behind the last sequence


def test_read_back_of_every_code_and_scale():
    """code * 2^(byte - 127) rounded to bf16, every code under a sweep of bytes."""
    codes = np.tile(np.arange(256, dtype=np.uint8), 16).reshape(1, 2, 16, 128)
    k = torch.from_numpy(codes).cuda()
    b = np.linspace(0, 254, 32).astype(np.uint8).reshape(1, 2, 16)
    ks = torch.from_numpy(b).cuda()
    out, _ = fb.paged_kv_read_e4m3(k, k, ks, ks, _i32([[0]]), _i32([16]), _i32([0, 16]), 16)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(E.values(codes, b)[0].transpose(1, 0, 2).astype(np.float32))
    assert torch.equal(out.cpu().view(torch.int16) & 0x7f80 == 0x7f80,
                       ~torch.isfinite(want.bfloat16()))
    fin = torch.isfinite(want.bfloat16())
    assert torch.equal(out.cpu()[fin], want.bfloat16()[fin])


# -------------------------------------------------------------------- decode
def _decode_check(c, q, window=0, sinks=0, what=""):
    """q bf16 CPU tensor [S,H,d]."""
    scale = E.softmax_scale(c.d)
    o, lse = fb.paged_decode_e4m3(q.cuda(), *c.gpu(), scale, window=window, sinks=sinks)
    o, lse, qd = _f64(o), _f64(lse), q.double().numpy()
    for s in range(len(c.lens)):
        ref = E.attend(qd[s:s + 1], c.rows["k"][s], c.rows["v"][s], scale, True, window, sinks,
                       c.vexp[s])
        E.check(o[s:s + 1], lse[s:s + 1], ref, c.d, W_ROUND, f"{what} sequence {s}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 8, 9, 16, 20, 32])
def test_decode_groups_and_lengths(d, group):
    rng = np.random.default_rng(100 + group)
    lens = [0, 1, 15, 16, 17, 33, 257, 640]
    c = _cache(rng, lens, 2, d, max_blocks=48)
    q = E.bf16(rng.standard_normal((len(lens), 2 * group, d)))[0]
    _decode_check(c, q)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 4), (100, 0), (100, 20),
                                          (128, 16), (130, 300), (639, 4), (640, 0), (5000, 7)])
def test_decode_window_and_sinks(window, sinks):
    rng = np.random.default_rng(window + sinks)
    lens = [0, 1, 16, 17, 100, 101, 129, 257, 640]
    c = _cache(rng, lens, 2, 128)
    q = E.bf16(rng.standard_normal((len(lens), 8, 128)))[0]
    _decode_check(c, q, window, sinks)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("num_seqs", [1, 2, 7, 40, 300])
def test_decode_batch_sizes(num_seqs):
    """Cluster sizes from 8 down to 1, ranked and unranked launches."""
    rng = np.random.default_rng(num_seqs)
    lens = rng.integers(1, 400, num_seqs)
    c = _cache(rng, lens, 4, 64)
    q = E.bf16(rng.standard_normal((num_seqs, 4, 64)))[0]
    _decode_check(c, q)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("d,group", [(128, 4), (64, 2), (128, 12), (64, 20)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (900, 5)])
def test_decode_shares_of_a_few_long_sequences(d, group, window, sinks):
    """A few long sequences cut into equal shares (with a workspace): a warp's piece starts and ends
    anywhere and may span several units, where the lengths are short; and the same without one."""
    rng = np.random.default_rng(d + group)
    lens, Hkv = [20, 3000, 0, 1, 17, 4096], 3
    c = _cache(rng, lens, Hkv, d, max_blocks=400)
    q = E.bf16(rng.standard_normal((len(lens), Hkv * group, d)))[0]
    scale, t = E.softmax_scale(d), c.gpu()
    _decode_check(c, q, window, sinks)
    S, H = q.shape[:2]
    o = torch.full((S, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((S, H), device="cuda")
    fb.fa_paged_decode_e4m3(q.cuda(), *t, o, lse, S, H, Hkv, d, 16, c.num_pages, 400, scale, window,
                            sinks)                       # no workspace: clusters
    qd = q.double().numpy()
    for s in range(S):
        ref = E.attend(qd[s:s + 1], c.rows["k"][s], c.rows["v"][s], scale, True, window, sinks, c.vexp[s])
        E.check(_f64(o[s:s + 1]), _f64(lse[s:s + 1]), ref, d, W_ROUND)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("num_seqs,lo,hi,window", [(20, 300, 3000, 0), (80, 40, 600, 0), (80, 700, 800, 300)])
def test_decode_batches_of_many_units(num_seqs, lo, hi, window):
    """Units by the hundred: clusters of several sizes, longest first."""
    rng = np.random.default_rng(num_seqs + lo)
    lens = rng.integers(lo, hi, num_seqs)
    c = _cache(rng, lens, 8, 128, max_blocks=200)
    q = E.bf16(rng.standard_normal((num_seqs, 16, 128)))[0]
    _decode_check(c, q, window, 4)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("num_seqs", [77, 255, 256, 257])
@pytest.mark.parametrize("equal", [True, False])
def test_decode_order_by_length(num_seqs, equal):
    """Sequences counted into classes of length: all in one class, empty ones among them, a part of
    the last 32, as many as are ordered and one more."""
    rng = np.random.default_rng(num_seqs)
    lens = [20] * num_seqs if equal else [int(x) for x in rng.integers(0, 70, num_seqs)]
    c = _cache(rng, lens, 8, 64)
    q = E.bf16(rng.standard_normal((num_seqs, 8, 64)))[0]
    _decode_check(c, q)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 3)])
def test_one_long_sequence_is_shared_by_every_warp(window, sinks):
    rng = np.random.default_rng(50)
    c = _cache(rng, [20001], 1, 128, max_blocks=10000)
    q = E.bf16(rng.standard_normal((1, 4, 128)))[0]
    _decode_check(c, q, window, sinks)
    q = E.bf16(rng.standard_normal((5, 4, 128)))[0]
    _chunk_check(c, q, [5], True, window, sinks)
    assert fb.fa_get_device_status() == 0


def test_shares_of_short_chunks_skip_bad_sequences():
    """As the cluster form: bad sequences set the status and leave their rows alone."""
    rng = np.random.default_rng(51)
    new = np.array([3, 0, 4, 1, 2, 4])
    lens = rng.integers(900, 2500, 6)
    c = _cache(rng, lens, 2, 128, max_blocks=160)
    q = E.bf16(rng.standard_normal((int(new.sum()), 8, 128)))[0]
    _chunk_check(c, q, list(new), True, 400, 4)
    cu = np.concatenate([[0], np.cumsum(new)])
    t = c.gpu()
    t[5][2], t[5][4] = 160 * 16 + 1, -5
    t[4][0, 3] = c.num_pages
    ws = torch.empty(fb.fa_paged_e4m3_workspace_size(6, 4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o = torch.full((int(cu[-1]), 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, int(cu[-1])), 9.0, device="cuda")
    for i in range(2):
        fb.fa_paged_prefill_e4m3(q.cuda(), *t, _i32(cu), o, lse, 6, int(cu[-1]), 4, 8, 2, 128, 16,
                                 c.num_pages, 160, 0.1, workspace=ws, workspace_bytes=ws.numel())
        assert fb.fa_get_device_status() in (fb.FA_ERR_INVALID_ARG, fb.FA_ERR_BAD_BLOCK_TABLE)
        for s in range(6):
            r = slice(cu[s], cu[s + 1])
            if s in (2, 4):
                assert (o[r] == 9.0).all() and (lse[:, r] == 9.0).all()
            elif s != 0:
                ref = E.attend(q[r].double().numpy(), c.rows["k"][s], c.rows["v"][s],
                               float(np.float32(0.1)), True, 0, 0, c.vexp[s])
                E.check(_f64(o[r]), _f64(lse[:, r]).T, ref, 128, W_ROUND, f"sequence {s}")


def test_timeout_in_a_share_is_recorded(monkeypatch):
    rng = np.random.default_rng(52)
    c = _cache(rng, [900] * 4, 8, 64, max_blocks=200)
    q = E.bf16(rng.standard_normal((4, 8, 64)))[0]
    monkeypatch.setenv("FA_TEST_FORCE_WAIT_TIMEOUT", "1")
    fb.paged_decode_e4m3(q.cuda(), *c.gpu(), 0.1)
    assert fb.fa_get_device_status() == fb.FA_ERR_TIMEOUT
    monkeypatch.delenv("FA_TEST_FORCE_WAIT_TIMEOUT")
    _decode_check(c, q)
    assert fb.fa_get_device_status() == 0


def test_hidden_keys_are_never_used():
    """NaN codes and infinite scales outside the window and the sinks, and freed pages (table
    entries -1 or past the pool) there, change nothing and set no status."""
    rng = np.random.default_rng(5)
    lens, window, sinks = [300, 77, 40], 37, 5
    c = _cache(rng, lens, 2, 128)
    for s, L in enumerate(lens):
        pos = np.arange(sinks, max(sinks, L - window))
        for x in "kv":
            c.codes[x][c.table[s, pos // 16], :, pos % 16] = 0x7f
            c.scales[x][c.table[s, pos // 16], :, pos % 16] = 255
    c.table[0, 1:(300 - 37) // 16] = -1
    c.table[1, 1:2] = 1 << 30
    q = E.bf16(rng.standard_normal((3, 8, 128)))[0]
    _decode_check(c, q, window, sinks)
    assert fb.fa_get_device_status() == 0


def test_scales_far_apart():
    """Rows whose powers of two differ by up to 2^40, zero rows, hot scores: the V scales ride on
    the weights, so a long tail of small rows beside a large one keeps its share."""
    rng = np.random.default_rng(6)
    L, Hkv, d = 500, 2, 128
    k = rng.standard_normal((L, Hkv, d)) * np.exp2(rng.integers(-12, 2, (L, Hkv, 1)))
    v = rng.standard_normal((L, Hkv, d)) * np.exp2(rng.integers(-20, 21, (L, Hkv, 1)))
    k[7], v[9], v[100:150] = 0.0, 0.0, 0.0
    c = E.Cache(rng, [k, k[:260], k], [v, np.zeros((260, Hkv, d)), v * 2.0 ** -90])
    q = rng.standard_normal((3, 8, d))
    q[0, 1] *= 20.0
    q[0, 2] *= 2.0 ** -30
    q[1, 3] = 0.0
    _decode_check(c, E.bf16(q)[0])


def test_large_v_row_with_no_weight():
    """A V row 2^30 larger than the rest whose weight is 2^-100: the rest decides O."""
    rng = np.random.default_rng(7)
    L, d = 200, 128
    q = np.zeros((1, 1, d))
    q[0, 0, 0] = 64.0
    k = rng.standard_normal((L, 1, d)) * 0.1
    k[:, 0, 0] = 8.0
    v = rng.standard_normal((L, 1, d))
    for at in (0, 90, 199):
        k[at, 0, 0], v[at] = -6.0, 2.0 ** 30 * rng.standard_normal(d)
    _decode_check(E.Cache(rng, [k], [v]), E.bf16(q)[0])


def test_bad_page_ids_and_lengths_set_the_status():
    rng = np.random.default_rng(8)
    c = _cache(rng, [100, 50, 70], 2, 128)
    q = E.bf16(rng.standard_normal((3, 4, 128)))[0]
    t = c.gpu()
    t[4][0, 2] = c.num_pages
    scale = E.softmax_scale(128)
    o, lse = fb.paged_decode_e4m3(q.cuda(), *t, scale)
    assert fb.fa_get_device_status() == fb.FA_ERR_BAD_BLOCK_TABLE
    # that page's keys are left out, the other sequences are untouched
    keep = np.r_[0:32, 48:100]
    ref = E.attend(q[:1].double().numpy(), c.rows["k"][0][keep], c.rows["v"][0][keep], scale, True,
                   0, 0, c.vexp[0][keep])
    E.check(_f64(o[:1]), _f64(lse[:1]), ref, 128, W_ROUND)
    ref = E.attend(q[1:2].double().numpy(), c.rows["k"][1], c.rows["v"][1], scale, True, 0, 0,
                   c.vexp[1])
    E.check(_f64(o[1:2]), _f64(lse[1:2]), ref, 128, W_ROUND)
    t = c.gpu()
    t[5][1] = 16 * c.table.shape[1] + 1
    t[5][2] = -1
    o, lse = fb.paged_decode_e4m3(q.cuda(), *t, scale)
    assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG
    assert (o[1:] == 0).all() and torch.isneginf(lse[1:]).all() and torch.isfinite(lse[0]).all()


def test_decode_timeout_is_recorded_and_the_next_call_runs(monkeypatch):
    """The test hook keeps each warp's first page from being requested: its bounded wait runs out,
    FA_ERR_TIMEOUT is recorded, and the next call is a normal one."""
    rng = np.random.default_rng(9)
    c = _cache(rng, [100, 900], 2, 128)
    q = E.bf16(rng.standard_normal((2, 8, 128)))[0]
    monkeypatch.setenv("FA_TEST_FORCE_WAIT_TIMEOUT", "1")
    fb.paged_decode_e4m3(q.cuda(), *c.gpu(), 0.1)
    assert fb.fa_get_device_status() == fb.FA_ERR_TIMEOUT
    monkeypatch.delenv("FA_TEST_FORCE_WAIT_TIMEOUT")
    _decode_check(c, q)
    assert fb.fa_get_device_status() == 0


# --------------------------------------------------------------------- chunks
def _chunk_check(c, q, new, causal=True, window=0, sinks=0, rounding=None, what=""):
    """With a workspace (the keys of few units are split) and without one."""
    scale = E.softmax_scale(c.d)
    cu = np.concatenate([[0], np.cumsum(new)])
    S, (Tq, H, d), mq, t = len(c.lens), q.shape, int(max(new)), c.gpu()
    rounding = rounding or _rounding(mq, H // c.Hkv, d)
    refs = []
    qd = q.double().numpy()
    for s in range(S):
        refs.append(E.attend(qd[cu[s]:cu[s + 1]], c.rows["k"][s], c.rows["v"][s], scale, causal, window,
                             sinks, c.vexp[s]))
    need = fb.fa_paged_e4m3_workspace_size(S, mq, H, c.Hkv, d)
    for ws in [None] + ([torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")] if need else []):
        o = torch.full((Tq, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((H, Tq), 9.0, device="cuda")
        fb.fa_paged_prefill_e4m3(q.cuda(), *t, _i32(cu), o, lse, S, Tq, mq, H, c.Hkv, d, 16, c.num_pages,
                                 c.table.shape[1], scale, causal, window, sinks, ws,
                                 0 if ws is None else need)
        o, lse = _f64(o), _f64(lse).T
        for s in range(S):
            r = slice(cu[s], cu[s + 1])
            E.check(o[r], lse[r], refs[s], c.d, rounding, f"{what} sequence {s} workspace {need if ws is not None else 0}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 4, 16])
@pytest.mark.parametrize("causal", [True, False])
def test_short_chunks(d, group, causal):
    rng = np.random.default_rng(group + d)
    lens, new = [1, 16, 17, 130, 0, 300, 5], [1, 4, 3, 8, 2, 0, 8]   # the last: more queries than keys
    c = _cache(rng, lens, 2, d)
    q = E.bf16(rng.standard_normal((sum(new), 2 * group, d)))[0]
    _chunk_check(c, q, new, causal, rounding=_rounding(8, group, d))
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (16, 4), (33, 0), (60, 40), (400, 3)])
def test_short_chunks_window(window, sinks):
    rng = np.random.default_rng(window)
    lens, new = [9, 40, 17, 130, 300], [5, 4, 8, 8, 7]
    c = _cache(rng, lens, 2, 128)
    q = E.bf16(rng.standard_normal((sum(new), 6, 128)))[0]
    _chunk_check(c, q, new, True, window, sinks)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 4, 16, 32])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(d, group, causal):
    rng = np.random.default_rng(3 * group + d)
    # partial pages and tiles, more queries than keys, no keys, no queries, single tokens
    lens, new = [1, 128, 129, 700, 0, 300, 60, 259], [1, 64, 129, 40, 2, 0, 90, 1]
    c = _cache(rng, lens, 2, d)
    q = E.bf16(rng.standard_normal((sum(new), 2 * group, d)))[0]
    _chunk_check(c, q, new, causal, rounding=P_ROUND)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("group", [1, 4, 6])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 4), (128, 0), (129, 128), (200, 129),
                                          (300, 400), (511, 1), (4000, 9)])
def test_chunks_window(window, sinks, group):
    rng = np.random.default_rng(window + group)
    lens, new = [900, 257, 40, 130, 1200], [300, 257, 70, 1, 129]
    c = _cache(rng, lens, 2, 128)
    q = E.bf16(rng.standard_normal((sum(new), 2 * group, 128)))[0]
    _chunk_check(c, q, new, True, window, sinks, P_ROUND)
    assert fb.fa_get_device_status() == 0


def test_chunk_equals_the_bf16_prefill_of_the_read_back_cache():
    """Widening a tile is exact, so with one query head per kv head (no packing) the LSE's bits are
    those of fa_paged_prefill on the rows read back into a bf16 cache, and at d = 64 O's too.  At
    d = 128 O's divisor is the exact sum here, the rounded weights' there: 2^-9 apart, before each
    is rounded to bf16 (half a step, 2^-8)."""
    rng = np.random.default_rng(30)
    lens, new = [300, 77, 513, 20], [200, 77, 60, 33]
    for d in (64, 128):
        c = _cache(rng, lens, 4, d, spread=2.0)
        q = E.bf16(rng.standard_normal((sum(new), 4, d)))[0].cuda()
        t, cu = c.gpu(), _i32(np.concatenate([[0], np.cumsum(new)]))
        kc, vc = (torch.from_numpy(E.values(c.codes[x], np.where(c.scales[x] == 255, 0, c.scales[x]))
                                   .astype(np.float32)).bfloat16().cuda() for x in "kv")
        o1, l1 = torch.empty_like(q), torch.empty((4, sum(new)), device="cuda")
        fb.fa_paged_prefill_e4m3(q, *t, cu, o1, l1, 4, sum(new), max(new), 4, 4, d, 16, c.num_pages,
                                 c.table.shape[1], 0.1)
        o2, l2 = fb.paged_prefill(q, kc, vc, t[4], t[5], cu, max(new), 0.1)
        assert torch.equal(l1.view(torch.int32), l2.view(torch.int32))
        if d == 64:
            assert torch.equal(o1.view(torch.int16), o2.view(torch.int16))
        else:
            o1, o2 = _f64(o1), _f64(o2)
            assert (np.abs(o1 - o2) <= (2.0 ** -9 + 2 * 2.0 ** -8) * 1.01 * np.abs(o2)).all()
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("d,group,new", [(128, 4, [40]), (64, 2, [64]), (128, 1, [90]), (128, 8, [5, 9]),
                                         (64, 6, [33, 0, 20])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
def test_chunks_split_over_long_contexts(d, group, new, window, sinks):
    """A chunk of few units whose K/V tiles are cut into parts, merged by a second launch: parts with
    no tile, parts whose only tile one query tile skips, sequences shorter than the parts are many."""
    rng = np.random.default_rng(d + group)
    lens = [5000, 100, 2300][:len(new)]
    c = _cache(rng, lens, 2, d, max_blocks=320)
    q = E.bf16(rng.standard_normal((sum(new), 2 * group, d)))[0]
    assert fb.fa_paged_e4m3_workspace_size(len(new), max(new), 2 * group, 2, d) > 0
    _chunk_check(c, q, new, True, window, sinks, P_ROUND)
    if not window:
        _chunk_check(c, q, new, False, 0, 0, P_ROUND)
    assert fb.fa_get_device_status() == 0


def test_chunk_hidden_keys_are_never_used():
    rng = np.random.default_rng(31)
    lens, new, window, sinks = [700, 400, 300], [100, 60, 300], 150, 5
    c = _cache(rng, lens, 2, 128)
    for s, (L, n) in enumerate(zip(lens, new)):
        pos = np.arange(sinks, max(sinks, L - n - window + 1))    # before the first query's window
        for x in "kv":
            c.codes[x][c.table[s, pos // 16], :, pos % 16] = 0x7f
            c.scales[x][c.table[s, pos // 16], :, pos % 16] = 255
    c.table[0, 1:(700 - 100 - 150) // 16] = -1
    c.table[1, 1:3] = 1 << 30
    q = E.bf16(rng.standard_normal((sum(new), 8, 128)))[0]
    _chunk_check(c, q, new, True, window, sinks, P_ROUND)
    assert fb.fa_get_device_status() == 0


def test_chunks_of_many_sequences():
    """More (sequence, query pair) combinations than the sorted list holds: one CTA per unit."""
    rng = np.random.default_rng(32)
    new = rng.integers(0, 50, 300)
    lens = new + rng.integers(0, 60, 300)
    c = _cache(rng, lens, 1, 64)
    q = E.bf16(rng.standard_normal((int(new.sum()), 4, 64)))[0]
    _chunk_check(c, q, list(new), True, 70, 3, P_ROUND)
    assert fb.fa_get_device_status() == 0


def test_chunk_scales_far_apart():
    """Power-of-two scales from 2^-60 to 2^40: inside and outside the widening's f16 range."""
    rng = np.random.default_rng(33)
    L, n, d = 400, 120, 128
    k = rng.standard_normal((L, 1, d)) * np.exp2(rng.integers(-12, 2, (L, 1, 1)))
    v = rng.standard_normal((L, 1, d)) * np.exp2(rng.integers(-40, 41, (L, 1, 1)))
    v[20:40], k[30] = 0.0, 0.0
    c = E.Cache(rng, [k, k * 2.0 ** -40], [v, v * 2.0 ** -20])
    q = rng.standard_normal((2 * n, 2, d))
    q[n:] *= 2.0 ** 40
    _chunk_check(c, E.bf16(q)[0], [n, n], True, 0, 0, P_ROUND)


def test_chunk_status():
    """Bad page ids, lengths, offsets and counts set the status; the other sequences' rows are
    right and a skipped sequence's rows are left alone."""
    rng = np.random.default_rng(34)
    lens, new = [100, 200, 150], [40, 50, 60]
    c = _cache(rng, lens, 2, 128, max_blocks=13)
    q = E.bf16(rng.standard_normal((150, 8, 128)))[0]
    cu, scale = [0, 40, 90, 150], E.softmax_scale(128)

    def run(t, cu, mq=60):
        o = torch.full((150, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((8, 150), 9.0, device="cuda")
        fb.fa_paged_prefill_e4m3(q.cuda(), *t, _i32(cu), o, lse, 3, 150, mq, 8, 2, 128, 16,
                                 c.num_pages, 13, scale)
        st = fb.fa_get_device_status()
        good = []
        for s in range(3):
            r = slice(cu[s], cu[s + 1])
            ref = E.attend(q[r].double().numpy(), c.rows["k"][s], c.rows["v"][s], scale)
            try:
                E.check(_f64(o[r]), _f64(lse[:, r]).T, ref, 128, P_ROUND)
                good.append(s)
            except AssertionError:
                pass
        return st, good, [s for s in range(3) if (o[cu[s]:cu[s + 1]] == 9.0).all()]

    t = c.gpu()
    assert run(t, cu) == (0, [0, 1, 2], [])
    t[4][1, 3] = c.num_pages
    st, good, left = run(t, cu)     # (that sequence's rows are unspecified)
    assert st == fb.FA_ERR_BAD_BLOCK_TABLE and {0, 2} <= set(good)
    for bad_len in (-1, 13 * 16 + 1):
        t = c.gpu()
        t[5][2] = bad_len
        assert run(t, cu) == (fb.FA_ERR_INVALID_ARG, [0, 1], [2])
    assert run(c.gpu(), cu, mq=55) == (fb.FA_ERR_INVALID_ARG, [0, 1], [2])
    assert run(c.gpu(), [0, 40, 90, 151])[0] == fb.FA_ERR_INVALID_ARG


def test_chunk_of_one_token_is_the_decode():
    rng = np.random.default_rng(12)
    lens = [5, 100, 333]
    c = _cache(rng, lens, 2, 128)
    q = E.bf16(rng.standard_normal((3, 8, 128)))[0].cuda()
    t = c.gpu()
    for w, sk in ((0, 0), (50, 3)):
        o1, l1 = fb.paged_decode_e4m3(q, *t, 0.1, window=w, sinks=sk)
        o2, l2 = fb.paged_prefill_e4m3(q, *t, _i32([0, 1, 2, 3]), 1, 0.1, window=w, sinks=sk)
        assert torch.equal(o1, o2) and torch.equal(l1, l2.T)


# ---------------------------------------------------------- the loop together
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_serving_loop(window, sinks):
    """Prompts in two chunks, then single tokens: each step writes its rows to the cache and
    attends from them; every step's output is held to the rows quantised so far."""
    rng = np.random.default_rng(20)
    S, H, Hkv, d = 3, 8, 2, 128
    steps = [[37, 5, 64], [20, 0, 33], [2, 1, 2]] + [[1, 1, 1]] * 4
    full = np.array(steps).sum(0)
    blocks = int((full.max() + 15) // 16)
    table = rng.permutation(S * blocks).reshape(S, blocks).astype(np.int32)
    kc, vc = (torch.zeros((S * blocks, Hkv, 16, d), device="cuda").to(torch.float8_e4m3fn) for _ in "kv")
    ks, vs = (torch.zeros((S * blocks, Hkv, 16), dtype=torch.uint8, device="cuda") for _ in "kv")
    rows = {"k": [np.zeros((0, Hkv, d))] * S, "v": [np.zeros((0, Hkv, d))] * S}
    vexp = [np.zeros((0, Hkv))] * S
    scale = E.softmax_scale(d)
    lens = np.zeros(S, np.int32)
    for new in steps:
        n = sum(new)
        qkv = E.bf16(rng.standard_normal((n, H + 2 * Hkv, d)))[0].cuda()
        q, k, v = qkv[:, :H].contiguous(), qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        lens = lens + np.array(new, np.int32)
        cu = np.concatenate([[0], np.cumsum(new)])
        cache = (kc, vc, ks, vs, _i32(table), _i32(lens))
        fb.paged_kv_write_e4m3(k, v, *cache, _i32(cu))
        if max(new) == 1:
            o, lse = fb.paged_decode_e4m3(q, *cache, scale, window=window, sinks=sinks)
            lse = lse.T
        else:
            o, lse = fb.paged_prefill_e4m3(q, *cache, _i32(cu), max(new), scale, window=window,
                                           sinks=sinks)
        o, lse, qd = _f64(o), _f64(lse).T, _f64(q)
        for s in range(S):
            r = slice(cu[s], cu[s + 1])
            for name, x in (("k", k), ("v", v)):
                code, b = E.quantise(_f64(x[r]))
                rows[name][s] = np.concatenate([rows[name][s], E.values(code, b)])
                if name == "v":
                    vexp[s] = np.concatenate([vexp[s], b.astype(float) - 127])
            ref = E.attend(qd[r], rows["k"][s], rows["v"][s], scale, True, window, sinks, vexp[s])
            E.check(o[r], lse[r], ref, d, P_ROUND, f"step {new} sequence {s}")
        back, _ = fb.paged_kv_read_e4m3(*cache, _i32(np.concatenate([[0], np.cumsum(lens)])),
                                        int(lens.sum()))
        assert np.array_equal(_f64(back), np.concatenate(rows["k"]))
    assert fb.fa_get_device_status() == 0


def test_captured_step_replays_and_streams_do_not_mix():
    """write + decode captured into two graphs and replayed in turn on two streams: no workspace
    is shared, so the bits are those of calls made one after the other."""
    rng = np.random.default_rng(21)
    c = _cache(rng, [100, 900, 30], 2, 128)
    graphs, outs, want = [], [], []
    fb.paged_decode_e4m3(E.bf16(rng.standard_normal((3, 8, 128)))[0].cuda(), *c.gpu(), 0.1)
    for i in range(2):
        t = c.gpu()
        q = E.bf16(rng.standard_normal((3, 8, 128)))[0].cuda()
        k = E.bf16(rng.standard_normal((3, 2, 128)))[0].cuda()
        cu = _i32([0, 1, 2, 3])
        fb.paged_kv_write_e4m3(k, k, *t, cu)
        want.append(fb.paged_decode_e4m3(q, *t, 0.1, window=64, sinks=4))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            fb.paged_kv_write_e4m3(k, k, *t, cu)
            o, lse = fb.paged_decode_e4m3(q, *t, 0.1, window=64, sinks=4)
        graphs.append((g, side, t, q, k, cu))
        outs.append((o, lse))
    for _ in range(20):
        for g, side, *_ in graphs:
            with torch.cuda.stream(side):
                g.replay()
    torch.cuda.synchronize()
    for (o, lse), (ow, lw) in zip(outs, want):
        assert torch.equal(o, ow) and torch.equal(lse, lw)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("Hkv", [1, 2, 3, 4, 5, 8, 12])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("offset", [0, 8])
def test_heads_and_alignments_of_the_rows(Hkv, d, offset):
    """Every split of the heads over warps, inputs and outputs 16 and 32 bytes aligned, rows in
    front of the first and behind the last sequence left alone."""
    rng = np.random.default_rng(Hkv + d + offset)
    c = _cache(rng, [40, 7], Hkv, d)
    kc, vc, ks, vs, bt, sl = c.gpu()
    new = [33, 7]
    T = sum(new) + 3
    src = [torch.zeros(T * Hkv * d + offset, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = (x[offset:].view(T, Hkv, d) for x in src)
    for x in (k, v):
        x.copy_(E.bf16(rng.standard_normal((T, Hkv, d)))[0])
    k[5, 0, 3], v[9, Hkv - 1, 1] = float("inf"), float("nan")
    cu = _i32([1, 34, 41])
    fb.paged_kv_write_e4m3(k, v, kc, vc, ks, vs, bt, sl, cu)
    out = [torch.full((T * Hkv * d + offset,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ko, vo = (x[offset:].view(T, Hkv, d) for x in out)
    fb.fa_paged_kv_read_e4m3(kc, vc, ks, vs, bt, sl, cu, ko, vo, 2, T, Hkv, d, 16, c.num_pages,
                             c.table.shape[1])
    assert fb.fa_get_device_status() == 0
    for x, y, buf in ((k, ko, out[0]), (v, vo, out[1])):
        assert (buf[:offset] == 7.0).all() and (y[0] == 7.0).all() and (y[41:] == 7.0).all()
        a, b = x[1:41].double(), y[1:41].double()
        bad = ~torch.isfinite(a)
        assert torch.equal(torch.isnan(b), bad)
        # half a step of 4 significant bits, or of the row's smallest code (2^-9 of the scale, whose
        # 448-fold is below twice the row's largest)
        top = torch.where(bad, 0.0, a).abs().amax(-1, keepdim=True)
        err = torch.where(bad, 0.0, a - b).abs()
        assert (err <= torch.maximum(a.abs().nan_to_num(posinf=0) * 2.0 ** -4, top / 224 * 2.0 ** -10)).all()


def test_split_calls_captured_and_replayed():
    """The two-launch forms (equal shares, cut chunks) in one graph, replayed beside eager calls on
    another stream with a workspace of their own."""
    rng = np.random.default_rng(23)
    c = _cache(rng, [3000, 2500], 2, 128)
    t = c.gpu()
    q1 = E.bf16(rng.standard_normal((2, 8, 128)))[0].cuda()
    q2 = E.bf16(rng.standard_normal((60, 8, 128)))[0].cuda()
    cu = _i32([0, 20, 60])

    def step():
        return fb.paged_decode_e4m3(q1, *t, 0.1) + fb.paged_prefill_e4m3(q2, *t, cu, 40, 0.1, window=900)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step()
    for _ in range(10):
        with torch.cuda.stream(side):
            g.replay()
        eager = step()
    torch.cuda.synchronize()
    for a, b, e in zip(want, got, eager):
        assert torch.equal(a, b) and torch.equal(a, e)
    assert fb.fa_get_device_status() == 0


@pytest.mark.parametrize("bound", [8, 40, 512, 8192, 2 ** 31 - 1])
def test_workspace_of_a_larger_bound_on_the_chunk(bound):
    """max_seqlen_q may be any upper bound (a captured step's), with the workspace sized for it,
    although the form that the rows at hand take may want a larger one."""
    rng = np.random.default_rng(25)
    c = _cache(rng, [2500], 1, 128)
    q = E.bf16(rng.standard_normal((8, 8, 128)))[0].cuda()
    cu = _i32([0, 8])
    ref = E.attend(_f64(q), c.rows["k"][0], c.rows["v"][0], 0.1, True, 0, 0, c.vexp[0])
    need = fb.fa_paged_e4m3_workspace_size(1, bound, 8, 1, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    for w in (ws, None):
        o, lse = fb.paged_prefill_e4m3(q, *c.gpu(), cu, bound, 0.1, workspace=w)
        E.check(_f64(o), _f64(lse).T, ref, 128, P_ROUND)
    assert fb.fa_get_device_status() == 0


def test_widest_windows_and_wild_offsets():
    """Windows and sinks up to 2^31 - 1 mean what they say, with more queries than keys too; offsets
    whose sums pass 32 bits are refused on the device and nothing is written."""
    rng = np.random.default_rng(24)
    big = 2 ** 31 - 1
    c = _cache(rng, [100, 300], 2, 128, max_blocks=64)
    for group in (1, 8):
        q = E.bf16(rng.standard_normal((170, 2 * group, 128)))[0]
        for w, s in ((big, 0), (big, big), (1023, big), (50, big)):
            _chunk_check(c, q, [120, 50], True, w, s, P_ROUND)
    q = E.bf16(rng.standard_normal((2, 8, 128)))[0]
    _decode_check(c, q, big, big)
    _decode_check(c, q, 40, big)
    for n in (8, 90):           # short chunks and long ones
        q = E.bf16(rng.standard_normal((2 * n, 8, 128)))[0].cuda()
        for cu in ([0, big - 4, big], [0, -5, n], [big, 2, n], [-big, big, n], [big - 3, -big, n]):
            o = torch.full((2 * n, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
            fb.fa_paged_prefill_e4m3(q, *c.gpu(), _i32(cu), o, None, 2, 2 * n, n, 8, 2, 128, 16,
                                     c.num_pages, 64, 0.1)
            assert fb.fa_get_device_status() == fb.FA_ERR_INVALID_ARG, cu
            assert (o[n:] == 9.0).all(), cu


def test_offsets_past_32_bits():
    """Pages whose byte offset passes 2^32 are written, read back and attended."""
    pages, Hkv, d = 270000, 8, 128                 # 4.4 GB a cache
    kc, vc = (torch.empty((pages, Hkv, 16, d), dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros((pages, Hkv, 16), dtype=torch.uint8, device="cuda") for _ in "kv")
    rng = np.random.default_rng(22)
    L, new = 40, 40
    table = _i32([[pages - 1, 131075, pages - 9]])
    k = E.bf16(rng.standard_normal((new, Hkv, d)))[0]
    v = E.bf16(rng.standard_normal((new, Hkv, d)))[0]
    cache = (kc, vc, ks, vs, table, _i32([L]))
    fb.paged_kv_write_e4m3(k.cuda(), v.cuda(), *cache, _i32([0, new]))
    rows = [E.values(*E.quantise(x.double().numpy())) for x in (k, v)]
    got = fb.paged_kv_read_e4m3(*cache, _i32([0, L]), L)
    assert np.array_equal(_f64(got[0]), rows[0]) and np.array_equal(_f64(got[1]), rows[1])
    q = E.bf16(rng.standard_normal((1, 16, d)))[0]
    o, lse = fb.paged_decode_e4m3(q.cuda(), *cache, 0.1)
    ref = E.attend(q.double().numpy(), *rows, float(np.float32(0.1)), True, 0, 0,
                   E.quantise(v.double().numpy())[1].astype(float) - 127)
    E.check(_f64(o), _f64(lse), ref, d, W_ROUND)
    assert fb.fa_get_device_status() == 0


def test_binding_refuses_tensors_the_c_entry_cannot_tell_apart():
    rng = np.random.default_rng(40)
    c = _cache(rng, [20, 30], 2, 64)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    good = c.gpu()

    def refused(i=None, t=None, q=q):
        a = list(good)
        if i is not None:
            a[i] = t
        with pytest.raises(fb.FaError) as e:
            fb.paged_decode_e4m3(q, *a, 0.1)
        return e.value.status == fb.FA_ERR_INVALID_ARG

    fb.paged_decode_e4m3(q, *good, 0.1)
    assert refused(0, good[0].cpu())
    assert refused(0, good[0].view(torch.uint8).to(torch.int16))
    assert refused(1, good[1][:-1])
    assert refused(2, good[2].view(torch.uint8).bool())
    assert refused(3, good[3].transpose(1, 2))
    assert refused(0, good[0].view(torch.float8_e5m2))
    assert refused(4, good[4].long())
    assert refused(4, good[4][:, ::2]) if good[4].shape[1] > 1 else True
    assert refused(5, good[5][:1])
    assert refused(q=q.float())
    assert refused(q=q.transpose(1, 2))
    assert refused(q=q.cpu())
    for ws in (torch.empty(64, dtype=torch.uint8, device="cuda"), torch.empty(1 << 24, dtype=torch.uint8),
               torch.empty((1 << 24, 2), dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(fb.FaError) as e:
            fb.paged_decode_e4m3(q, *good, 0.1, workspace=ws)
        assert e.value.status == fb.FA_ERR_WORKSPACE
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (k.float(), k[:1], k.cpu(), k.transpose(0, 1).contiguous().transpose(0, 1),
                torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")[:, :, ::2]):
        with pytest.raises(fb.FaError):
            fb.paged_kv_write_e4m3(k, bad, *good, _i32([0, 1, 2]))
