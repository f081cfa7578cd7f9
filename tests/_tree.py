"""Plain 64-bit forms of the operators on drafted token trees, and the bounds that the kernels'
outputs are held to."""
import numpy as np
import torch

PAGE = 16
BF16 = 2.0 ** -8      # half a step, relative
STREAMS = "kv"


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def table(rng, lens, pool, width=None):
    """Block table of distinct pages; entries that no token needs are out of range."""
    need = [(n + PAGE - 1) // PAGE for n in lens]
    width = width or max(need + [1])
    ids = rng.permutation(pool)[:sum(need)]
    bt = np.full((len(lens), width), -7, np.int32)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = ids[at:at + n]
        at += n
    return bt


def random_parents(rng, n):
    return np.array([rng.integers(-1, t) for t in range(n)], np.int32).reshape(n)


def ancestors(parents):
    """[n, n] truth values (row sees column) and depths."""
    n = len(parents)
    see, depth = np.zeros((n, n), bool), np.zeros(n, np.int64)
    for t in range(n):
        at = t
        while at >= 0:
            see[t, at] = True
            at = parents[at]
        depth[t] = see[t].sum() - 1
    return see, depth


def pack(see, words):
    """Rows of bits as int32 words."""
    n = see.shape[0]
    out = np.zeros((n, words), np.int64)
    for t in range(see.shape[1]):
        out[:, t // 32] |= see[:, t].astype(np.int64) << (t % 32)
    return out.astype(np.uint32).view(np.int32)


def rotate(x, w, table_rows, rot, interleaved, eps):
    """x [T, heads, d], table_rows [T, rot / 2, 2] in f64 -> the value, and the sum of magnitudes that
    its roundings are relative to."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y, mag = x.copy(), np.abs(x)
    if rot:
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        c, s = table_rows[:, None, :, 0], table_rows[:, None, :, 1]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        mag[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, mag


def check_rows(got, want, mag, what=""):
    """One rounding to bf16, and fp32 steps relative to the terms: d additions of the mean, the square
    root and its reciprocal, two products of the norm, two products and a sum of the rotation (fewer
    than 150 half steps of 2^-24)."""
    tol = BF16 * np.abs(want) + 150 * 2.0 ** -24 * mag + 2.0 ** -133
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want)[bad].max()))


def attend(q, k, v, scale, see):
    """q [n, G, d], k, v [L, d], see [n, L] -> o, lse, and their bounds."""
    n, G, d = q.shape
    o, lse = np.zeros((n, G, d)), np.full((n, G), -np.inf)
    tol_o, tol_l = np.zeros((n, G, d)), np.zeros((n, G))
    for i in range(n):
        j = np.nonzero(see[i])[0]
        if len(j) == 0:
            continue
        x = q[i] @ k[j].T * scale                       # [G, keys]
        m = x.max(-1, keepdims=True)
        p = np.exp(x - m)
        l = p.sum(-1, keepdims=True)
        w = p / l
        o[i] = w @ v[j]
        lse[i] = (m + np.log(l))[:, 0]
        # score: d products accumulated in fp32 (a step of 2^-23 each, should the tensor core truncate),
        # its scaling and the subtraction of the reference (at most 2^8 away from the maximum)
        mag = (np.abs(q[i]) @ np.abs(k[j]).T).max(-1) * scale
        e = (d + 2) * 2.0 ** -23 * mag + 2.0 ** -23 * (np.abs(m[:, 0]) + 8)
        # weights: rounded to bf16 (product and divisor use the same ones), 2^-22 of the exponential;
        # then |sum w (1 + u) v / sum w (1 + u) - o| <= max u / (1 - max u) * sum w |v - o|
        u = BF16 + e + 2.0 ** -20
        spread = np.stack([w[g] @ np.abs(v[j] - o[i, g]) for g in range(G)])
        # fp32 accumulation of P V over the keys, tile by tile
        acc = (len(j) + 64) * 2.0 ** -23 * (w @ np.abs(v[j]))
        tol_o[i] = (u / (1 - u))[:, None] * spread + acc + BF16 * np.abs(o[i]) + 2.0 ** -133
        tol_l[i] = e + (len(j) + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse[i])
    return o, lse, tol_o, tol_l


def check_attention(o, lse, ref, what=""):
    """o [n, G, d] and lse [n, G] in f64 against attend()."""
    want_o, want_l, tol_o, tol_l = ref
    empty = np.isneginf(want_l)
    assert (np.isneginf(lse) == empty).all(), what
    err = np.abs(o - want_o)
    assert (err <= tol_o).all(), (what, float(err.max()), float((err - tol_o).max()))
    err = np.abs(lse[~empty] - want_l[~empty])
    assert (err <= tol_l[~empty]).all(), (what, float(err.max()))
    assert (o[empty] == 0).all(), what


class Cache:
    """bf16 caches with sequences' rows in them; other slots hold NaN."""

    def __init__(self, rng, lens, Hkv, d, spread=0.5, extra=5, width=None, gen=1):
        g = torch.Generator(device="cuda").manual_seed(gen)
        self.lens = list(lens)
        pool = sum((n + PAGE - 1) // PAGE for n in lens) + extra
        self.bt = table(rng, lens, pool, width)
        self.k, self.v = (torch.full((pool, Hkv, PAGE, d), float("nan"), dtype=torch.bfloat16, device="cuda")
                          for _ in STREAMS)
        self.rows = []      # per sequence: k, v [L, Hkv, d] in f64
        for s, n in enumerate(lens):
            pair = []
            for c in (self.k, self.v):
                x = torch.randn((n, Hkv, d), device="cuda", generator=g)
                x *= torch.exp2(spread * torch.randn((n, 1, 1), device="cuda", generator=g))
                x = x.bfloat16()
                pos = torch.arange(n, device="cuda")
                if n:
                    c[torch.from_numpy(self.bt[s]).cuda().long()[pos // PAGE], :, pos % PAGE] = x
                pair.append(f64(x))
            self.rows.append(pair)

    def args(self):
        return self.k, self.v, i32(self.bt), i32(self.lens)
