"""Timing cases of drafted token trees over the paged cache.

Five operators, as a serving loop that drafts trees of tokens uses them together:

  layout        the tree's parents to ancestor bits and rotary positions
  rope          q and k of each head normalised and rotated in one pass; k and v
                written into the bf16 paged cache, or k left dense
  tree          attention of the drafted tokens over the cache: each sees the
                context and its own ancestors
  accept        the K/V rows of the accepted path moved to the front of the
                drafted tail, in every layer
  copy          whole pages copied for forked sequences, in every layer

A sequence's n drafted tokens are the last n of its L cached ones; drafted token
t of sequence s is row cu[s] + t of the packed tensors.  Row i of the mask holds
bit t (word t / 32, bit t % 32) when drafted token i sees drafted token t.
"""
import math
import random

import torch

own = False

PAGE = 16
F8 = torch.float8_e4m3fn
EPS = 1e-6
MAX_POS = 8192     # rows of the rotary table
BASE = 10000.0


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    c = {"op": op, "seqs": 1, "lo": 1, "hi": 1, "new_lo": 1, "new_hi": 1, "H": 32, "Hkv": 8,
         "d": 128, "pick": 1, "paged": True, "norm": True, "rot": 128, "interleaved": False,
         "axes": 1, "layers": 1, "e4m3": False, "pairs": 0}
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # the trees of one drafting step of a small batch
        _case("layout 8x24", "layout", seqs=8, lo=512, hi=8192, new_lo=24, new_hi=24, pick=61),
        # wide trees of a full batch, ragged
        _case("layout 64x256", "layout", seqs=64, lo=512, hi=8192, new_lo=100, new_hi=256, pick=62),
        # one new token of 64 sequences on its way into the cache: latency
        _case("rope step 64", "rope", seqs=64, lo=512, hi=8192, pick=63),
        # ragged prompts with time, height and width positions
        _case("rope prompts 16 axes", "rope", seqs=16, lo=1, hi=4096, new_lo=1, new_hi=4096,
              axes=3, pick=64),
        # one interactive sequence, a small tree: latency
        _case("tree 1x1000 8", "tree", seqs=1, lo=1000, hi=1000, new_lo=8, new_hi=8, pick=65),
        # a full batch, contexts uniform on [512, 8192], 16 drafted tokens each
        _case("tree 64x16", "tree", seqs=64, lo=512, hi=8192, new_lo=16, new_hi=16, pick=42),
        # ragged trees of a smaller model, three query heads a kv head
        _case("tree 16x64 d64", "tree", seqs=16, lo=512, hi=8192, new_lo=20, new_hi=64, H=24, d=64,
              rot=64, pick=66),
        # a few long documents with wide trees
        _case("tree 4x64 long", "tree", seqs=4, lo=16384, hi=65536, new_lo=48, new_hi=64, pick=67),
        # accepted paths of a small batch, one layer
        _case("accept 16", "accept", seqs=16, lo=40, hi=400, new_lo=16, new_hi=32, pick=68),
        # accepted paths of a full batch, all layers of the cache in one call
        _case("accept 64 layers 8", "accept", seqs=64, lo=70, hi=128, new_lo=16, new_hi=64, layers=8,
              pick=69),
        # the last pages of eight forked sequences, one layer
        _case("copy 8", "copy", pairs=8, pick=70),
        # a pool put in order: many pages in all layers of an e4m3 cache
        _case("copy 512 layers 8 e4m3", "copy", pairs=512, layers=8, e4m3=True, pick=71),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_LARGEST = None


def _largest():
    """The largest listed work of each operator: a drawn case costs no more."""
    global _LARGEST
    if _LARGEST is None:
        _LARGEST = {}
        for c in listed():
            w = work(c)
            b, f = _LARGEST.get(c["op"], (0, 0))
            _LARGEST[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    return _LARGEST


def draw(rng):
    while True:
        op = rng.choice(("layout", "rope", "tree", "tree", "accept", "copy"))
        Hkv = rng.choice((1, 2, 4, 8))
        d = rng.choice((64, 128))
        kw = dict(H=Hkv * rng.choice((1, 2, 3, 4, 5, 8)), Hkv=Hkv, d=d, pick=rng.randrange(1 << 20),
                  rot=rng.choice((d, d, d // 2)))
        if op == "layout":
            new = _spread(rng, 1, 256)
            c = _case(None, op, seqs=_spread(rng, 1, 64), lo=new, hi=MAX_POS,
                      new_lo=1 + rng.randrange(new), new_hi=new, **kw)
        elif op == "rope":
            hi = _spread(rng, 1, 4096)
            new = _spread(rng, 1, hi)
            c = _case(None, op, seqs=_spread(rng, 1, 64), lo=1 + rng.randrange(hi), hi=hi,
                      new_lo=1 + rng.randrange(new), new_hi=new, paged=rng.random() < 0.6,
                      norm=rng.random() < 0.8, interleaved=rng.random() < 0.3,
                      axes=rng.choice((1, 1, 2, 3)), **kw)
        elif op == "tree":
            hi = _spread(rng, 16, 65536)
            new = _spread(rng, 1, min(hi, 200))
            c = _case(None, op, seqs=_spread(rng, 1, 64), lo=max(new, 1 + rng.randrange(hi)), hi=hi,
                      new_lo=1 + rng.randrange(new), new_hi=new, **kw)
        elif op == "accept":
            new = _spread(rng, 1, 64)
            hi = new + rng.randrange(200)
            c = _case(None, op, seqs=_spread(rng, 1, 64), lo=new, hi=hi, new_lo=1 + rng.randrange(new),
                      new_hi=new, layers=rng.randint(1, 8), e4m3=rng.random() < 0.4, **kw)
        else:
            c = _case(None, op, pairs=_spread(rng, 1, 512), layers=rng.randint(1, 8),
                      e4m3=rng.random() < 0.4, **kw)
        c["lo"] = min(c["lo"], c["hi"])
        w, (b, f) = work(c), _largest()[op]
        lens, new, _, _ = _lengths(c)
        scores = c["seqs"] * c["H"] * max(new) * max(lens) if op == "tree" else 0
        held = c["seqs"] * c["Hkv"] * c["d"] * max(lens) if op == "tree" else 0
        if w["bytes"] <= b and w["flops"] <= f and scores <= 4e8 and held <= 6e8:
            return c


def _lengths(c):
    """Context and new-token lengths of the sequences, and the longest of each."""
    r = random.Random(c["pick"])
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    new = [min(n, r.randint(c["new_lo"], c["new_hi"])) for n in lens]
    return lens, new, max(new), max(lens)


def _paths(c):
    """How many tokens of each tree are accepted, and the first of them.  The rest of a path lies
    behind the places its rows move to, as in a tree listed level by level: passes may repeat."""
    r = random.Random(c["pick"] + 1)
    out = []
    for n in _lengths(c)[1]:
        k = r.randint(0, min(8, (n + 1) // 2))
        out.append([] if k == 0 else [0] + sorted(r.sample(range(k, n), k - 1)) if r.random() < 0.5
                   else sorted(r.sample(range(k, n), min(k, n - k))))
    return out


def _row_bytes(c):
    """Bytes of one K and one V row."""
    return 2 * c["d"] + 2 if c["e4m3"] else 4 * c["d"]


def work(case):
    lens, new, nmax, _ = _lengths(case)
    H, Hkv, d, op = case["H"], case["Hkv"], case["d"], case["op"]
    total = sum(new)
    if op == "layout":
        words = (nmax + 31) // 32
        return {"bytes": 4 * total * (words + 2) + 8 * len(new), "flops": 0}
    if op == "rope":
        heads = H + (2 if case["paged"] else 1) * Hkv
        angles = min(total * case["axes"], MAX_POS) * 4 * case["rot"]
        return {"bytes": total * (4 * heads * d + 4 * case["axes"]) + angles,
                "flops": total * (H + Hkv) * d * 8}
    if op == "tree":
        pairs = sum(n * (L - n) + n * 4 for L, n in zip(lens, new))   # (about four ancestors a token)
        pages = sum((L + PAGE - 1) // PAGE for L in lens)
        io = total * H * (4 * d + 4) + 4 * total * ((nmax + 31) // 32)
        return {"bytes": sum(lens) * Hkv * 4 * d + io + 4 * pages, "flops": 4.0 * d * H * pairs}
    if op == "accept":
        moved = sum(1 for p in _paths(case) for a, t in enumerate(p) if t != a)
        accepted = sum(len(p) for p in _paths(case))
        return {"bytes": 2 * moved * Hkv * _row_bytes(case) * case["layers"] + 4 * accepted + 12 * len(new),
                "flops": 0}
    return {"bytes": case["pairs"] * (2 * PAGE * Hkv * _row_bytes(case) * case["layers"] + 8), "flops": 0}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tables(case, g):
    lens, new, _, _ = _lengths(case)
    need = [(n + PAGE - 1) // PAGE for n in lens]
    pool = sum(need) + max(4, sum(need) // 10)
    perm = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    at = torch.arange(max(need), device="cuda")[None, :]
    n = torch.tensor(need, device="cuda")[:, None]
    start = n.cumsum(0) - n
    bt = torch.where(at < n, perm[(start + at).clamp(max=pool - 1)], -1).to(torch.int32)
    cu = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    return pool, bt.contiguous(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu


def _rows(g, shape, spread):
    """Rows with channels and tokens of different size, as projections give them."""
    x = torch.randn(shape, device="cuda", generator=g)
    x *= 1 + 3 * (torch.rand(shape[-1], device="cuda", generator=g) < 0.05)
    x *= torch.exp2(spread * torch.randn(shape[:-1] + (1,), device="cuda", generator=g))
    return x


def _sections(case):
    """Rotary pairs of each axis: the first axis has what the others leave."""
    half = case["rot"] // 2
    rest = [half * 3 // 8] * (case["axes"] - 1)
    return [half - sum(rest)] + rest


def _cache(case, g, pool):
    shape = (case["layers"], pool, case["Hkv"], PAGE, case["d"])
    if not case["e4m3"]:
        return [torch.randn(shape, device="cuda", generator=g).bfloat16() for _ in "kv"] + [None, None]
    codes = [torch.randn(shape, device="cuda", generator=g).mul_(80).to(F8) for _ in "kv"]
    return codes + [torch.randint(110, 130, shape[:4], device="cuda", generator=g).to(torch.uint8) for _ in "kv"]


def prepare(case, seed):
    g = _gen(seed)
    lens, new, nmax, longest = _lengths(case)
    H, Hkv, d, total, op = case["H"], case["Hkv"], case["d"], sum(new), case["op"]
    s = dict(case, total=total, nmax=nmax, longest=longest, words=(nmax + 31) // 32)
    if op == "copy":
        pool = 2 * case["pairs"] + 64
        s["kc"], s["vc"], s["ks"], s["vs"] = _cache(case, g, pool)
        perm = torch.randperm(pool, device="cuda", generator=g)[:2 * case["pairs"]]
        s["list"] = perm.view(-1, 2).to(torch.int32)
        return s
    pool, s["bt"], s["lens"], s["cu"] = _tables(case, g)
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device="cuda"), n, output_size=total)
    t = torch.arange(total, device="cuda") - s["cu"][seq].long()
    if op in ("layout", "tree"):
        # a parent uniform over the context's last token (-1) and the earlier drafted tokens
        u = torch.rand(total, device="cuda", generator=g, dtype=torch.float64)
        s["parents"] = ((u * (t + 1)).floor().clamp(max=t.double()) - 1).to(torch.int32)
    if op == "layout":
        return s
    if op == "rope":
        qkv = _rows(g, (total, H + 2 * Hkv, d), 0.5).bfloat16()   # one projection's output
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(d, device="cuda", generator=g)).bfloat16() if case["norm"]
                            else None for _ in "qk")
        half = case["rot"] // 2
        freq = BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * freq
        s["table"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        pos = (s["lens"][seq].long() - n[seq] + t)[None]
        if case["axes"] > 1:    # the other axes walk over an image's rows and columns
            side = 1 + int(torch.randint(8, 64, (1,), device="cuda", generator=g).item())
            pos = torch.stack([pos[0], t // side, t % side][:case["axes"]])
        s["pos"] = pos.to(torch.int32).contiguous()
        s["sections"] = _sections(case)
        if case["paged"]:
            shape = (pool, Hkv, PAGE, d)
            s["kc"], s["vc"] = (torch.zeros(shape, device="cuda", dtype=torch.bfloat16) for _ in "kv")
        return s
    if op == "tree":
        s["scale"] = float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32))
        shape = (pool, Hkv, PAGE, d)
        s["kc"] = _rows(g, shape, 0.3).bfloat16()
        s["vc"] = _rows(g, shape, 0.7).bfloat16()
        s["q"] = torch.randn((total, H, d), device="cuda", generator=g).bfloat16()
        s["mask"], _ = _plain_layout(s)
        if own:     # a serving loop keeps one workspace
            from tiled_online_softmax_sm_gb300 import binding as fb
            need = fb.fa_paged_tree_workspace_size(case["seqs"], nmax, H, Hkv, d)
            s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        return s
    s["kc"], s["vc"], s["ks"], s["vs"] = _cache(case, g, pool)
    paths = _paths(case)
    s["deepest"] = max(1, max(len(p) for p in paths))
    s["path"] = torch.tensor([p + [-1] * (s["deepest"] - len(p)) for p in paths], dtype=torch.int32, device="cuda")
    s["path_lens"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------ plain forms
def _where(s):
    """Sequence of each packed row, its place in it and its position in the context."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(s["seqs"], device="cuda"), n, output_size=s["total"])
    t = torch.arange(s["total"], device="cuda") - s["cu"][seq].long()
    return n, seq, t, s["lens"][seq].long() - n[seq] + t


def _plain_layout(s):
    n, seq, t, _ = _where(s)
    N = s["nmax"]
    reach = torch.zeros((s["seqs"], N, N + 1), device="cuda")    # column N: the context
    reach[seq, t, t] = 1
    up = s["parents"].long()
    reach[seq, t, torch.where(up < 0, N, up)] = 1
    reach = reach[:, :, :N].contiguous()
    for _ in range(max(1, N - 1).bit_length()):
        reach = (torch.matmul(reach, reach) > 0).float()
    depth = reach.sum(-1)[seq, t].long() - 1
    bits = torch.zeros((s["seqs"], N, 32 * s["words"]), device="cuda", dtype=torch.int64)
    bits[:, :, :N] = reach.long()
    weight = torch.bitwise_left_shift(torch.ones(32, device="cuda", dtype=torch.int64), torch.arange(32, device="cuda"))
    word = (bits.view(s["seqs"], N, s["words"], 32) * weight).sum(-1)[seq, t]
    mask = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
    return mask, (s["lens"][seq].long() - n[seq] + depth).to(torch.int32)


def _plain_rope(s, x, w):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    rot, half = s["rot"], s["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(s["axes"], device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=half)
    angle = s["table"][s["pos"].long()[axis].T, torch.arange(half, device="cuda")]    # [total, half, 2]
    c, n = angle[:, None, :, 0], angle[:, None, :, 1]
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["interleaved"] else (x[..., :half], x[..., half:rot])
    first, second = a * c - b * n, b * c + a * n
    if s["interleaved"]:
        y[..., 0:rot:2], y[..., 1:rot:2] = first, second
    else:
        y[..., :half], y[..., half:rot] = first, second
    return y.bfloat16()


def _plain_tree(s):
    n, seq, t, _ = _where(s)
    S, H, Hkv, d, N = s["seqs"], s["H"], s["Hkv"], s["d"], s["nmax"]
    ids = s["bt"].long().clamp(min=0)
    k, v = (s[x][ids].permute(0, 1, 3, 2, 4).reshape(S, -1, Hkv, d).float() for x in ("kc", "vc"))
    L = k.shape[1]
    j = torch.arange(L, device="cuda")
    lens = s["lens"].long()
    start = (lens - n)[:, None, None]
    bits = torch.zeros((S, N, s["words"]), device="cuda", dtype=torch.int64)
    bits[seq, t] = s["mask"].long()
    drafted = (j[None, None] - start).clamp(0, 32 * s["words"] - 1).expand(S, N, L)
    bit = torch.bitwise_right_shift(torch.gather(bits, 2, drafted // 32), drafted % 32) & 1
    see = (j[None, None] < start) | ((bit == 1) & (j[None, None] < lens[:, None, None]))
    v = torch.where((j < lens[:, None])[:, :, None, None], v, 0.0)
    q = torch.zeros((S, N, H, d), device="cuda")
    q[seq, t] = s["q"].float()
    q = q.reshape(S, N, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).reshape(S, Hkv, H // Hkv, N, L)
    x = torch.where(see[:, None, None], x * s["scale"], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(S, Hkv, -1, L), v.permute(0, 2, 1, 3)).reshape(S, H, N, d)
    o = o / torch.where(l > 0, l, 1.0).reshape(S, H, N, 1)
    lse = (m + torch.log(l)).reshape(S, H, N)
    return {"o": o.permute(0, 2, 1, 3)[seq, t].bfloat16(), "lse": lse[seq, :, t].T.contiguous()}


def _caches(s):
    return {x: s[y] for x, y in (("k_cache", "kc"), ("v_cache", "vc"), ("k_scale", "ks"), ("v_scale", "vs"))
            if s[y] is not None}


def _bytes(x):
    return x.view(torch.uint8) if x.dtype is F8 else x


def _plain(s):
    op = s["op"]
    if op == "layout":
        mask, pos = _plain_layout(s)
        return {"mask": mask, "positions": pos}
    if op == "rope":
        out = {"q": _plain_rope(s, s["q"], s["qw"])}
        k = _plain_rope(s, s["k"], s["kw"])
        if not s["paged"]:
            return dict(out, k=k)
        _, seq, _, pos = _where(s)
        page, at = s["bt"][seq, pos // PAGE].long(), pos % PAGE
        s["kc"][page, :, at] = k
        s["vc"][page, :, at] = s["v"]
        return dict(out, k_cache=s["kc"], v_cache=s["vc"])
    if op == "tree":
        return _plain_tree(s)
    if op == "copy":
        src, dst = s["list"][:, 0].long(), s["list"][:, 1].long()
        for x in _caches(s).values():
            _bytes(x)[:, dst] = _bytes(x)[:, src]
        return _caches(s)
    first = s["lens"].long() - (s["cu"][1:] - s["cu"][:-1]).long()
    a = torch.arange(s["deepest"], device="cuda")
    live = a < s["path_lens"][:, None]
    seq, a = live.nonzero(as_tuple=True)
    src, dst = first[seq] + s["path"][seq, a].long(), first[seq] + a
    page_s, page_d = s["bt"][seq, src // PAGE].long(), s["bt"][seq, dst // PAGE].long()
    for x in _caches(s).values():
        b = _bytes(x)
        b[:, page_d, :, dst % PAGE] = b[:, page_s, :, src % PAGE]
    return dict(_caches(s), seq_lens=(first + s["path_lens"]).to(torch.int32))


def run(state):
    if not own:
        return _plain(state)
    from tiled_online_softmax_sm_gb300 import binding as fb
    s, op = state, state["op"]
    if op == "layout":
        mask, pos = fb.tree_layout(s["parents"], s["lens"], s["cu"], s["words"])
        return {"mask": mask, "positions": pos}
    if op == "rope":
        if not s["paged"]:
            q, k = fb.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["table"], s["pos"], EPS, s["sections"],
                                   s["interleaved"])
            return {"q": q, "k": k}
        q = fb.paged_qkv_write(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["table"], s["pos"], s["kc"], s["vc"],
                               s["bt"], s["lens"], s["cu"], EPS, s["sections"], s["interleaved"])
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    if op == "tree":
        o, lse = fb.paged_tree_attention(s["q"], s["kc"], s["vc"], s["bt"], s["lens"], s["cu"], s["nmax"],
                                         s["mask"], s["scale"], workspace=s["ws"])
        return {"o": o, "lse": lse}
    if op == "copy":
        fb.paged_copy_pages(s["kc"], s["vc"], s["list"], s["ks"], s["vs"])
        return _caches(s)
    lens = fb.paged_kv_accept(s["kc"], s["vc"], s["bt"], s["lens"], s["cu"], s["path"], s["path_lens"],
                              s["ks"], s["vs"])
    return dict(_caches(s), seq_lens=lens)


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    lens, new, _, _ = _lengths(case)
    H, Hkv, d, op = case["H"], case["Hkv"], case["d"], case["op"]
    if op == "copy":
        out = {x: (y.double() if y.dtype is not torch.uint8 else y.clone()) for x, y in _caches(s).items()}
        for src, dst in s["list"].tolist():
            for x in out.values():
                x[:, dst] = x[:, src].clone()
        return out
    cu = s["cu"].tolist()
    if op == "layout":
        up, W = s["parents"].tolist(), s["words"]
        mask, pos = [], []
        for i in range(case["seqs"]):
            for t in range(new[i]):
                row, at, depth = 0, t, -1
                while at >= 0:
                    row, at, depth = row | 1 << at, up[cu[i] + at], depth + 1
                words = [row >> 32 * w & 0xffffffff for w in range(W)]
                mask.append([x - (1 << 32) if x >> 31 else x for x in words])
                pos.append(lens[i] - new[i] + depth)
        return {"mask": torch.tensor(mask, dtype=torch.int32), "positions": torch.tensor(pos, dtype=torch.int32)}
    bt = s["bt"].long()
    if op == "rope":
        half, rot = case["rot"] // 2, case["rot"]
        owner = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
        angle = torch.stack([s["table"].double()[s["pos"][owner[p]].long(), p] for p in range(half)], 1)
        z = torch.complex(angle[..., 0], angle[..., 1])[:, None]

        def turned(x, w):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + EPS) * w.double()
            r = x[..., :rot]
            pair = r.unflatten(-1, (half, 2)) if case["interleaved"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            y = y if case["interleaved"] else y.transpose(-1, -2)
            return torch.cat([y.flatten(-2), x[..., rot:]], -1)

        q, k = turned(s["q"], s["qw"]), turned(s["k"], s["kw"])
        if not case["paged"]:
            return {"q": q, "k": k}
        out = {"q": q, "k_cache": s["kc"].double(), "v_cache": s["vc"].double()}
        for i in range(case["seqs"]):
            pos = torch.arange(lens[i] - new[i], lens[i], device="cuda")
            out["k_cache"][bt[i, pos // PAGE], :, pos % PAGE] = k[cu[i]:cu[i + 1]]
            out["v_cache"][bt[i, pos // PAGE], :, pos % PAGE] = s["v"][cu[i]:cu[i + 1]].double()
        return out
    if op == "accept":
        out = {x: (y.double() if y.dtype is not torch.uint8 else y.clone()) for x, y in _caches(s).items()}
        table, paths = bt.tolist(), _paths(case)
        for i, p in enumerate(paths):
            first = lens[i] - new[i]
            for x in out.values():
                old = [x[:, table[i][(first + t) // PAGE], :, (first + t) % PAGE].clone() for t in p]
                for a, row in enumerate(old):
                    x[:, table[i][(first + a) // PAGE], :, (first + a) % PAGE] = row
        out["seq_lens"] = torch.tensor([L - n + len(p) for L, n, p in zip(lens, new, paths)], dtype=torch.int32)
        return out
    o = torch.zeros((s["total"], H, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total"], H), dtype=torch.float64, device="cuda")
    G = H // Hkv
    up = s["parents"].tolist()
    for i in range(case["seqs"]):
        L, n = lens[i], new[i]
        hide = torch.ones((n, n), dtype=torch.bool)
        for t in range(n):
            at = t
            while at >= 0:
                hide[t, at] = False
                at = up[cu[i] + at]
        hide = torch.cat([torch.zeros((n, L - n), dtype=torch.bool), hide], 1).cuda()
        ids = bt[i, :(L + PAGE - 1) // PAGE]
        for h in range(Hkv):
            k, v = (s[x][ids, h].reshape(-1, d)[:L].double() for x in ("kc", "vc"))
            rows, heads = slice(cu[i], cu[i + 1]), slice(h * G, (h + 1) * G)
            x = torch.einsum("ngd,jd->ngj", s["q"][rows, heads].double(), k) * s["scale"]
            x = x.masked_fill(hide[:, None, :], -math.inf)
            z = torch.logsumexp(x, -1)
            lse[rows, heads] = z
            o[rows, heads] = torch.einsum("ngj,jd->ngd", torch.exp(x - z[..., None]), v)
    return {"o": o, "lse": lse.T.contiguous()}
