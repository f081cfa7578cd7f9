"""Timing cases of the quantised paged KV cache and of sliding-window attention.

Five operators, as a serving loop uses them together:

  write         new K/V rows quantised to e4m3 as they go into the paged cache
  read          cached rows read back as bf16
  decode        one query token a sequence over the quantised cache
  chunk         several new query tokens a sequence over the quantised cache
  window        bf16 attention over prompts, packed or dense

decode, chunk and window take a sliding window with a few first tokens that
stay visible (sinks): the query at position p sees key j when j <= p and
(j > p - window or j < sinks); window 0 means no window.

Cache format: codes [pages][kv heads][16][d] in e4m3 and one scale byte per row
[pages][kv heads][16], row = codes * 2^(byte - 127), with the smallest exponent
e >= -127 for which the row's largest finite magnitude is at most 448 * 2^e.
"""
import math
import random

import torch

own = False

PAGE = 16
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    c = {"op": op, "seqs": 1, "lo": 1, "hi": 1, "new_lo": 1, "new_hi": 1, "H": 32, "Hkv": 8,
         "d": 128, "window": 0, "sinks": 0, "causal": True, "dense": False, "pick": 1}
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # the cache write of one decode step: 64 sequences, one new token each
        _case("write step 64", "write", seqs=64, lo=512, hi=8192, pick=42),
        # the cache write behind a batch of ragged prompts
        _case("write prompts 16", "write", seqs=16, lo=1, hi=4096, new_lo=1, new_hi=4096, pick=43),
        # a few short prefixes read back, to be copied or checked
        _case("read short 4 d64", "read", seqs=4, lo=30, hi=700, new_lo=30, new_hi=700, Hkv=4,
              H=16, d=64, pick=44),
        # every cached prefix of a full batch read back (a move to a bf16 consumer)
        _case("read prefixes 64", "read", seqs=64, lo=512, hi=8192, new_lo=8192, new_hi=8192,
              pick=42),
        # interactive decoding of one sequence: latency
        _case("decode 1x1000", "decode", seqs=1, lo=1000, hi=1000, pick=45),
        # a full decode batch, contexts uniform on [512, 8192]
        _case("decode 64", "decode", seqs=64, lo=512, hi=8192, pick=42),
        # a full batch of long streams, each kept to a window and four sinks
        _case("decode 64 window", "decode", seqs=64, lo=8192, hi=32768, window=2048, sinks=4,
              pick=46),
        # draft tokens of 16 sequences checked in one pass
        _case("chunk draft 16x4", "chunk", seqs=16, lo=512, hi=8192, new_lo=4, new_hi=4, pick=47),
        # chunked prefill: 512 new tokens of 16 sequences
        _case("chunk 16x512", "chunk", seqs=16, lo=512, hi=8192, new_lo=512, new_hi=512, pick=48),
        # long documents in chunks of 2048 under a window
        _case("chunk 4x2048 window", "chunk", seqs=4, lo=8000, hi=16384, new_lo=2048, new_hi=2048,
              window=4096, sinks=4, pick=49),
        # one long prompt under a window with sinks
        _case("window dense 8192", "window", seqs=1, lo=8192, hi=8192, new_lo=8192, new_hi=8192,
              Hkv=32, window=1024, sinks=4, dense=True, pick=50),
        # ragged prompts of a smaller model, short window
        _case("window ragged d64", "window", seqs=16, lo=1, hi=4096, new_lo=4096, new_hi=4096,
              H=16, Hkv=4, d=64, window=256, sinks=0, pick=51),
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
        op = rng.choice(("write", "read", "decode", "chunk", "window"))
        Hkv = rng.choice((1, 2, 4, 8))
        G = rng.choice((1, 2, 3, 4, 5, 8))
        d = rng.choice((64, 128))
        window = rng.choice((0, _spread(rng, 1, 8192))) if op != "window" else _spread(rng, 1, 4096)
        sinks = rng.choice((0, 4, rng.randint(1, 200))) if window else 0
        kw = dict(H=Hkv * G, Hkv=Hkv, d=d, pick=rng.randrange(1 << 20))
        if op in ("write", "read"):
            hi = _spread(rng, 1, 8192)
            new = 1 if op == "write" and rng.random() < 0.4 else hi
            c = _case(None, op, seqs=_spread(rng, 1, 64), lo=1 + rng.randrange(hi), hi=hi,
                      new_lo=1, new_hi=new, **kw)
        elif op == "decode":
            hi = _spread(rng, 1, 32768)
            c = _case(None, op, seqs=_spread(rng, 1, 64), lo=1 + rng.randrange(hi), hi=hi,
                      window=window, sinks=sinks, **kw)
        elif op == "chunk":
            hi = _spread(rng, 16, 16384)
            new = _spread(rng, 2, min(hi, 2048))
            c = _case(None, op, seqs=_spread(rng, 1, 16), lo=1 + rng.randrange(hi), hi=hi,
                      new_lo=1 + rng.randrange(new), new_hi=new, window=window, sinks=sinks,
                      causal=window > 0 or rng.random() < 0.8, **kw)
        else:
            dense = rng.random() < 0.5
            n = _spread(rng, 17, 8192 if dense else 4096)
            c = _case(None, op, seqs=_spread(rng, 1, 4 if dense else 16),
                      lo=n if dense else 1 + rng.randrange(n), hi=n,
                      new_lo=n, new_hi=n, window=window, sinks=sinks, dense=dense, **kw)
        c["lo"] = min(c["lo"], c["hi"])
        w, (b, f) = work(c), _largest()[op]
        scores = c["seqs"] * c["H"] * _lengths(c)[2] * _lengths(c)[3]
        if w["bytes"] <= b and w["flops"] <= f and scores <= 4.4e9:
            return c


def _lengths(c):
    """Context and new-token lengths of the sequences, and the longest of each."""
    r = random.Random(c["pick"])
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    new = [min(n, r.randint(c["new_lo"], c["new_hi"])) for n in lens]
    return lens, new, max(new), max(lens)


def _visible(L, n, window, sinks, causal):
    """(query, key) pairs that n queries at the end of L keys see, and how many keys any of them sees."""
    if not causal:
        return n * L, L
    if window <= 0:
        return sum(range(L - n + 1, L + 1)), L
    pairs = sum(min(p + 1, window) + min(sinks, max(0, p + 1 - window)) for p in range(L - n, L))
    first = max(0, L - n + 1 - window)
    return pairs, L - first + min(sinks, first)


def work(case):
    lens, new, _, _ = _lengths(case)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    total, op = sum(new), case["op"]
    pages = sum((n + PAGE - 1) // PAGE for n in lens)
    if op in ("write", "read"):
        touched = sum((L + PAGE - 1) // PAGE - (L - n) // PAGE for L, n in zip(lens, new))
        return {"bytes": total * Hkv * 2 * (3 * d + 1) + 4 * (touched + 2 * len(lens)), "flops": total * Hkv * 2 * d}
    seen = [_visible(L, n, case["window"], case["sinks"], case["causal"]) for L, n in zip(lens, new)]
    pairs, keys = sum(s[0] for s in seen), sum(s[1] for s in seen)
    row = 2 * d + 2 if op != "window" else 4 * d
    io = total * H * (4 * d + 4)
    table = 4 * pages if op != "window" else 0
    return {"bytes": keys * Hkv * row + io + table, "flops": 4.0 * d * H * pairs}


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """Rows of x (any float type) to e4m3 codes and scale bytes; plain operations."""
    x = x.float()
    finite = torch.isfinite(x)
    amax = torch.where(finite, x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(amax)                 # amax = m * 2^e, m in [0.5, 1)
    e = e - 9 + (m > 0.875).to(e.dtype)      # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, -127).clamp(min=-127)
    # 2^-e in two factors: both stay inside the normal range
    y = torch.ldexp(torch.ldexp(x, (-e // 2)[..., None]), (-e - (-e // 2))[..., None])
    y = torch.where(finite, y, float("nan"))
    return y.to(F8), (e + 127).to(torch.uint8)


def _values(codes, scale):
    """What the codes stand for, in fp32."""
    return torch.ldexp(codes.float(), (scale.to(torch.int32) - 127)[..., None])


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tables(case, g):
    lens, new, _, longest = _lengths(case)
    need = [(n + PAGE - 1) // PAGE for n in lens]
    pool = sum(need) + max(4, sum(need) // 10)
    perm = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    width = max(need)
    at = torch.arange(width, device="cuda")[None, :]
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


def prepare(case, seed):
    g = _gen(seed)
    _, new, nmax, longest = _lengths(case)
    H, Hkv, d, total = case["H"], case["Hkv"], case["d"], sum(new)
    s = dict(case, scale=float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32)), total=total,
             nmax=nmax, longest=longest)
    if case["op"] == "window":
        lens, _, _, _ = _lengths(case)
        Tk = sum(lens)
        lead = (case["seqs"], nmax) if case["dense"] else (total,)
        kead = (case["seqs"], longest) if case["dense"] else (Tk,)
        s["q"] = torch.randn(lead + (H, d), device="cuda", generator=g).bfloat16()
        s["k"] = torch.randn(kead + (Hkv, d), device="cuda", generator=g).bfloat16()
        s["v"] = torch.randn(kead + (Hkv, d), device="cuda", generator=g).bfloat16()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
        s["cu_k"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        return s
    pool, s["bt"], s["lens"], s["cu"] = _tables(case, g)
    shape = (pool, Hkv, PAGE, d)
    if case["op"] == "write":
        s["k"] = _rows(g, (total, Hkv, d), 0.7).bfloat16()
        s["v"] = _rows(g, (total, Hkv, d), 0.7).bfloat16()
        s["kc"], s["vc"] = (torch.zeros(shape, device="cuda").to(F8) for _ in range(2))
        s["ks"], s["vs"] = (torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2))
        return s
    s["kc"], s["ks"] = _quantise(_rows(g, shape, 0.3).bfloat16())
    s["vc"], s["vs"] = _quantise(_rows(g, shape, 0.7).bfloat16())
    s["q"] = torch.randn((total, H, d), device="cuda", generator=g).bfloat16()
    return s


# ------------------------------------------------------------ plain forms
def _slots(s):
    """Page and place in it of each new row: row cu[i] + t is token lens[i] - n_i + t."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(s["seqs"], device="cuda"), n, output_size=s["total"])
    t = torch.arange(s["total"], device="cuda") - s["cu"][seq].long()
    pos = s["lens"][seq].long() - n[seq] + t
    return s["bt"][seq, pos // PAGE].long(), pos % PAGE, seq, t, pos


def _attend(s, q, k, v, pos, valid):
    """q [S,n,H,d], k, v [S,L,Hkv,d] in fp32, query positions [S,n], valid keys [S]; o and lse."""
    S, n, H, d = q.shape
    L, Hkv = k.shape[1], k.shape[2]
    j = torch.arange(L, device="cuda")
    see = (j < valid[:, None])[:, None, :]
    if s["causal"]:
        p = pos[:, :, None]
        see = see & (j <= p)
        if s["window"] > 0:
            see = see & ((j > p - s["window"]) | (j < s["sinks"]))
    see = see.expand(S, n, L)
    v = torch.where((j < valid[:, None])[:, :, None, None], v, 0.0)
    q = q.reshape(S, n, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).reshape(S, Hkv, H // Hkv, n, L)
    x = torch.where(see[:, None, None], x * s["scale"], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(S, Hkv, -1, L), v.permute(0, 2, 1, 3)).reshape(S, H, n, d)
    o = o / torch.where(l > 0, l, 1.0).reshape(S, H, n, 1)
    lse = (m + torch.log(l)).reshape(S, H, n)
    return o.permute(0, 2, 1, 3), lse


def _plain(s):
    op = s["op"]
    if op == "write":
        page, at, _, _, _ = _slots(s)
        for_k, for_v = _quantise(s["k"]), _quantise(s["v"])
        s["kc"].view(torch.uint8)[page, :, at] = for_k[0].view(torch.uint8)
        s["vc"].view(torch.uint8)[page, :, at] = for_v[0].view(torch.uint8)
        s["ks"][page, :, at] = for_k[1]
        s["vs"][page, :, at] = for_v[1]
        return {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if op == "read":
        page, at, _, _, _ = _slots(s)
        k = _values(s["kc"].view(torch.uint8)[page, :, at].view(F8), s["ks"][page, :, at])
        v = _values(s["vc"].view(torch.uint8)[page, :, at].view(F8), s["vs"][page, :, at])
        return {"k": k.bfloat16(), "v": v.bfloat16()}
    S, H, Hkv, d = s["seqs"], s["H"], s["Hkv"], s["d"]
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), n, output_size=s["total"])
    t = torch.arange(s["total"], device="cuda") - s["cu"][seq].long()
    q = torch.zeros((S, s["nmax"], H, d), device="cuda")
    q[seq, t] = s["q"].reshape(s["total"], H, d).float()
    if op == "window":
        L = s["longest"]
        at = (s["cu_k"][:-1, None].long() + torch.arange(L, device="cuda")).clamp(max=s["cu_k"][-1].long() - 1)
        k = s["k"].reshape(-1, Hkv, d)[at].float()
        v = s["v"].reshape(-1, Hkv, d)[at].float()
    else:
        ids = s["bt"].long().clamp(min=0)
        k = _values(s["kc"].view(torch.uint8)[ids].view(F8), s["ks"][ids])
        v = _values(s["vc"].view(torch.uint8)[ids].view(F8), s["vs"][ids])
        k, v = (x.permute(0, 1, 3, 2, 4).reshape(S, -1, Hkv, d) for x in (k, v))
    pos = s["lens"].long()[:, None] - n[:, None] + torch.arange(s["nmax"], device="cuda")
    o, lse = _attend(s, q, k, v, pos, s["lens"].long())
    if op == "window" and s["dense"]:
        return {"o": o.bfloat16(), "lse": lse}
    o, lse = o[seq, t].bfloat16(), lse[seq, :, t]
    return {"o": o, "lse": lse if op == "decode" else lse.T.contiguous()}


def run(state):
    if not own:
        return _plain(state)
    from tiled_online_softmax_sm_gb300 import binding as fb
    s, op = state, state["op"]
    if op == "write":
        fb.paged_kv_write_e4m3(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"],
                               s["lens"], s["cu"])
        return {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if op == "read":
        k, v = fb.paged_kv_read_e4m3(s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["lens"],
                                     s["cu"], s["total"])
        return {"k": k, "v": v}
    if op == "decode":
        o, lse = fb.paged_decode_e4m3(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"],
                                      s["lens"], s["scale"], window=s["window"], sinks=s["sinks"])
    elif op == "chunk":
        o, lse = fb.paged_prefill_e4m3(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"],
                                       s["lens"], s["cu"], s["nmax"], s["scale"],
                                       causal=s["causal"], window=s["window"], sinks=s["sinks"])
    elif s["dense"]:
        o, lse = fb.forward_window(s["q"], s["k"], s["v"], s["scale"], s["window"], s["sinks"])
    else:
        o, lse = fb.forward_varlen_window(s["q"], s["k"], s["v"], s["cu"], s["cu_k"], s["nmax"],
                                          s["longest"], s["scale"], s["window"], s["sinks"])
    return {"o": o, "lse": lse}


# ------------------------------------------------- the definition in 64 bits
def _exact_codes(x):
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax / 448)).clamp(min=-127)
    e = torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, e).clamp(min=-127)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs())).clamp(min=-6) - 3)
    return torch.round(y / step) * step, (e[..., 0] + 127)


def exact(case, seed):
    s = prepare(case, seed)
    lens, new, _, _ = _lengths(case)
    cu, bt = s["cu"].tolist(), s["bt"].long() if "bt" in s else None
    S, H, Hkv, d = case["seqs"], case["H"], case["Hkv"], case["d"]

    def where(i):
        pos = torch.arange(lens[i] - new[i], lens[i], device="cuda")
        return bt[i, pos // PAGE], pos % PAGE

    if case["op"] == "write":
        out = {"k_cache": s["kc"].double(), "v_cache": s["vc"].double(),
               "k_scale": s["ks"].double(), "v_scale": s["vs"].double()}
        for i in range(S):
            page, at = where(i)
            for x in ("k", "v"):
                c, e = _exact_codes(s[x][cu[i]:cu[i + 1]])
                out[x + "_cache"][page, :, at] = c
                out[x + "_scale"][page, :, at] = e
        return dict(out, k_scale=out["k_scale"].to(torch.uint8), v_scale=out["v_scale"].to(torch.uint8))
    if case["op"] == "read":
        out = {x: torch.empty((s["total"], Hkv, d), dtype=torch.float64, device="cuda") for x in "kv"}
        for i in range(S):
            page, at = where(i)
            for x in "kv":
                c = s[x + "c"].view(torch.uint8)[page, :, at].view(F8).double()
                out[x][cu[i]:cu[i + 1]] = c * torch.exp2(s[x + "s"][page, :, at].double() - 127)[..., None]
        return out
    o = torch.zeros((s["total"], H, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total"], H), dtype=torch.float64, device="cuda")
    q, G, ck = s["q"].reshape(-1, H, d), H // Hkv, 0
    for i in range(S):
        L, n = lens[i], new[i]
        if case["op"] == "window":
            kv = [s[x].reshape(-1, Hkv, d)[ck:ck + L].double() for x in "kv"]
            ck += L
        else:
            ids = bt[i, :(L + PAGE - 1) // PAGE]
            kv = [(s[x + "c"].view(torch.uint8)[ids].view(F8).double()
                   * torch.exp2(s[x + "s"][ids].double() - 127)[..., None]).transpose(1, 2).reshape(-1, Hkv, d)[:L]
                  for x in "kv"]
        for r0 in range(0, n, 1024):
            r1 = min(n, r0 + 1024)
            p = torch.arange(L - n + r0, L - n + r1, device="cuda")[:, None]
            first, last = 0, L      # the keys any of these queries sees, beside the sinks
            if case["causal"]:
                last = L - n + r1
                first = max(0, L - n + r0 - case["window"] + 1) if case["window"] > 0 else 0
            j = torch.cat([torch.arange(min(case["sinks"], first), device="cuda"),
                           torch.arange(first, last, device="cuda")])
            hide = torch.zeros((r1 - r0, j.numel()), dtype=torch.bool, device="cuda")
            if case["causal"]:
                hide = j[None, :] > p
                if case["window"] > 0:
                    hide = hide | ((j[None, :] <= p - case["window"]) & (j[None, :] >= case["sinks"]))
            for h in range(Hkv):
                k, v = kv[0][j, h], kv[1][j, h]
                rows = slice(cu[i] + r0, cu[i] + r1)
                x = torch.einsum("ngd,jd->ngj", q[rows, h * G:(h + 1) * G].double(), k) * s["scale"]
                x = x.masked_fill(hide[:, None, :], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[rows, h * G:(h + 1) * G] = z
                o[rows, h * G:(h + 1) * G] = torch.einsum("ngj,jd->ngd", torch.exp(x - z[..., None]), v)
    if case["op"] == "decode":
        return {"o": o, "lse": lse}
    if case["dense"]:
        n = case["hi"]
        return {"o": o.reshape(S, n, H, d), "lse": lse.reshape(S, n, H).permute(0, 2, 1).contiguous()}
    return {"o": o, "lse": lse.T.contiguous()}
