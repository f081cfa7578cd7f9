"""Plain float64 forms of the e4m3 paged cache and of windowed attention, and
the error bounds the GPU tests hold the kernels to."""
import math

import numpy as np

PAGE = 16
# the values of codes 0x00 .. 0x7e, ascending (0x7f is NaN)
CODE_VALUES = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                        for c in range(127)])


def quantise(x):
    """x [..., d] float64 -> (codes uint8, scale bytes uint8)."""
    x = np.asarray(x, np.float64)
    finite = np.isfinite(x)
    amax = np.where(finite, np.abs(x), 0.0).max(-1)
    e = np.full(amax.shape, -127)
    some = amax > 0
    e[some] = np.ceil(np.log2(amax[some] / 448)).astype(int)
    e[some] -= amax[some] <= 448 * 2.0 ** (e[some] - 1.0)     # log2's own rounding
    e[some] += amax[some] > 448 * 2.0 ** e[some].astype(float)
    e = np.maximum(e, -127)
    y = np.where(finite, np.abs(x), 0.0) / 2.0 ** e[..., None].astype(float)
    hi = np.clip(np.searchsorted(CODE_VALUES, y), 0, 126)     # first value >= y
    lo = np.maximum(hi - 1, 0)
    up, down = CODE_VALUES[hi] - y, y - CODE_VALUES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (up == 0), hi, lo)
    code = np.where(finite, code, 0x7f) | np.where(np.signbit(x), 0x80, 0)
    return code.astype(np.uint8), (e + 127).astype(np.uint8)


def values(codes, scale):
    """What codes and scale bytes stand for (NaN codes as NaN)."""
    mag = codes & 0x7f
    v = np.where(mag == 0x7f, np.nan, CODE_VALUES[np.minimum(mag, 126)])
    return np.where(codes & 0x80, -v, v) * 2.0 ** (scale[..., None].astype(float) - 127)


def visible(n, L, causal, window, sinks):
    """[n, L] mask: n queries at the end of L keys."""
    p = L - n + np.arange(n)[:, None]
    j = np.arange(L)[None, :]
    see = np.ones((n, L), bool)
    if causal:
        see = j <= p
        if window > 0:
            see &= (j > p - window) | (j < sinks)
    return see


def attend(q, k, v, scale, causal=True, window=0, sinks=0, vexp=None):
    """q [n,H,d], k, v [L,Hkv,d] float64 -> dict of o [n,H,d], lse [n,H] and, per output,
    what the bounds need: a = sum w|v| / l, ds = error unit of a row's scores, big = the
    largest weight times its V row's power of two (with vexp [L,Hkv]) over l."""
    n, H, d = q.shape
    L, Hkv = k.shape[:2]
    G = H // Hkv
    see = visible(n, L, causal, window, sinks)
    used = see.any(0)
    k, v = np.where(used[:, None, None], k, 0.0), np.where(used[:, None, None], v, 0.0)
    out = {"o": np.zeros((n, H, d)), "lse": np.full((n, H), -np.inf), "a": np.zeros((n, H, d)),
           "ds": np.zeros((n, H)), "big": np.zeros((n, H)), "keys": see.sum(1)}
    if L == 0:
        return out
    for h in range(H):
        x = np.where(see, q[:, h] @ k[:, h // G].T * scale, -np.inf)
        mag = np.where(see, np.abs(q[:, h]) @ np.abs(k[:, h // G]).T * scale, 0.0)
        m = x.max(1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        w = np.exp(x - m)
        l = w.sum(1)
        some = l > 0
        ls = np.where(some, l, 1.0)[:, None]
        out["o"][:, h] = w @ v[:, h // G] / ls
        out["a"][:, h] = w @ np.abs(v[:, h // G]) / ls
        with np.errstate(divide="ignore"):
            out["lse"][:, h] = np.where(some, m[:, 0] + np.log(l), -np.inf)
        out["ds"][:, h] = mag.max(1)
        if vexp is not None:
            out["big"][:, h] = (w * 2.0 ** vexp[None, :, h // G]).max(1) / ls[:, 0]
    return out


def bounds(ref, d, rounding):
    """Error bounds (o, lse) of a kernel that keeps scores, sums and accumulators in fp32 and
    rounds each softmax weight by `rounding` (relative) before the value product.

    A score is a sum of d products in fp32 scaled twice: off by at most (d + 4) 2^-24 of the sum
    of magnitudes; that and the exponential's 2^-21 (argument rounding included: |x - m| below
    2^5 where a weight matters) are relative errors of a weight, in numerator and divisor alike.
    Sums of up to `keys` fp32 terms add keys 2^-24.  O is rounded once to bf16 (2^-8)."""
    eps = 2 * ((d + 4) * 2.0 ** -24 * ref["ds"] + 2.0 ** -21) + ref["keys"][:, None] * 2.0 ** -23
    o = (2.0 ** -8 * np.abs(ref["o"]) + (1 + 2.0 ** -8) * (rounding + eps)[..., None] * ref["a"]
         # weights below f16's normal range: half its subnormal step, at codes of up to 448,
         # against a reference that lags the largest weight by 8 at most
         + (ref["keys"][:, None] * 2.0 ** -25 * 448 * ref["big"])[..., None] + 1e-30)
    lse = eps + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)))
    return o, lse


def check(got_o, got_lse, ref, d, rounding, what=""):
    """got_o [n,H,d], got_lse [n,H] against attend()'s answer."""
    bo, bl = bounds(ref, d, rounding)
    err = np.abs(got_o - ref["o"])
    assert np.isfinite(got_o).all(), f"{what}: non-finite O"
    assert (err <= bo).all(), f"{what}: O off by {(err / bo).max():.2f} of its bound, {err.max():.2e}"
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(ref["lse"])), f"{what}: -inf rows of LSE"
    fin = np.isfinite(ref["lse"])
    err = np.abs(got_lse[fin] - ref["lse"][fin])
    assert np.isfinite(got_lse[fin]).all()
    assert (err <= bl[fin]).all(), f"{what}: LSE off by {(err / bl[fin]).max():.2f} of its bound"


class Cache:
    """A page pool holding the sequences' rows k, v (lists of [L,Hkv,d] float64), every other
    slot NaN codes under an infinite scale; block-table entries past a sequence are -1."""

    def __init__(self, rng, k, v, extra=5, max_blocks=None):
        self.lens = np.array([len(x) for x in k], np.int32)
        self.Hkv, self.d = k[0].shape[1:]
        need = (self.lens + PAGE - 1) // PAGE
        self.num_pages = int(need.sum()) + extra
        width = max_blocks or max(1, int(need.max()))
        perm = rng.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((len(k), width), -1, np.int32)
        shape = (self.num_pages, self.Hkv, PAGE, self.d)
        self.codes = {x: np.full(shape, 0x7f, np.uint8) for x in "kv"}
        self.scales = {x: np.full(shape[:3], 255, np.uint8) for x in "kv"}
        self.rows = {"k": [], "v": []}     # what the cache stands for
        self.vexp = []
        at = 0
        for s, n in enumerate(need):
            ids = perm[at:at + n]
            at += n
            self.table[s, :n] = ids
            pos = np.arange(self.lens[s])
            for name, x in (("k", k[s]), ("v", v[s])):
                c, b = quantise(x)
                self.codes[name][ids[pos // PAGE], :, pos % PAGE] = c
                self.scales[name][ids[pos // PAGE], :, pos % PAGE] = b
                self.rows[name].append(values(c, b))
                if name == "v":
                    self.vexp.append(b.astype(float) - 127)

    def gpu(self):
        """(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens) on the GPU."""
        import torch
        t = [torch.from_numpy(self.codes[x]).cuda().view(torch.float8_e4m3fn) for x in "kv"]
        t += [torch.from_numpy(self.scales[x]).cuda() for x in "kv"]
        return t + [torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda()]


def bf16(x):
    """float64 -> (torch bf16 CPU tensor, its exact float64 values)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


def softmax_scale(d):
    return float(np.float32(1 / math.sqrt(d)))
