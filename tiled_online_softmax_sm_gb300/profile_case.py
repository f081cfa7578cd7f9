"""Run a few launches of one named workload on resident inputs, for profilers.

  python -m tiled_online_softmax_sm_gb300.profile_case fwd_c3 [--reps 2]

Workloads (sizes as in the bench and the parity tests):
  fwd_c3     causal bf16 forward, B=1 H=32 n=m=8192 d=128 (192 MB of inputs)
  fwd_c2     non-causal bf16 forward, B=4 H=16 n=m=2048 d=128
  fwd_c2c    causal bf16 forward, B=4 H=16 n=m=2048 d=128
  varlen_c5  ragged causal bf16 varlen forward, 16 sequences, d=128
  varlen_c5_d64  the same at d=64
  decode_c4  paged grouped-head decode, 64 sequences, H=32 Hkv=8, 8 splits (1.3 GB KV)
  fp8_c3     causal e4m3 forward, B=1 H=32 n=m=8192 d=128
  prefill_c4 paged prefill: 512-token chunks of 16 sequences of the decode pool
  fwd_f32    fp32 forward, n=m=256 d=64
  write_e4m3, read_e4m3  the decode pool's K/V rows into and out of an e4m3 paged cache
  decode_e4m3  paged grouped-head decode over it, 64 sequences, H=32 Hkv=8
  draft_e4m3   4 new tokens of 16 sequences over an e4m3 cache
  prefill_e4m3 512-token chunks of those sequences
  window_c3    causal bf16 forward, n=m=8192 H=32 d=128, window 1024 with 4 sinks
  tree_c4      attention of 16 drafted nodes of each of the decode pool's 64 sequences
  tree_e4m3    the same over an e4m3 cache
  tree_long    64 drafted nodes of 4 sequences of [16384, 65536] tokens
  tree_d64     64 drafted nodes of 16 sequences of [512, 8192] tokens, 24 heads of 8, d=64
  qkv_rows     q, k and v rows of 16 x 1024 new tokens: norms, rotation and cache write
  copy_pages   2048 pages of a bf16 cache (64 KB each with K and V) copied
Inputs come from the same seeded generators; nothing is checked here.
"""
from __future__ import annotations

import argparse
import sys

import numpy as np
import torch

from . import binding as fb
from . import inputs as I


def _dev(t):
    if t.dtype == "bf16":
        return torch.from_numpy(t.data.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(t.data).cuda()


def e4m3_cache(seed: int, S: int, Hkv: int = 8, d: int = 128):
    """Random K/V rows of S sequences of [512, 8192] tokens, an empty e4m3 paged cache with room for
    them (randomly ordered pages, table 512 wide), and the sequences' lengths and offsets."""
    g = torch.Generator(device="cuda").manual_seed(I.BASE_SEED)
    lens = I.uniform_lengths(seed, S, 512, 8192)
    need = (lens + 15) // 16
    pages, T = int(need.sum()), int(lens.sum())
    table = np.full((S, 512), -1, np.int32)
    ids = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    for s, at in enumerate(np.cumsum(need) - need):
        table[s, :need[s]] = ids[at:at + need[s]]
    k, v = (torch.randn((T, Hkv, d), device="cuda", generator=g).bfloat16() for _ in range(2))
    cache = [torch.zeros((pages, Hkv, 16, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.zeros((pages, Hkv, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda()]
    return k, v, cache, offsets(lens), lens


def offsets(n):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()


def bf16_cache(lens, Hkv: int = 8, d: int = 128, seed: int = I.BASE_SEED):
    """Random pages for sequences of these lengths, their table (randomly ordered pages) and lengths."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = (np.asarray(lens) + 15) // 16
    table = np.full((len(lens), int(need.max())), -1, np.int32)
    ids = np.random.default_rng(seed).permutation(int(need.sum())).astype(np.int32)
    for s, at in enumerate(np.cumsum(need) - need):
        table[s, :need[s]] = ids[at:at + need[s]]
    shape = (int(need.sum()), Hkv, 16, d)
    k, v = (torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16) for _ in range(2))
    return k, v, torch.from_numpy(table).cuda(), torch.from_numpy(np.asarray(lens, np.int32)).cuda()


def drafted(sl, n: int, H: int = 32, d: int = 128, seed: int = I.BASE_SEED):
    """Random trees of n nodes at the end of each sequence: q rows, offsets, ancestor bits, positions."""
    rng = np.random.default_rng(seed)
    S = len(sl)
    parents = np.concatenate([[rng.integers(-1, i) for i in range(n)] for _ in range(S)]).astype(np.int32)
    cu = offsets([n] * S)
    mask, pos = fb.tree_layout(torch.from_numpy(parents).cuda(), sl, cu, (n + 31) // 32)
    return torch.randn((S * n, H, d), device="cuda").bfloat16(), cu, mask, pos


def make(name: str, splits: int = 8):
    if name in ("fwd_c3", "fwd_c2", "fwd_c2c"):
        c = I.c3_bf16() if name == "fwd_c3" else I.c2_bf16(causal=name == "fwd_c2c")
        q, k, v = _dev(c.q), _dev(c.k), _dev(c.v)
        o = torch.empty((c.B, c.n, c.H, c.dv), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((c.B, c.H, c.n), dtype=torch.float32, device="cuda")
        return lambda: fb.fa_forward(q, k, v, o, lse, c.B, c.H, c.Hkv, c.n, c.m, c.d, c.dv,
                                     c.scale, int(c.causal))
    if name in ("varlen_c5", "varlen_c5_d64"):
        c = I.c5_varlen(64 if name.endswith("d64") else 128)
        q, k, v = _dev(c.q), _dev(c.k), _dev(c.v)
        cu = torch.from_numpy(c.cu_seqlens).cuda()
        T = int(c.cu_seqlens[-1])
        mx = int(c.lens.max())
        o = torch.empty((T, c.H, c.dv), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((c.H, T), dtype=torch.float32, device="cuda")
        return lambda: fb.fa_forward_varlen(q, k, v, o, lse, cu, cu, len(c.lens), T, T, mx, mx,
                                            c.H, c.Hkv, c.d, c.dv, c.scale, 1)
    if name == "decode_c4":
        c = I.c4_decode()
        q, kc, vc = _dev(c.q), _dev(c.k_cache), _dev(c.v_cache)
        bt = torch.from_numpy(c.block_table).cuda()
        sl = torch.from_numpy(c.seq_lens).cuda()
        S = len(c.seq_lens)
        need = fb.fa_paged_decode_workspace_size(S, c.H, c.dv, splits)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        o = torch.empty((S, c.H, c.dv), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((S, c.H), dtype=torch.float32, device="cuda")
        return lambda: fb.fa_paged_decode(q, kc, vc, bt, sl, o, lse, S, c.H, c.Hkv, c.d, c.dv,
                                          c.page_size, c.num_pages, c.max_blocks, splits, c.scale,
                                          ws, need)
    if name == "fp8_c3":
        g = I.rng(I.BASE_SEED, 3)
        ts = [I.Tensor.from_f32(I.normal_f32(g, (1, 8192, 32, 128)), "e4m3") for _ in range(3)]
        q, k, v = (torch.from_numpy(t.data).cuda() for t in ts)
        o = torch.empty((1, 8192, 32, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((1, 32, 8192), dtype=torch.float32, device="cuda")
        sc = I.fp32_scale(128)
        return lambda: fb.fa_forward_fp8(q, k, v, o, lse, 1, 32, 32, 8192, 8192, 128, 128, sc,
                                         ts[0].descale, ts[1].descale, ts[2].descale, 1)
    if name == "prefill_c4":
        lens = I.uniform_lengths(63, 16, 512, 8192)
        ql = np.minimum(lens, 512)
        kv = I.decode_case(63, num_seqs=16, H=32, Hkv=8, d=128, lens=lens, max_blocks=512)
        cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
        T = int(cu[-1])
        q = _dev(I.Tensor.from_f32(I.normal_f32(I.rng(63, 51), (T, 32, 128)), "bf16"))
        kc, vc = _dev(kv.k_cache), _dev(kv.v_cache)
        bt = torch.from_numpy(kv.block_table).cuda()
        sl = torch.from_numpy(kv.seq_lens).cuda()
        cut = torch.from_numpy(cu).cuda()
        o = torch.empty((T, 32, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((32, T), dtype=torch.float32, device="cuda")
        return lambda: fb.fa_paged_prefill(q, kc, vc, bt, sl, cut, o, lse, 16, T, 512, 32, 8, 128,
                                           128, 16, kv.num_pages, 512, kv.scale, 1)
    if name == "fwd_f32":
        c = I.c1_fp32()
        q, k, v = _dev(c.q), _dev(c.k), _dev(c.v)
        o = torch.empty((c.B, c.n, c.H, c.dv), dtype=torch.float32, device="cuda")
        lse = torch.empty((c.B, c.H, c.n), dtype=torch.float32, device="cuda")
        return lambda: fb.fa_forward_f32(q, k, v, o, lse, c.B, c.H, c.Hkv, c.n, c.m, c.d, c.dv,
                                         c.scale, 0)
    if name in ("write_e4m3", "read_e4m3", "decode_e4m3", "draft_e4m3", "prefill_e4m3"):
        S, seed, n = {"draft_e4m3": (16, 63, 4), "prefill_e4m3": (16, 63, 512)}.get(
            name, (64, I.BASE_SEED, 1))
        k, v, cache, cu, lens = e4m3_cache(seed, S)
        write = lambda: fb.paged_kv_write_e4m3(k, v, *cache, cu)  # noqa: E731
        write()
        nq = np.minimum(lens, n)
        q = torch.randn((int(nq.sum()), 32, 128), device="cuda").bfloat16()
        sc, cuq = I.fp32_scale(128), offsets(nq)
        return {"write_e4m3": write,
                "read_e4m3": lambda: fb.paged_kv_read_e4m3(*cache, cu, int(lens.sum())),
                "decode_e4m3": lambda: fb.paged_decode_e4m3(q, *cache, sc)}.get(
                    name, lambda: fb.paged_prefill_e4m3(q, *cache, cuq, n, sc))
    if name == "window_c3":
        q, k, v = (torch.randn((1, 8192, 32, 128), device="cuda").bfloat16() for _ in range(3))
        return lambda: fb.forward_window(q, k, v, I.fp32_scale(128), 1024, 4)
    if name in ("tree_c4", "tree_long", "tree_d64"):
        S, n, at, H, d = {"tree_c4": (64, 16, (512, 8192), 32, 128), "tree_long": (4, 64, (16384, 65536), 32, 128),
                          "tree_d64": (16, 64, (512, 8192), 24, 64)}[name]
        cache = bf16_cache(I.uniform_lengths(I.BASE_SEED, S, *at), d=d)
        q, cu, mask, _ = drafted(cache[3], n, H, d)
        return lambda: fb.paged_tree_attention(q, *cache, cu, n, mask, I.fp32_scale(d))
    if name == "tree_e4m3":
        k, v, cache, cu, _ = e4m3_cache(I.BASE_SEED, 64)
        fb.paged_kv_write_e4m3(k, v, *cache, cu)
        q, cu, mask, _ = drafted(cache[5], 16)
        return lambda: fb.paged_tree_attention_e4m3(q, *cache, cu, 16, mask, I.fp32_scale(128))
    if name == "qkv_rows":
        lens = np.full(16, 1024)
        k_cache, v_cache, bt, sl = bf16_cache(lens)
        T, cu = int(lens.sum()), offsets(lens)
        q, k, v = (torch.randn((T, h, 128), device="cuda").bfloat16() for h in (32, 8, 8))
        wq, wk = (torch.ones(128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        angles = torch.arange(1024, device="cuda")[:, None] / 10000.0 ** (torch.arange(64, device="cuda") / 64)
        cos_sin = torch.stack([angles.cos(), angles.sin()], -1).float().contiguous()
        pos = torch.arange(1024, dtype=torch.int32, device="cuda").repeat(16)[None].contiguous()
        return lambda: fb.paged_qkv_write(q, k, v, wq, wk, cos_sin, pos, k_cache, v_cache, bt, sl, cu)
    if name == "copy_pages":
        k_cache, v_cache = bf16_cache([16 * 4096])[:2]
        ids = np.random.default_rng(I.BASE_SEED).permutation(4096).astype(np.int32).reshape(2048, 2)
        pairs = torch.from_numpy(ids).cuda()
        return lambda: fb.paged_copy_pages(k_cache, v_cache, pairs)
    raise SystemExit(f"unknown workload {name}")


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("workload")
    ap.add_argument("--reps", type=int, default=2)
    ap.add_argument("--splits", type=int, default=8)
    a = ap.parse_args(argv)
    fn = make(a.workload, a.splits)
    for _ in range(a.reps):
        fn()
    torch.cuda.synchronize()
    st = fb.fa_get_device_status()
    print(f"{a.workload}: {a.reps} launches, device status {st}")
    return 0 if st == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
