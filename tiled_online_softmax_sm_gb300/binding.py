"""ctypes binding of libfa_gb300.so (the C ABI of include/fa.h).

Argument marshalling only: every function here converts its arguments to
pointers and ints and calls the entry point of the same name; all the
arithmetic runs in the library's CUDA kernels.  Pointer arguments may be torch
tensors (their data_ptr is passed), plain ints, or None.  A non-zero status
raises FaError with the library's message.  There is no fallback: if the
library is missing or cannot be loaded, the first call raises.

The helpers at the end (``forward``, ``forward_f32``, ``forward_varlen``,
``paged_decode``, ``paged_decode_fused``, the e4m3 cache's ``paged_..._e4m3``,
``split_combine``) allocate outputs with torch and then call the same entry
points.  Only they and a call's default stream import torch: the entry points
themselves, with plain addresses and a given stream, do without it.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
# FA_LIBRARY selects another build of the same ABI (the debug build,
# libfa_gb300_debug.so, for instance); by default the in-tree library.
LIB_PATH = os.environ.get("FA_LIBRARY") or os.path.join(HERE, "libfa_gb300.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_WORKSPACE = 3
FA_ERR_CUDA = 4
FA_ERR_TIMEOUT = 5
FA_ERR_BAD_BLOCK_TABLE = 6
FA_ERR_DEBUG_CHECK = 7

EXPORTED = ("fa_forward", "fa_forward_fp8", "fa_forward_f32", "fa_forward_varlen", "fa_paged_prefill",
            "fa_paged_decode_workspace_size",
            "fa_paged_decode", "fa_paged_decode_fused", "fa_paged_decode_noalloc", "fa_paged_gather", "fa_split_combine",
            "fa_forward_window", "fa_forward_varlen_window",
            "fa_paged_kv_write_e4m3", "fa_paged_kv_read_e4m3", "fa_paged_e4m3_workspace_size",
            "fa_paged_e4m3_workspace_used", "fa_paged_decode_e4m3", "fa_paged_prefill_e4m3",
            "fa_last_error",
            "fa_get_device_status")
FA_NOALLOC_SCRATCH_BYTES = 16 << 20


class FaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"fa status {status}: {message}")
        self.status = status


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load the library (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise FaError(FA_ERR_UNSUPPORTED,
                          f"{path} is missing: build it with tiled_online_softmax_sm_gb300.build")
        lib = ctypes.CDLL(path)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_forward.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, I, P]
        lib.fa_forward_f32.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, I, P]
        lib.fa_forward_fp8.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, F, F, F, I, P]
        lib.fa_forward_varlen.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P]
        lib.fa_forward_window.argtypes = [P] * 5 + [I, I, I, I, I, I, I, F, I, I, P]
        lib.fa_forward_varlen_window.argtypes = [P] * 7 + [I] * 9 + [F, I, I, P]
        lib.fa_paged_prefill.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, I, P]
        lib.fa_paged_decode_workspace_size.argtypes = [I, I, I, I]
        lib.fa_paged_decode_workspace_size.restype = Z
        lib.fa_paged_decode.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P, Z, P]
        lib.fa_paged_decode_fused.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P, Z, P]
        lib.fa_paged_decode_noalloc.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P]
        lib.fa_paged_gather.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, P]
        lib.fa_split_combine.argtypes = [P, P, P, P, P, I, I, I, I, P]
        LL = ctypes.c_longlong
        lib.fa_paged_kv_write_e4m3.argtypes = [P] * 9 + [I, I, I, I, LL, LL, I, I, I, P]
        lib.fa_paged_kv_read_e4m3.argtypes = [P] * 9 + [I, I, I, I, I, I, I, P]
        lib.fa_paged_decode_e4m3.argtypes = [P] * 9 + [I, I, I, I, I, I, I, F, I, I, P, Z, P]
        lib.fa_paged_prefill_e4m3.argtypes = [P] * 10 + [I, I, I, I, I, I, I, I, I, F, I, I, I, P, Z, P]
        lib.fa_paged_e4m3_workspace_size.argtypes = [I] * 5
        lib.fa_paged_e4m3_workspace_size.restype = Z
        lib.fa_paged_e4m3_workspace_used.argtypes = [I] * 9
        lib.fa_paged_e4m3_workspace_used.restype = Z
        lib.fa_last_error.argtypes = []
        lib.fa_last_error.restype = ctypes.c_char_p
        lib.fa_get_device_status.argtypes = [P, ctypes.POINTER(I)]
        for name in ("fa_forward", "fa_forward_fp8", "fa_forward_f32", "fa_forward_varlen",
                     "fa_paged_prefill",
                     "fa_paged_decode", "fa_paged_decode_fused",
                     "fa_paged_decode_noalloc", "fa_paged_gather", "fa_split_combine",
                     "fa_forward_window", "fa_forward_varlen_window",
                     "fa_paged_kv_write_e4m3", "fa_paged_kv_read_e4m3", "fa_paged_decode_e4m3",
                     "fa_paged_prefill_e4m3", "fa_get_device_status"):
            getattr(lib, name).restype = I
        _lib = lib
        return lib


def _p(x):
    """Pointer of a tensor / int / None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        # the handle alone: building a Stream object takes 3 us
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class _Torch:
    """Stands for torch until its first use, which imports it."""

    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _Torch()

# Set by _bind_torch, before the e4m3 helpers' first check: the current stream of a device that is
# known to be the current one, the current device once there are tensors on one, and the types of
# the e4m3 cache's codes and scales.
_current_raw_stream = _current_device = _CODES = _SCALES = None


def _bind_torch():
    global _current_raw_stream, _current_device, _CODES, _SCALES
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _SCALES = frozenset((torch.uint8, torch.int8) +
                        ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ()))
    _CODES = frozenset((torch.float8_e4m3fn, torch.uint8, torch.int8))


def _check(rc: int):
    if rc != FA_OK:
        msg = load().fa_last_error()
        raise FaError(rc, msg.decode() if msg else "")


# ------------------------------------------------------------ C entry points
def fa_forward(q, k, v, o, lse, B, H, Hkv, n, m, d, dv, scale, causal, stream=None):
    _check(load().fa_forward(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, Hkv, n, m, d, dv,
                             float(scale), int(causal), _stream(stream)))


def fa_forward_fp8(q, k, v, o, lse, B, H, Hkv, n, m, d, dv, scale, q_descale, k_descale,
                   v_descale, causal, stream=None):
    _check(load().fa_forward_fp8(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, Hkv, n, m, d, dv,
                                 float(scale), float(q_descale), float(k_descale),
                                 float(v_descale), int(causal), _stream(stream)))


def fa_forward_f32(q, k, v, o, lse, B, H, Hkv, n, m, d, dv, scale, causal, stream=None):
    _check(load().fa_forward_f32(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, Hkv, n, m, d, dv,
                                 float(scale), int(causal), _stream(stream)))


def fa_forward_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                      max_seqlen_q, max_seqlen_k, H, Hkv, d, dv, scale, causal, stream=None):
    _check(load().fa_forward_varlen(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_seqlens_q),
                                    _p(cu_seqlens_k), num_seqs, total_q, total_k, max_seqlen_q,
                                    max_seqlen_k, H, Hkv, d, dv, float(scale), int(causal),
                                    _stream(stream)))


def fa_forward_window(q, k, v, o, lse, B, H, Hkv, n, m, d, dv, scale, window, sinks=0,
                      stream=None):
    _check(load().fa_forward_window(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, Hkv, n, m, d, dv,
                                    float(scale), int(window), int(sinks), _stream(stream)))


def fa_forward_varlen_window(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q,
                             total_k, max_seqlen_q, max_seqlen_k, H, Hkv, d, dv, scale, window,
                             sinks=0, stream=None):
    _check(load().fa_forward_varlen_window(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_seqlens_q),
                                           _p(cu_seqlens_k), num_seqs, total_q, total_k,
                                           max_seqlen_q, max_seqlen_k, H, Hkv, d, dv, float(scale),
                                           int(window), int(sinks), _stream(stream)))


def fa_paged_prefill(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, o, lse, num_seqs,
                     total_q, max_seqlen_q, H, Hkv, d, dv, page_size, num_pages,
                     max_blocks_per_seq, scale, causal, stream=None):
    _check(load().fa_paged_prefill(_p(q), _p(k_cache), _p(v_cache), _p(block_table), _p(seq_lens),
                                   _p(cu_seqlens_q), _p(o), _p(lse), num_seqs, total_q,
                                   max_seqlen_q, H, Hkv, d, dv, page_size, num_pages,
                                   max_blocks_per_seq, float(scale), int(causal), _stream(stream)))


def fa_paged_decode_workspace_size(num_seqs, H, dv, num_splits) -> int:
    return int(load().fa_paged_decode_workspace_size(num_seqs, H, dv, num_splits))


def fa_paged_decode(q, k_cache, v_cache, block_table, seq_lens, o, lse, num_seqs, H, Hkv, d, dv,
                    page_size, num_pages, max_blocks_per_seq, num_splits, scale, workspace,
                    workspace_bytes, stream=None):
    _check(load().fa_paged_decode(_p(q), _p(k_cache), _p(v_cache), _p(block_table), _p(seq_lens),
                                  _p(o), _p(lse), num_seqs, H, Hkv, d, dv, page_size, num_pages,
                                  max_blocks_per_seq, num_splits, float(scale), _p(workspace),
                                  int(workspace_bytes), _stream(stream)))


def fa_paged_decode_fused(q, k_cache, v_cache, block_table, seq_lens, o, lse, num_seqs, H, Hkv, d,
                          dv, page_size, num_pages, max_blocks_per_seq, num_splits, scale,
                          workspace, workspace_bytes, stream=None):
    _check(load().fa_paged_decode_fused(_p(q), _p(k_cache), _p(v_cache), _p(block_table),
                                        _p(seq_lens), _p(o), _p(lse), num_seqs, H, Hkv, d, dv,
                                        page_size, num_pages, max_blocks_per_seq, num_splits,
                                        float(scale), _p(workspace), int(workspace_bytes),
                                        _stream(stream)))


def fa_paged_decode_noalloc(q, k_cache, v_cache, block_table, seq_lens, o, lse, num_seqs, H, Hkv,
                            d, dv, page_size, num_pages, max_blocks_per_seq, num_splits, scale,
                            stream=None):
    """fa_paged_decode without a workspace: for callers that may not allocate
    device memory themselves.  The split partials live in the library's own
    fixed device array (FA_NOALLOC_SCRATCH_BYTES); calls share it, so calls
    that overlap on the GPU must not be issued."""
    _check(load().fa_paged_decode_noalloc(_p(q), _p(k_cache), _p(v_cache), _p(block_table),
                                          _p(seq_lens), _p(o), _p(lse), num_seqs, H, Hkv, d, dv,
                                          page_size, num_pages, max_blocks_per_seq, num_splits,
                                          float(scale), _stream(stream)))


def fa_paged_gather(k_cache, v_cache, block_table, seq_lens, k_out, v_out, num_seqs, Hkv, d,
                    page_size, num_pages, max_blocks_per_seq, num_splits, stream=None):
    _check(load().fa_paged_gather(_p(k_cache), _p(v_cache), _p(block_table), _p(seq_lens),
                                  _p(k_out), _p(v_out), num_seqs, Hkv, d, page_size, num_pages,
                                  max_blocks_per_seq, num_splits, _stream(stream)))


def fa_paged_kv_write_e4m3(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                           cu_seqlens, num_seqs, total, Hkv, d, k_stride, v_stride, page_size,
                           num_pages, max_blocks_per_seq, stream=None):
    _check(load().fa_paged_kv_write_e4m3(_p(k), _p(v), _p(k_cache), _p(v_cache), _p(k_scale),
                                         _p(v_scale), _p(block_table), _p(seq_lens),
                                         _p(cu_seqlens), num_seqs, total, Hkv, d, k_stride,
                                         v_stride, page_size, num_pages, max_blocks_per_seq,
                                         _stream(stream)))


def fa_paged_kv_read_e4m3(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens,
                          k, v, num_seqs, total, Hkv, d, page_size, num_pages,
                          max_blocks_per_seq, stream=None):
    _check(load().fa_paged_kv_read_e4m3(_p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale),
                                        _p(block_table), _p(seq_lens), _p(cu_seqlens), _p(k),
                                        _p(v), num_seqs, total, Hkv, d, page_size, num_pages,
                                        max_blocks_per_seq, _stream(stream)))


def fa_paged_e4m3_workspace_size(num_seqs, max_seqlen_q, H, Hkv, d) -> int:
    return int(load().fa_paged_e4m3_workspace_size(num_seqs, max_seqlen_q, H, Hkv, d))


def fa_paged_e4m3_workspace_used(num_seqs, max_seqlen_q, H, Hkv, d, max_blocks_per_seq, causal=True,
                                 window=0, sinks=0) -> int:
    return int(load().fa_paged_e4m3_workspace_used(num_seqs, max_seqlen_q, H, Hkv, d,
                                                   max_blocks_per_seq, int(causal), int(window),
                                                   int(sinks)))


def fa_paged_decode_e4m3(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, o, lse,
                         num_seqs, H, Hkv, d, page_size, num_pages, max_blocks_per_seq, scale,
                         window=0, sinks=0, workspace=None, workspace_bytes=0, stream=None):
    _check(load().fa_paged_decode_e4m3(_p(q), _p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale),
                                       _p(block_table), _p(seq_lens), _p(o), _p(lse), num_seqs, H,
                                       Hkv, d, page_size, num_pages, max_blocks_per_seq,
                                       float(scale), int(window), int(sinks), _p(workspace),
                                       int(workspace_bytes), _stream(stream)))


def fa_paged_prefill_e4m3(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                          cu_seqlens_q, o, lse, num_seqs, total_q, max_seqlen_q, H, Hkv, d,
                          page_size, num_pages, max_blocks_per_seq, scale, causal=True, window=0,
                          sinks=0, workspace=None, workspace_bytes=0, stream=None):
    _check(load().fa_paged_prefill_e4m3(_p(q), _p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale),
                                        _p(block_table), _p(seq_lens), _p(cu_seqlens_q), _p(o),
                                        _p(lse), num_seqs, total_q, max_seqlen_q, H, Hkv, d,
                                        page_size, num_pages, max_blocks_per_seq, float(scale),
                                        int(causal), int(window), int(sinks), _p(workspace),
                                        int(workspace_bytes), _stream(stream)))


def fa_split_combine(part_m, part_l, part_o, o, lse, num_seqs, H, num_splits, dv, stream=None):
    _check(load().fa_split_combine(_p(part_m), _p(part_l), _p(part_o), _p(o), _p(lse), num_seqs, H,
                                   num_splits, dv, _stream(stream)))


def fa_get_device_status(stream=None) -> int:
    st = ctypes.c_int(0)
    _check(load().fa_get_device_status(_stream(stream), ctypes.byref(st)))
    return st.value


def fa_last_error() -> str:
    msg = load().fa_last_error()
    return msg.decode() if msg else ""


# ------------------------------------------------ torch-allocating helpers
def _given(stream):
    """Makes a given stream (a torch stream, or a handle) torch's current one, for the helpers of the
    windowed forward and of the e4m3 cache: outputs and workspace then belong to it, and a block that
    torch gets back from another stream's work is not given out to this one's before that is done."""
    raw = _stream(stream)
    if isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(raw) if raw else torch.cuda.default_stream())


def forward(q, k, v, scale, causal=False, stream=None):
    """q [B,n,H,d], k [B,m,Hkv,d], v [B,m,Hkv,dv] bf16 CUDA tensors -> (o bf16, lse fp32 [B,H,n])."""
    B, n, H, d = q.shape
    _, m, Hkv, dv = v.shape
    o = torch.empty((B, n, H, dv), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, H, n), dtype=torch.float32, device=q.device)
    fa_forward(q, k, v, o, lse, B, H, Hkv, n, m, d, dv, scale, causal, stream)
    return o, lse


def forward_fp8(q, k, v, scale, q_descale, k_descale, v_descale, causal=False, stream=None):
    """e4m3 q [B,n,H,d], k/v [B,m,Hkv,d] (uint8 or float8 tensors) -> (o bf16, lse fp32)."""
    B, n, H, d = q.shape
    _, m, Hkv, dv = v.shape
    o = torch.empty((B, n, H, dv), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, H, n), dtype=torch.float32, device=q.device)
    fa_forward_fp8(q, k, v, o, lse, B, H, Hkv, n, m, d, dv, scale, q_descale, k_descale, v_descale,
                   causal, stream)
    return o, lse


def forward_f32(q, k, v, scale, causal=False, stream=None):
    B, n, H, d = q.shape
    _, m, Hkv, dv = v.shape
    o = torch.empty((B, n, H, dv), dtype=torch.float32, device=q.device)
    lse = torch.empty((B, H, n), dtype=torch.float32, device=q.device)
    fa_forward_f32(q, k, v, o, lse, B, H, Hkv, n, m, d, dv, scale, causal, stream)
    return o, lse


def forward_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale,
                   causal=True, stream=None):
    """Packed q [Tq,H,d], k/v [Tk,Hkv,d] -> (o [Tq,H,dv] bf16, lse [H,Tq] fp32)."""
    Tq, H, d = q.shape
    Tk, Hkv, dv = v.shape
    S = cu_seqlens_q.shape[0] - 1
    o = torch.empty((Tq, H, dv), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((H, Tq), dtype=torch.float32, device=q.device)
    fa_forward_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, S, Tq, Tk, max_seqlen_q,
                      max_seqlen_k, H, Hkv, d, dv, scale, causal, stream)
    return o, lse


def forward_window(q, k, v, scale, window, sinks=0, stream=None):
    """q [B,n,H,d], k/v [B,m,Hkv,d] bf16, causal under a sliding window with sinks
    -> (o [B,n,H,d] bf16, lse [B,H,n] fp32)."""
    if stream is not None:
        with _given(stream):
            return forward_window(q, k, v, scale, window, sinks)
    B, n, H, d = q.shape
    m, Hkv = k.shape[1:3]
    _check_tensors("forward_window", q.get_device(), ("q", q, torch.bfloat16, (B, n, H, d)),
             ("k", k, torch.bfloat16, (B, m, Hkv, d)), ("v", v, torch.bfloat16, (B, m, Hkv, d)))
    o = torch.empty_like(q)
    lse = torch.empty((B, H, n), dtype=torch.float32, device=q.device)
    fa_forward_window(q, k, v, o, lse, B, H, Hkv, n, m, d, d, scale, window, sinks)
    return o, lse


def forward_varlen_window(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale,
                          window, sinks=0, stream=None):
    """Packed q [Tq,H,d], k/v [Tk,Hkv,d] bf16, causal under a sliding window with sinks
    -> (o [Tq,H,d] bf16, lse [H,Tq] fp32)."""
    if stream is not None:
        with _given(stream):
            return forward_varlen_window(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                                         max_seqlen_k, scale, window, sinks)
    Tq, H, d = q.shape
    Tk, Hkv = k.shape[:2]
    S = cu_seqlens_q.shape[0] - 1
    _check_tensors("forward_varlen_window", q.get_device(), ("q", q, torch.bfloat16, (Tq, H, d)),
             ("k", k, torch.bfloat16, (Tk, Hkv, d)), ("v", v, torch.bfloat16, (Tk, Hkv, d)),
             ("cu_seqlens_q", cu_seqlens_q, torch.int32, (S + 1,)),
             ("cu_seqlens_k", cu_seqlens_k, torch.int32, (S + 1,)))
    o = torch.empty_like(q)
    lse = torch.empty((H, Tq), dtype=torch.float32, device=q.device)
    fa_forward_varlen_window(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, S, Tq, Tk, max_seqlen_q,
                             max_seqlen_k, H, Hkv, d, d, scale, window, sinks)
    return o, lse


def paged_prefill(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q, scale,
                  causal=True, stream=None):
    """q [Tq,H,d] packed by cu_seqlens_q; caches [P,Hkv,page,d] -> (o [Tq,H,dv], lse [H,Tq])."""
    Tq, H, d = q.shape
    P, Hkv, page, dv = v_cache.shape
    S = cu_seqlens_q.shape[0] - 1
    o = torch.empty((Tq, H, dv), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((H, Tq), dtype=torch.float32, device=q.device)
    fa_paged_prefill(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, o, lse, S, Tq,
                     max_seqlen_q, H, Hkv, d, dv, page, P, block_table.shape[1], scale, causal,
                     stream)
    return o, lse


def paged_decode(q, k_cache, v_cache, block_table, seq_lens, num_splits, scale, workspace=None,
                 stream=None):
    """q [S,H,d]; caches [P,Hkv,page,d]; block_table [S,max_blocks] int32; seq_lens [S] int32."""
    S, H, d = q.shape
    P, Hkv, page, dv = v_cache.shape
    need = fa_paged_decode_workspace_size(S, H, dv, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    o = torch.empty((S, H, dv), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((S, H), dtype=torch.float32, device=q.device)
    fa_paged_decode(q, k_cache, v_cache, block_table, seq_lens, o, lse, S, H, Hkv, d, dv, page, P,
                    block_table.shape[1], num_splits, scale, workspace, workspace.numel(), stream)
    return o, lse


def paged_decode_fused(q, k_cache, v_cache, block_table, seq_lens, num_splits, scale,
                       workspace=None, stream=None):
    """As paged_decode, in one launch; a workspace passed in must have had its
    ticket words zeroed once (a new one is zeroed here)."""
    S, H, d = q.shape
    P, Hkv, page, dv = v_cache.shape
    need = fa_paged_decode_workspace_size(S, H, dv, num_splits)
    if workspace is None:
        workspace = torch.zeros(max(need, 1), dtype=torch.uint8, device=q.device)
    o = torch.empty((S, H, dv), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((S, H), dtype=torch.float32, device=q.device)
    fa_paged_decode_fused(q, k_cache, v_cache, block_table, seq_lens, o, lse, S, H, Hkv, d, dv,
                          page, P, block_table.shape[1], num_splits, scale, workspace,
                          workspace.numel(), stream)
    return o, lse


def _refuse(fn, device, *named):
    """Raise for the first of (name, tensor, types, shape) that is not a contiguous tensor of one of
    those types and that shape on the current CUDA device: the C entry sees only its address."""
    current = torch.cuda.current_device()
    if device != current:
        raise FaError(FA_ERR_INVALID_ARG, f"{fn}: the tensors are on device {device}, the current "
                                          f"one is {current}")
    for name, t, kinds, shape in named:
        if t.get_device() != device:
            raise FaError(FA_ERR_INVALID_ARG, f"{fn}: {name} is on {t.device}, not cuda:{device}")
        if t.dtype not in kinds:
            raise FaError(FA_ERR_INVALID_ARG, f"{fn}: {name} has type {t.dtype}")
        if t.shape != shape or not t.is_contiguous():
            raise FaError(FA_ERR_INVALID_ARG, f"{fn}: {name} has shape {tuple(t.shape)} and strides "
                                              f"{t.stride()}, wanted contiguous {tuple(shape)}")
    raise FaError(FA_ERR_INVALID_ARG, f"{fn}: tensors do not fit together")


def _check_tensors(fn, device, *named):
    """As _refuse, for good tensors too: (name, tensor, type, shape)."""
    ok = device == torch.cuda.current_device()
    for _, t, kind, shape in named:
        ok = ok and t.dtype is kind and t.shape == shape and t.get_device() == device and \
            t.is_contiguous()
    if not ok:
        _refuse(fn, device, *((name, t, (kind,), shape) for name, t, kind, shape in named))


def _check_cache(fn, device, kc, vc, ks, vs, bt, sl):
    """The paged e4m3 cache's tensors: code and scale caches, block table and lengths.  (Written
    out: it runs on every call of the serving path, where a loop over them takes twice as long.)"""
    if _CODES is None:
        _bind_torch()
    shape, table = kc.shape, bt.shape
    if len(shape) != 4 or len(table) != 2:
        raise FaError(FA_ERR_INVALID_ARG, f"{fn}: k_cache has shape {tuple(shape)}, block_table "
                                          f"{tuple(table)}, wanted 4 and 2 dimensions")
    rows = shape[:3]
    if not (kc.dtype in _CODES and vc.dtype in _CODES and ks.dtype in _SCALES and vs.dtype in _SCALES
            and bt.dtype is torch.int32 and sl.dtype is torch.int32 and vc.shape == shape
            and ks.shape == rows and vs.shape == rows and sl.shape == table[:1]
            and kc.get_device() == device and vc.get_device() == device and ks.get_device() == device
            and vs.get_device() == device and bt.get_device() == device and sl.get_device() == device
            and kc.is_contiguous() and vc.is_contiguous() and ks.is_contiguous()
            and vs.is_contiguous() and bt.is_contiguous() and sl.is_contiguous()
            and device >= 0 and device == _current_device()):
        _refuse(fn, device, ("k_cache", kc, _CODES, shape), ("v_cache", vc, _CODES, shape),
                ("k_scale", ks, _SCALES, rows), ("v_scale", vs, _SCALES, rows),
                ("block_table", bt, (torch.int32,), table),
                ("seq_lens", sl, (torch.int32,), table[:1]))


def _check_rows(fn, device, name, t, kind, shape):
    if not (t.dtype is kind and t.shape == shape and t.get_device() == device and t.is_contiguous()):
        _refuse(fn, device, (name, t, (kind,), shape))


def paged_kv_write_e4m3(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                        cu_seqlens, stream=None):
    """Quantise new rows k, v [T,Hkv,d] bf16 (token strides may be larger than Hkv*d) into the
    cache [P,Hkv,16,d] (float8_e4m3fn, uint8 or int8) and its scale bytes [P,Hkv,16]."""
    fn = "paged_kv_write_e4m3"
    device = k.get_device()
    _check_cache(fn, device, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens)
    P, Hkv, page, d = k_cache.shape
    S, max_blocks = block_table.shape
    _check_rows(fn, device, "cu_seqlens", cu_seqlens, torch.int32, (S + 1,))
    T = k.shape[0]
    strides = []
    for name, t in (("k", k), ("v", v)):
        st = t.stride()
        if t.shape != (T, Hkv, d) or st[2] != 1 or (Hkv > 1 and st[1] != d) or \
                t.dtype is not torch.bfloat16 or t.get_device() != device:
            raise FaError(FA_ERR_INVALID_ARG, f"{fn}: {name} is {t.dtype} on {t.device} of shape "
                                              f"{tuple(t.shape)} and strides {st}, wanted bf16 "
                                              f"{(T, Hkv, d)} with dense heads")
        strides.append(st[0] if T > 1 else Hkv * d)
    lib = _lib or load()
    _check(lib.fa_paged_kv_write_e4m3(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens.data_ptr(), S,
        T, Hkv, d, strides[0], strides[1], page, P, max_blocks,
        _current_raw_stream(device) if stream is None else _stream(stream)))


def paged_kv_read_e4m3(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens,
                       total, stream=None):
    """The last n_s cached rows of every sequence -> (k, v) [total,Hkv,d] bf16."""
    if stream is not None:
        with _given(stream):
            return paged_kv_read_e4m3(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                      cu_seqlens, total)
    fn = "paged_kv_read_e4m3"
    device = k_cache.get_device()
    _check_cache(fn, device, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens)
    P, Hkv, page, d = k_cache.shape
    S, max_blocks = block_table.shape
    _check_rows(fn, device, "cu_seqlens", cu_seqlens, torch.int32, (S + 1,))
    k = torch.empty((total, Hkv, d), dtype=torch.bfloat16, device=k_cache.device)
    v = torch.empty_like(k)
    lib = _lib or load()
    _check(lib.fa_paged_kv_read_e4m3(
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens.data_ptr(), k.data_ptr(),
        v.data_ptr(), S, total, Hkv, d, page, P, max_blocks, _current_raw_stream(device)))
    return k, v


@functools.lru_cache(maxsize=4096)
def _e4m3_workspace_used(*sizes):
    """fa_paged_e4m3_workspace_used, which depends on the sizes alone (asked for every call of the
    serving path, where the C call would take 1 us each time)."""
    return int(load().fa_paged_e4m3_workspace_used(*sizes))


def _e4m3_workspace(fn, workspace, q, S, max_q, H, Hkv, d, max_blocks, causal, window, sinks):
    """Address and bytes of the caller's workspace, of a new one where the call uses it, or of none;
    and the tensor, to be kept until the call is queued."""
    if workspace is None:
        need = _e4m3_workspace_used(S, int(max_q), H, Hkv, d, max_blocks, causal, int(window),
                                    int(sinks))
        if not need:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != q.get_device() or not workspace.is_contiguous():
        raise FaError(FA_ERR_WORKSPACE, f"{fn}: the workspace is on {workspace.device} with strides "
                                        f"{workspace.stride()}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def paged_decode_e4m3(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale,
                      window=0, sinks=0, workspace=None, stream=None):
    """q [S,H,d]; e4m3 cache [P,Hkv,16,d] with scale bytes [P,Hkv,16] -> (o [S,H,d], lse [S,H])."""
    if stream is not None:
        with _given(stream):
            return paged_decode_e4m3(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                     scale, window, sinks, workspace)
    fn = "paged_decode_e4m3"
    device = q.get_device()
    _check_cache(fn, device, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens)
    P, Hkv, page, d = k_cache.shape
    S, max_blocks = block_table.shape
    H = q.shape[1]
    _check_rows(fn, device, "q", q, torch.bfloat16, (S, H, d))
    o = torch.empty_like(q)
    lse = torch.empty((S, H), dtype=torch.float32, device=q.device)
    ws, ws_bytes, keep = _e4m3_workspace(fn, workspace, q, S, 1, H, Hkv, d, max_blocks, 1, window,
                                         sinks)
    lib = _lib or load()
    _check(lib.fa_paged_decode_e4m3(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
        lse.data_ptr(), S, H, Hkv, d, page, P, max_blocks, scale, window, sinks, ws, ws_bytes,
        _current_raw_stream(device)))
    return o, lse


def paged_prefill_e4m3(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens_q,
                       max_seqlen_q, scale, causal=True, window=0, sinks=0, workspace=None,
                       stream=None):
    """q [Tq,H,d] packed by cu_seqlens_q over the e4m3 cache -> (o [Tq,H,d], lse [H,Tq]).
    max_seqlen_q may be any upper bound of the sequences' query counts."""
    if stream is not None:
        with _given(stream):
            return paged_prefill_e4m3(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                      cu_seqlens_q, max_seqlen_q, scale, causal, window, sinks,
                                      workspace)
    fn = "paged_prefill_e4m3"
    device = q.get_device()
    _check_cache(fn, device, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens)
    P, Hkv, page, d = k_cache.shape
    S, max_blocks = block_table.shape
    Tq, H = q.shape[:2]
    _check_rows(fn, device, "q", q, torch.bfloat16, (Tq, H, d))
    _check_rows(fn, device, "cu_seqlens_q", cu_seqlens_q, torch.int32, (S + 1,))
    o = torch.empty_like(q)
    lse = torch.empty((H, Tq), dtype=torch.float32, device=q.device)
    if workspace is None:   # (a caller's own is sized for the caller's bound)
        max_seqlen_q = min(max_seqlen_q, Tq)
    ws, ws_bytes, keep = _e4m3_workspace(fn, workspace, q, S, max_seqlen_q, H, Hkv, d, max_blocks,
                                         1 if causal else 0, window, sinks)
    lib = _lib or load()
    _check(lib.fa_paged_prefill_e4m3(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens_q.data_ptr(),
        o.data_ptr(), lse.data_ptr(), S, Tq, max_seqlen_q, H, Hkv, d, page, P, max_blocks, scale,
        1 if causal else 0, window, sinks, ws, ws_bytes, _current_raw_stream(device)))
    return o, lse


def split_combine(part_m, part_l, part_o, stream=None):
    S, H, X, dv = part_o.shape
    o = torch.empty((S, H, dv), dtype=torch.bfloat16, device=part_o.device)
    lse = torch.empty((S, H), dtype=torch.float32, device=part_o.device)
    fa_split_combine(part_m, part_l, part_o, o, lse, S, H, X, dv, stream)
    return o, lse


def decode_workspace_views(workspace, num_seqs, H, dv, num_splits):
    """Views (part_m, part_l, part_o) of a decode workspace, for inspection."""

    def r256(x):
        return (x + 255) // 256 * 256
    tri = num_seqs * H * num_splits
    ws = workspace.view(torch.uint8)[r256(num_seqs * H * 4):]   # past the ticket words
    a = r256(tri * 4)
    pm = ws[:tri * 4].view(torch.float32).view(num_seqs, H, num_splits)
    pl = ws[a:a + tri * 4].view(torch.float32).view(num_seqs, H, num_splits)
    po = ws[2 * a:2 * a + tri * dv * 4].view(torch.float32).view(num_seqs, H, num_splits, dv)
    return pm, pl, po
