"""ctypes binding of libfa_gb300.so (the C ABI of include/fa.h).

Argument marshalling only: every function here converts its arguments to
pointers and ints and calls the entry point of the same name; all the
arithmetic runs in the library's CUDA kernels.  Pointer arguments may be torch
tensors (their data_ptr is passed), plain ints, or None.  A non-zero status
raises FaError with the library's message.  There is no fallback: if the
library is missing or cannot be loaded, the first call raises.

The helpers at the end (``forward``, ``forward_f32``, ``forward_varlen``,
``paged_decode``, ``paged_decode_fused``, the e4m3 cache's ``paged_..._e4m3``,
``split_combine``, and those of drafted trees: ``tree_layout``, ``qk_norm_rope``,
``paged_qkv_write``, ``paged_tree_attention``,
``paged_tree_attention_e4m3``, ``paged_kv_accept``,
``paged_copy_pages``) allocate outputs with torch and then call the same entry
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
            "fa_tree_layout", "fa_qk_norm_rope", "fa_paged_qkv_write", "fa_paged_tree_workspace_size",
            "fa_paged_tree_attention", "fa_paged_tree_attention_e4m3", "fa_paged_kv_accept",
            "fa_paged_copy_pages", "fa_last_error",
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
        lib.fa_tree_layout.argtypes = [P] * 5 + [I, I, I, P]
        lib.fa_qk_norm_rope.argtypes = [P] * 8 + [I, I, I, I, LL, LL, I, I, I, P, I, F, P]
        lib.fa_paged_qkv_write.argtypes = [P] * 13 + [I] * 5 + [LL, LL, LL, I, I, I, P, I, F, I, I, I, P]
        lib.fa_paged_tree_workspace_size.argtypes = [I] * 5
        lib.fa_paged_tree_workspace_size.restype = Z
        lib.fa_paged_tree_attention.argtypes = [P] * 9 + [I] * 10 + [F, P, Z, P]
        lib.fa_paged_tree_attention_e4m3.argtypes = [P] * 11 + [I] * 10 + [F, P, Z, P]
        lib.fa_paged_kv_accept.argtypes = [P] * 10 + [I] * 9 + [P]
        lib.fa_paged_copy_pages.argtypes = [P] * 5 + [I] * 6 + [P]
        lib.fa_last_error.argtypes = []
        lib.fa_last_error.restype = ctypes.c_char_p
        lib.fa_get_device_status.argtypes = [P, ctypes.POINTER(I)]
        for name in ("fa_forward", "fa_forward_fp8", "fa_forward_f32", "fa_forward_varlen",
                     "fa_paged_prefill",
                     "fa_paged_decode", "fa_paged_decode_fused",
                     "fa_paged_decode_noalloc", "fa_paged_gather", "fa_split_combine",
                     "fa_forward_window", "fa_forward_varlen_window",
                     "fa_paged_kv_write_e4m3", "fa_paged_kv_read_e4m3", "fa_paged_decode_e4m3",
                     "fa_paged_prefill_e4m3", "fa_tree_layout", "fa_qk_norm_rope", "fa_paged_qkv_write",
                     "fa_paged_tree_attention", "fa_paged_kv_accept", "fa_paged_copy_pages",
                     "fa_get_device_status"):
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

# Set by _bind_torch, before the e4m3 and tree helpers' first check: the current stream of a device
# that is known to be the current one, the current device once there are tensors on one, the types of
# the e4m3 cache's codes and scales, torch's own types under names that cost one look-up, and new
# memory on the current device, (size, strides, type) -> tensor: past torch's dispatcher where torch
# offers that (behind a launch, whose code has pushed the dispatcher out of the caches, the two
# outputs of an attention take 4.3 us instead of 7.8).
_current_raw_stream = _current_device = _CODES = _SCALES = _I32 = _BF16 = _F32 = _U8 = _new = None


def _bind_torch():
    global _current_raw_stream, _current_device, _CODES, _SCALES, _I32, _BF16, _F32, _U8, _new
    _I32, _BF16, _F32, _U8 = torch.int32, torch.bfloat16, torch.float32, torch.uint8
    guards = getattr(getattr(torch._C, "_dynamo", None), "guards", None)
    short = getattr(guards, "_empty_strided_cuda", None)
    _new = short if short is not None and _fits(short, "cuda") else _new_strided
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _SCALES = frozenset((torch.uint8, torch.int8) +
                        ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ()))
    _CODES = frozenset((torch.float8_e4m3fn, torch.uint8, torch.int8))


def _new_strided(size, strides, dtype):
    return torch.empty_strided(size, strides, dtype=dtype, device="cuda")


def _fits(new, device):
    """Whether new(size, strides, type) gives what the helpers expect: it is no public function of torch's."""
    try:
        t = new((2, 3), (1, 2), torch.int32)
        return t.shape == (2, 3) and t.stride() == (1, 2) and t.dtype is torch.int32 and t.device.type == device
    except Exception:
        return False


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


def fa_tree_layout(parents, seq_lens, cu_seqlens, mask, positions, num_seqs, total, mask_words, stream=None):
    _check(load().fa_tree_layout(_p(parents), _p(seq_lens), _p(cu_seqlens), _p(mask), _p(positions),
                                 num_seqs, total, mask_words, _stream(stream)))


@functools.lru_cache(maxsize=256)
def _ints(values):
    """The host array of a tuple of ints."""
    return (ctypes.c_int * len(values))(*values)


def fa_qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out, total, H, Hkv, d,
                    q_stride, k_stride, rot_dim, interleaved, num_axes, sections, max_positions, eps,
                    stream=None):
    """sections: the axes' pairs (a sequence of ints), or None with one axis."""
    _check(load().fa_qk_norm_rope(_p(q), _p(k), _p(q_weight), _p(k_weight), _p(cos_sin), _p(positions),
                                  _p(q_out), _p(k_out), total, H, Hkv, d, q_stride, k_stride, rot_dim,
                                  1 if interleaved else 0, num_axes, _sections(sections, num_axes),
                                  max_positions, eps, _stream(stream)))


def fa_paged_qkv_write(q, k, v, q_weight, k_weight, cos_sin, positions, q_out, k_cache, v_cache,
                       block_table, seq_lens, cu_seqlens, num_seqs, total, H, Hkv, d, q_stride, k_stride,
                       v_stride, rot_dim, interleaved, num_axes, sections, max_positions, eps, page_size,
                       num_pages, max_blocks_per_seq, stream=None):
    _check(load().fa_paged_qkv_write(_p(q), _p(k), _p(v), _p(q_weight), _p(k_weight), _p(cos_sin),
                                     _p(positions), _p(q_out), _p(k_cache), _p(v_cache),
                                     _p(block_table), _p(seq_lens), _p(cu_seqlens), num_seqs, total, H,
                                     Hkv, d, q_stride, k_stride, v_stride, rot_dim,
                                     1 if interleaved else 0, num_axes, _sections(sections, num_axes),
                                     max_positions, eps, page_size, num_pages, max_blocks_per_seq,
                                     _stream(stream)))


def _sections(sections, num_axes):
    """The host array of the axes' sections, of the length that the entry reads."""
    if sections is None:
        return None
    sections = tuple(sections)
    if len(sections) != num_axes:
        raise FaError(FA_ERR_INVALID_ARG, f"{len(sections)} sections for {num_axes} axes")
    return _ints(sections)


def fa_paged_tree_workspace_size(num_seqs, max_seqlen_q, H, Hkv, d) -> int:
    return int(load().fa_paged_tree_workspace_size(num_seqs, max_seqlen_q, H, Hkv, d))


def fa_paged_tree_attention(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, mask, o, lse,
                            num_seqs, total_q, max_seqlen_q, mask_words, H, Hkv, d, page_size, num_pages,
                            max_blocks_per_seq, scale, workspace, workspace_bytes, stream=None):
    _check(load().fa_paged_tree_attention(_p(q), _p(k_cache), _p(v_cache), _p(block_table), _p(seq_lens),
                                          _p(cu_seqlens_q), _p(mask), _p(o), _p(lse), num_seqs, total_q,
                                          max_seqlen_q, mask_words, H, Hkv, d, page_size, num_pages,
                                          max_blocks_per_seq, scale, _p(workspace), workspace_bytes,
                                          _stream(stream)))


def fa_paged_tree_attention_e4m3(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                 cu_seqlens_q, mask, o, lse, num_seqs, total_q, max_seqlen_q, mask_words,
                                 H, Hkv, d, page_size, num_pages, max_blocks_per_seq, scale, workspace,
                                 workspace_bytes, stream=None):
    _check(load().fa_paged_tree_attention_e4m3(_p(q), _p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale),
                                               _p(block_table), _p(seq_lens), _p(cu_seqlens_q), _p(mask),
                                               _p(o), _p(lse), num_seqs, total_q, max_seqlen_q, mask_words,
                                               H, Hkv, d, page_size, num_pages, max_blocks_per_seq, scale,
                                               _p(workspace), workspace_bytes, _stream(stream)))


def fa_paged_kv_accept(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, path,
                       path_lens, new_seq_lens, num_seqs, total, max_path, num_layers, Hkv, d, page_size,
                       num_pages, max_blocks_per_seq, stream=None):
    _check(load().fa_paged_kv_accept(_p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale), _p(block_table),
                                     _p(seq_lens), _p(cu_seqlens), _p(path), _p(path_lens),
                                     _p(new_seq_lens), num_seqs, total, max_path, num_layers, Hkv, d,
                                     page_size, num_pages, max_blocks_per_seq, _stream(stream)))


def fa_paged_copy_pages(k_cache, v_cache, k_scale, v_scale, pairs, num_pairs, num_layers, Hkv, d,
                        page_size, num_pages, stream=None):
    _check(load().fa_paged_copy_pages(_p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale), _p(pairs),
                                      num_pairs, num_layers, Hkv, d, page_size, num_pages,
                                      _stream(stream)))


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


# ------------------------------------------------------ drafted token trees
# (The checks are written out: these helpers run on every step of a serving loop, whose kernels take a
# few us, where a loop over the tensors or a call for each of them would take twice as long.)
def _refuse_ints(fn, device, *named):
    _refuse(fn, device, *((name, t, (_I32,), shape) for name, t, shape in named))


def tree_layout(parents, seq_lens, cu_seqlens, mask_words, stream=None):
    """parents [T] int32 (-1: child of the context) -> (mask [T,mask_words] int32 of ancestor bits,
    positions [T] int32)."""
    if stream is not None:
        with _given(stream):
            return tree_layout(parents, seq_lens, cu_seqlens, mask_words)
    if _CODES is None:
        _bind_torch()
    i32, device = _I32, parents.get_device()
    T, S = parents.shape[0], seq_lens.shape[0]
    if not (parents.dtype is i32 and seq_lens.dtype is i32 and cu_seqlens.dtype is i32
            and parents.dim() == 1 and seq_lens.dim() == 1 and cu_seqlens.shape == (S + 1,)
            and seq_lens.get_device() == device and cu_seqlens.get_device() == device
            and parents.is_contiguous() and seq_lens.is_contiguous() and cu_seqlens.is_contiguous()
            and device >= 0 and device == _current_device()):
        _refuse_ints("tree_layout", device, ("parents", parents, (T,)), ("seq_lens", seq_lens, (S,)),
                     ("cu_seqlens", cu_seqlens, (S + 1,)))
    if mask_words < 0:
        raise FaError(FA_ERR_INVALID_ARG, f"tree_layout: mask_words={mask_words}")
    mask = _new((T, mask_words), (mask_words, 1), i32)
    positions = _new((T,), (1,), i32)
    lib = _lib or load()
    rc = lib.fa_tree_layout(parents.data_ptr(), seq_lens.data_ptr(), cu_seqlens.data_ptr(), mask.data_ptr(),
                            positions.data_ptr(), S, T, mask_words, _current_raw_stream(device))
    if rc:
        _check(rc)
    return mask, positions


def _heads_stride(fn, name, t, shape, device):
    """Token stride of bf16 rows [T,heads,d] whose heads are dense."""
    st = t.stride()
    if t.shape != shape or st[2] != 1 or (st[1] != shape[2] and shape[1] > 1) or t.dtype is not _BF16 or \
            t.get_device() != device:
        raise FaError(FA_ERR_INVALID_ARG, f"{fn}: {name} is {t.dtype} on {t.device} of shape "
                                          f"{tuple(t.shape)} and strides {st}, wanted bf16 "
                                          f"{tuple(shape)} with dense heads")
    return st[0] if shape[0] > 1 else shape[1] * shape[2]


def _rotary(fn, device, T, d, q_weight, k_weight, cos_sin, positions, sections):
    """Addresses of the weights, the table and the positions, and (rot_dim, axes, rows of the table, host
    sections) of the rotation; its tensors checked."""
    qw = kw = cs = at = None
    if q_weight is not None:
        if not (q_weight.dtype is _BF16 and q_weight.shape == (d,) and q_weight.get_device() == device
                and q_weight.is_contiguous()):
            _refuse(fn, device, ("q_weight", q_weight, (_BF16,), (d,)))
        qw = q_weight.data_ptr()
    if k_weight is not None:
        if not (k_weight.dtype is _BF16 and k_weight.shape == (d,) and k_weight.get_device() == device
                and k_weight.is_contiguous()):
            _refuse(fn, device, ("k_weight", k_weight, (_BF16,), (d,)))
        kw = k_weight.data_ptr()
    if cos_sin is None:
        return qw, kw, None, None, 0, 1, 0, None
    if positions is None or cos_sin.dim() != 3 or positions.dim() != 2:
        raise FaError(FA_ERR_INVALID_ARG, f"{fn}: a rotation takes cos_sin [positions,rot_dim/2,2] and "
                                          "positions [axes,T]")
    rows, half, two = cos_sin.shape
    axes, tokens = positions.shape
    if not (cos_sin.dtype is _F32 and positions.dtype is _I32 and two == 2 and tokens == T
            and cos_sin.get_device() == device and positions.get_device() == device
            and cos_sin.is_contiguous() and positions.is_contiguous()):
        _refuse(fn, device, ("cos_sin", cos_sin, (_F32,), (rows, half, 2)),
                ("positions", positions, (_I32,), (axes, T)))
    return qw, kw, cos_sin.data_ptr(), positions.data_ptr(), 2 * half, axes, rows, \
        None if sections is None else _sections(sections, axes)


def qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps=1e-6, sections=None,
                 interleaved=False, stream=None):
    """q [T,H,d], k [T,Hkv,d] bf16 (parts of one projection allowed), weights [d] bf16 or None, cos_sin
    [positions,rot_dim/2,2] fp32 or None, positions [axes,T] int32 -> (q [T,H,d], k [T,Hkv,d])."""
    if stream is not None:
        with _given(stream):
            return qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps, sections, interleaved)
    if _CODES is None:
        _bind_torch()
    fn = "qk_norm_rope"
    device = q.get_device()
    T, H, d = q.shape
    shape, k_shape = (T, H, d), (T, k.shape[1], d)
    if device < 0 or device != _current_device():
        _refuse(fn, device)
    qs, ks = _heads_stride(fn, "q", q, shape, device), _heads_stride(fn, "k", k, k_shape, device)
    qw, kw, cs, at, rot, axes, rows, host = _rotary(fn, device, T, d, q_weight, k_weight, cos_sin, positions,
                                                    sections)
    q_out = _new(shape, (H * d, d, 1), _BF16)
    k_out = _new(k_shape, (k_shape[1] * d, d, 1), _BF16)
    lib = _lib or load()
    rc = lib.fa_qk_norm_rope(q.data_ptr(), k.data_ptr(), qw, kw, cs, at, q_out.data_ptr(), k_out.data_ptr(), T,
                             H, k_shape[1], d, qs, ks, rot, 1 if interleaved else 0, axes, host, rows, eps,
                             _current_raw_stream(device))
    if rc:
        _check(rc)
    return q_out, k_out


def _check_paged(fn, device, kc, vc, bt, sl, cu):
    """The bf16 paged cache's tensors; the shapes of the cache and of the block table."""
    if _CODES is None:
        _bind_torch()
    shape, table, kind, i32 = kc.shape, bt.shape, _BF16, _I32
    if len(shape) != 4 or len(table) != 2:
        raise FaError(FA_ERR_INVALID_ARG, f"{fn}: k_cache has shape {tuple(shape)}, block_table "
                                          f"{tuple(table)}, wanted 4 and 2 dimensions")
    S = table[0]
    if not (kc.dtype is kind and vc.dtype is kind and bt.dtype is i32 and sl.dtype is i32
            and cu.dtype is i32 and vc.shape == shape and sl.shape == (S,) and cu.shape == (S + 1,)
            and kc.get_device() == device and vc.get_device() == device and bt.get_device() == device
            and sl.get_device() == device and cu.get_device() == device and kc.is_contiguous()
            and vc.is_contiguous() and bt.is_contiguous() and sl.is_contiguous()
            and cu.is_contiguous() and device >= 0 and device == _current_device()):
        _refuse(fn, device, ("k_cache", kc, (kind,), shape), ("v_cache", vc, (kind,), shape),
                ("block_table", bt, (i32,), table), ("seq_lens", sl, (i32,), (S,)),
                ("cu_seqlens", cu, (i32,), (S + 1,)))
    return shape, table


def paged_qkv_write(q, k, v, q_weight, k_weight, cos_sin, positions, k_cache, v_cache, block_table,
                    seq_lens, cu_seqlens, eps=1e-6, sections=None, interleaved=False, stream=None):
    """As qk_norm_rope, with K and V going into the bf16 paged cache [P,Hkv,16,d] -> q [T,H,d]."""
    if stream is not None:
        with _given(stream):
            return paged_qkv_write(q, k, v, q_weight, k_weight, cos_sin, positions, k_cache, v_cache,
                                   block_table, seq_lens, cu_seqlens, eps, sections, interleaved)
    fn = "paged_qkv_write"
    device = q.get_device()
    (P, Hkv, page, d), (S, max_blocks) = _check_paged(fn, device, k_cache, v_cache, block_table, seq_lens,
                                                      cu_seqlens)
    T, H, _ = q.shape
    shape, kv_shape = (T, H, d), (T, Hkv, d)
    qs, ks, vs = (_heads_stride(fn, "q", q, shape, device), _heads_stride(fn, "k", k, kv_shape, device),
                  _heads_stride(fn, "v", v, kv_shape, device))
    qw, kw, cs, at, rot, axes, rows, host = _rotary(fn, device, T, d, q_weight, k_weight, cos_sin, positions,
                                                    sections)
    q_out = _new(shape, (H * d, d, 1), _BF16)
    lib = _lib or load()
    rc = lib.fa_paged_qkv_write(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), qw, kw, cs, at, q_out.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens.data_ptr(), S, T, H, Hkv, d,
        qs, ks, vs, rot, 1 if interleaved else 0, axes, host, rows, eps, page, P, max_blocks,
        _current_raw_stream(device))
    if rc:
        _check(rc)
    return q_out


@functools.lru_cache(maxsize=4096)
def _tree_workspace(*sizes):
    """fa_paged_tree_workspace_size, which depends on the sizes alone."""
    return fa_paged_tree_workspace_size(*sizes)


def paged_tree_attention(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q, mask,
                         scale, workspace=None, stream=None):
    """Drafted nodes q [T,H,d] packed by cu_seqlens_q over the bf16 cache, mask [T,words] int32 of the
    nodes that each node sees beside the context -> (o [T,H,d] bf16, lse [H,T] fp32).  A max_seqlen_q of 0
    counts as 1, with a workspace of the call's own."""
    if stream is not None:
        with _given(stream):
            return paged_tree_attention(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q,
                                        max_seqlen_q, mask, scale, workspace)
    fn = "paged_tree_attention"
    device = q.get_device()
    (P, Hkv, page, d), (S, max_blocks) = _check_paged(fn, device, k_cache, v_cache, block_table, seq_lens,
                                                      cu_seqlens_q)
    T, H, width = q.shape
    words = mask.shape[-1]
    if not (q.dtype is _BF16 and mask.dtype is _I32 and width == d and mask.shape == (T, words)
            and mask.get_device() == device and q.is_contiguous() and mask.is_contiguous()):
        _refuse(fn, device, ("q", q, (_BF16,), (T, H, d)), ("mask", mask, (_I32,), (T, words)))
    if max_seqlen_q == 0:   # (the entry would look at no sequence, and say nothing of one with nodes)
        max_seqlen_q, workspace = 1, None
    if workspace is None:   # (a caller's own is sized for the caller's bound)
        max_seqlen_q = min(max_seqlen_q, T)
        size = _tree_workspace(S, max_seqlen_q, H, Hkv, d)
        workspace = _new((size,), (1,), _U8)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise FaError(FA_ERR_WORKSPACE, f"{fn}: the workspace is on {workspace.device} with strides "
                                        f"{workspace.stride()}")
    else:
        size = workspace.nbytes
    o = _new((T, H, d), (H * d, d, 1), _BF16)
    lse = _new((H, T), (T, 1), _F32)
    lib = _lib or load()
    rc = lib.fa_paged_tree_attention(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        cu_seqlens_q.data_ptr(), mask.data_ptr(), o.data_ptr(), lse.data_ptr(), S, T, max_seqlen_q, words,
        H, Hkv, d, page, P, max_blocks, scale, workspace.data_ptr(), size, _current_raw_stream(device))
    if rc:
        _check(rc)
    return o, lse


def paged_tree_attention_e4m3(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens_q,
                              max_seqlen_q, mask, scale, workspace=None, stream=None):
    """paged_tree_attention over the e4m3 cache [P,Hkv,16,d] with scale bytes [P,Hkv,16]."""
    if stream is not None:
        with _given(stream):
            return paged_tree_attention_e4m3(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                             cu_seqlens_q, max_seqlen_q, mask, scale, workspace)
    fn = "paged_tree_attention_e4m3"
    device = q.get_device()
    _check_cache(fn, device, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens)
    P, Hkv, page, d = k_cache.shape
    S, max_blocks = block_table.shape
    T, H = q.shape[:2]
    words = mask.shape[-1]
    _check_rows(fn, device, "q", q, torch.bfloat16, (T, H, d))
    _check_rows(fn, device, "mask", mask, torch.int32, (T, words))
    _check_rows(fn, device, "cu_seqlens_q", cu_seqlens_q, torch.int32, (S + 1,))
    if max_seqlen_q == 0:   # (the entry would look at no sequence, and say nothing of one with nodes)
        max_seqlen_q, workspace = 1, None
    if workspace is None:   # (a caller's own is sized for the caller's bound)
        max_seqlen_q = min(max_seqlen_q, T)
        size = _tree_workspace(S, max_seqlen_q, H, Hkv, d)
        workspace = _new((size,), (1,), _U8)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise FaError(FA_ERR_WORKSPACE, f"{fn}: the workspace is on {workspace.device} with strides "
                                        f"{workspace.stride()}")
    else:
        size = workspace.nbytes
    o = _new((T, H, d), (H * d, d, 1), _BF16)
    lse = _new((H, T), (T, 1), _F32)
    lib = _lib or load()
    rc = lib.fa_paged_tree_attention_e4m3(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens_q.data_ptr(), mask.data_ptr(), o.data_ptr(),
        lse.data_ptr(), S, T, max_seqlen_q, words, H, Hkv, d, page, P, max_blocks, scale,
        workspace.data_ptr(), size, _current_raw_stream(device))
    if rc:
        _check(rc)
    return o, lse


def _check_layers(fn, device, kc, vc, ks, vs):
    """Caches [P,Hkv,16,d], or [layers,P,Hkv,16,d], bf16 or (with scales) e4m3; their layers and a layer's
    shape."""
    if _CODES is None:
        _bind_torch()
    shape = kc.shape
    if len(shape) not in (4, 5) or (ks is None) != (vs is None):
        raise FaError(FA_ERR_INVALID_ARG, f"{fn}: k_cache has shape {tuple(shape)}, wanted 4 dimensions, or "
                                          "5 with layers first, and both scales or none")
    ok = vc.shape == shape and kc.is_contiguous() and vc.is_contiguous() and vc.get_device() == device and \
        device >= 0 and device == _current_device()
    if ks is None:
        if not (ok and kc.dtype is _BF16 and vc.dtype is _BF16):
            _refuse(fn, device, ("k_cache", kc, (_BF16,), shape), ("v_cache", vc, (_BF16,), shape))
    elif not (ok and kc.dtype in _CODES and vc.dtype in _CODES and ks.dtype in _SCALES and vs.dtype in _SCALES
              and ks.shape == shape[:-1] and vs.shape == shape[:-1] and ks.is_contiguous()
              and vs.is_contiguous() and ks.get_device() == device and vs.get_device() == device):
        _refuse(fn, device, ("k_cache", kc, _CODES, shape), ("v_cache", vc, _CODES, shape),
                ("k_scale", ks, _SCALES, shape[:-1]), ("v_scale", vs, _SCALES, shape[:-1]))
    return (1, *shape) if len(shape) == 4 else shape


def paged_kv_accept(k_cache, v_cache, block_table, seq_lens, cu_seqlens, path, path_lens, k_scale=None,
                    v_scale=None, stream=None):
    """The rows of the accepted nodes path [S,max_path] int32 (path_lens [S] of them) moved behind the
    context, in caches [P,Hkv,16,d] or [layers,P,Hkv,16,d] -> the new lengths [S] int32."""
    if stream is not None:
        with _given(stream):
            return paged_kv_accept(k_cache, v_cache, block_table, seq_lens, cu_seqlens, path, path_lens,
                                   k_scale, v_scale)
    fn = "paged_kv_accept"
    device = k_cache.get_device()
    layers, P, Hkv, page, d = _check_layers(fn, device, k_cache, v_cache, k_scale, v_scale)
    if layers == 0:   # (the entry would do nothing, and the new lengths hold anything)
        raise FaError(FA_ERR_INVALID_ARG, f"{fn}: caches without layers")
    S, max_blocks = block_table.shape
    max_path, i32 = path.shape[-1], _I32
    if not (block_table.dtype is i32 and seq_lens.dtype is i32 and cu_seqlens.dtype is i32
            and path.dtype is i32 and path_lens.dtype is i32 and seq_lens.shape == (S,)
            and cu_seqlens.shape == (S + 1,) and path.shape == (S, max_path) and path_lens.shape == (S,)
            and block_table.get_device() == device and seq_lens.get_device() == device
            and cu_seqlens.get_device() == device and path.get_device() == device
            and path_lens.get_device() == device and block_table.is_contiguous()
            and seq_lens.is_contiguous() and cu_seqlens.is_contiguous() and path.is_contiguous()
            and path_lens.is_contiguous()):
        _refuse_ints(fn, device, ("block_table", block_table, (S, max_blocks)), ("seq_lens", seq_lens, (S,)),
                     ("cu_seqlens", cu_seqlens, (S + 1,)), ("path", path, (S, max_path)),
                     ("path_lens", path_lens, (S,)))
    new_lens = _new((S,), (1,), i32)
    lib = _lib or load()
    rc = lib.fa_paged_kv_accept(
        k_cache.data_ptr(), v_cache.data_ptr(), None if k_scale is None else k_scale.data_ptr(),
        None if v_scale is None else v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        cu_seqlens.data_ptr(), path.data_ptr(), path_lens.data_ptr(), new_lens.data_ptr(), S, 0x7fffffff,
        max_path, layers, Hkv, d, page, P, max_blocks, _current_raw_stream(device))
    if rc:
        _check(rc)
    return new_lens


def paged_copy_pages(k_cache, v_cache, pairs, k_scale=None, v_scale=None, stream=None):
    """Pages pairs[:, 0] copied to pages pairs[:, 1] ([N,2] int32) of caches [P,Hkv,16,d] or
    [layers,P,Hkv,16,d], and of their scales."""
    fn = "paged_copy_pages"
    device = k_cache.get_device()
    layers, P, Hkv, page, d = _check_layers(fn, device, k_cache, v_cache, k_scale, v_scale)
    N = pairs.shape[0]
    if not (pairs.dtype is _I32 and pairs.shape == (N, 2) and pairs.get_device() == device
            and pairs.is_contiguous()):
        _refuse_ints(fn, device, ("pairs", pairs, (N, 2)))
    lib = _lib or load()
    rc = lib.fa_paged_copy_pages(k_cache.data_ptr(), v_cache.data_ptr(),
                                 None if k_scale is None else k_scale.data_ptr(),
                                 None if v_scale is None else v_scale.data_ptr(), pairs.data_ptr(), N, layers,
                                 Hkv, d, page, P,
                                 _current_raw_stream(device) if stream is None else _stream(stream))
    if rc:
        _check(rc)


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
