"""Fused exact attention for B200 (sm_100a): the Python binding of libfa.so.

The binding marshals arguments only; every step of the computation runs in the CUDA
kernels behind the C ABI of ``include/fa.h``.  The C entry points are mirrored one to one
(``fa_fwd``, ``fa_bwd``, ``fa_fwd_ex``, ``fa_bwd_ex``, ``fa_bwd_workspace_bytes``,
``fa_bwd_workspace_bytes_ex``, ``fa_bwd_workspace_bytes_split``, ``fa_bwd_splitq_choose``, ``fa_bwd_noalloc``, ``fa_fwd_partial``, ``fa_lse_merge``, ``fa_fwd_splitkv``,
``fa_fwd_splitkv_workspace_bytes``, ``fa_splitkv_choose``, ``fa_fwd_fp8``, ``fa_fwd_fp8_workspace_bytes``, ``fa_selftest_wait_timeout``, ``fa_selftest_exp2_poly``, ``fa_check_status``,
``fa_cache_append``, ``fa_cache_read``, ``fa_cache_keep``, ``fa_fwd_tree``, ``fa_fwd_tree_workspace_bytes``,
``fa_status_string``, ``fa_last_launch_count``); they take torch tensors (or raw device
addresses as ints).  ``attention_forward`` / ``attention_backward`` /
``attention_forward_splitkv`` / ``attention_forward_partial`` / ``lse_merge`` and
``FlashAttention`` add output allocation with torch on top.

Serving: ``KVCache`` describes a paged key/value cache (16-bit, or E4M3 quantised as it is
written); ``cache_append`` writes new tokens' rows, ``attention_forward_tree`` lets the new tokens (one, a
chain, or a tree of drafted tokens, ``tree_mask``) attend over it, ``cache_keep`` keeps the accepted
ones, ``cache_read`` reads it back as dense tensors:

    cache_append(cache, k, v, cu, lens)
    o, lse = attention_forward_tree(q, cache, cu, lens, max_new, tree_mask=tree_mask(parents, cu))
    cache_keep(cache, lens, kept, counts);  lens += counts

``stream``: the stream (or its handle) a call's kernels run on, torch's current one by default.  What a
call allocates belongs to that stream; what the caller passes has to be ready on it, and to live until it is
done.

There is no fallback: if ``libfa.so`` is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import struct

__all__ = [
    "FAError", "fa_fwd", "fa_bwd", "fa_fwd_ex", "fa_bwd_ex", "fa_bwd_workspace_bytes",
    "fa_check_status", "fa_status_string", "fa_last_launch_count", "fa_bwd_noalloc", "lib", "library_path",
    "attention_forward", "attention_backward", "FlashAttention", "FA_BF16", "FA_FP16", "FA_FP32",
    "fa_fwd_partial", "fa_lse_merge", "fa_fwd_splitkv", "fa_fwd_splitkv_workspace_bytes",
    "fa_splitkv_choose", "attention_forward_splitkv", "attention_forward_partial", "lse_merge",
    "FA_MAX_PARTS", "fa_bwd_workspace_bytes_ex", "fa_bwd_workspace_bytes_split", "fa_bwd_splitq_choose", "FA_ERR_RANGE", "fa_fwd_fp8", "fa_fwd_fp8_workspace_bytes",
    "attention_forward_fp8", "fa_selftest_wait_timeout", "fa_selftest_exp2_poly",
    "FA_E4M3", "KVCache", "fa_cache_append", "fa_cache_read", "fa_cache_keep", "fa_fwd_tree",
    "fa_fwd_tree_workspace_bytes", "cache_append", "cache_read", "cache_keep", "attention_forward_tree", "tree_mask",
]

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_WORKSPACE, FA_ERR_RANGE = range(7)
FA_BF16, FA_FP16, FA_FP32, FA_E4M3 = 0, 1, 2, 3
TILE = 128
FA_MAX_PARTS = 64

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libfa.so")
_lib = None
_torch = None          # set by the first KVCache, which every serving call needs

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_ll = ctypes.c_longlong
_bytes = ctypes.c_char_p


class FwdArgs(ctypes.Structure):
    """Mirror of fa_fwd_args."""
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("lse", _vp),
                ("B", _i), ("H", _i), ("N", _i), ("d", _i), ("scale", _f), ("causal", _i),
                ("blockmask", _vp), ("dtype", _i), ("o_fp32", _i), ("visit_log", _vp),
                ("stream", _vp), ("dropout_p", _f), ("dropout_seed", ctypes.c_ulonglong)]


class BwdArgs(ctypes.Structure):
    """Mirror of fa_bwd_args."""
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("lse", _vp), ("dout", _vp),
                ("dq", _vp), ("dk", _vp), ("dv", _vp),
                ("B", _i), ("H", _i), ("N", _i), ("d", _i), ("scale", _f), ("causal", _i),
                ("blockmask", _vp), ("dtype", _i), ("visit_log", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("stream", _vp),
                ("main_start_event", _vp), ("main_stop_event", _vp), ("deterministic", _i),
                ("dropout_p", _f), ("dropout_seed", ctypes.c_ulonglong), ("query_splits", _i)]


class PartialArgs(ctypes.Structure):
    """Mirror of fa_fwd_partial_args."""
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("o_part", _vp), ("lse_part", _vp),
                ("B", _i), ("H", _i), ("N", _i), ("Nk", _i), ("d", _i), ("key_offset", _i),
                ("scale", _f), ("causal", _i), ("blockmask", _vp), ("dtype", _i), ("stream", _vp)]


class Fp8Args(ctypes.Structure):
    """Mirror of fa_fwd_fp8_args."""
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("descale_q", _f), ("descale_k", _f), ("descale_v", _f),
                ("o", _vp), ("lse", _vp), ("B", _i), ("H", _i), ("N", _i), ("d", _i), ("scale", _f),
                ("causal", _i), ("blockmask", _vp), ("o_fp32", _i), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("stream", _vp)]


class CacheArgs(ctypes.Structure):
    """Mirror of fa_cache."""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("page_table", _vp),
                ("pages", _i), ("Hk", _i), ("page_size", _i), ("d", _i), ("dtype", _i),
                ("B", _i), ("max_pages", _i), ("table_stride", _i)]


class CacheAppendArgs(ctypes.Structure):
    """Mirror of fa_cache_append_args."""
    _fields_ = [("cache", CacheArgs), ("k_new", _vp), ("v_new", _vp),
                ("k_token_stride", _ll), ("k_head_stride", _ll), ("v_token_stride", _ll), ("v_head_stride", _ll),
                ("cu_new", _vp), ("lens", _vp), ("total", _i), ("dtype", _i), ("stream", _vp)]


class CacheReadArgs(ctypes.Structure):
    """Mirror of fa_cache_read_args."""
    _fields_ = [("cache", CacheArgs), ("lens", _vp), ("k_out", _vp), ("v_out", _vp), ("N", _i), ("dtype", _i),
                ("stream", _vp)]


class CacheKeepArgs(ctypes.Structure):
    """Mirror of fa_cache_keep_args."""
    _fields_ = [("cache", CacheArgs), ("lens", _vp), ("kept", _vp), ("counts", _vp), ("width", _i), ("stream", _vp)]


class TreeArgs(ctypes.Structure):
    """Mirror of fa_fwd_tree_args."""
    _fields_ = [("cache", CacheArgs), ("q", _vp), ("o", _vp), ("lse", _vp),
                ("q_token_stride", _ll), ("q_head_stride", _ll), ("o_token_stride", _ll), ("o_head_stride", _ll),
                ("cu_new", _vp), ("lens", _vp), ("tree_mask", _vp), ("mask_words", _i),
                ("total", _i), ("Hq", _i), ("max_new", _i), ("dtype", _i), ("scale", _f),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("stream", _vp)]


class FAError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {fa_status_string(code)} ({code})")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libfa.so (built in-tree by exact_attention_111_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"{library_path} is not built; run `python -m exact_attention_111_b200.build`")
    L = ctypes.CDLL(library_path)
    L.fa_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _vp]
    L.fa_fwd.restype = _i
    L.fa_bwd.argtypes = [_vp] * 9 + [_i, _i, _i, _i, _f, _i, _vp, _vp, ctypes.c_size_t, _vp]
    L.fa_bwd.restype = _i
    L.fa_fwd_ex.argtypes = [ctypes.POINTER(FwdArgs)]
    L.fa_fwd_ex.restype = _i
    L.fa_bwd_ex.argtypes = [ctypes.POINTER(BwdArgs)]
    L.fa_bwd_ex.restype = _i
    L.fa_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i]
    L.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
    L.fa_bwd_workspace_bytes_ex.argtypes = [_i, _i, _i, _i, _i]
    L.fa_bwd_workspace_bytes_ex.restype = ctypes.c_size_t
    L.fa_bwd_workspace_bytes_split.argtypes = [_i, _i, _i, _i, _i]
    L.fa_bwd_workspace_bytes_split.restype = ctypes.c_size_t
    L.fa_bwd_splitq_choose.argtypes = [_i, _i, _i, _i, _i]
    L.fa_bwd_splitq_choose.restype = _i
    L.fa_check_status.argtypes = [_vp]
    L.fa_check_status.restype = _i
    L.fa_status_string.argtypes = [_i]
    L.fa_status_string.restype = ctypes.c_char_p
    L.fa_bwd_noalloc.argtypes = [_vp] * 9 + [_i, _i, _i, _i, _f, _i, _vp, _vp]
    L.fa_bwd_noalloc.restype = _i
    L.fa_last_launch_count.argtypes = []
    L.fa_last_launch_count.restype = _i
    L.fa_fwd_partial.argtypes = [ctypes.POINTER(PartialArgs)]
    L.fa_fwd_partial.restype = _i
    L.fa_lse_merge.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_vp), _i, _vp, _vp, _i, _i, _i, _i, _i, _vp]
    L.fa_lse_merge.restype = _i
    L.fa_fwd_splitkv.argtypes = [_vp] * 5 + [_i, _i, _i, _i, _f, _i, _vp, _i, _vp, ctypes.c_size_t, _vp]
    L.fa_fwd_splitkv.restype = _i
    L.fa_fwd_splitkv_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
    L.fa_fwd_splitkv_workspace_bytes.restype = ctypes.c_size_t
    L.fa_splitkv_choose.argtypes = [_i, _i, _i, _i, _i]
    L.fa_splitkv_choose.restype = _i
    L.fa_fwd_fp8.argtypes = [ctypes.POINTER(Fp8Args)]
    L.fa_fwd_fp8.restype = _i
    L.fa_fwd_fp8_workspace_bytes.argtypes = [_i, _i, _i, _i]
    L.fa_fwd_fp8_workspace_bytes.restype = ctypes.c_size_t
    L.fa_selftest_wait_timeout.argtypes = [ctypes.c_uint, _vp, _vp]
    L.fa_selftest_wait_timeout.restype = _i
    L.fa_selftest_exp2_poly.argtypes = [_vp, _vp, _i, _vp]
    L.fa_selftest_exp2_poly.restype = _i
    L.fa_cache_append.argtypes = [_bytes]                # the bytes of a CacheAppendArgs
    L.fa_cache_append.restype = _i
    L.fa_cache_read.argtypes = [_bytes]                # the bytes of a CacheReadArgs
    L.fa_cache_read.restype = _i
    L.fa_cache_keep.argtypes = [_bytes]                # the bytes of a CacheKeepArgs
    L.fa_cache_keep.restype = _i
    L.fa_fwd_tree.argtypes = [_bytes]                    # the bytes of a TreeArgs
    L.fa_fwd_tree.restype = _i
    L.fa_fwd_tree_workspace_bytes.argtypes = [_i, _i, _i, _i]
    L.fa_fwd_tree_workspace_bytes.restype = ctypes.c_size_t
    _lib = L
    return L


def _ptr(x):
    """Device address of a tensor (or None / int passed through)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _made_on(stream, device):
    """Context for the tensors that a call on `stream` makes for itself: torch's allocator keeps a block
    for the stream that was current when it was made, and gives it to that stream alone.  Made
    under another stream than the kernels', a result could lie where earlier work is not done, and a
    scratch block would be given away while the kernels still use it."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):                          # (an external stream of handle 0 would be a new stream)
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _check(rc: int, what: str):
    if rc != FA_OK:
        raise FAError(rc, what)


def fa_status_string(code: int) -> str:
    return lib().fa_status_string(code).decode()


def fa_last_launch_count() -> int:
    return lib().fa_last_launch_count()


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return lib().fa_bwd_workspace_bytes(B, H, N, d)


def fa_bwd_workspace_bytes_ex(B: int, H: int, N: int, d: int, deterministic: bool) -> int:
    return lib().fa_bwd_workspace_bytes_ex(B, H, N, d, int(bool(deterministic)))


def fa_bwd_workspace_bytes_split(B: int, H: int, N: int, d: int, query_splits: int) -> int:
    return lib().fa_bwd_workspace_bytes_split(B, H, N, d, int(query_splits))


def fa_bwd_splitq_choose(B: int, H: int, N: int, causal: bool, num_sms: int) -> int:
    return lib().fa_bwd_splitq_choose(B, H, N, int(bool(causal)), num_sms)


def fa_check_status(stream=None):
    _check(lib().fa_check_status(_stream(stream)), "fa_check_status")


def fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, blockmask, stream=None):
    _check(lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, scale,
                        int(bool(causal)), _ptr(blockmask), _stream(stream)), "fa_fwd")


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, scale, causal, blockmask,
           workspace, workspace_bytes, stream=None):
    _check(lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                        _ptr(dk), _ptr(dv), B, H, N, d, scale, int(bool(causal)), _ptr(blockmask),
                        _ptr(workspace), workspace_bytes, _stream(stream)), "fa_bwd")


def fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, scale, causal, blockmask,
                   stream=None):
    """fa_bwd without a workspace argument, for callers that cannot allocate device memory
    at call time; uses the library's fixed 64 MiB per-device scratch (see include/fa.h)."""
    _check(lib().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                                _ptr(dk), _ptr(dv), B, H, N, d, scale, int(bool(causal)),
                                _ptr(blockmask), _stream(stream)), "fa_bwd_noalloc")


def fa_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal=False, blockmask=None, dtype=FA_BF16,
              o_fp32=False, visit_log=None, stream=None, dropout_p=0.0, dropout_seed=0):
    a = FwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, scale, int(bool(causal)),
                _ptr(blockmask), dtype, int(bool(o_fp32)), _ptr(visit_log), _stream(stream),
                float(dropout_p), int(dropout_seed))
    _check(lib().fa_fwd_ex(ctypes.byref(a)), "fa_fwd_ex")


def fa_fwd_partial(q, k, v, o_part, lse_part, B, H, N, Nk, d, key_offset, scale, causal=False,
                   blockmask=None, dtype=FA_BF16, stream=None):
    a = PartialArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(o_part), _ptr(lse_part), B, H, N, Nk, d, key_offset,
                    scale, int(bool(causal)), _ptr(blockmask), dtype, _stream(stream))
    _check(lib().fa_fwd_partial(ctypes.byref(a)), "fa_fwd_partial")


def fa_lse_merge(o_parts, lse_parts, o, lse, B, H, N, d, out_dtype=FA_BF16, stream=None):
    """o_parts / lse_parts: sequences of device tensors (or addresses), one per part."""
    n = len(o_parts)
    if len(lse_parts) != n:
        raise ValueError("o_parts and lse_parts differ in length")
    po = (_vp * max(n, 1))(*[_ptr(x) for x in o_parts])
    pl = (_vp * max(n, 1))(*[_ptr(x) for x in lse_parts])
    _check(lib().fa_lse_merge(po, pl, n, _ptr(o), _ptr(lse), B, H, N, d, out_dtype, _stream(stream)),
           "fa_lse_merge")


def fa_fwd_splitkv_workspace_bytes(B: int, H: int, N: int, d: int, num_splits: int) -> int:
    return lib().fa_fwd_splitkv_workspace_bytes(B, H, N, d, num_splits)


def fa_splitkv_choose(B: int, H: int, N: int, causal: bool, num_sms: int) -> int:
    return lib().fa_splitkv_choose(B, H, N, int(bool(causal)), num_sms)


def fa_fwd_splitkv(q, k, v, o, lse, B, H, N, d, scale, causal, blockmask, num_splits, workspace,
                   workspace_bytes, stream=None):
    _check(lib().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, scale,
                                int(bool(causal)), _ptr(blockmask), num_splits, _ptr(workspace),
                                workspace_bytes, _stream(stream)), "fa_fwd_splitkv")


def fa_selftest_wait_timeout(limit_us: int, waited_ok=None, stream=None):
    """Runs the bounded-wait diagnostic (include/fa.h); fa_check_status then reports
    FA_ERR_TIMEOUT."""
    _check(lib().fa_selftest_wait_timeout(int(limit_us), _ptr(waited_ok), _stream(stream)), "fa_selftest_wait_timeout")


def fa_selftest_exp2_poly(x, y, n: int, stream=None):
    """y[:n] = 2^x[:n] by the kernels' FMA-pipe polynomial (the diagnostic of include/fa.h)."""
    _check(lib().fa_selftest_exp2_poly(_ptr(x), _ptr(y), int(n), _stream(stream)), "fa_selftest_exp2_poly")


def fa_fwd_fp8_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return lib().fa_fwd_fp8_workspace_bytes(B, H, N, d)


def fa_fwd_fp8(q8, k8, v8, descale_q, descale_k, descale_v, o, lse, B, H, N, d, scale, causal=False,
               blockmask=None, o_fp32=False, workspace=None, workspace_bytes=0, stream=None):
    a = Fp8Args(_ptr(q8), _ptr(k8), _ptr(v8), float(descale_q), float(descale_k), float(descale_v), _ptr(o),
                _ptr(lse), B, H, N, d, scale, int(bool(causal)), _ptr(blockmask), int(bool(o_fp32)),
                _ptr(workspace), workspace_bytes, _stream(stream))
    _check(lib().fa_fwd_fp8(ctypes.byref(a)), "fa_fwd_fp8")


# The serving calls are made once per layer and token, so their argument blocks are packed as bytes
# (the structs' native layout, the cache's block first) instead of through ctypes fields.
_pack_append = struct.Struct("@PPqqqqPPiiP").pack
_pack_read = struct.Struct("@PPPiiP").pack
_pack_keep = struct.Struct("@PPPiP").pack
_pack_tree = struct.Struct("@PPPqqqqPPPiiiiifPNP").pack


def fa_cache_append(cache, k_new, v_new, k_strides, v_strides, cu_new, lens, total, dtype, stream=None):
    """cache: the bytes of a CacheArgs; strides: (token, head) in elements."""
    rc = lib().fa_cache_append(cache + _pack_append(_ptr(k_new), _ptr(v_new), *k_strides, *v_strides, _ptr(cu_new),
                                                    _ptr(lens), total, dtype, _stream(stream)))
    if rc:
        raise FAError(rc, "fa_cache_append")


def fa_cache_read(cache, lens, k_out, v_out, N, dtype, stream=None):
    rc = lib().fa_cache_read(cache + _pack_read(_ptr(lens), _ptr(k_out), _ptr(v_out), N, dtype, _stream(stream)))
    if rc:
        raise FAError(rc, "fa_cache_read")


def fa_cache_keep(cache, lens, kept, counts, width, stream=None):
    rc = lib().fa_cache_keep(cache + _pack_keep(_ptr(lens), _ptr(kept), _ptr(counts), width, _stream(stream)))
    if rc:
        raise FAError(rc, "fa_cache_keep")


def fa_fwd_tree_workspace_bytes(total: int, Hq: int, Hk: int, d: int) -> int:
    return lib().fa_fwd_tree_workspace_bytes(total, Hq, Hk, d)


def fa_fwd_tree(cache, q, o, lse, q_strides, o_strides, cu_new, lens, tree_mask, mask_words, total, Hq, max_new,
                dtype, scale, workspace, workspace_bytes, stream=None):
    """cache: the bytes of a CacheArgs; strides: (token, head) in elements."""
    rc = lib().fa_fwd_tree(cache + _pack_tree(_ptr(q), _ptr(o), _ptr(lse), *q_strides, *o_strides, _ptr(cu_new),
                                              _ptr(lens), _ptr(tree_mask) or 0, mask_words, total, Hq, max_new,
                                              dtype, scale, _ptr(workspace), workspace_bytes, _stream(stream)))
    if rc:
        raise FAError(rc, "fa_fwd_tree")


def _event(e):
    if e is None or isinstance(e, int):
        return e
    return e.cuda_event  # torch.cuda.Event (created lazily by torch on first use)


def fa_bwd_ex(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, scale, causal=False, blockmask=None,
              dtype=FA_BF16, visit_log=None, workspace=None, workspace_bytes=0, stream=None,
              main_start_event=None, main_stop_event=None, deterministic=False, dropout_p=0.0, dropout_seed=0,
              query_splits=0):
    a = BwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                _ptr(dv), B, H, N, d, scale, int(bool(causal)), _ptr(blockmask), dtype,
                _ptr(visit_log), _ptr(workspace), workspace_bytes, _stream(stream),
                _event(main_start_event), _event(main_stop_event), int(bool(deterministic)),
                float(dropout_p), int(dropout_seed), int(query_splits))
    _check(lib().fa_bwd_ex(ctypes.byref(a)), "fa_bwd_ex")


# ----------------------------------------------------------------------------------------
# torch conveniences (allocation only; the arithmetic is in the kernels)
# ----------------------------------------------------------------------------------------

def _dtype_code(t):
    import torch
    if t.dtype is torch.bfloat16:
        return FA_BF16
    if t.dtype is torch.float16:
        return FA_FP16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check_qkv(*ts):
    for t in ts:
        if not (t.is_cuda and t.is_contiguous() and t.dim() == 4):
            raise ValueError("expected contiguous CUDA tensors of shape [B, H, N, d]")


def attention_forward(q, k, v, causal=False, blockmask=None, scale=None, o_fp32=False,
                      visit_log=None, stream=None, dropout_p=0.0, dropout_seed=0):
    """Returns (O, LSE) for [B, H, N, d] CUDA tensors (bf16 or fp16).  ``dropout_p`` > 0 drops
    probabilities with the Philox mask of ``dropout_seed`` (include/fa.h)."""
    import torch
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    scale = (1.0 / d ** 0.5) if scale is None else scale
    with _made_on(stream, q.device):
        o = torch.empty(q.shape, dtype=torch.float32 if o_fp32 else q.dtype, device=q.device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, blockmask, _dtype_code(q), o_fp32,
              visit_log, stream, dropout_p=dropout_p, dropout_seed=dropout_seed)
    return o, lse


def attention_forward_splitkv(q, k, v, causal=False, blockmask=None, scale=None, num_splits=None,
                              workspace=None, stream=None):
    """fa_fwd_splitkv on bf16 [B, H, N, d] tensors.  ``num_splits=None`` takes
    fa_splitkv_choose for this GPU's SM count.  Returns (O, LSE, num_splits)."""
    import torch
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    scale = (1.0 / d ** 0.5) if scale is None else scale
    if num_splits is None:
        sms = torch.cuda.get_device_properties(q.device).multi_processor_count
        num_splits = fa_splitkv_choose(B, H, N, causal, sms)
    nbytes = fa_fwd_splitkv_workspace_bytes(B, H, N, d, num_splits)
    with _made_on(stream, q.device):
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
        if workspace is None and num_splits > 1:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    fa_fwd_splitkv(q, k, v, o, lse, B, H, N, d, scale, causal, blockmask, num_splits, workspace,
                   0 if workspace is None else workspace.numel(), stream)
    return o, lse, num_splits


def attention_forward_partial(q, k, v, key_offset=0, causal=False, blockmask=None, scale=None,
                              stream=None):
    """Attention of all query rows of q [B, H, N, d] over the keys k, v [B, H, Nk, d] that sit
    at query-sequence positions key_offset.. (fa_fwd_partial).  Returns fp32 (O_part, LSE_part)."""
    import torch
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    Nk = k.shape[2]
    scale = (1.0 / d ** 0.5) if scale is None else scale
    with _made_on(stream, q.device):
        o = torch.empty((B, H, N, d), dtype=torch.float32, device=q.device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fwd_partial(q, k, v, o, lse, B, H, N, Nk, d, key_offset, scale, causal, blockmask,
                   _dtype_code(q), stream)
    return o, lse


def lse_merge(o_parts, lse_parts, out_dtype=None, stream=None):
    """Merge fp32 partial results [B, H, N, d] / [B, H, N] over disjoint key slices
    (fa_lse_merge).  ``out_dtype``: torch dtype of O (bf16 default, fp16 or fp32)."""
    import torch
    B, H, N, d = o_parts[0].shape
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    code = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16, torch.float32: FA_FP32}[out_dtype]
    for t in list(o_parts) + list(lse_parts):
        if not (t.is_cuda and t.is_contiguous() and t.dtype == torch.float32):
            raise ValueError("parts must be contiguous fp32 CUDA tensors")
    with _made_on(stream, o_parts[0].device):
        o = torch.empty((B, H, N, d), dtype=out_dtype, device=o_parts[0].device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=o_parts[0].device)
    fa_lse_merge(list(o_parts), list(lse_parts), o, lse, B, H, N, d, code, stream)
    return o, lse


def attention_forward_fp8(q8, k8, v8, descale_q, descale_k, descale_v, causal=False, blockmask=None, scale=None,
                          o_fp32=False, workspace=None, stream=None):
    """FP8 forward on E4M3 tensors [B, H, N, 128] (torch.float8_e4m3fn or uint8 codes) with
    per-tensor dequantisation factors.  Returns (O bf16 or fp32, LSE)."""
    import torch
    for t in (q8, k8, v8):
        if not (t.is_cuda and t.is_contiguous() and t.dim() == 4 and t.element_size() == 1):
            raise ValueError("expected contiguous 8-bit CUDA tensors of shape [B, H, N, 128]")
    B, H, N, d = q8.shape
    scale = (1.0 / d ** 0.5) if scale is None else scale
    with _made_on(stream, q8.device):
        o = torch.empty((B, H, N, d), dtype=torch.float32 if o_fp32 else torch.bfloat16, device=q8.device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
        if workspace is None:
            workspace = torch.empty(max(fa_fwd_fp8_workspace_bytes(B, H, N, d), 1), dtype=torch.uint8, device=q8.device)
    fa_fwd_fp8(q8, k8, v8, descale_q, descale_k, descale_v, o, lse, B, H, N, d, scale, causal, blockmask, o_fp32,
               workspace, workspace.numel(), stream)
    return o, lse


def attention_backward(q, k, v, o, lse, dout, causal=False, blockmask=None, scale=None,
                       workspace=None, visit_log=None, stream=None, deterministic=False, dropout_p=0.0,
                       dropout_seed=0, query_splits=0):
    """Returns (dQ, dK, dV) for the gradient ``dout`` of O.  ``deterministic``: bitwise
    repeatable dQ through the int64 fixed-point accumulator; ``query_splits`` S >= 2: each key
    tile's query range cut into S ranges (include/fa.h)."""
    import torch
    _check_qkv(q, k, v, o, dout)
    B, H, N, d = q.shape
    scale = (1.0 / d ** 0.5) if scale is None else scale
    nbytes = (fa_bwd_workspace_bytes_split(B, H, N, d, query_splits) if query_splits > 1
              else fa_bwd_workspace_bytes_ex(B, H, N, d, deterministic))
    with _made_on(stream, q.device):
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        dq = torch.empty_like(q)
        dk = torch.empty_like(k)
        dv = torch.empty_like(v)
    fa_bwd_ex(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, scale, causal, blockmask,
              _dtype_code(q), visit_log, workspace, workspace.numel(), stream, deterministic=deterministic,
              dropout_p=dropout_p, dropout_seed=dropout_seed, query_splits=query_splits)
    return dq, dk, dv


class KVCache:
    """A paged key/value cache (fa_cache of include/fa.h): the caller's tensors and their checks.

    ``k``, ``v``: [pages, Hk, page_size, d] CUDA tensors, contiguous, bf16 or fp16, or E4M3 codes
    (torch.float8_e4m3fn or uint8) with ``k_scale``, ``v_scale`` [pages, Hk, page_size] E8M0 codes
    (torch.float8_e8m0fnu or uint8).  ``page_table``: int32 [B, max_pages]; its contents may change
    between calls.  The object keeps the tensors alive and allocates nothing.  These
    attributes cannot be set: the calls use the addresses and sizes taken here, so another table or other
    pages need another KVCache."""

    _fixed = frozenset(("k", "v", "k_scale", "v_scale", "page_table", "device", "index", "dtype", "pages", "Hk",
                        "page_size", "d", "B", "max_pages", "args", "_per_sequence", "_bounds"))

    def __setattr__(self, name, value):
        if name in self._fixed:
            raise AttributeError(f"a KVCache's {name} cannot be set: make another KVCache")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        if name in self._fixed:
            raise AttributeError(f"a KVCache's {name} cannot be deleted")
        object.__delattr__(self, name)

    def __reduce__(self):                                # a copy has the addresses of its own tensors
        return KVCache, (self.k, self.v, self.page_table, self.k_scale, self.v_scale)

    def __init__(self, k, v, page_table, k_scale=None, v_scale=None):
        global _torch
        import torch
        _torch = torch
        for t in (k, v):
            if not (t.is_cuda and t.is_contiguous() and t.dim() == 4 and t.shape == k.shape and t.dtype == k.dtype):
                raise ValueError("expected k and v as contiguous CUDA tensors of one type, [pages, Hk, page_size, d]")
        if k.element_size() == 1:
            if k.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise TypeError(f"unsupported cache dtype {k.dtype}")
            for t in (k_scale, v_scale):
                if t is None or not (t.is_cuda and t.is_contiguous() and t.element_size() == 1
                                     and t.shape == k.shape[:3]):
                    raise ValueError("an E4M3 cache needs k_scale and v_scale, [pages, Hk, page_size] E8M0 codes")
            dtype = FA_E4M3
        else:
            if k_scale is not None or v_scale is not None:
                raise ValueError("scales belong to an E4M3 cache")
            dtype = _dtype_code(k)
        if not (page_table.is_cuda and page_table.dtype == torch.int32 and page_table.dim() == 2
                and (page_table.shape[1] == 1 or page_table.stride(1) == 1)):
            raise ValueError("expected page_table as an int32 CUDA tensor [B, max_pages]")
        for t in (v, k_scale, v_scale, page_table):
            if t is not None and t.device != k.device:
                raise ValueError("the cache's tensors are on different devices")
        pages, Hk, page_size, d = k.shape
        B, max_pages = page_table.shape
        args = CacheArgs(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), pages, Hk, page_size, d, dtype,
                         B, max_pages, page_table.stride(0) if B > 1 else max(max_pages, 1))
        self.__dict__.update(
            k=k, v=v, k_scale=k_scale, v_scale=v_scale, page_table=page_table, device=k.device, index=k.get_device(),
            dtype=dtype, pages=pages, Hk=Hk, page_size=page_size, d=d, B=B, max_pages=max_pages, args=bytes(args),
            _per_sequence=(B,), _bounds=(B + 1,))

    def _ints(self, name, t, shape):
        """The address of an int32 tensor after its checks."""
        if t.dtype is _torch.int32 and t.shape == shape and t.is_contiguous() and t.get_device() == self.index:
            return t.data_ptr()
        raise ValueError(f"expected {name} as a contiguous int32 tensor {list(shape)} on the cache's device")

    def _rows(self, name, t, heads):
        """(token, head) strides of a [total, heads, d] tensor."""
        shape = t.shape
        if len(shape) == 3 and shape[1] == heads and shape[2] == self.d and t.get_device() == self.index:
            st, sh, sd = t.stride()
            if sd == 1:
                return st if shape[0] > 1 else 0, sh if heads > 1 else 0
        raise ValueError(f"expected {name} as [total, {heads}, {self.d}] on the cache's device, its last dimension contiguous")

    def _type(self, t):
        code = _dtype_code(t)
        if self.dtype != FA_E4M3 and code != self.dtype:
            raise TypeError(f"{t.dtype} tensors with a cache of {self.k.dtype}")
        return code

    def _raw_stream(self, stream):
        """The stream's handle; the current stream of the cache's device by default."""
        if stream is None:
            return _torch._C._cuda_getCurrentRawStream(self.index)
        return _stream(stream)

    def _call(self, name, payload):
        """Call an entry point with the cache's device current (CUDA launches go to it)."""
        f = getattr(_lib or lib(), name)
        if self.index == _torch._C._cuda_getDevice():
            rc = f(self.args + payload)
        else:
            with _torch.cuda.device(self.index):
                rc = f(self.args + payload)
        if rc:
            raise FAError(rc, name)


def cache_append(cache, k_new, v_new, cu_new, lens, stream=None):
    """Write the rows of new tokens, k_new and v_new [total, Hk, d] (bf16 or fp16; strided views
    will do), behind what each sequence holds (fa_cache_append): token cu_new[b] + i goes to position
    lens[b] + i of sequence b.  ``lens`` is not changed.  An E4M3 cache quantises them."""
    kt, kh = cache._rows("k_new", k_new, cache.Hk)
    vt, vh = cache._rows("v_new", v_new, cache.Hk)
    total = k_new.shape[0]
    if v_new.shape[0] != total or v_new.dtype is not k_new.dtype:
        raise ValueError("k_new and v_new differ in shape or type")
    cache._call("fa_cache_append", _pack_append(
        k_new.data_ptr(), v_new.data_ptr(), kt, kh, vt, vh, cache._ints("cu_new", cu_new, cache._bounds),
        cache._ints("lens", lens, cache._per_sequence), total, cache._type(k_new), cache._raw_stream(stream)))


def cache_read(cache, lens, N, dtype=None, k_out=None, v_out=None, stream=None):
    """The cache as dense (K, V), [B, Hk, N, d] 16-bit tensors with zeros past lens[b]
    (fa_cache_read).  ``dtype``: of an E4M3 cache's result, torch.bfloat16 (default) or float16;
    ``k_out``, ``v_out``: tensors to write to."""
    at = cache._ints("lens", lens, cache._per_sequence)
    shape = (cache.B, cache.Hk, N, cache.d)
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else _torch.bfloat16 if cache.dtype == FA_E4M3 else cache.k.dtype
    with _made_on(stream, cache.device):
        if k_out is None:
            k_out = _torch.empty(shape, dtype=dtype, device=cache.device)
        if v_out is None:
            v_out = _torch.empty(shape, dtype=dtype, device=cache.device)
    for t in (k_out, v_out):
        if not (t.get_device() == cache.index and t.shape == shape and t.is_contiguous() and t.dtype is dtype):
            raise ValueError(f"expected k_out and v_out as contiguous {dtype} tensors {list(shape)}")
    cache._call("fa_cache_read", _pack_read(at, k_out.data_ptr(), v_out.data_ptr(), N,
                                            cache._type(k_out), cache._raw_stream(stream)))
    return k_out, v_out


def cache_keep(cache, lens, kept, counts, stream=None):
    """Keep accepted rows of drafted tokens (fa_cache_keep): row lens[b] + kept[b, i] moves to row
    lens[b] + i, i < counts[b].  ``kept`` int32 [B, width], strictly increasing along a row; ``counts``
    int32 [B].  ``lens`` is not changed."""
    if kept.dim() != 2:
        raise ValueError("expected kept as [B, width]")
    width = kept.shape[1]
    cache._call("fa_cache_keep", _pack_keep(
        cache._ints("lens", lens, cache._per_sequence), cache._ints("kept", kept, (cache.B, width)),
        cache._ints("counts", counts, cache._per_sequence), width, cache._raw_stream(stream)))


def attention_forward_tree(q, cache, cu_new, lens, max_new, tree_mask=None, scale=None, workspace=None, o=None,
                           lse=None, stream=None):
    """Attention of new tokens q [total, Hq, d] over the cache that already holds their rows
    (fa_fwd_tree).  ``tree_mask``: None for a chain (token t sees new tokens j <= t), or int64
    [total, words] visibility bits (see ``tree_mask``).  ``max_new``: at least every sequence's number of
    new tokens.  ``o``, ``lse``, ``workspace``: tensors to use instead of new ones, which belong to
    ``stream``.  Returns (O, LSE), [total, Hq, d] and fp32 [total, Hq]."""
    index = cache.index
    shape = q.shape
    if len(shape) != 3 or shape[1] < 1 or shape[1] % cache.Hk:
        raise ValueError(f"expected q as [total, a multiple of {cache.Hk} heads, {cache.d}]")
    total, Hq, d = shape
    qt, qh = cache._rows("q", q, Hq)
    code = cache._type(q)
    bits = words = 0
    if tree_mask is not None:
        if not (tree_mask.get_device() == index and tree_mask.dtype is _torch.int64 and tree_mask.dim() == 2
                and tree_mask.is_contiguous() and tree_mask.shape[0] == total):
            raise ValueError("expected tree_mask as a contiguous int64 tensor [total, words] on the cache's device")
        bits, words = tree_mask.data_ptr(), tree_mask.shape[1]
    if o is None or lse is None or workspace is None:
        with _made_on(stream, cache.device):
            if o is None:
                o = _torch.empty(shape, dtype=q.dtype, device=cache.device)
            if lse is None:
                lse = _torch.empty((total, Hq), dtype=_torch.float32, device=cache.device)
            if workspace is None:
                workspace = _torch.empty(fa_fwd_tree_workspace_bytes(total, Hq, cache.Hk, d), dtype=_torch.uint8,
                                         device=cache.device)
    if o.shape != shape or o.dtype is not q.dtype:
        raise ValueError("o and q differ in shape or type")
    ot, oh = cache._rows("o", o, Hq)
    if not (lse.get_device() == index and lse.dtype is _torch.float32 and lse.shape == (total, Hq)
            and lse.is_contiguous()):
        raise ValueError("expected lse as a contiguous float32 tensor [total, Hq]")
    if not (workspace.get_device() == index and workspace.is_contiguous()):
        raise ValueError("expected workspace as a contiguous tensor on the cache's device")
    cache._call("fa_fwd_tree", _pack_tree(
        q.data_ptr(), o.data_ptr(), lse.data_ptr(), qt, qh, ot, oh, cache._ints("cu_new", cu_new, cache._bounds),
        cache._ints("lens", lens, cache._per_sequence), bits, words, total, Hq, max_new, code,
        1.0 / d ** 0.5 if scale is None else scale, workspace.data_ptr(), workspace.nbytes, cache._raw_stream(stream)))
    return o, lse


def tree_mask(parents, cu_new, words=None):
    """Visibility bits of drafted trees: int64 [total, words] with bit j of token t's row set iff new
    token j of its sequence is t itself or one of its ancestors.  ``parents``: int [total], the
    parent's index within the sequence's new tokens, smaller than the token's own, or -1 (only the prefix above
    it); ``cu_new`` as for attention_forward_tree.  Computed on the host (trees are
    drafted there or are fixed); the result is on ``cu_new``'s device."""
    import torch
    par = parents.tolist() if isinstance(parents, torch.Tensor) else [int(x) for x in parents]
    cu = cu_new.tolist()
    most = max([b - a for a, b in zip(cu, cu[1:])] + [1])
    words = (most + 63) // 64 if words is None else words
    if 64 * words < most:
        raise ValueError(f"{words} words hold no {most} tokens")
    rows = [0] * len(par)
    for a, b in zip(cu, cu[1:]):
        for t in range(a, b):
            if not -1 <= par[t] < t - a:
                raise ValueError(f"token {t - a}'s parent {par[t]} does not precede it")
            rows[t] = (rows[a + par[t]] if par[t] >= 0 else 0) | 1 << (t - a)
    full = (1 << 64) - 1
    vals = [[((r >> 64 * w & full) ^ 1 << 63) - (1 << 63) for w in range(words)] for r in rows]
    return torch.tensor(vals, dtype=torch.int64, device=cu_new.device).reshape(len(par), words)


def _make_autograd():
    import torch

    class FlashAttention(torch.autograd.Function):
        """autograd glue: forward saves (q, k, v, O, LSE); backward calls fa_bwd."""

        @staticmethod
        def forward(ctx, q, k, v, causal=False, blockmask=None, scale=None):
            o, lse = attention_forward(q, k, v, causal, blockmask, scale)
            ctx.save_for_backward(q, k, v, o, lse)
            ctx.causal, ctx.blockmask, ctx.scale = causal, blockmask, scale
            return o

        @staticmethod
        def backward(ctx, do):
            q, k, v, o, lse = ctx.saved_tensors
            dq, dk, dv = attention_backward(q, k, v, o, lse, do.contiguous(), ctx.causal,
                                            ctx.blockmask, ctx.scale)
            return dq, dk, dv, None, None, None

    return FlashAttention


def __getattr__(name):
    if name == "FlashAttention":
        fn = _make_autograd()
        globals()["FlashAttention"] = fn
        return fn
    raise AttributeError(name)
