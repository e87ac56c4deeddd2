"""Binding of the attention operators (include/bitlinear.h, "attention between the
projections"): per-head norms with the position rotation, attention over packed
sequences with a window and visible first tokens, and attention of one new token
over a paged key-value cache.

    table = bl.rope_table(4096, 128)                                   # once
    q, k, v = bl.qk_norm_rope(Y, 32, 8, 128, pos, table, gq, gk)       # Y: the Q/K/V projection's rows
    out, lse = bl.attention(q, k, v, cu, cu, max_q)                    # prompts, training
    q = bl.qk_norm_rope_append(Y, 32, 8, 128, pos, table, gq, gk, kcache, vcache, slots)
    out = bl.paged_attention(q, kcache, vcache, pages, lens, ws=ws)    # one new token per sequence

Calls run on the current stream of the tensors' device.  The tensors are checked and
passed on by csrc/torch_binding.cpp; the structs below mirror the header for callers of
the C ABI itself.
"""
from __future__ import annotations

import ctypes

from . import _check, _P, _I64, _SZ, _F, _I, _torch, load

_I32 = ctypes.c_int32


class QkvRows(ctypes.Structure):
    """bl_qkv_rows (field order and types as in the header)."""
    _fields_ = [("M", _I64), ("Hq", _I32), ("Hkv", _I32), ("D", _I32), ("q", _P), ("k", _P), ("v", _P),
                ("ldq", _I64), ("ldk", _I64), ("ldv", _I64), ("pos", _P), ("table", _P), ("P", _I64), ("R", _I32),
                ("interleaved", _I32), ("gq", _P), ("gk", _P), ("eps", _F)]


class KvPages(ctypes.Structure):
    """bl_kv_pages (field order and types as in the header)."""
    _fields_ = [("t", _I), ("k", _P), ("v", _P), ("pages", _I64), ("page", _I32), ("Hkv", _I32), ("D", _I32)]


class AttnCall(ctypes.Structure):
    """bl_attn_call (field order and types as in the header)."""
    _fields_ = [("t", _I), ("Hq", _I32), ("Hkv", _I32), ("D", _I32), ("q", _P), ("k", _P), ("v", _P), ("ldq", _I64),
                ("ldk", _I64), ("ldv", _I64), ("Tq", _I64), ("Tk", _I64), ("cu_q", _P), ("cu_k", _P), ("B", _I32),
                ("max_q", _I32), ("max_k", _I32), ("window", _I32), ("sinks", _I32), ("scale", _F)]


_ROWS, _PAGES, _CALL = (ctypes.POINTER(c) for c in (QkvRows, KvPages, AttnCall))
SIGNATURES = {
    "bl_rope_table": (_I, [_P, _I64, _I, ctypes.c_double, _P]),
    "bl_qk_norm_rope": (_I, [_ROWS, _I, _P, _P, _P, _P]),
    "bl_qk_norm_rope_append": (_I, [_ROWS, _P, _PAGES, _P, _P]),
    "bl_qk_norm_rope_plan": (_I, [_ROWS, _I, ctypes.POINTER(_I)]),
    "bl_qk_norm_rope_backward_workspace_size": (_SZ, [_ROWS]),
    "bl_qk_norm_rope_backward": (_I, [_ROWS, _I, _P, _P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _SZ, _P]),
    "bl_attention": (_I, [_CALL, _P, _P, _P]),
    "bl_attention_ex": (_I, [_CALL, _P, _P, _I, _P]),
    "bl_attention_backward_workspace_size": (_SZ, [_CALL]),
    "bl_attention_backward": (_I, [_CALL, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bl_attention_backward_ex": (_I, [_CALL, _P, _P, _P, _P, _P, _P, _P, _SZ, _I, _P]),
    "bl_paged_attention_workspace_size": (_SZ, [_I64, _I, _PAGES]),
    "bl_paged_attention": (_I, [_P, _I64, _I, _PAGES, _P, _I64, _P, _I32, _I32, _F, _I, _P, _P, _SZ, _P]),
}

_TYPES = {"torch.float32": 0, "torch.float16": 1, "torch.bfloat16": 2}     # bl_dtype, by the dtype's name
_binding = None


def _native():
    """The tensor binding over the loaded library (raises if it has not been built for the PyTorch and Python
    that run)."""
    global _binding
    if _binding is None:
        from . import build
        lib = load()
        _torch()
        if not build.binding_fits():
            raise RuntimeError("_binding.so is missing or built for another PyTorch or Python: build it with "
                               "python -m int8_row_absmax_b200.build")
        from . import _binding as module
        module.use(lib._handle)
        _binding = module
    return _binding


def _code(dtype):
    code = _TYPES.get(str(dtype))
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    return code


def rope_table(positions: int, rot: int, base: float = 10000.0, device=None):
    """cos | sin of position * base^(-2i/rot), float32 [positions, rot]."""
    torch, lib = _torch(), load()
    table = torch.empty((positions, rot), dtype=torch.float32, device="cuda" if device is None else device)
    if not table.is_cuda:
        raise ValueError("the table must be on a CUDA device")
    with torch.cuda.device(table.device):
        _check("bl_rope_table", lib.bl_rope_table(table.data_ptr(), positions, rot, base,
                                                  torch.cuda.current_stream(table.device).cuda_stream))
    return table


def qk_norm_rope(qkv, heads: int, kv_heads: int, dim: int, pos, table, gq=None, gk=None, eps: float = 1e-6,
                 dtype=None, interleaved: bool = False):
    """RMSNorm of each query and key head (gains gq, gk [dim]), rotated by its position; values converted.
    qkv: the projection's float32 rows [M, (heads + 2 kv_heads) dim], or a tuple of three [M, .] tensors.
    Returns q [M, heads, dim], k and v [M, kv_heads, dim] of `dtype` (bfloat16 by default).  table None: no
    rotation.  Rows of a position outside the table are undefined (sync_status() then says BL_ERR_RANGE)."""
    return _native().qk_norm_rope(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps,
                                  2 if dtype is None else _code(dtype), interleaved)


def qk_norm_rope_append(qkv, heads: int, kv_heads: int, dim: int, pos, table, gq, gk, kcache, vcache, slots,
                        eps: float = 1e-6, interleaved: bool = False):
    """qk_norm_rope with the keys and values stored in a paged cache [pages, kv_heads, page, dim] at
    slots [M] int64 (page number * page + place; negative: not stored).  Returns q of the cache's type (rows
    of a position outside the table are undefined)."""
    return _native().qk_norm_rope_append(qkv, heads, kv_heads, dim, pos, table, gq, gk, kcache, vcache, slots, eps,
                                         interleaved)


def qk_norm_rope_backward(dq, dk, dv, qkv, heads: int, kv_heads: int, dim: int, pos, table, gq=None, gk=None,
                          eps: float = 1e-6, interleaved: bool = False, ws=None):
    """Gradients of qk_norm_rope: (dqkv float32 [M, (heads + 2 kv_heads) dim], dgq, dgk float32 [dim]).
    dgq and dgk are sums over all M rows, padding included, whose dq and dk have to be zero, as
    attention_backward leaves them.  Rows of a position outside the table are undefined and not summed."""
    return _native().qk_norm_rope_backward(dq, dk, dv, qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved,
                                           ws)


def attention(q, k, v, cu_q, cu_k, max_q: int, window: int = 0, sinks: int = 0, scale=None, out=None, lse=None):
    """softmax(scale q k^T over the visible keys) v over sequences packed end to end: q [Tq, heads, D],
    k and v [Tk, kv_heads, D] (float16 or bfloat16), cu_q and cu_k [B + 1] int32 offsets, max_q at least the
    longest query length.  A query sees the keys up to its own position within `window` tokens (0: all) and
    the first `sinks` tokens.  Returns (out [Tq, heads, D], lse float32 [heads, Tq]).  Rows of no sequence
    (before cu_q[0], behind cu_q[-1]) keep what `out` and `lse` hold when given, else they are 0 and -inf;
    those of a sequence that is left out (BL_ERR_RANGE) are undefined."""
    return _native().attention(q, k, v, cu_q, cu_k, max_q, window, sinks, scale, out, lse)


def attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, max_q: int, max_k: int, window: int = 0, sinks: int = 0,
                       scale=None, ws=None, grads=None):
    """Gradients (dq, dk, dv) of attention() from its out and lse; written into `grads` when given (rows of no
    sequence then keep what they hold, else they are 0)."""
    dq, dk, dv = (None, None, None) if grads is None else grads
    return _native().attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, max_q, max_k, window, sinks, scale, ws, dq,
                                        dk, dv)


def paged_attention_workspace_size(batch: int, heads: int, kcache) -> int:
    """Bytes of the zero-filled `ws` that paged_attention needs (allocate it once with workspace())."""
    n, hk, page, d = kcache.shape
    c = KvPages(_code(kcache.dtype), 16, 16, n, page, hk, d)
    return int(load().bl_paged_attention_workspace_size(batch, heads, ctypes.byref(c)))


def paged_attention(q, kcache, vcache, pages, lens, window: int = 0, sinks: int = 0, scale=None,
                    out_dtype=None, ws=None, out=None):
    """Attention of one new token per sequence over a paged cache [pages, kv_heads, page, D]: q [B, heads, D]
    of the cache's type, pages [B, n] int32 page numbers, lens [B] int32 tokens of each sequence (the new one
    included).  out float32 (the default) or the cache's type, [B, heads, D].  ws:
    workspace(paged_attention_workspace_size(...)), kept by the caller between calls; allocated and cleared in
    the call when None."""
    return _native().paged_attention(q, kcache, vcache, pages, lens, window, sinks, scale,
                                     0 if out_dtype is None else _code(out_dtype), ws, out)
