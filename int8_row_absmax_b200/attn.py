"""Binding of the attention operators (include/bitlinear.h, "attention between the
projections"): per-head norms with the position rotation, attention over packed
sequences with a window and visible first tokens, and attention of one new token
over a paged key-value cache.

    table = bl.rope_table(4096, 128)                                   # once
    q, k, v = bl.qk_norm_rope(Y, 32, 8, 128, pos, table, gq, gk)       # Y: the Q/K/V projection's rows
    out, lse = bl.attention(q, k, v, cu, cu, max_q)                    # prompts, training
    q = bl.qk_norm_rope_append(Y, 32, 8, 128, pos, table, gq, gk, kcache, vcache, slots)
    out = bl.paged_attention(q, kcache, vcache, pages, lens, ws=ws)    # one new token per sequence

Calls run on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _check, _P, _I64, _SZ, _F, _I, load, workspace

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
    "bl_qk_norm_rope_backward_workspace_size": (_SZ, [_ROWS]),
    "bl_qk_norm_rope_backward": (_I, [_ROWS, _I, _P, _P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _SZ, _P]),
    "bl_attention": (_I, [_CALL, _P, _P, _P]),
    "bl_attention_backward_workspace_size": (_SZ, [_CALL]),
    "bl_attention_backward": (_I, [_CALL, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bl_paged_attention_workspace_size": (_SZ, [_I64, _I, _PAGES]),
    "bl_paged_attention": (_I, [_P, _I64, _I, _PAGES, _P, _I64, _P, _I32, _I32, _F, _I, _P, _P, _SZ, _P]),
}

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}     # bl_dtype


class _on:
    """The device of `t` made current for a call (only when it is not already)."""
    __slots__ = ("dev", "guard")

    def __init__(self, t):
        self.dev, self.guard = t.device, None

    def __enter__(self):
        if self.dev.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.dev)
            self.guard.__enter__()
        return torch.cuda.current_stream(self.dev).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _need(t, name, dtype, shape, dev):
    """The pointer of a contiguous tensor of this type and shape on `dev`."""
    if t.device != dev or t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {shape} on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t.device


def _half(t, name):
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"{name}: expected float16 or bfloat16, got {t.dtype}")
    return _TYPES[t.dtype]


def _rows3(t, name, dtype, dev, shape=None):
    """(pointer, elements between tokens) of [tokens, heads, D] rows whose heads are D apart."""
    if t.device != dev or t.dtype != dtype or t.dim() != 3 or (shape is not None and tuple(t.shape) != shape):
        raise ValueError(f"{name}: expected {dtype} [tokens, heads, D] {shape or ''} on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    n, h, d = t.shape
    if t.is_contiguous():
        return t.data_ptr(), h * d
    if t.stride(2) != 1 or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous, strides are {t.stride()}")
    return t.data_ptr(), t.stride(0) if n > 1 else h * d


def rope_table(positions: int, rot: int, base: float = 10000.0, device=None):
    """cos | sin of position * base^(-2i/rot), float32 [positions, rot]."""
    lib = load()
    table = torch.empty((positions, rot), dtype=torch.float32, device="cuda" if device is None else device)
    with _on(table) as stream:
        _check("bl_rope_table", lib.bl_rope_table(table.data_ptr(), positions, rot, base, stream))
    return table


def _qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved, values=True):
    """The bl_qkv_rows of a fused projection [M, (heads + 2 kv_heads) dim] or of three separate ones."""
    wq, wk = heads * dim, kv_heads * dim
    parts = (qkv, qkv, qkv) if isinstance(qkv, torch.Tensor) else tuple(qkv)
    fused = parts[0] is qkv
    dev, m = _cuda(parts[0], "qkv"), parts[0].shape[0]
    ptrs, lds = [], []
    for t, w in zip(parts, (wq, wk, wk)):
        if t is None and not values and len(ptrs) == 2:
            ptrs.append(0)
            lds.append(0)
            continue
        w = wq + 2 * wk if fused else w
        if t.device != dev or t.dtype != torch.float32 or t.dim() != 2 or tuple(t.shape) != (m, w) or \
                (w > 1 and t.stride(1) != 1):
            raise ValueError(f"qkv: expected float32 rows [{m}, {w}] on {dev}, got {t.dtype} {tuple(t.shape)} "
                             f"strides {t.stride()} on {t.device}")
        ptrs.append(t.data_ptr())
        lds.append(t.stride(0) if m > 1 else w)
    if fused:
        ptrs = [ptrs[0], ptrs[0] + 4 * wq, ptrs[0] + 4 * (wq + wk)]
    p, rot = (0, 0) if table is None else table.shape
    r = QkvRows(m, heads, kv_heads, dim, ptrs[0], ptrs[1], ptrs[2], lds[0], lds[1], lds[2],
                _need(pos, "pos", torch.int32, (m,), dev) if rot else 0,
                _need(table, "table", torch.float32, (p, rot), dev) if rot else 0, p, rot, 1 if interleaved else 0,
                0 if gq is None else _need(gq, "gq", torch.float32, (dim,), dev),
                0 if gk is None else _need(gk, "gk", torch.float32, (dim,), dev), eps)
    return r, dev, m


def qk_norm_rope(qkv, heads: int, kv_heads: int, dim: int, pos, table, gq=None, gk=None, eps: float = 1e-6,
                 dtype=torch.bfloat16, interleaved: bool = False):
    """RMSNorm of each query and key head (gains gq, gk [dim]), rotated by its position; values converted.
    qkv: the projection's float32 rows [M, (heads + 2 kv_heads) dim], or a tuple of three [M, .] tensors.
    Returns q [M, heads, dim], k and v [M, kv_heads, dim] of `dtype`.  table None: no rotation."""
    lib = load()
    if dtype not in _TYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    r, dev, m = _qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved)
    q = torch.empty((m, heads, dim), dtype=dtype, device=dev)
    k = torch.empty((m, kv_heads, dim), dtype=dtype, device=dev)
    v = torch.empty((m, kv_heads, dim), dtype=dtype, device=dev)
    with _on(q) as stream:
        _check("bl_qk_norm_rope", lib.bl_qk_norm_rope(ctypes.byref(r), _TYPES[dtype], q.data_ptr(), k.data_ptr(),
                                                      v.data_ptr(), stream))
    return q, k, v


def _cache(kcache, vcache, dev):
    if kcache.dim() != 4:
        raise ValueError("a cache is [pages, kv_heads, page, dim]")
    t = _half(kcache, "kcache")
    n, hk, page, d = kcache.shape
    return KvPages(t, _need(kcache, "kcache", kcache.dtype, (n, hk, page, d), dev),
                   _need(vcache, "vcache", kcache.dtype, (n, hk, page, d), dev), n, page, hk, d)


def qk_norm_rope_append(qkv, heads: int, kv_heads: int, dim: int, pos, table, gq, gk, kcache, vcache, slots,
                        eps: float = 1e-6, interleaved: bool = False):
    """qk_norm_rope with the keys and values stored in a paged cache [pages, kv_heads, page, dim] at
    slots [M] int64 (page number * page + place; negative: not stored).  Returns q of the cache's type."""
    lib = load()
    r, dev, m = _qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved)
    c = _cache(kcache, vcache, dev)
    at = _need(slots, "slots", torch.int64, (m,), dev)
    q = torch.empty((m, heads, dim), dtype=kcache.dtype, device=dev)
    with _on(q) as stream:
        _check("bl_qk_norm_rope_append", lib.bl_qk_norm_rope_append(ctypes.byref(r), q.data_ptr(), ctypes.byref(c), at,
                                                                    stream))
    return q


def qk_norm_rope_backward(dq, dk, dv, qkv, heads: int, kv_heads: int, dim: int, pos, table, gq=None, gk=None,
                          eps: float = 1e-6, interleaved: bool = False, ws=None):
    """Gradients of qk_norm_rope: (dqkv float32 [M, (heads + 2 kv_heads) dim], dgq, dgk float32 [dim])."""
    lib = load()
    r, dev, m = _qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved, values=False)
    if dq.dtype not in _TYPES:
        raise ValueError(f"unsupported dtype {dq.dtype}")
    pq = _need(dq, "dq", dq.dtype, (m, heads, dim), dev)
    pk = _need(dk, "dk", dq.dtype, (m, kv_heads, dim), dev)
    pv = _need(dv, "dv", dq.dtype, (m, kv_heads, dim), dev)
    wq, wk = heads * dim, kv_heads * dim
    wide = wq + 2 * wk
    dx = torch.empty((m, wide), dtype=torch.float32, device=dev)
    dg = torch.empty((2, dim), dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(lib.bl_qk_norm_rope_backward_workspace_size(ctypes.byref(r)), dtype=torch.uint8, device=dev)
    at, ag = dx.data_ptr(), dg.data_ptr()
    with _on(dx) as stream:
        _check("bl_qk_norm_rope_backward", lib.bl_qk_norm_rope_backward(
            ctypes.byref(r), _TYPES[dq.dtype], pq, pk, pv, at, wide, at + 4 * wq, wide, at + 4 * (wq + wk), wide, ag,
            ag + 4 * dim, ws.data_ptr(), ws.numel(), stream))
    return dx, dg[0], dg[1]


def _attn_call(q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale):
    dev = _cuda(q, "q")
    t = _half(q, "q")
    pq, ldq = _rows3(q, "q", q.dtype, dev)
    pk, ldk = _rows3(k, "k", q.dtype, dev)
    pv, ldv = _rows3(v, "v", q.dtype, dev, tuple(k.shape))
    if k.shape[2] != q.shape[2]:
        raise ValueError("q and k differ in head size")
    n = cu_q.shape[0]
    if n < 1:
        raise ValueError("cu_q needs at least one entry")
    return AttnCall(t, q.shape[1], k.shape[1], q.shape[2], pq, pk, pv, ldq, ldk, ldv, q.shape[0], k.shape[0],
                    _need(cu_q, "cu_q", torch.int32, (n,), dev), _need(cu_k, "cu_k", torch.int32, (n,), dev), n - 1,
                    max_q, max_k, window, sinks, 1.0 / math.sqrt(q.shape[2]) if scale is None else scale), dev


def attention(q, k, v, cu_q, cu_k, max_q: int, window: int = 0, sinks: int = 0, scale=None, out=None, lse=None):
    """softmax(scale q k^T over the visible keys) v over sequences packed end to end: q [Tq, heads, D],
    k and v [Tk, kv_heads, D] (float16 or bfloat16), cu_q and cu_k [B + 1] int32 offsets, max_q at least the
    longest query length.  A query sees the keys up to its own position within `window` tokens (0: all) and
    the first `sinks` tokens.  Returns (out [Tq, heads, D], lse float32 [heads, Tq])."""
    lib = load()
    c, dev = _attn_call(q, k, v, cu_q, cu_k, max_q, 0, window, sinks, scale)
    n, h, d = q.shape
    out = torch.empty((n, h, d), dtype=q.dtype, device=dev) if out is None else out
    lse = torch.empty((h, n), dtype=torch.float32, device=dev) if lse is None else lse
    po, pl = _need(out, "out", q.dtype, (n, h, d), dev), _need(lse, "lse", torch.float32, (h, n), dev)
    with _on(q) as stream:
        _check("bl_attention", lib.bl_attention(ctypes.byref(c), po, pl, stream))
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, max_q: int, max_k: int, window: int = 0, sinks: int = 0,
                       scale=None, ws=None, grads=None):
    """Gradients (dq, dk, dv) of attention() from its out and lse; written into `grads` when given."""
    lib = load()
    c, dev = _attn_call(q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale)
    n, h, d = q.shape
    po, pg = _need(out, "out", q.dtype, (n, h, d), dev), _need(dout, "dout", q.dtype, (n, h, d), dev)
    pl = _need(lse, "lse", torch.float32, (h, n), dev)
    if grads is None:
        grads = (torch.empty((n, h, d), dtype=q.dtype, device=dev),
                 torch.empty(tuple(k.shape), dtype=q.dtype, device=dev),
                 torch.empty(tuple(k.shape), dtype=q.dtype, device=dev))
    pd = [_need(g, "grads", q.dtype, tuple(x.shape), dev) for g, x in zip(grads, (q, k, k))]
    if ws is None:
        ws = torch.empty(lib.bl_attention_backward_workspace_size(ctypes.byref(c)), dtype=torch.uint8, device=dev)
    with _on(q) as stream:
        _check("bl_attention_backward", lib.bl_attention_backward(
            ctypes.byref(c), po, pl, pg, pd[0], pd[1], pd[2], ws.data_ptr(), ws.numel(), stream))
    return tuple(grads)


def paged_attention_workspace_size(batch: int, heads: int, kcache) -> int:
    """Bytes of the zero-filled `ws` that paged_attention needs (allocate it once with workspace())."""
    n, hk, page, d = kcache.shape
    c = KvPages(_half(kcache, "kcache"), 16, 16, n, page, hk, d)
    return int(load().bl_paged_attention_workspace_size(batch, heads, ctypes.byref(c)))


def paged_attention(q, kcache, vcache, pages, lens, window: int = 0, sinks: int = 0, scale=None,
                    out_dtype=torch.float32, ws=None, out=None):
    """Attention of one new token per sequence over a paged cache [pages, kv_heads, page, D]: q [B, heads, D]
    of the cache's type, pages [B, n] int32 page numbers, lens [B] int32 tokens of each sequence (the new one
    included).  out float32 or the cache's type, [B, heads, D].  ws: workspace(paged_attention_workspace_size(
    ...)), kept by the caller between calls; allocated and cleared in the call when None."""
    lib = load()
    dev = _cuda(q, "q")
    c = _cache(kcache, vcache, dev)
    if q.dim() != 3:
        raise ValueError("q is [batch, heads, dim]")
    b, h, d = q.shape
    if d != c.D:
        raise ValueError("q and the cache differ in head size")
    if out_dtype not in _TYPES:
        raise ValueError(f"unsupported out_dtype {out_dtype}")
    pq = _need(q, "q", kcache.dtype, (b, h, d), dev)
    if pages.dim() != 2:
        raise ValueError("pages is [batch, n]")
    pp = _need(pages, "pages", torch.int32, (b, pages.shape[1]), dev)
    pl = _need(lens, "lens", torch.int32, (b,), dev)
    out = torch.empty((b, h, d), dtype=out_dtype, device=dev) if out is None else out
    po = _need(out, "out", out_dtype, (b, h, d), dev)
    if ws is None:
        ws = workspace(lib.bl_paged_attention_workspace_size(b, h, ctypes.byref(c)), dev)
    elif ws.device != dev:
        raise ValueError(f"ws: expected a tensor on {dev}, got {ws.device}")
    with _on(q) as stream:
        _check("bl_paged_attention", lib.bl_paged_attention(
            pq, b, h, ctypes.byref(c), pp, pages.shape[1], pl, window, sinks,
            1.0 / math.sqrt(d) if scale is None else scale, _TYPES[out_dtype], po, ws.data_ptr(), ws.numel(), stream))
    return out
