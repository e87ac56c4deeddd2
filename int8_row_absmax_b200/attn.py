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
import struct

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


# Small calls are bound by the host's time, so the structs are packed in one step (the
# same native layout as the classes above) and passed by address.
_pack_rows = struct.Struct("@q3i3P3q2Pq2i2Pf4x").pack
_pack_pages = struct.Struct("@i2Pq3i4x").pack
_pack_call = struct.Struct("@4i3P5q2P5if").pack

SIGNATURES = {
    "bl_rope_table": (_I, [_P, _I64, _I, ctypes.c_double, _P]),
    "bl_qk_norm_rope": (_I, [_P, _I, _P, _P, _P, _P]),
    "bl_qk_norm_rope_append": (_I, [_P, _P, _P, _P, _P]),
    "bl_qk_norm_rope_backward_workspace_size": (_SZ, [_P]),
    "bl_qk_norm_rope_backward": (_I, [_P, _I, _P, _P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _SZ, _P]),
    "bl_attention": (_I, [_P, _P, _P, _P]),
    "bl_attention_backward_workspace_size": (_SZ, [_P]),
    "bl_attention_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bl_paged_attention_workspace_size": (_SZ, [_I64, _I, _P]),
    "bl_paged_attention": (_I, [_P, _I64, _I, _P, _P, _I64, _P, _I32, _I32, _F, _I, _P, _P, _SZ, _P]),
}

_F32 = torch.float32
_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}     # bl_dtype
_HALF = {torch.float16: 1, torch.bfloat16: 2}


def _call(fn, name, dev, args):
    """fn(*args, the device's current stream) with that device current."""
    if dev == torch.cuda.current_device():
        code = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if code:
        _check(name, code)


def _need(t, name, dtype, shape, dev):
    """The pointer of a contiguous tensor of this type and shape on device `dev`."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _cuda(t, name):
    """The index of the tensor's device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    return dev


def _half(t, name):
    code = _HALF.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: expected float16 or bfloat16, got {t.dtype}")
    return code


def _rows3(t, name, dtype, dev):
    """(pointer, elements between tokens) of [tokens, heads, D] rows whose heads are D apart."""
    if t.get_device() != dev or t.dtype is not dtype or t.dim() != 3:
        raise ValueError(f"{name}: expected {dtype} [tokens, heads, D] on cuda:{dev}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    n, h, d = t.shape
    if t.is_contiguous():
        return t.data_ptr(), h * d
    if t.stride(2) != 1 or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous, strides are {t.stride()}")
    return t.data_ptr(), t.stride(0) if n > 1 else h * d


def rope_table(positions: int, rot: int, base: float = 10000.0, device=None):
    """cos | sin of position * base^(-2i/rot), float32 [positions, rot]."""
    lib = load()
    table = torch.empty((positions, rot), dtype=_F32, device="cuda" if device is None else device)
    _call(lib.bl_rope_table, "bl_rope_table", _cuda(table, "table"), (table.data_ptr(), positions, rot, base))
    return table


def _qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved, values=True):
    """(the packed bl_qkv_rows, device, tokens) of a fused projection [M, (heads + 2 kv_heads) dim] or of three
    separate ones."""
    wq, wk = heads * dim, kv_heads * dim
    if isinstance(qkv, torch.Tensor):
        dev, shape = _cuda(qkv, "qkv"), qkv.shape
        if qkv.dtype is not _F32 or len(shape) != 2 or shape[1] != wq + 2 * wk or not (
                qkv.is_contiguous() or qkv.stride(1) == 1):
            raise ValueError(f"qkv: expected float32 rows of {wq + 2 * wk}, got {qkv.dtype} {tuple(shape)} strides "
                             f"{qkv.stride()}")
        m = shape[0]
        ldq = ldk = ldv = qkv.stride(0) if m > 1 else wq + 2 * wk
        q = qkv.data_ptr()
        k = q + 4 * wq
        v = k + 4 * wk
    else:
        parts = tuple(qkv)
        dev, m = _cuda(parts[0], "qkv"), parts[0].shape[0]
        ptrs, lds = [], []
        for t, w in zip(parts, (wq, wk, wk)):
            if t is None and not values and len(ptrs) == 2:
                ptrs.append(0)
                lds.append(0)
                continue
            if t.get_device() != dev or t.dtype is not _F32 or t.shape != (m, w) or (w > 1 and t.stride(1) != 1):
                raise ValueError(f"qkv: expected float32 rows [{m}, {w}] on cuda:{dev}, got {t.dtype} "
                                 f"{tuple(t.shape)} strides {t.stride()} on {t.device}")
            ptrs.append(t.data_ptr())
            lds.append(t.stride(0) if m > 1 else w)
        (q, k, v), (ldq, ldk, ldv) = ptrs, lds
    if table is None:
        p = rot = pp = pt = 0
    else:
        p, rot = table.shape
        pt = _need(table, "table", _F32, (p, rot), dev)
        pp = _need(pos, "pos", torch.int32, (m,), dev)
    return _pack_rows(m, heads, kv_heads, dim, q, k, v, ldq, ldk, ldv, pp, pt, p, rot, 1 if interleaved else 0,
                      0 if gq is None else _need(gq, "gq", _F32, (dim,), dev),
                      0 if gk is None else _need(gk, "gk", _F32, (dim,), dev), eps), dev, m


def qk_norm_rope(qkv, heads: int, kv_heads: int, dim: int, pos, table, gq=None, gk=None, eps: float = 1e-6,
                 dtype=torch.bfloat16, interleaved: bool = False):
    """RMSNorm of each query and key head (gains gq, gk [dim]), rotated by its position; values converted.
    qkv: the projection's float32 rows [M, (heads + 2 kv_heads) dim], or a tuple of three [M, .] tensors.
    Returns q [M, heads, dim], k and v [M, kv_heads, dim] of `dtype`.  table None: no rotation."""
    lib = load()
    code = _TYPES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    r, dev, m = _qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved)
    device = torch.device("cuda", dev)
    q = torch.empty((m, heads, dim), dtype=dtype, device=device)
    k = torch.empty((m, kv_heads, dim), dtype=dtype, device=device)
    v = torch.empty((m, kv_heads, dim), dtype=dtype, device=device)
    _call(lib.bl_qk_norm_rope, "bl_qk_norm_rope", dev, (r, code, q.data_ptr(), k.data_ptr(), v.data_ptr()))
    return q, k, v


def _cache(kcache, vcache, dev):
    """(the packed bl_kv_pages, kv_heads, dim)."""
    if kcache.dim() != 4:
        raise ValueError("a cache is [pages, kv_heads, page, dim]")
    t, shape, dtype = _half(kcache, "kcache"), kcache.shape, kcache.dtype
    n, hk, page, d = shape
    return _pack_pages(t, _need(kcache, "kcache", dtype, shape, dev), _need(vcache, "vcache", dtype, shape, dev), n,
                       page, hk, d), hk, d


def qk_norm_rope_append(qkv, heads: int, kv_heads: int, dim: int, pos, table, gq, gk, kcache, vcache, slots,
                        eps: float = 1e-6, interleaved: bool = False):
    """qk_norm_rope with the keys and values stored in a paged cache [pages, kv_heads, page, dim] at
    slots [M] int64 (page number * page + place; negative: not stored).  Returns q of the cache's type."""
    lib = load()
    r, dev, m = _qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved)
    c, _, _ = _cache(kcache, vcache, dev)
    at = _need(slots, "slots", torch.int64, (m,), dev)
    q = kcache.new_empty((m, heads, dim))
    _call(lib.bl_qk_norm_rope_append, "bl_qk_norm_rope_append", dev, (r, q.data_ptr(), c, at))
    return q


def qk_norm_rope_backward(dq, dk, dv, qkv, heads: int, kv_heads: int, dim: int, pos, table, gq=None, gk=None,
                          eps: float = 1e-6, interleaved: bool = False, ws=None):
    """Gradients of qk_norm_rope: (dqkv float32 [M, (heads + 2 kv_heads) dim], dgq, dgk float32 [dim])."""
    lib = load()
    r, dev, m = _qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved, values=False)
    dtype = dq.dtype
    code = _TYPES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    pq = _need(dq, "dq", dtype, (m, heads, dim), dev)
    pk = _need(dk, "dk", dtype, (m, kv_heads, dim), dev)
    pv = _need(dv, "dv", dtype, (m, kv_heads, dim), dev)
    wq, wk = heads * dim, kv_heads * dim
    wide = wq + 2 * wk
    device = torch.device("cuda", dev)
    dx = torch.empty((m, wide), dtype=_F32, device=device)
    dg = torch.empty((2, dim), dtype=_F32, device=device)
    if ws is None:
        ws = torch.empty(lib.bl_qk_norm_rope_backward_workspace_size(r), dtype=torch.uint8, device=device)
    else:
        _need(ws, "ws", ws.dtype, ws.shape, dev)
    at, ag = dx.data_ptr(), dg.data_ptr()
    _call(lib.bl_qk_norm_rope_backward, "bl_qk_norm_rope_backward", dev,
          (r, code, pq, pk, pv, at, wide, at + 4 * wq, wide, at + 4 * (wq + wk), wide, ag, ag + 4 * dim, ws.data_ptr(),
           ws.nbytes))
    dgq, dgk = dg.unbind()
    return dx, dgq, dgk


def _attn_call(q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale):
    dev, dtype = _cuda(q, "q"), q.dtype
    t = _half(q, "q")
    pq, ldq = _rows3(q, "q", dtype, dev)
    pk, ldk = _rows3(k, "k", dtype, dev)
    pv, ldv = _rows3(v, "v", dtype, dev)
    tq, h, d = q.shape
    tk, hk, dk = k.shape
    if v.shape != k.shape or dk != d:
        raise ValueError(f"q, k and v do not fit together: {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    n = cu_q.shape
    if len(n) != 1 or n[0] < 1:
        raise ValueError("cu_q holds at least one offset")
    return _pack_call(t, h, hk, d, pq, pk, pv, ldq, ldk, ldv, tq, tk, _need(cu_q, "cu_q", torch.int32, n, dev),
                      _need(cu_k, "cu_k", torch.int32, n, dev), n[0] - 1, max_q, max_k, window, sinks,
                      1.0 / math.sqrt(d) if scale is None else scale), dev


def attention(q, k, v, cu_q, cu_k, max_q: int, window: int = 0, sinks: int = 0, scale=None, out=None, lse=None):
    """softmax(scale q k^T over the visible keys) v over sequences packed end to end: q [Tq, heads, D],
    k and v [Tk, kv_heads, D] (float16 or bfloat16), cu_q and cu_k [B + 1] int32 offsets, max_q at least the
    longest query length.  A query sees the keys up to its own position within `window` tokens (0: all) and
    the first `sinks` tokens.  Returns (out [Tq, heads, D], lse float32 [heads, Tq])."""
    lib = load()
    c, dev = _attn_call(q, k, v, cu_q, cu_k, max_q, 0, window, sinks, scale)
    shape = q.shape
    n, h, _ = shape
    if out is None:
        out = q.new_empty(shape)
    if lse is None:
        lse = q.new_empty((h, n), dtype=_F32)
    _call(lib.bl_attention, "bl_attention", dev,
          (c, _need(out, "out", q.dtype, shape, dev), _need(lse, "lse", _F32, (h, n), dev)))
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, max_q: int, max_k: int, window: int = 0, sinks: int = 0,
                       scale=None, ws=None, grads=None):
    """Gradients (dq, dk, dv) of attention() from its out and lse; written into `grads` when given."""
    lib = load()
    c, dev = _attn_call(q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale)
    dtype, shape, kshape = q.dtype, q.shape, k.shape
    po, pg = _need(out, "out", dtype, shape, dev), _need(dout, "dout", dtype, shape, dev)
    pl = _need(lse, "lse", _F32, (shape[1], shape[0]), dev)
    if grads is None:
        dq, dk, dv = q.new_empty(shape), q.new_empty(kshape), q.new_empty(kshape)
    else:
        dq, dk, dv = grads
    if ws is None:
        ws = q.new_empty(lib.bl_attention_backward_workspace_size(c), dtype=torch.uint8)
    else:
        _need(ws, "ws", ws.dtype, ws.shape, dev)
    _call(lib.bl_attention_backward, "bl_attention_backward", dev,
          (c, po, pl, pg, _need(dq, "dq", dtype, shape, dev), _need(dk, "dk", dtype, kshape, dev),
           _need(dv, "dv", dtype, kshape, dev), ws.data_ptr(), ws.nbytes))
    return dq, dk, dv


def paged_attention_workspace_size(batch: int, heads: int, kcache) -> int:
    """Bytes of the zero-filled `ws` that paged_attention needs (allocate it once with workspace())."""
    n, hk, page, d = kcache.shape
    return int(load().bl_paged_attention_workspace_size(batch, heads, _pack_pages(_half(kcache, "kcache"), 16, 16, n,
                                                                                  page, hk, d)))


def paged_attention(q, kcache, vcache, pages, lens, window: int = 0, sinks: int = 0, scale=None,
                    out_dtype=torch.float32, ws=None, out=None):
    """Attention of one new token per sequence over a paged cache [pages, kv_heads, page, D]: q [B, heads, D]
    of the cache's type, pages [B, n] int32 page numbers, lens [B] int32 tokens of each sequence (the new one
    included).  out float32 or the cache's type, [B, heads, D].  ws: workspace(paged_attention_workspace_size(
    ...)), kept by the caller between calls; allocated and cleared in the call when None."""
    lib = load()
    dev, shape = _cuda(q, "q"), q.shape
    c, _, d = _cache(kcache, vcache, dev)
    if len(shape) != 3 or shape[2] != d:
        raise ValueError(f"q is [batch, heads, {d}], got {tuple(shape)}")
    b, h, _ = shape
    code = _TYPES.get(out_dtype)
    if code is None:
        raise ValueError(f"unsupported out_dtype {out_dtype}")
    pq = _need(q, "q", kcache.dtype, shape, dev)
    width = pages.shape
    if len(width) != 2 or width[0] != b:
        raise ValueError(f"pages is [{b}, n], got {tuple(width)}")
    pp = _need(pages, "pages", torch.int32, width, dev)
    pl = _need(lens, "lens", torch.int32, (b,), dev)
    if out is None:
        out = q.new_empty(shape, dtype=out_dtype)
    po = _need(out, "out", out_dtype, shape, dev)
    if ws is None:
        ws = workspace(lib.bl_paged_attention_workspace_size(b, h, c), q.device)
    else:
        _need(ws, "ws", ws.dtype, ws.shape, dev)
    _call(lib.bl_paged_attention, "bl_paged_attention", dev,
          (pq, b, h, c, pp, width[1], pl, window, sinks, 1.0 / math.sqrt(d) if scale is None else scale, code, po,
           ws.data_ptr(), ws.nbytes))
    return out
