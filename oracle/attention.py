"""Attention between the projections, in float64 (plain and slow).

"ultragraph -- when the graph is the 1-bit LLM, part 2", section "attention, as
graph ops": heads, softmax(Q K^T / sqrt(d) + mask) V, RMSNorm(x) = x /
sqrt(mean(x^2) + eps) * g; RoPE and the KV cache of "ultragraph-1bit 0.12.0"
(PyPI).  A token at position p sees the keys j <= p with j > p - window (window 0:
all of them) or j < sinks.
"""
import numpy as np

F64 = np.float64


def rope_table(positions, rot, base=10000.0):
    """cos | sin of p * base^(-2i/rot): float32 [positions, rot]."""
    ang = np.arange(positions, dtype=F64)[:, None] * base ** (-2.0 * np.arange(rot // 2, dtype=F64) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def rotation_pairs(rot, interleaved):
    """The two members of each rotated pair of a head's elements."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(y, pos, table, interleaved, back=False):
    """Rows y [M, heads, D]: (a, b) -> (a cos - b sin, a sin + b cos); `back`: the transposed rotation."""
    rot = table.shape[1]
    a, b = rotation_pairs(rot, interleaved)
    t = table.astype(F64)[pos][:, None, :]
    cos, sin = t[..., :rot // 2], t[..., rot // 2:] * (-1 if back else 1)
    z = y.astype(F64).copy()
    z[..., a] = y[..., a] * cos - y[..., b] * sin
    z[..., b] = y[..., a] * sin + y[..., b] * cos
    return z


def norm_rope(x, pos, table, g, eps, interleaved=False):
    """x [M, heads, D] -> the normed and rotated heads."""
    x = x.astype(F64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if g is None else g.astype(F64))
    return y if table is None else rotate(y, pos, table, interleaved)


def norm_rope_backward(dz, x, pos, table, g, eps, interleaved=False):
    """(dx, dg) of norm_rope."""
    x, dz = x.astype(F64), dz.astype(F64)
    dy = dz if table is None else rotate(dz, pos, table, interleaved, back=True)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    gy = dy * (1.0 if g is None else g.astype(F64))
    dx = r * gy - x * r ** 3 * (x * gy).mean(-1, keepdims=True)
    return dx, (dy * x * r).sum((0, 1))


def visible(nq, nk, window=0, sinks=0):
    """Truth values [nq, nk]; query i stands at position i + nk - nq."""
    p = np.arange(nq)[:, None] + nk - nq
    j = np.arange(nk)[None]
    see = j <= p
    return see & ((j > p - window) | (j < sinks)) if window else see


def attention(q, k, v, window=0, sinks=0, scale=None):
    """One sequence: q [nq, Hq, D], k, v [nk, Hkv, D] -> (out [nq, Hq, D], lse [Hq, nq], p [Hq, nq, nk])."""
    q, k, v = (t.astype(F64) for t in (q, k, v))
    nq, hq, d = q.shape
    nk, hkv, _ = k.shape
    scale = 1 / np.sqrt(d) if scale is None else scale
    see = visible(nq, nk, window, sinks)
    out, lse, ps = np.zeros((nq, hq, d)), np.full((hq, nq), -np.inf), np.zeros((hq, nq, nk))
    some = see.any(1)
    for h in range(hq):
        u = h // (hq // hkv)
        kk, vv = np.where(see.any(0)[:, None], k[:, u], 0), np.where(see.any(0)[:, None], v[:, u], 0)
        x = np.where(see, q[:, h] @ kk.T * scale, -np.inf)
        top = np.where(some, x.max(1, initial=-np.inf), 0)
        e = np.exp(x - top[:, None])
        s = e.sum(1)
        ps[h] = e / np.where(some, s, 1)[:, None]
        lse[h, some] = top[some] + np.log(s[some])
        out[:, h] = ps[h] @ vv
    return out, lse, ps


def attention_backward(dout, q, k, v, out, lse, window=0, sinks=0, scale=None):
    """One sequence: (dq, dk, dv) from the given out [nq, Hq, D] and lse [Hq, nq]."""
    q, k, v, dout, out, lse = (t.astype(F64) for t in (q, k, v, dout, out, lse))
    nq, hq, d = q.shape
    nk, hkv, _ = k.shape
    scale = 1 / np.sqrt(d) if scale is None else scale
    see = visible(nq, nk, window, sinks)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(hq):
        u = h // (hq // hkv)
        low = np.where(np.isfinite(lse[h]), lse[h], 0)[:, None]
        p = np.where(see, np.exp(np.where(see, q[:, h] @ k[:, u].T * scale, 0) - low), 0)
        delta = (dout[:, h] * out[:, h]).sum(1, keepdims=True)
        ds = p * (dout[:, h] @ v[:, u].T - delta) * scale
        dq[:, h] = ds @ k[:, u]
        dk[:, u] += ds.T @ q[:, h]
        dv[:, u] += p.T @ dout[:, h]
    return dq, dk, dv


def paged_rows(cache, pages, n):
    """The first n tokens [n, Hkv, D] of a sequence whose pages [.] lie in cache [pages, Hkv, page, D]."""
    page = cache.shape[2]
    rows = [cache[pages[j // page], :, j % page] for j in range(n)]
    return np.stack(rows) if rows else np.zeros((0, cache.shape[1], cache.shape[3]), cache.dtype)
